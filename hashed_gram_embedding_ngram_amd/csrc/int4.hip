// Weights in 4 bits with a scale (and a zero) for each group of columns, for
// MI355X (gfx950): ngram_quant_int4, ngram_dequant_int4 and the product
// ngram_project_int4.  The formats and formulas are in include/ngram.h.  Times in comments are on the
// card: of one kernel, or of a call replayed in a graph.
#include "common8.h"

#include <algorithm>

namespace ng8 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kChunk = 128;             // columns that a wavefront takes at a time: 16 bytes of codes a lane

inline int64_t int4_ld(int64_t cols) { return (cols + 31) / 32 * 16; }
inline int64_t int4_groups(int64_t cols, int group) { return (cols + group - 1) / group; }
inline int64_t int4_sld(int64_t cols, int group) { return (int4_groups(cols, group) + 3) / 4 * 4; }

bool shape_ok(int64_t rows, int64_t cols, int group) {
    return rows >= 0 && rows <= NGRAM_INT4_MAX_ROWS && cols >= 0 && cols <= NGRAM_INT4_MAX_COLS && cols % kVec == 0 &&
           (group == 32 || group == 64 || group == 128);
}

int check_int4(const ngram_int4* q, const char* what) {
    if (!q) return fail(NGRAM_EINVAL, "%s is NULL", what);
    if (q->rows < 0 || q->cols < 0 || q->cols % kVec != 0)
        return fail(NGRAM_EINVAL, "%s: rows=%lld and cols=%lld must not be negative, cols a multiple of %d", what, (long long)q->rows,
                    (long long)q->cols, kVec);
    if (q->group != 32 && q->group != 64 && q->group != 128) return fail(NGRAM_EINVAL, "%s: group=%d must be 32, 64 or 128", what, q->group);
    if (q->scale_dtype != NGRAM_F32 && q->scale_dtype != NGRAM_BF16)
        return fail(NGRAM_EINVAL, "%s: scale_dtype=%d is not an ngram_value", what, q->scale_dtype);
    if (q->rows > NGRAM_INT4_MAX_ROWS || q->cols > NGRAM_INT4_MAX_COLS)
        return fail(NGRAM_ERANGE, "%s: rows=%lld above %d or cols=%lld above %d", what, (long long)q->rows, NGRAM_INT4_MAX_ROWS,
                    (long long)q->cols, NGRAM_INT4_MAX_COLS);
    if (q->rows > 0 && q->cols > 0) {
        if (!q->codes || !q->scales) return fail(NGRAM_EINVAL, "%s: codes or scales is NULL", what);
        if (!aligned(q->codes, 16) || !aligned(q->scales, 16) || !aligned(q->zeros, 4))
            return fail(NGRAM_EALIGN, "%s: codes and scales must be 16-byte and zeros 4-byte aligned", what);
    }
    return NGRAM_OK;
}

// ---------------------------------------------------------------------------
// Quantising and reading back.  A lane takes eight columns, a group is 4, 8 or
// 16 neighbouring lanes: its lowest and highest value go round by lane moves.
// 151936 x 2560 bf16 with zeros and bf16 scales (991 MB): quantising 226 to 256 us,
// bound by some 200 instructions for eight columns (a division for each weight
// 325, two corrections of each quotient 265); reading back 163 to 170, bound by
// memory at 6 TB/s.
struct QuantArgs {
    const void* x;          // quantising: [rows][cols] fp32 or bf16
    void* y;                // reading back: the same
    uint8_t* codes;
    void* scales;
    uint8_t* zeros;         // or NULL: 8
    int64_t row0;           // the launch's first row
    int64_t ld, sld;
    uint32_t units;         // eights of columns a row, up to whole groups
    uint32_t count;         // of the launch, below 2^31
    uint32_t magic, shift;  // t / units = (t * magic) >> (32 + shift) for t < 2^31
    int32_t cols, group, sf32;
};

__device__ __forceinline__ float min_lanes(float x, int lanes) {
    x = fminf(x, __uint_as_float(dpp<0xB1>(__float_as_uint(x))));
    x = fminf(x, __uint_as_float(dpp<0x4E>(__float_as_uint(x))));
    if (lanes > 4) x = fminf(x, __uint_as_float(dpp<0x141>(__float_as_uint(x))));
    if (lanes > 8) x = fminf(x, __uint_as_float(dpp<0x140>(__float_as_uint(x))));
    return x;
}

__device__ __forceinline__ uint32_t div_units(const QuantArgs& a, uint32_t t) {
    return a.units == 1 ? t : static_cast<uint32_t>((static_cast<uint64_t>(t) * a.magic) >> 32) >> a.shift;
}

// a / b correctly rounded from y = 1 / b, which is: a product, and twice the remainder times y.  The first
// makes the quotient one of the two fp32 numbers around the true one, and from such a one and a correctly
// rounded y the second gives the nearest (Markstein's theorem).  Where a and b have eight bits once is enough:
// a / b then is an fp32 number or 2^-9 of a step and more from the middle of two (a whole number over b's, 2^-24
// and 2^-8), and the first leaves an error below 2^-22 of a step before it rounds.
template <bool TWICE>
__device__ __forceinline__ float quotient(float a, float b, float y) {
    float v = a * y;
    v = __builtin_fmaf(__builtin_fmaf(-v, b, a), y, v);
    if (TWICE) v = __builtin_fmaf(__builtin_fmaf(-v, b, a), y, v);
    return v;
}

template <bool F32, bool ASYM, bool SF32>
__global__ void __launch_bounds__(256) quant_int4_kernel(const QuantArgs a) {
    const uint32_t t = blockIdx.x * 256 + threadIdx.x;
    const bool on = t < a.count;                            // whole groups are on or off
    const uint32_t r = div_units(a, t), u = t - r * a.units;
    const int64_t row = a.row0 + r;
    const int col = static_cast<int>(u) * kVec;
    Raw8<F32> raw;
    if (on && col < a.cols) raw.load_stream(a.x, row * a.cols + col); else raw.zero();
    float w[8];
    raw.get(w);
    // lowest and highest value, both from minima; a NaN or an infinity anywhere makes the sum of 0 * w a NaN
    float lo = 0.0f, nhi = 0.0f, bad = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        lo = fminf(lo, w[k]);
        nhi = fminf(nhi, -w[k]);
        bad = __builtin_fmaf(w[k], 0.0f, bad);
    }
    const int lanes = a.group / kVec;
    lo = min_lanes(lo, lanes);
    nhi = min_lanes(nhi, lanes);
    constexpr float steps = ASYM ? 15.0f : 7.0f, one = 1.0f / steps;
    const float range = ASYM ? -nhi - lo : fmaxf(-lo, -nhi);
    float s = quotient<true>(range, steps, one);
    if (__builtin_expect(__ballot(!(range > 0x1p-90f && range < 0x1p90f)) != 0, 0)) s = range / steps;
    if (!SF32) s = __uint_as_float(bf16_pair(s, s) << 16);
    // a group with a value that is not finite, or too wide for a finite scale, is NaN throughout
    const uint64_t odd = __ballot(!(bad == 0.0f));
    const int first = (threadIdx.x & 63) & ~(lanes - 1);
    const bool nan = ((odd >> first) & ((1u << lanes) - 1)) != 0 || !(s < __uint_as_float(kInfBits));
    if (s == 0.0f) s = 1.0f;
    const float y = 1.0f / s;
    float z = 8.0f, q[8];
    if (ASYM) z = rintf(quotient<F32 || SF32>(-lo, s, y));
#pragma unroll
    for (int k = 0; k < 8; ++k) q[k] = rintf(quotient<F32 || SF32>(w[k], s, y));
    if (__builtin_expect(__ballot(!(s > 0x1p-100f && s < 0x1p100f)) != 0, 0)) {     // where 1 / s or a remainder leaves the range
        if (ASYM) z = rintf(-lo / s);
#pragma unroll
        for (int k = 0; k < 8; ++k) q[k] = rintf(w[k] / s);
    }
    if (ASYM) z = fminf(fmaxf(z, 0.0f), 15.0f);
    // four codes in a whole number below 2^16, Horner's way, the zero added to all of them at once
    float half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v = 0.0f;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
            const float c = __builtin_amdgcn_fmed3f(q[4 * h + k], -z, 15.0f - z);
            v = k == 3 ? c : __builtin_fmaf(v, 16.0f, c);
        }
        half[h] = __builtin_fmaf(z, 4369.0f, v);
    }
    uint32_t code = static_cast<uint32_t>(half[0]) | static_cast<uint32_t>(half[1]) << 16;
    if (nan) {
        s = __uint_as_float(0x7FC00000u);
        z = 8.0f;
        code = 0x88888888u;
    }
    if (!on) return;
    if (4 * static_cast<int64_t>(u) < a.ld) reinterpret_cast<uint32_t*>(a.codes + row * a.ld)[u] = code;
    if ((u & (lanes - 1)) == 0) {
        const int64_t at = row * a.sld + u / lanes;
        if (SF32) static_cast<float*>(a.scales)[at] = s;
        else static_cast<uint16_t*>(a.scales)[at] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
        if (ASYM) a.zeros[at] = static_cast<uint8_t>(z);
        // the places past the last group, to whole fours: scale 1, zero 8
        if (u + lanes == a.units) {
            for (int64_t e = at + 1; e < (row + 1) * a.sld; ++e) {
                if (SF32) static_cast<float*>(a.scales)[e] = 1.0f;
                else static_cast<uint16_t*>(a.scales)[e] = 0x3F80;
                if (ASYM) a.zeros[e] = 8;
            }
        }
    }
}

__device__ __forceinline__ float scale_at(const void* s, int64_t i, int f32) {
    return f32 ? static_cast<const float*>(s)[i] : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(s)[i]) << 16);
}

template <bool F32>
__global__ void __launch_bounds__(256) dequant_int4_kernel(const QuantArgs a) {
    const uint32_t t = blockIdx.x * 256 + threadIdx.x;
    if (t >= a.count) return;
    const uint32_t r = div_units(a, t), u = t - r * a.units;
    const int64_t row = a.row0 + r;
    const int col = static_cast<int>(u) * kVec;
    const uint32_t code = reinterpret_cast<const uint32_t*>(a.codes + row * a.ld)[u];
    const int64_t at = row * a.sld + col / a.group;
    const float s = scale_at(a.scales, at, a.sf32);
    const float z = a.zeros ? static_cast<float>(a.zeros[at]) : 8.0f;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = (static_cast<float>((code >> (4 * k)) & 15) - z) * s;
    const int64_t to = row * a.cols + col;
    if (F32) {
        u32x4* const p = reinterpret_cast<u32x4*>(static_cast<float*>(a.y) + to);
        u32x4 lo, hi;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            lo[k] = __float_as_uint(v[k]);
            hi[k] = __float_as_uint(v[4 + k]);
        }
        __builtin_nontemporal_store(lo, p);
        __builtin_nontemporal_store(hi, p + 1);
    } else {
        u32x4 b;
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = bf16_pair(v[2 * k], v[2 * k + 1]);
        __builtin_nontemporal_store(b, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.y) + to));
    }
}

// ---------------------------------------------------------------------------
// The product.  Per group G of columns
//   sum over j in G of x[i][j] s (q - z) = s (sum of x (16 + q) - (16 + z) sum of x).
// 16 + q is a bf16 number that costs a shift, an and and an or for two codes
// (the code's four bits are the upper four of the seven behind the leading
// one), so the matrix cores take 16 + q, and the accumulator starts each
// group at -(16 + z) times the group's sum of x.  Sums are fp32; the 16 costs
// them less than three bits of a group's own sum, far below a bf16 result's
// rounding and about what a different order of an fp32 sum costs.
//
// x is the first operand of v_mfma_f32_16x16x32_bf16 (16 rows), 16 weight rows
// the second, so lane l holds codes, scale and zero of weight row l & 15, and
// the results of its column for x rows 4 (l >> 4) .. + 3.  A lane loads 16
// bytes, 32 consecutive columns of its row; the four quarters of a wavefront
// hold 128 columns, and a 4 x 4 transposition of words between the quarters
// (four lane swaps) makes word f of quarter q columns 32 f + 8 q .. + 7, so
// that one instruction sums over 32 consecutive columns, all of one group.
//
// fp32 x is three bf16 parts (upper eight bits, next eight, last eight),
// whose products are exact, added into the same accumulator.
//
// The weights' bytes bound the head's product (32 x 2560 x 151936: 43 us); three
// kernels share the formula, and launch_group has the figures that choose.
struct ProductArgs {
    const void* x;          // [n][k]
    const uint8_t* codes;   // [o][ld]
    const void* scales;     // [o][sld]
    const uint8_t* zeros;
    void* y;                // [n][o]
    int64_t n, o;
    int64_t ld, sld;
    int32_t k;
    int32_t chunks;         // of kChunk columns
    int32_t sf32, yf32;
    int64_t otiles;         // workgroups along the weight rows
    int64_t first;          // the launch's first x tile
};

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// Word i of quarter q becomes word q of quarter i.
__device__ __forceinline__ void transpose4(u32x4& w) {
    uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    swap32(a, c);
    swap32(b, d);
    swap16(a, b);
    swap16(c, d);
    w = u32x4{a, b, c, d};
}

// Eight codes as the bf16 numbers 16 + q, in the order 0 4 1 5 2 6 3 7: two
// instructions for two codes, with both constants in registers.
struct Widen {
    uint32_t mask = 0x00780078u, sixteen = 0x41804180u;
    __device__ __forceinline__ Widen() { asm("" : "+s"(mask), "+v"(sixteen)); }
    __device__ __forceinline__ bf16x8 operator()(uint32_t w) const {
        u32x4 r;
        r[0] = ((w << 3) & mask) | sixteen;
        r[1] = ((w >> 1) & mask) | sixteen;
        r[2] = ((w >> 5) & mask) | sixteen;
        r[3] = ((w >> 9) & mask) | sixteen;
        return __builtin_bit_cast(bf16x8, r);
    }
};

// Eight values of x, as 1 or 3 bf16 operands in the order 0 4 1 5 2 6 3 7.
template <bool F32>
__device__ __forceinline__ void parts_of(const Raw8<F32>& x, bf16x8* out) {
    u32x4 r;
    if (!F32) {
        r[0] = __builtin_amdgcn_perm(x.a[2], x.a[0], 0x05040100u);
        r[1] = __builtin_amdgcn_perm(x.a[2], x.a[0], 0x07060302u);
        r[2] = __builtin_amdgcn_perm(x.a[3], x.a[1], 0x05040100u);
        r[3] = __builtin_amdgcn_perm(x.a[3], x.a[1], 0x07060302u);
        out[0] = __builtin_bit_cast(bf16x8, r);
        return;
    }
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = x.at(k);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = __float_as_uint(v[k]), hi = __float_as_uint(v[4 + k]);
            r[k] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
            v[k] = v[k] - __uint_as_float(lo & 0xFFFF0000u);
            v[4 + k] = v[4 + k] - __uint_as_float(hi & 0xFFFF0000u);
        }
        out[p] = __builtin_bit_cast(bf16x8, r);
    }
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// What a lane holds of a chunk of its weight row: codes, and the scales and
// -(16 + zero) of the chunk's groups.  16 rows' addresses are one uniform base and
// a 32-bit distance.
struct WeightRows {
    const uint8_t* codes;
    const char* scales;
    const uint8_t* zeros;
    uint32_t row, srow;         // the lane's row from the base, in bytes and in scales
    uint32_t ld, quarter;
    int sf32;
    __device__ __forceinline__ WeightRows(const ProductArgs& a, int64_t tile, int lane) {
        const int64_t r0 = min(tile * 16, a.o - 1);
        const uint32_t r = static_cast<uint32_t>(min(tile * 16 + (lane & 15), a.o - 1) - r0);
        sf32 = a.sf32;
        codes = a.codes + r0 * a.ld;
        scales = static_cast<const char*>(a.scales) + r0 * a.sld * (sf32 ? 4 : 2);
        zeros = a.zeros ? a.zeros + r0 * a.sld : nullptr;
        ld = static_cast<uint32_t>(a.ld);
        row = r * ld;
        srow = r * static_cast<uint32_t>(a.sld);
        quarter = static_cast<uint32_t>(lane >> 4) * 16;
    }
};
template <int GROUP>
struct Weights {
    static constexpr int G = kChunk / GROUP;
    u32x4 w;
    u32x4 s;
    uint32_t z;
    __device__ __forceinline__ void load(const WeightRows& r, int chunk) {
        // past the row's last 16 bytes: any codes will do, x is 0 there
        w = *reinterpret_cast<const u32x4*>(r.codes + (r.row + min(static_cast<uint32_t>(chunk) * 64 + r.quarter, r.ld - 16)));
        const uint32_t g = r.srow + static_cast<uint32_t>(chunk) * G;
        if (r.sf32) {
            const char* const p = r.scales + g * 4;
            if (G == 4) s = *reinterpret_cast<const u32x4*>(p);
            else if (G == 2) { const u32x2 v = *reinterpret_cast<const u32x2*>(p); s[0] = v[0]; s[1] = v[1]; }
            else s[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            const char* const p = r.scales + g * 2;
            if (G == 4) { const u32x2 v = *reinterpret_cast<const u32x2*>(p); s[0] = v[0]; s[1] = v[1]; }
            else if (G == 2) s[0] = *reinterpret_cast<const uint32_t*>(p);
            else s[0] = *reinterpret_cast<const uint16_t*>(p);
        }
        z = 0x08080808u;
        if (r.zeros) {
            const uint8_t* const p = r.zeros + g;
            z = G == 4 ? *reinterpret_cast<const uint32_t*>(p) : G == 2 ? *reinterpret_cast<const uint16_t*>(p) : *p;
        }
    }
    __device__ __forceinline__ float scale(int i, int sf32) const {
        if (sf32) return __uint_as_float(s[i]);
        return __uint_as_float(i & 1 ? s[i >> 1] & 0xFFFF0000u : s[i >> 1] << 16);
    }
    __device__ __forceinline__ float start(int i) const { return -16.0f - static_cast<float>((z >> (8 * i)) & 255); }
};

__device__ __forceinline__ void store_y(const ProductArgs& a, int64_t row, int64_t col, float v) {
    if (row >= a.n || col >= a.o) return;
    if (a.yf32) static_cast<float*>(a.y)[row * a.o + col] = v;
    else static_cast<uint16_t*>(a.y)[row * a.o + col] = static_cast<uint16_t>(bf16_pair(v, v));
}

constexpr int kSplitWaves = 8;

// Few weight rows: a workgroup has 16 of them, its wavefronts share the
// columns and join their sums in LDS in a fixed order.  100 x 2560 x 4096 bf16: 22
// us, four passes of widening for 64 rows of x each and x read from L2 by every
// workgroup.
template <int MT, int GROUP, bool F32>
__global__ void __launch_bounds__(64 * kSplitWaves) project_int4_split_kernel(const ProductArgs a) {
    constexpr int G = kChunk / GROUP, PARTS = F32 ? 3 : 1, F = GROUP / 32;
    __shared__ f32x4 part[kSplitWaves][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, quarter = lane >> 4;
    const int64_t mtile = a.first + blockIdx.x / a.otiles, otile = blockIdx.x % a.otiles;
    const int64_t wrow = otile * 16 + lr;
    const WeightRows rows(a, otile, lane);
    const Widen widen4;
    const int64_t m0 = mtile * 16 * MT;
    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = static_cast<__bf16>(1.0f);
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = wave; c < a.chunks; c += kSplitWaves) {
        Weights<GROUP> w;
        w.load(rows, c);
        Raw8<F32> x[MT][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int64_t m = m0 + 16 * t + lr;
                const int col = c * kChunk + 32 * f + 8 * quarter;
                if (m < a.n && col < a.k) x[t][f].load(a.x, m * a.k + col); else x[t][f].zero();
            }
        }
        transpose4(w.w);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            bf16x8 b[F];
#pragma unroll
            for (int f = 0; f < F; ++f) b[f] = widen4(w.w[g * F + f]);
            // past the last group there may be anything
            const float s = c * kChunk + g * GROUP < a.k ? w.scale(g, a.sf32) : 0.0f, z = w.start(g);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f}, d;
                bf16x8 p[F][PARTS];
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    parts_of<F32>(x[t][g * F + f], p[f]);
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) sum = mfma(p[f][q], ones, sum);
                }
                d = sum * z;
#pragma unroll
                for (int f = 0; f < F; ++f)
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) d = mfma(p[f][q], b[f], d);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(s, d[i], acc[t][i]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += kSplitWaves) {
        f32x4 v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < kSplitWaves; ++w) v += part[w][t][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) store_y(a, m0 + 16 * t + 4 * quarter + i, wrow, v[i]);
    }
}

// Few rows of x: they stay in registers.  The wavefronts of a workgroup share
// the columns, PER chunks each, and walk over tiles of 16 weight rows; a tile's
// sums are joined in LDS, in a fixed order, by MT of the wavefronts in turn.
//
// Each wavefront brings its own codes, scales and zeros into LDS, SLOTS - 1
// tiles ahead, so that its products wait for nothing but its own loads.  Through LDS
// because the matrix operand wants neighbouring lanes in different rows, and a load whose
// neighbouring lanes lie in different rows takes four times as long: here four
// lanes read the 64 bytes of a row.  A row's four parts lie rotated by half its
// number, so that reads have no bank conflicts.
//
// 32 x 2560 x 151936 bf16: 70 to 73 us, 3.2 TB/s; the chain of load, LDS read,
// widening, products and barrier of each 16 weight rows bounds it, on 10
// wavefronts a unit (x in registers and 12 KB of LDS a wavefront allow no more; 16 x 2560 x 151936 60 us, 4 x 1032 x 151936 29).
// Codes straight to registers instead 180 us, two tiles a turn 90.
template <int MT, int GROUP, bool F32, bool SF32, int PER>
struct RowsShape {
    static constexpr int G = kChunk / GROUP, PARTS = F32 ? 3 : 1, F = GROUP / 32;
    static constexpr int SLOTS = PER == 4 ? 2 : PER == 2 || MT * PARTS == 1 ? 3 : 4;       // of one chunk and 16 bf16 rows 3 let two workgroups fit
    static constexpr int SD = PER * G * (SF32 ? 4 : 2) < 4 ? 1 : PER * G * (SF32 ? 4 : 2) / 4;      // words of scales a row
    static constexpr int ZD = PER * G < 4 ? 1 : PER * G / 4;                                        // words of zeros a row
    static constexpr int SL = (16 * SD + 63) / 64, ZL = (16 * ZD + 63) / 64;                        // loads of them
    static constexpr int Slot = PER * 1024 + (SL + ZL) * 256;
    static constexpr int Part = MT * 1024;
    static constexpr int Simd = PER * MT * PARTS == 1 ? 6 : PER * MT * PARTS <= 3 ? 4 : 3;      // wavefronts a SIMD that registers allow
    static constexpr int bytes(int waves) { return waves * (SLOTS * Slot + 2 * Part); }
};

template <int MT, int GROUP, bool F32, bool SF32, int PER, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, (RowsShape<MT, GROUP, F32, SF32, PER>::Simd)) project_int4_rows_kernel(const ProductArgs a) {
    typedef RowsShape<MT, GROUP, F32, SF32, PER> S;
    constexpr int G = S::G, PARTS = S::PARTS, F = S::F, SLOTS = S::SLOTS;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int lr = lane & 15, quarter = lane >> 4;
    uint8_t* const mine = lds + wave * SLOTS * S::Slot;
    uint8_t* const part = lds + waves * SLOTS * S::Slot;            // [2][waves][MT][64 lanes][16]
    const int64_t m0 = a.first * 16 * MT;
    const Widen widen4;
    const int c0 = wave * PER;
    const uint32_t ld = static_cast<uint32_t>(a.ld), sld = static_cast<uint32_t>(a.sld);
    // this lane's place in its row of codes, for each chunk, and in the rows of scales and zeros
    uint32_t at[PER];
#pragma unroll
    for (int c = 0; c < PER; ++c)       // past the row's last 16 bytes: any codes will do, x is 0 there
        at[c] = min(static_cast<uint32_t>(c0 + c) * 64 + 16 * ((lane & 3) ^ ((lane >> 3) & 3)), ld - 16);
    const auto load = [&](int64_t tile, int slot) {
        const int64_t r0 = min(tile, a.otiles - 1) * 16;
        const uint32_t last = static_cast<uint32_t>(min(a.o - 1 - r0, INT64_C(15)));
        uint8_t* const to = mine + slot * S::Slot;
        const uint8_t* const codes = a.codes + r0 * a.ld;
        const uint32_t row = min(static_cast<uint32_t>(lane >> 2), last) * ld;
#pragma unroll
        for (int h = 0; h < S::SL; ++h) {
            const uint32_t i = h * 64 + lane, r = min(i / S::SD, last), words = sld * (SF32 ? 4 : 2) / 4;
            const uint32_t w = min(static_cast<uint32_t>(c0) * G * (SF32 ? 4 : 2) / 4 + i % S::SD, words - 1);
            const char* const s = static_cast<const char*>(a.scales) + r0 * a.sld * (SF32 ? 4 : 2);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(s + (r * words + w) * 4),
                                             (__attribute__((address_space(3))) void*)(to + PER * 1024 + h * 256), 4, 0, 0);
        }
        if (a.zeros) {
#pragma unroll
            for (int h = 0; h < S::ZL; ++h) {
                const uint32_t i = h * 64 + lane, r = min(i / S::ZD, last);
                const uint32_t w = min(static_cast<uint32_t>(c0) * G / 4 + i % S::ZD, sld / 4 - 1);
                const uint8_t* const s = a.zeros + r0 * a.sld;
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(s + r * sld + w * 4),
                                                 (__attribute__((address_space(3))) void*)(to + PER * 1024 + (S::SL + h) * 256), 4, 0, 0);
            }
        }
#pragma unroll
        for (int c = 0; c < PER; ++c)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(codes + (row + at[c])),
                                             (__attribute__((address_space(3))) void*)(to + c * 1024), 16, 0, 0);
    };
    bf16x8 x[PER][MT][4][PARTS];
    f32x4 sx[PER][G][MT];
    {
        Raw8<F32> raw[PER][MT][4];
#pragma unroll
        for (int c = 0; c < PER; ++c)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int64_t m = m0 + 16 * t + lr;
                    const int col = (c0 + c) * kChunk + 32 * f + 8 * quarter;
                    if (m < a.n && col < a.k) raw[c][t][f].load(a.x, m * a.k + col); else raw[c][t][f].zero();
                }
        bf16x8 ones;
#pragma unroll
        for (int i = 0; i < 8; ++i) ones[i] = static_cast<__bf16>(1.0f);
#pragma unroll
        for (int c = 0; c < PER; ++c)
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        parts_of<F32>(raw[c][t][g * F + f], x[c][t][g * F + f]);
#pragma unroll
                        for (int q = 0; q < PARTS; ++q) s = mfma(x[c][t][g * F + f][q], ones, s);
                    }
                    sx[c][g][t] = s;
                }
    }
    const int64_t step = static_cast<int64_t>(gridDim.x);
    int64_t tile = blockIdx.x;
#pragma unroll
    for (int h = 0; h < SLOTS - 1; ++h)
        if (tile + h * step < a.otiles) load(tile + h * step, h);
    int slot = 0, turn = 0;
    for (; tile < a.otiles; tile += step, ++turn) {
        f32x4 acc[MT];
        {
            // into the slot whose reads ended with the last tile's products; loads of zeros may be missing from the count
            if (tile + (SLOTS - 1) * step < a.otiles) {
                load(tile + (SLOTS - 1) * step, (slot + SLOTS - 1) % SLOTS);
                __asm__ volatile("s_waitcnt vmcnt(%0)" ::"i"((SLOTS - 1) * (PER + S::SL)) : "memory");
            } else {
                __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
            }
            const uint8_t* const from = mine + slot * S::Slot;
            // this lane's scales and zeros; one alone in its word is moved to the word's start
            constexpr int SB = PER * G * (SF32 ? 4 : 2), ZB = PER * G;
            uint32_t sw[S::SD], zw[S::ZD];
#pragma unroll
            for (int i = 0; i < S::SD; ++i) sw[i] = reinterpret_cast<const uint32_t*>(from + PER * 1024 + lr * S::SD * 4)[i];
#pragma unroll
            for (int i = 0; i < S::ZD; ++i)
                zw[i] = a.zeros ? reinterpret_cast<const uint32_t*>(from + PER * 1024 + S::SL * 256 + lr * S::ZD * 4)[i] : 0x08080808u;
            if (SB < 4) sw[0] >>= 8 * ((c0 * G * (SF32 ? 4 : 2)) & 3);
            if (ZB < 4) zw[0] >>= 8 * ((c0 * G) & 3);
#pragma unroll
            for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < PER; ++c) {
                u32x4 w = *reinterpret_cast<const u32x4*>(from + c * 1024 + lr * 64 + 16 * (quarter ^ ((lr >> 1) & 3)));
                transpose4(w);
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int i = c * G + g;
                    const float sv = __uint_as_float(SF32 ? sw[SF32 ? i : 0] : i & 1 ? sw[i >> 1] & 0xFFFF0000u : sw[i >> 1] << 16);
                    const float z = -16.0f - static_cast<float>((zw[i >> 2] >> (8 * (i & 3))) & 255);
                    bf16x8 b[F];
#pragma unroll
                    for (int f = 0; f < F; ++f) b[f] = widen4(w[g * F + f]);
                    // past the last group there may be anything
                    const float s = (c0 + c) * kChunk + g * GROUP < a.k ? sv : 0.0f;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        f32x4 d = sx[c][g][t] * z;
#pragma unroll
                        for (int f = 0; f < F; ++f)
#pragma unroll
                            for (int q = 0; q < PARTS; ++q) d = mfma(x[c][t][g * F + f][q], b[f], d);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[t][e] = __builtin_fmaf(s, d[e], acc[t][e]);
                    }
                }
            }
            slot = slot + 1 == SLOTS ? 0 : slot + 1;
        }
        f32x4* const sum = reinterpret_cast<f32x4*>(part + (turn & 1) * waves * S::Part);
#pragma unroll
        for (int t = 0; t < MT; ++t) sum[(wave * MT + t) * 64 + lane] = acc[t];
        __syncthreads();
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            if ((turn * MT + t) % waves != wave) continue;
            f32x4 v = sum[t * 64 + lane];
            for (int i = 1; i < waves; ++i) v += sum[(i * MT + t) * 64 + lane];
#pragma unroll
            for (int e = 0; e < 4; ++e) store_y(a, m0 + 16 * t + 4 * quarter + e, tile * 16 + lr, v[e]);
        }
    }
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");            // loads into LDS end before the workgroup does
}

constexpr int kTileWaves = 8;

// Many weight rows and more rows of x than registers hold: a workgroup has 128
// weight rows, 16 a wavefront, and walks the columns KS chunks at a time; x
// goes through LDS in operand order, with its sums over groups, one step ahead,
// and the weights' loads are a step ahead too.  100 x 2560 x 32768 bf16: 49 us, bound
// by loads whose neighbouring lanes lie in different rows; more
// loads ahead gained nothing.
template <int MT, int GROUP, bool F32, int KS>
__global__ void __launch_bounds__(64 * kTileWaves) project_int4_tile_kernel(const ProductArgs a) {
    constexpr int G = kChunk / GROUP, PARTS = F32 ? 3 : 1, F = GROUP / 32;
    constexpr int PAIRS = KS * G * MT, PER = (PAIRS + kTileWaves - 1) / kTileWaves;     // groups of 16 rows of x: (group in the step, rows)
    __shared__ bf16x8 xs[2][PAIRS][F][PARTS][64];
    __shared__ f32x4 sums[2][PAIRS][4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, quarter = lane >> 4;
    const int64_t mtile = a.first + blockIdx.x / a.otiles, otile = (blockIdx.x % a.otiles) * kTileWaves + wave;
    const WeightRows rows(a, otile, lane);
    const Widen widen4;
    const int64_t m0 = mtile * 16 * MT;
    const int steps = (a.chunks + KS - 1) / KS;
    Raw8<F32> x[PER][F];
    const auto fetch = [&](int step) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int pair = wave + j * kTileWaves;
            const int64_t m = m0 + 16 * (pair % MT) + lr;
#pragma unroll
            for (int f = 0; f < F; ++f) {
                const int col = step * KS * kChunk + (pair / MT) * GROUP + 32 * f + 8 * quarter;
                if (pair < PAIRS && m < a.n && col < a.k) x[j][f].load(a.x, m * a.k + col); else x[j][f].zero();
            }
        }
    };
    const auto put = [&](int buf) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int pair = wave + j * kTileWaves;
            if (pair >= PAIRS) break;
            float s = 0.0f;
#pragma unroll
            for (int f = 0; f < F; ++f) {
                bf16x8 p[PARTS];
                parts_of<F32>(x[j][f], p);
#pragma unroll
                for (int q = 0; q < PARTS; ++q) xs[buf][pair][f][q][lane] = p[q];
                float v[8];
                x[j][f].get(v);
                s += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (quarter == 0) reinterpret_cast<float*>(&sums[buf][pair][0])[lr] = s;
        }
    };
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // loads come back in order: x, which is waited for first, is asked for before the weights
    Weights<GROUP> w[KS], next[KS];
    fetch(0);
#pragma unroll
    for (int c = 0; c < KS; ++c) next[c].load(rows, min(c, a.chunks - 1));
    put(0);
    __syncthreads();
    for (int step = 0; step < steps; ++step) {
#pragma unroll
        for (int c = 0; c < KS; ++c) w[c] = next[c];
        if (step + 1 < steps) {
            fetch(step + 1);
#pragma unroll
            for (int c = 0; c < KS; ++c) next[c].load(rows, min((step + 1) * KS + c, a.chunks - 1));
        }
        const int buf = step & 1;
#pragma unroll
        for (int c = 0; c < KS; ++c) {
            transpose4(w[c].w);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                bf16x8 b[F];
#pragma unroll
                for (int f = 0; f < F; ++f) b[f] = widen4(w[c].w[g * F + f]);
                // past the last group there may be anything
                const float s = (step * KS + c) * kChunk + g * GROUP < a.k ? w[c].scale(g, a.sf32) : 0.0f, z = w[c].start(g);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    const int pair = (c * G + g) * MT + t;
                    f32x4 d = sums[buf][pair][quarter] * z;
#pragma unroll
                    for (int f = 0; f < F; ++f)
#pragma unroll
                        for (int q = 0; q < PARTS; ++q) d = mfma(xs[buf][pair][f][q][lane], b[f], d);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(s, d[i], acc[t][i]);
                }
            }
        }
        if (step + 1 < steps) put(buf ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) store_y(a, m0 + 16 * t + 4 * quarter + i, otile * 16 + lr, acc[t][i]);
}

template <int MT, int GROUP, bool F32>
int launch_product(ProductArgs a, hipStream_t st) {
    const int64_t mtiles = (a.n + 16 * MT - 1) / (16 * MT), tiles = (a.o + 16 * kTileWaves - 1) / (16 * kTileWaves);
    // Tiles of 128 weight rows where there are enough of them (us, split and tile): 100 x 2560 x 4096 bf16 22 and 38,
    // x 8192 37 and 39, x 12288 52 and 40, x 16384 68 and 41, 200 x 2560 x 8192 69 and 39; fp32 20 x 2560 x 12288
    // 28 and 35, 40 x 2560 x 12288 50 and 37, 40 x 1032 x 12288 21 and 17.
    const bool split = tiles * mtiles < 192;
    const int threads = split ? 64 * kSplitWaves : 64 * kTileWaves;
    a.otiles = split ? (a.o + 15) / 16 : tiles;
    const int64_t most = most_groups(threads) / a.otiles;
    for (a.first = 0; a.first < mtiles; a.first += most) {
        const dim3 grid(static_cast<uint32_t>(std::min(most, mtiles - a.first) * a.otiles));
        if (split) hipLaunchKernelGGL((project_int4_split_kernel<MT, GROUP, F32>), grid, dim3(threads), 0, st, a);
        else hipLaunchKernelGGL((project_int4_tile_kernel<MT, GROUP, F32, MT * (F32 ? 2 : 1) >= 4 ? 1 : 2>), grid, dim3(threads), 0, st, a);
    }
    return hip_status("ngram_project_int4");
}

template <int MT, int GROUP, bool F32, bool SF32, int PER, int WAVES>
int launch_rows_of(ProductArgs a, hipStream_t st) {
    typedef RowsShape<MT, GROUP, F32, SF32, PER> S;
    const int waves = (a.chunks + PER - 1) / PER, lds = S::bytes(waves);
    if (lds > 160 * 1024) return 1;             // the caller takes another kernel
    const auto kernel = project_int4_rows_kernel<MT, GROUP, F32, SF32, PER, WAVES>;
    a.otiles = (a.o + 15) / 16;
    // workgroups a unit: two, whose barriers are not each other's, or 16 wavefronts (4 x 1032 x 151936 bf16 29 us, one
    // workgroup 43; 8 x 2048 x 40000 14.8 and 16.4; 8 x 1536 x 40000 13.0 and 15.4; but 4 x 512 x 151936 with 24 wavefronts
    // 19.1, with 16 15.1, with 12 16.3)
    const int fit = std::min(4 * S::Simd / waves, 160 * 1024 / lds);
    const int64_t at_once = 256 * std::max(1, std::min(fit, std::max(16 / waves, 2)));
    const dim3 grid(static_cast<uint32_t>(std::min(a.otiles, at_once))), block(64 * waves);
    for (a.first = 0; a.first * 16 * MT < a.n; ++a.first) hipLaunchKernelGGL(kernel, grid, block, lds, st, a);
    return hip_status("ngram_project_int4");
}
template <int MT, int GROUP, bool F32, int PER, int WAVES>
int launch_rows(const ProductArgs& a, hipStream_t st) {
    return a.sf32 ? launch_rows_of<MT, GROUP, F32, true, PER, WAVES>(a, st) : launch_rows_of<MT, GROUP, F32, false, PER, WAVES>(a, st);
}

template <int GROUP, bool F32>
int launch_group(const ProductArgs& a, hipStream_t st) {
    // x in registers where they hold it and, but for the last, where that is faster (us, so and without): bf16 1 x
    // 2560 x 2560 4.5 and 4.8, 16 x 2560 x 151936 60 and 102, 16 x 6144 x 5120 13 and 22, 32 x 1536 x 40000 18 and 26,
    // 48 x 2560 x 8192 19 and 20, 64 x 2560 x 16384 27 and 44; but 64 x 1032 x 4096 8.5 and 6.0, 40 x 2560 x 4096 14 and 10;
    // fp32 16 x 1536 x 40000 18 and 25, 11 x 1032 x 151936 48 and 51; two chunks a wavefront lose, 16 x 2560 x 151936
    // 130 and 113.
    int rc = 1;
    if (a.n <= 16) {
        if (a.chunks <= 12) rc = launch_rows<1, GROUP, F32, 1, 12>(a, st);
        else if (!F32 && a.chunks <= 24) rc = launch_rows<1, GROUP, false, 2, 12>(a, st);
        else if (!F32 && a.chunks <= 48) rc = launch_rows<1, GROUP, false, 4, 12>(a, st);
    } else if (!F32 && (a.n <= 32 || (a.n <= 64 && a.chunks > 12 && a.o >= 8192))) {
        if (a.chunks <= 12) rc = launch_rows<2, GROUP, false, 1, 12>(a, st);
        else if (a.chunks <= 24) rc = launch_rows<2, GROUP, false, 2, 12>(a, st);
    }
    if (rc != 1) return rc;
    if (a.n <= 16) return launch_product<1, GROUP, F32>(a, st);
    return F32 || a.n <= 32 ? launch_product<2, GROUP, F32>(a, st) : launch_product<F32 ? 2 : 4, GROUP, F32>(a, st);
}

// A launch for the rows from row0 on; fills magic and shift.
template <typename L>
int in_rows(QuantArgs a, int64_t rows, L launch, const char* what) {
    a.shift = 31 - __builtin_clz(a.units);
    a.magic = static_cast<uint32_t>(((UINT64_C(1) << (32 + a.shift)) + a.units - 1) / a.units);
    if (a.units > 1 && (a.units & (a.units - 1)) == 0) {    // 2^32 does not fit, its half with one shift less does
        a.magic = 0x80000000u;
        a.shift -= 1;
    }
    const int64_t most = INT64_C(0x7FFF0000) / a.units;
    for (int64_t r = 0; r < rows; r += most) {
        a.row0 = r;
        a.count = static_cast<uint32_t>(std::min(most, rows - r) * a.units);
        launch(a, dim3((a.count + 255) / 256));
    }
    return hip_status(what);
}

}  // namespace
}  // namespace ng8

using namespace ng8;

extern "C" {

int64_t ngram_int4_code_bytes(int64_t rows, int64_t cols) { return shape_ok(rows, cols, 32) ? rows * int4_ld(cols) : -1; }

int64_t ngram_int4_scales(int64_t rows, int64_t cols, int32_t group) { return shape_ok(rows, cols, group) ? rows * int4_sld(cols, group) : -1; }

int ngram_quant_int4(const void* x, int32_t x_dtype, int64_t n, int32_t d, const ngram_int4* q, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    const int rc = check_int4(q, "q");
    if (rc) return rc;
    if (x_dtype != NGRAM_F32 && x_dtype != NGRAM_BF16) return fail(NGRAM_EINVAL, "x_dtype=%d is not an ngram_value", x_dtype);
    if (q->rows != n || q->cols != d) return fail(NGRAM_EINVAL, "q is %lld x %lld, x %lld x %d", (long long)q->rows, (long long)q->cols, (long long)n, d);
    if (n == 0 || d == 0) return NGRAM_OK;
    if (!x) return fail(NGRAM_EINVAL, "x is NULL");
    if (!aligned(x, 16)) return fail(NGRAM_EALIGN, "x must be 16-byte aligned");
    QuantArgs a = {};
    a.x = x; a.codes = q->codes; a.scales = q->scales; a.zeros = q->zeros;
    a.ld = int4_ld(d); a.sld = int4_sld(d, q->group);
    a.units = static_cast<uint32_t>(int4_groups(d, q->group) * (q->group / kVec));
    a.cols = d; a.group = q->group; a.sf32 = q->scale_dtype == NGRAM_F32;
    const bool f32 = x_dtype == NGRAM_F32, asym = q->zeros != nullptr;
    const auto launch = [&](auto kernel) {
        return in_rows(a, n, [&](const QuantArgs& b, dim3 grid) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, b); }, "ngram_quant_int4");
    };
    if (f32) {
        if (asym) return a.sf32 ? launch(quant_int4_kernel<true, true, true>) : launch(quant_int4_kernel<true, true, false>);
        return a.sf32 ? launch(quant_int4_kernel<true, false, true>) : launch(quant_int4_kernel<true, false, false>);
    }
    if (asym) return a.sf32 ? launch(quant_int4_kernel<false, true, true>) : launch(quant_int4_kernel<false, true, false>);
    return a.sf32 ? launch(quant_int4_kernel<false, false, true>) : launch(quant_int4_kernel<false, false, false>);
}

int ngram_dequant_int4(const ngram_int4* q, void* y, int32_t y_dtype, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    const int rc = check_int4(q, "q");
    if (rc) return rc;
    if (y_dtype != NGRAM_F32 && y_dtype != NGRAM_BF16) return fail(NGRAM_EINVAL, "y_dtype=%d is not an ngram_value", y_dtype);
    if (q->rows == 0 || q->cols == 0) return NGRAM_OK;
    if (!y) return fail(NGRAM_EINVAL, "y is NULL");
    if (!aligned(y, 16)) return fail(NGRAM_EALIGN, "y must be 16-byte aligned");
    QuantArgs a = {};
    a.y = y; a.codes = q->codes; a.scales = q->scales; a.zeros = q->zeros;
    a.ld = int4_ld(q->cols); a.sld = int4_sld(q->cols, q->group);
    a.units = static_cast<uint32_t>(q->cols / kVec);
    a.cols = static_cast<int32_t>(q->cols); a.group = q->group; a.sf32 = q->scale_dtype == NGRAM_F32;
    return in_rows(a, q->rows, [&](const QuantArgs& b, dim3 grid) {
        if (y_dtype == NGRAM_F32) hipLaunchKernelGGL((dequant_int4_kernel<true>), grid, dim3(256), 0, stream, b);
        else hipLaunchKernelGGL((dequant_int4_kernel<false>), grid, dim3(256), 0, stream, b);
    }, "ngram_dequant_int4");
}

int ngram_project_int4(const void* x, int32_t x_dtype, int64_t n, const ngram_int4* W, void* y, int32_t y_dtype, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    const int rc = check_int4(W, "W");
    if (rc) return rc;
    if (x_dtype != NGRAM_F32 && x_dtype != NGRAM_BF16) return fail(NGRAM_EINVAL, "x_dtype=%d is not an ngram_value", x_dtype);
    if (y_dtype != NGRAM_F32 && y_dtype != NGRAM_BF16) return fail(NGRAM_EINVAL, "y_dtype=%d is not an ngram_value", y_dtype);
    if (n < 0) return fail(NGRAM_EINVAL, "n=%lld is negative", (long long)n);
    if (n > NGRAM_FP8_MAX) return fail(NGRAM_ERANGE, "n=%lld above %d", (long long)n, NGRAM_FP8_MAX);
    if (W->cols < 1) return fail(NGRAM_EINVAL, "W has no columns");
    if (n == 0 || W->rows == 0) return NGRAM_OK;
    if (!x || !y) return fail(NGRAM_EINVAL, "x or y is NULL");
    if (!aligned(x, 16) || !aligned(y, 16)) return fail(NGRAM_EALIGN, "x and y must be 16-byte aligned");
    ProductArgs a = {};
    a.x = x; a.codes = W->codes; a.scales = W->scales; a.zeros = W->zeros; a.y = y;
    a.n = n; a.o = W->rows; a.ld = int4_ld(W->cols); a.sld = int4_sld(W->cols, W->group);
    a.k = static_cast<int32_t>(W->cols); a.chunks = static_cast<int32_t>((W->cols + kChunk - 1) / kChunk);
    a.sf32 = W->scale_dtype == NGRAM_F32; a.yf32 = y_dtype == NGRAM_F32;
    if (x_dtype == NGRAM_F32) {
        if (W->group == 32) return launch_group<32, true>(a, stream);
        return W->group == 64 ? launch_group<64, true>(a, stream) : launch_group<128, true>(a, stream);
    }
    if (W->group == 32) return launch_group<32, false>(a, stream);
    return W->group == 64 ? launch_group<64, false>(a, stream) : launch_group<128, false>(a, stream);
}

}  // extern "C"
