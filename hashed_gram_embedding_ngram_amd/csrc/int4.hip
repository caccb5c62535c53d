// Weights in 4 bits with a scale (and a zero) for each group of columns, for
// MI355X (gfx950): ngram_quant_int4, ngram_dequant_int4 and the product
// ngram_project_int4.  The formats and formulas are in include/ngram.h.
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
// Bound by memory.
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

template <bool F32, bool ASYM>
__global__ void __launch_bounds__(256) quant_int4_kernel(const QuantArgs a) {
    const uint32_t t = blockIdx.x * 256 + threadIdx.x;
    const bool on = t < a.count;                            // whole groups are on or off
    const uint32_t r = on ? div_units(a, t) : 0, u = on ? t - r * a.units : 0;
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
    float s;
    if (ASYM) s = (-nhi - lo) / 15.0f;
    else s = fmaxf(-lo, -nhi) / 7.0f;
    if (!a.sf32) s = __uint_as_float(bf16_pair(s, s) << 16);
    // a group with a value that is not finite, or too wide for a finite scale, is NaN throughout
    const uint64_t odd = __ballot(!(bad == 0.0f));
    const int first = (threadIdx.x & 63) & ~(lanes - 1);
    const bool nan = ((odd >> first) & ((1u << lanes) - 1)) != 0 || !(s < __uint_as_float(kInfBits));
    if (s == 0.0f) s = 1.0f;
    float z = 8.0f;
    if (ASYM) z = fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f);
    uint32_t code = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float q = fminf(fmaxf(rintf(w[k] / s) + z, 0.0f), 15.0f);
        code |= static_cast<uint32_t>(q) << (4 * k);
    }
    if (nan) {
        s = __uint_as_float(0x7FC00000u);
        z = 8.0f;
        code = 0x88888888u;
    }
    if (!on) return;
    if (4 * static_cast<int64_t>(u) < a.ld) reinterpret_cast<uint32_t*>(a.codes + row * a.ld)[u] = code;
    if ((u & (lanes - 1)) == 0) {
        const int64_t at = row * a.sld + u / lanes;
        if (a.sf32) static_cast<float*>(a.scales)[at] = s;
        else static_cast<uint16_t*>(a.scales)[at] = static_cast<uint16_t>(__float_as_uint(s) >> 16);
        if (ASYM) a.zeros[at] = static_cast<uint8_t>(z);
        // the places past the last group, to whole fours: scale 1, zero 8
        if (u + lanes == a.units) {
            for (int64_t e = at + 1; e < (row + 1) * a.sld; ++e) {
                if (a.sf32) static_cast<float*>(a.scales)[e] = 1.0f;
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

// Eight codes as the bf16 numbers 16 + q, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ bf16x8 widen4(uint32_t w) {
    u32x4 r;
    r[0] = ((w << 3) & 0x00780078u) | 0x41804180u;
    r[1] = ((w >> 1) & 0x00780078u) | 0x41804180u;
    r[2] = ((w >> 5) & 0x00780078u) | 0x41804180u;
    r[3] = ((w >> 9) & 0x00780078u) | 0x41804180u;
    return __builtin_bit_cast(bf16x8, r);
}

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
// -(16 + zero) of the chunk's groups.
template <int GROUP>
struct Weights {
    static constexpr int G = kChunk / GROUP;
    u32x4 w;
    u32x4 s;
    uint32_t z;
    // `row` is clamped by the caller; `col` the lane's first of 32 columns
    __device__ __forceinline__ void load(const ProductArgs& a, int64_t row, int chunk, int quarter) {
        const int at = chunk * 64 + quarter * 16;
        if (at < a.ld) w = *reinterpret_cast<const u32x4*>(a.codes + row * a.ld + at); else w = u32x4{0, 0, 0, 0};
        const int64_t g = row * a.sld + chunk * G;
        if (a.sf32) {
            const float* const p = static_cast<const float*>(a.scales) + g;
            if (G == 4) s = *reinterpret_cast<const u32x4*>(p);
            else if (G == 2) { const u32x2 v = *reinterpret_cast<const u32x2*>(p); s[0] = v[0]; s[1] = v[1]; }
            else s[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            const uint16_t* const p = static_cast<const uint16_t*>(a.scales) + g;
            if (G == 4) { const u32x2 v = *reinterpret_cast<const u32x2*>(p); s[0] = v[0]; s[1] = v[1]; }
            else if (G == 2) s[0] = *reinterpret_cast<const uint32_t*>(p);
            else s[0] = *p;
        }
        z = 0x08080808u;
        if (a.zeros) {
            const uint8_t* const p = a.zeros + g;
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
// columns and join their sums in LDS in a fixed order.
template <int MT, int GROUP, bool F32>
__global__ void __launch_bounds__(64 * kSplitWaves) project_int4_split_kernel(const ProductArgs a) {
    constexpr int G = kChunk / GROUP, PARTS = F32 ? 3 : 1, F = GROUP / 32;
    __shared__ f32x4 part[kSplitWaves][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, quarter = lane >> 4;
    const int64_t mtile = a.first + blockIdx.x / a.otiles, otile = blockIdx.x % a.otiles;
    const int64_t wrow = otile * 16 + lr;
    const int64_t row = min(wrow, a.o - 1);
    const int64_t m0 = mtile * 16 * MT;
    bf16x8 ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = static_cast<__bf16>(1.0f);
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = wave; c < a.chunks; c += kSplitWaves) {
        Weights<GROUP> w;
        w.load(a, row, c, quarter);
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

constexpr int kTileWaves = 8;

// Many weight rows: a workgroup has 128 of them, 16 a wavefront, and walks
// the columns; x goes through LDS in operand order, with its sums over
// 32 columns, one chunk ahead.
template <int MT, int GROUP, bool F32>
__global__ void __launch_bounds__(64 * kTileWaves) project_int4_tile_kernel(const ProductArgs a) {
    constexpr int G = kChunk / GROUP, PARTS = F32 ? 3 : 1, F = GROUP / 32, ITEMS = 4 * MT, PER = (ITEMS + kTileWaves - 1) / kTileWaves;
    __shared__ bf16x8 xs[2][ITEMS][PARTS][64];
    __shared__ float sums[2][ITEMS][16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15, quarter = lane >> 4;
    const int64_t mtile = a.first + blockIdx.x / a.otiles, otile = blockIdx.x % a.otiles;
    const int64_t wrow = (otile * kTileWaves + wave) * 16 + lr;
    const int64_t row = min(wrow, a.o - 1);
    const int64_t m0 = mtile * 16 * MT;
    Raw8<F32> x[PER];
    const auto fetch = [&](int c) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int item = wave + j * kTileWaves;
            const int64_t m = m0 + 16 * (item >> 2) + lr;
            const int col = c * kChunk + 32 * (item & 3) + 8 * quarter;
            if (item < ITEMS && m < a.n && col < a.k) x[j].load(a.x, m * a.k + col); else x[j].zero();
        }
    };
    const auto put = [&](int buf) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int item = wave + j * kTileWaves;
            if (item >= ITEMS) break;
            bf16x8 p[PARTS];
            parts_of<F32>(x[j], p);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) xs[buf][item][q][lane] = p[q];
            float v[8];
            x[j].get(v);
            float s = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (quarter == 0) sums[buf][item][lr] = s;
        }
    };
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Weights<GROUP> w, next;
    next.load(a, row, 0, quarter);
    fetch(0);
    put(0);
    __syncthreads();
    for (int c = 0; c < a.chunks; ++c) {
        w = next;
        if (c + 1 < a.chunks) {
            next.load(a, row, c + 1, quarter);
            fetch(c + 1);
        }
        const int buf = c & 1;
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
                f32x4 d = *reinterpret_cast<const f32x4*>(&sums[buf][4 * t + g * F][4 * quarter]);
#pragma unroll
                for (int f = 1; f < F; ++f) d += *reinterpret_cast<const f32x4*>(&sums[buf][4 * t + g * F + f][4 * quarter]);
                d *= z;
#pragma unroll
                for (int f = 0; f < F; ++f)
#pragma unroll
                    for (int q = 0; q < PARTS; ++q) d = mfma(xs[buf][4 * t + g * F + f][q][lane], b[f], d);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][i] = __builtin_fmaf(s, d[i], acc[t][i]);
            }
        }
        if (c + 1 < a.chunks) put(buf ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) store_y(a, m0 + 16 * t + 4 * quarter + i, wrow, acc[t][i]);
}

template <int MT, int GROUP, bool F32>
int launch_product(ProductArgs a, bool split, hipStream_t st) {
    const int threads = split ? 64 * kSplitWaves : 64 * kTileWaves;
    a.otiles = split ? (a.o + 15) / 16 : (a.o + 16 * kTileWaves - 1) / (16 * kTileWaves);
    const int64_t mtiles = (a.n + 16 * MT - 1) / (16 * MT), most = most_groups(threads) / a.otiles;
    for (a.first = 0; a.first < mtiles; a.first += most) {
        const dim3 grid(static_cast<uint32_t>(std::min(most, mtiles - a.first) * a.otiles));
        if (split) hipLaunchKernelGGL((project_int4_split_kernel<MT, GROUP, F32>), grid, dim3(threads), 0, st, a);
        else hipLaunchKernelGGL((project_int4_tile_kernel<MT, GROUP, F32>), grid, dim3(threads), 0, st, a);
    }
    return hip_status("ngram_project_int4");
}

template <int MT, bool F32>
int launch_group(const ProductArgs& a, int group, bool split, hipStream_t st) {
    if (group == 32) return launch_product<MT, 32, F32>(a, split, st);
    if (group == 64) return launch_product<MT, 64, F32>(a, split, st);
    return launch_product<MT, 128, F32>(a, split, st);
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
    const int64_t most = INT64_C(0x7FFFFF00) / a.units;
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
    return in_rows(a, n, [&](const QuantArgs& b, dim3 grid) {
        if (f32 && asym) hipLaunchKernelGGL((quant_int4_kernel<true, true>), grid, dim3(256), 0, stream, b);
        else if (f32) hipLaunchKernelGGL((quant_int4_kernel<true, false>), grid, dim3(256), 0, stream, b);
        else if (asym) hipLaunchKernelGGL((quant_int4_kernel<false, true>), grid, dim3(256), 0, stream, b);
        else hipLaunchKernelGGL((quant_int4_kernel<false, false>), grid, dim3(256), 0, stream, b);
    }, "ngram_quant_int4");
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
    const bool split = W->rows < 128 * 256;
    if (x_dtype == NGRAM_F32) return n <= 16 ? launch_group<1, true>(a, W->group, split, stream) : launch_group<2, true>(a, W->group, split, stream);
    if (n <= 16) return launch_group<1, false>(a, W->group, split, stream);
    if (n <= 32) return launch_group<2, false>(a, W->group, split, stream);
    return launch_group<4, false>(a, W->group, split, stream);
}

}  // extern "C"
