// Residual addition, root-mean-square norm and 8-bit quantisation for MI355X
// (gfx950): ngram_add_norm, ngram_add_norm_grad, ngram_quant_fp8 and the
// layout helpers of the 8-bit matrices.  The formulas are in
// include/ngram.h.  All of these are bound by HBM bandwidth.
#include "common8.h"

#include <algorithm>
#include <cmath>

namespace ng8 {

int fail(int status, const char* fmt, ...) {
    // ngram_last_error() returns the start of the calling thread's own
    // 512-byte message buffer, a plain char array: writing it from here keeps
    // one buffer for the whole library.
    char* const buffer = const_cast<char*>(ngram_last_error());
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buffer, 512, fmt, ap);
    va_end(ap);
    return status;
}

int hip_status(const char* what) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(NGRAM_EHIP, "%s: %s", what, hipGetErrorString(e));
    return NGRAM_OK;
}

int check_fp8(const ngram_fp8* q, const char* what) {
    if (!q) return fail(NGRAM_EINVAL, "%s is NULL", what);
    if (q->rows < 0 || q->cols < 0) return fail(NGRAM_EINVAL, "%s has a negative size", what);
    if (q->rows > NGRAM_FP8_MAX || q->cols > NGRAM_FP8_MAX)
        return fail(NGRAM_ERANGE, "%s: rows=%lld or cols=%lld above %lld", what, (long long)q->rows, (long long)q->cols,
                    (long long)NGRAM_FP8_MAX);
    if (q->block_rows != 1 && q->block_rows != kBlock)
        return fail(NGRAM_EINVAL, "%s: block_rows=%d must be 1 or %d", what, q->block_rows, kBlock);
    if (q->rows > 0 && q->cols > 0) {
        if (!q->codes || !q->scales) return fail(NGRAM_EINVAL, "%s: codes or scales is NULL", what);
        if (!aligned(q->codes, 16) || !aligned(q->scales, 4))
            return fail(NGRAM_EALIGN, "%s: codes must be 16-byte and scales 4-byte aligned", what);
    }
    return NGRAM_OK;
}

namespace {

// ---------------------------------------------------------------------------
// Residual addition and norm.
//
// A row of d columns is cut in chunks of 512: lane l of a wavefront holds
// columns 512 c + 8 l .. +7 of its chunks, so every load and store of a
// chunk is one 16-byte (bf16) or 8-byte (codes) access per lane over
// consecutive addresses, and a scale block of 128 columns is one group of 16
// lanes.  A wavefront takes one row of C chunks, every load of it issued
// before the first is used; with WIDE, the wavefronts of a workgroup share a
// row (wavefront w has chunks w C .. w C + C - 1) and join the sums of squares
// in LDS.
//
// Bound by memory: 32768 x 2560 from bf16 (7 bytes an element with the 8-bit
// output) 102 us, 5.8 TB/s, where a large copy reaches 5.5; 5003 x 1032 from
// fp32 with everything kept 10.9 us, 5.2 TB/s; 4 x 2560 2.7 us, which is an
// empty launch and one dependent load.
struct NormArgs {
    const void* x;
    const uint16_t* residual;
    const float* gamma;
    uint16_t* sum_out;
    uint16_t* y_out;
    uint8_t* codes;
    uint8_t* scales;
    float* r_out;
    int64_t n;
    int32_t d;
    int32_t ld;         // code columns
    int32_t sld;        // scale bytes per row
    float eps;
    float inv_d;
};

constexpr int kMaxWaves = 16;

// A store past the caches' usual keeping, or a plain one.  The sum and y are
// next read much later, and stream: us with and without, 32768 x 2560 101 /
// 106, 2048 x 8192 23.9 / 25.2, 1024 x 2560 5.4 / 5.9, 512 x 1032 3.5 / 3.2
// (rows shared by wavefronts stream from 2^20 elements on, whole rows, 2048
// and more, always).  The codes are read by the very next product and do not:
// streaming them too saves this kernel 1% (2048 x 8192 13%) and costs that
// product more (norm and product of 1024 x 2560 25.0 against 22.1 us, of 8192
// x 2560 100.1 / 96.4, of 32768 x 2560 297 / 295).
template <bool STREAM, typename V, typename P>
__device__ __forceinline__ void put(P* to, V v) {
    if (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<V*>(to));
    else *reinterpret_cast<V*>(to) = v;
}

template <int C, bool F32, bool WIDE, bool STREAM>
__global__ void __launch_bounds__(WIDE ? 64 * kMaxWaves : 256) add_norm_kernel(const NormArgs a) {
    __shared__ float part[kMaxWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int c0 = WIDE ? wave * C : 0;
    const int64_t row = WIDE ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * waves + wave;
    if (row >= a.n) return;
    Raw8<true> gam[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c0 + c) * kSlice + lane * kVec;
        if (col < a.d) gam[c].load(a.gamma, col); else gam[c].zero();
    }
    Raw8<F32> x[C];
    Raw8<false> res[C];
    const int64_t at = row * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c0 + c) * kSlice + lane * kVec;
        if (col < a.d) {
            x[c].load(a.x, at + col);
            if (a.residual) res[c].load(a.residual, at + col); else res[c].zero();
        } else {
            x[c].zero();
            res[c].zero();
        }
    }
    float s[C][8];
    float total = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c0 + c) * kSlice + lane * kVec;
        float u[8], v[8];
        x[c].get(u);
        res[c].get(v);
        u32x4 packed;
#pragma unroll
        for (int k = 0; k < 4; ++k) packed[k] = bf16_pair(u[2 * k] + v[2 * k], u[2 * k + 1] + v[2 * k + 1]);
        // the norm reads the rounded sum, so that the backward, which has
        // only the stored sum, differentiates what was computed
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s[c][2 * k] = bf16_lo(packed[k]);
            s[c][2 * k + 1] = bf16_hi(packed[k]);
        }
        if (a.sum_out && col < a.d) put<STREAM>(a.sum_out + at + col, packed);
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t = fmaf(s[c][k], s[c][k], t);
        total += t;
    }
    total = wave_sum(total);
    if (WIDE) {
        if (lane == 0) part[wave] = total;
        __syncthreads();
        total = 0.0f;
        for (int w = 0; w < waves; ++w) total += part[w];
    }
    const float r = 1.0f / sqrtf(total * a.inv_d + a.eps);
    if (a.r_out && lane == 0 && wave == (WIDE ? 0 : wave)) a.r_out[row] = r;
    uint32_t bytes = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c0 + c) * kSlice + lane * kVec;
        float y[8], gv[8];
        gam[c].get(gv);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = s[c][k] * r * gv[k];
        if (a.y_out && col < a.d) {
            u32x4 packed;
#pragma unroll
            for (int k = 0; k < 4; ++k) packed[k] = bf16_pair(y[2 * k], y[2 * k + 1]);
            put<STREAM>(a.y_out + at + col, packed);
        }
        if (a.codes) {
            if (col >= a.d) {       // past the row: zero codes, also where r is not finite
#pragma unroll
                for (int k = 0; k < 8; ++k) y[k] = 0.0f;
            }
            const uint32_t byte = block_scale16(y);
            const float inv = inverse_scale(byte);
            if (col < a.ld) {
                u32x2 q;
                q[0] = codes4(y[0], y[1], y[2], y[3], inv);
                q[1] = codes4(y[4], y[5], y[6], y[7], inv);
                put<false>(a.codes + row * a.ld + col, q);
            }
            const uint32_t b0 = __builtin_amdgcn_readlane(byte, 0), b1 = __builtin_amdgcn_readlane(byte, 16);
            const uint32_t b2 = __builtin_amdgcn_readlane(byte, 32), b3 = __builtin_amdgcn_readlane(byte, 48);
            const uint32_t word = b0 | b1 << 8 | b2 << 16 | b3 << 24;
            bytes = lane == c ? word : bytes;
        }
    }
    // chunk c's four scale bytes sit in lane c
    if (a.codes && lane < C && (c0 + lane) * 4 < a.sld)
        *reinterpret_cast<uint32_t*>(a.scales + row * a.sld + (c0 + lane) * 4) = bytes;
}

// ---------------------------------------------------------------------------
// Gradients of the norm: with h = gamma dy,
//   dx = r h - s (r^3 / d) sum(h s) + dsum,   dgamma = sum over rows of dy s r.
// A workgroup walks over rows, its wavefronts sharing each as in the wide
// forward (SLOTS: several narrow rows at once); a lane adds its columns' dgamma terms in registers, and one row of
// partial sums per workgroup goes to the workspace for the kernel below.
//
// Bound by memory, 8 bytes an element: 32768 x 2560 in bf16 112 us, 6.0 TB/s
// (5.8 with the column sums).
struct NormGradArgs {
    const void* dy;
    const uint16_t* sum;
    const float* r;
    const float* gamma;
    const uint16_t* dsum;
    uint16_t* dx;
    float* partial;     // [workgroups][d]
    int64_t n;
    int32_t d;
    int32_t waves;      // of a row, where a workgroup takes several at once
    float inv_d;
};

template <int C, bool F32, bool SLOTS>
__global__ void __launch_bounds__(64 * kMaxWaves) add_norm_grad_kernel(const NormGradArgs a) {
    static_assert(C == 1 || !SLOTS, "narrow rows have one chunk a wavefront");
    __shared__ float part[2][kMaxWaves];
    __shared__ __attribute__((aligned(16))) float joined[SLOTS ? kMaxWaves : 1][SLOTS ? kSlice : 4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = SLOTS ? a.waves : blockDim.x >> 6;
    const int slots = SLOTS ? (blockDim.x >> 6) / waves : 1, slot = SLOTS ? wave / waves : 0;
    const int first = slot * waves;     // the row's first wavefront
    const int c0 = (wave - first) * C;
    float gam[C][8], acc[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c0 + c) * kSlice + lane * kVec;
        Raw8<true> g;
        if (col < a.d) g.load(a.gamma, col); else g.zero();
        g.get(gam[c]);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[c][k] = 0.0f;
    }
    int it = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * slots; base < a.n; base += static_cast<int64_t>(gridDim.x) * slots, ++it) {
        const int64_t row = base + slot;
        const bool live = !SLOTS || row < a.n;
        Raw8<F32> dy[C];
        Raw8<false> s[C], ds[C];
        const int64_t at = row * a.d;
        const float r = live ? a.r[row] : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c0 + c) * kSlice + lane * kVec;
            if (live && col < a.d) {
                dy[c].load(a.dy, at + col);
                s[c].load(a.sum, at + col);
                if (a.dsum) ds[c].load(a.dsum, at + col); else ds[c].zero();
            } else {
                dy[c].zero();
                s[c].zero();
                ds[c].zero();
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float u[8], v[8];
            dy[c].get(u);
            s[c].get(v);
            float t = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                t = fmaf(u[k] * gam[c][k], v[k], t);
                acc[c][k] = fmaf(u[k], v[k] * r, acc[c][k]);
            }
            dot += t;
        }
        dot = wave_sum(dot);
        // two buffers in turn: a wavefront writes one while a slower one
        // still reads the other, so one barrier a row is enough
        float* const p = part[it & 1];
        if (lane == 0) p[wave] = dot;
        __syncthreads();
        dot = 0.0f;
        for (int w = 0; w < waves; ++w) dot += p[first + w];
        const float f = dot * r * r * r * a.inv_d;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c0 + c) * kSlice + lane * kVec;
            float u[8], v[8], w[8];
            dy[c].get(u);
            s[c].get(v);
            ds[c].get(w);
            u32x4 packed;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float o[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int j = 2 * k + q;
                    o[q] = (u[j] * gam[c][j] * r - v[j] * f) + w[j];
                }
                packed[k] = bf16_pair(o[0], o[1]);
            }
            if (live && col < a.d) put<true>(a.dx + at + col, packed);
        }
    }
    if constexpr (SLOTS) {              // the rows' sums, in the order of the slots
        float* const mine = joined[wave] + lane * kVec;
        *reinterpret_cast<f32x4*>(mine) = f32x4{acc[0][0], acc[0][1], acc[0][2], acc[0][3]};
        *reinterpret_cast<f32x4*>(mine + 4) = f32x4{acc[0][4], acc[0][5], acc[0][6], acc[0][7]};
        __syncthreads();
        if (slot > 0) return;
        for (int s = 1; s < slots; ++s)
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[0][k] += joined[s * waves + wave][lane * kVec + k];
    }
    float* const out = a.partial + static_cast<int64_t>(blockIdx.x) * a.d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c0 + c) * kSlice + lane * kVec;
        if (col < a.d) {
            *reinterpret_cast<f32x4*>(out + col) = f32x4{acc[c][0], acc[c][1], acc[c][2], acc[c][3]};
            *reinterpret_cast<f32x4*>(out + col + 4) = f32x4{acc[c][4], acc[c][5], acc[c][6], acc[c][7]};
        }
    }
}

// dgamma[col] = the sum of `rows` <= 512 rows of partial sums.  64 columns per
// workgroup: thread t has columns 4 (t & 15) .. +3 of every 64th row, at most
// eight loads that are all in flight at once, and LDS joins the 64 sums, each
// in a fixed order.  4.7 us over 2560 columns of 512 rows, of which a launch is
// 2.5; with four rows at a time it was 7.
constexpr int kPartialRows = 512;

__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int rows, int d,
                                                          float* __restrict__ out) {
    __shared__ float part[64][64];
    const int t = threadIdx.x, group = t >> 4, c4 = 4 * (t & 15);
    const int col = blockIdx.x * 64 + c4;
    f32x4 v[kPartialRows / 64];
#pragma unroll
    for (int i = 0; i < kPartialRows / 64; ++i) {
        const int r = group + 64 * i;
        v[i] = r < rows && col < d ? *reinterpret_cast<const f32x4*>(partial + static_cast<int64_t>(r) * d + col)
                                   : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    f32x4 s = v[0];
#pragma unroll
    for (int i = 1; i < kPartialRows / 64; ++i) s += v[i];
    *reinterpret_cast<f32x4*>(&part[group][c4]) = s;
    __syncthreads();
    // column t & 63: 16 threads add four sums each, then one adds the 16
    const int c = t & 63, w = t >> 6;
    const float q = (part[4 * w][c] + part[4 * w + 1][c]) + (part[4 * w + 2][c] + part[4 * w + 3][c]);
    __syncthreads();
    part[w][c] = q;
    __syncthreads();
    if (t < 64 && blockIdx.x * 64 + t < d) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += part[i][t];
        out[blockIdx.x * 64 + t] = sum;
    }
}

// Few rows, where launches are most of the time: dx and dgamma in one.  dgamma
// needs no result of dx's (r is given), so the first workgroups take 32
// columns each of all rows (thread t has columns 4 (t & 7) .. +3 of every
// 128th row, four rows in flight, and LDS joins the 128 sums in a fixed
// order), and the rest take rows once more, as many each as `waves` wavefronts
// to a row leave room for.  Bound by the launch and its chain of loads.  The second reading must find dy as it was, so a call whose dx
// replaces dy goes the other way.
constexpr int kFewGroups = 8 * kMaxWaves;       // row groups of a column workgroup

struct NormGradFewArgs {
    NormGradArgs g;     // without partial sums
    float* dgamma;
    int32_t column_groups;  // workgroups that take columns
    int32_t waves;          // of a row
};

template <bool F32>
__global__ void __launch_bounds__(64 * kMaxWaves) add_norm_grad_few_kernel(const NormGradFewArgs f) {
    __shared__ __attribute__((aligned(16))) float part[kFewGroups][32];
    const NormGradArgs& a = f.g;
    const int t = threadIdx.x, lane = t & 63;
    if (static_cast<int>(blockIdx.x) >= f.column_groups) {
        const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
        const int slots = kMaxWaves / f.waves, slot = wave / f.waves, col = (wave - slot * f.waves) * kSlice + lane * kVec;
        const int64_t row = static_cast<int64_t>(blockIdx.x - f.column_groups) * slots + slot;
        const bool live = slot < slots && row < a.n;
        const int64_t at = row * a.d + col;
        Raw8<F32> dy;
        Raw8<true> gam;
        Raw8<false> s, ds;
        dy.zero(); gam.zero(); s.zero(); ds.zero();
        const float r = live ? a.r[row] : 0.0f;
        if (live && col < a.d) {
            dy.load(a.dy, at);
            gam.load(a.gamma, col);
            s.load(a.sum, at);
            if (a.dsum) ds.load(a.dsum, at);
        }
        float u[8], v[8], w[8], h[8];
        dy.get(u);
        s.get(v);
        ds.get(w);
        gam.get(h);
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) dot = fmaf(u[k] * h[k], v[k], dot);
        dot = wave_sum(dot);
        if (lane == 0) part[0][wave] = dot;
        __syncthreads();
        if (!live) return;
        dot = 0.0f;
        for (int i = 0; i < f.waves; ++i) dot += part[0][slot * f.waves + i];
        const float scale = dot * r * r * r * a.inv_d;
        u32x4 packed;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            packed[k] = bf16_pair((u[2 * k] * h[2 * k] * r - v[2 * k] * scale) + w[2 * k],
                                  (u[2 * k + 1] * h[2 * k + 1] * r - v[2 * k + 1] * scale) + w[2 * k + 1]);
        if (col < a.d) put<false>(a.dx + at, packed);
        return;
    }
    const int first = blockIdx.x * 32, c4 = 4 * (t & 7), group = t >> 3, col = first + c4;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (col < a.d) {
        for (int64_t base = group; base < a.n; base += 4 * kFewGroups) {
            f32x4 u[4];
            u32x2 p[4] = {}, v[4];
            float r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t row = base + i * kFewGroups;
                const int64_t at = row * a.d + col;
                u[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                v[i] = u32x2{0, 0};
                r[i] = 0.0f;
                if (row < a.n) {
                    r[i] = a.r[row];
                    v[i] = *reinterpret_cast<const u32x2*>(a.sum + at);
                    if (F32) u[i] = *reinterpret_cast<const f32x4*>(static_cast<const float*>(a.dy) + at);
                    else p[i] = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(a.dy) + at);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!F32) u[i] = f32x4{bf16_lo(p[i][0]), bf16_hi(p[i][0]), bf16_lo(p[i][1]), bf16_hi(p[i][1])};
                acc[0] = fmaf(u[i][0], bf16_lo(v[i][0]) * r[i], acc[0]);
                acc[1] = fmaf(u[i][1], bf16_hi(v[i][0]) * r[i], acc[1]);
                acc[2] = fmaf(u[i][2], bf16_lo(v[i][1]) * r[i], acc[2]);
                acc[3] = fmaf(u[i][3], bf16_hi(v[i][1]) * r[i], acc[3]);
            }
        }
    }
    *reinterpret_cast<f32x4*>(&part[group][c4]) = acc;
    __syncthreads();
    // column t & 31: 32 threads add four sums each, then one adds the 32
    const int c = t & 31, w = t >> 5;
    const float q = (part[4 * w][c] + part[4 * w + 1][c]) + (part[4 * w + 2][c] + part[4 * w + 3][c]);
    __syncthreads();
    part[w][c] = q;
    __syncthreads();
    if (t < 32 && first + t < a.d) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += part[i][t];
        f.dgamma[first + t] = sum;
    }
}

// ---------------------------------------------------------------------------
// Quantisation of a matrix x[n][d]: codes and scales of its rows (a scale per
// 128 columns), of its transpose (a scale per 128 rows of x), or both from
// one read; with TILE one scale serves a 128 x 128 tile and both layouts.
//
// A workgroup owns a 128 x 128 tile.  Thread t holds the 8 x 8 patch of rows
// 8 (t >> 4) .. +7 and columns 8 (t & 15) .. +7: a row's 128 columns are a
// group of 16 lanes (row scales by lane moves), and the patch transposes in
// registers.  Column maxima go through LDS; so do the transposed codes, which
// then leave as whole 128-byte lines.
//
// Bound by memory, with the two barriers of a tile in the way: 8192 x 2560 in
// bf16, both outputs, 20.2 us, 4.2 TB/s (a large copy 5.5), the transposed one
// alone 14.4, the rows alone 12.3; among a layer's products 22 and 16.  128 x
// 128 tiles, both outputs: 2560 x 2560 in fp32 10.8 us, 3.6 TB/s (400 tiles for
// 256 compute units), 8192 x 8192 in bf16 55 us, 4.9 TB/s.  Streaming stores took
// 18.2 and 12.6 us where plain ones took 19.8 and 14.4, but the products that
// read the codes next took longer (a layer's two gradients 206 us against 199
// with the products of that time), so the stores are plain.
struct QuantArgs {
    const void* x;
    uint8_t *q, *qs, *qt, *qts;
    int64_t n;
    int32_t d;
    int64_t q_ld, q_sld, qt_ld, qt_sld;
    int32_t tiles_d;
    int32_t tile_scale;
};

template <bool F32>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(F32 ? 4 : 6))) quant_kernel(const QuantArgs a) {
    __shared__ u32x4 cmax[4][32];
    __shared__ __attribute__((aligned(16))) uint8_t codes[128 * 128];   // transposed
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int tr = t >> 4, tc = t & 15;
    const int64_t tile_r = blockIdx.x / a.tiles_d;
    const int tile_c = blockIdx.x - tile_r * a.tiles_d;
    const int64_t r0 = tile_r * 128 + 8 * tr;
    const int c0 = tile_c * 128 + 8 * tc;
    // kept as loaded and unpacked where used: fewer registers, more tiles in flight
    Raw8<F32> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (r0 + i < a.n && c0 < a.d) raw[i].load(a.x, (r0 + i) * a.d + c0); else raw[i].zero();
    }
    uint32_t tile_byte = 0;
    if (a.tile_scale) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x[8];
            raw[i].get(x);
            m = max(m, finite_amax_bits(x));
        }
        m = max16(m);
        m = max(max(__builtin_amdgcn_readlane(m, 0), __builtin_amdgcn_readlane(m, 16)),
                max(__builtin_amdgcn_readlane(m, 32), __builtin_amdgcn_readlane(m, 48)));
        if (lane == 0) cmax[wave][0][0] = m;
        __syncthreads();
        tile_byte = scale_byte(max(max(cmax[0][0][0], cmax[1][0][0]), max(cmax[2][0][0], cmax[3][0][0])));
    }
    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x[8];
            raw[i].get(x);
            const uint32_t byte = a.tile_scale ? tile_byte : block_scale16(x);
            const float inv = inverse_scale(byte);
            if (r0 + i < a.n) {
                u32x2 c;
                c[0] = codes4(x[0], x[1], x[2], x[3], inv);
                c[1] = codes4(x[4], x[5], x[6], x[7], inv);
                *reinterpret_cast<u32x2*>(a.q + (r0 + i) * a.q_ld + c0) = c;
                if (!a.tile_scale && tc == 0) a.qs[(r0 + i) * a.q_sld + tile_c] = static_cast<uint8_t>(byte);
                if (!a.tile_scale && tile_c == a.tiles_d - 1 && tc > 0 && tile_c + tc < a.q_sld)
                    a.qs[(r0 + i) * a.q_sld + tile_c + tc] = kUnitScale;
            }
        }
        if (a.tile_scale && t == 0) a.qs[tile_r * a.q_sld + tile_c] = static_cast<uint8_t>(tile_byte);
        if (a.tile_scale && tile_c == a.tiles_d - 1 && t > 0 && tile_c + t < a.q_sld)
            a.qs[tile_r * a.q_sld + tile_c + t] = kUnitScale;
    }
    if (!a.qt) return;
    uint32_t byte[8];
    if (a.tile_scale) {
#pragma unroll
        for (int k = 0; k < 8; ++k) byte[k] = tile_byte;
    } else {
        uint32_t m[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x[8];
            raw[i].get(x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t u = __float_as_uint(x[k]) & 0x7FFFFFFFu;
                m[k] = max(m[k], u < kInfBits ? u : 0u);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {       // over the wavefront's four groups of 16 lanes
            const auto p = __builtin_amdgcn_permlane16_swap(m[k], m[k], false, false);
            m[k] = max(p[0], p[1]);
            const auto q = __builtin_amdgcn_permlane32_swap(m[k], m[k], false, false);
            m[k] = max(q[0], q[1]);
        }
        if (lane < 16) {
            cmax[wave][2 * tc] = u32x4{m[0], m[1], m[2], m[3]};
            cmax[wave][2 * tc + 1] = u32x4{m[4], m[5], m[6], m[7]};
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 w0 = cmax[0][2 * tc + h], w1 = cmax[1][2 * tc + h], w2 = cmax[2][2 * tc + h], w3 = cmax[3][2 * tc + h];
#pragma unroll
            for (int k = 0; k < 4; ++k) byte[4 * h + k] = scale_byte(max(max(w0[k], w1[k]), max(w2[k], w3[k])));
        }
    }
    const int64_t last_r = (a.n - 1) / 128;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float inv = inverse_scale(byte[k]);
        u32x2 c;
        c[0] = codes4(raw[0].at(k), raw[1].at(k), raw[2].at(k), raw[3].at(k), inv);
        c[1] = codes4(raw[4].at(k), raw[5].at(k), raw[6].at(k), raw[7].at(k), inv);
        // column 8 tc + k, rows 8 tr .. +7: 8-byte unit tr ^ tc of LDS row
        // (8 tc + k) ^ (tc & 1), so that a store's 64 lanes spread over all banks
        *reinterpret_cast<u32x2*>(codes + ((8 * tc + k) ^ (tc & 1)) * 128 + 8 * (tr ^ tc)) = c;
        if (c0 + k < a.d && !a.tile_scale) {
            if (tr == 0) a.qts[static_cast<int64_t>(c0 + k) * a.qt_sld + tile_r] = static_cast<uint8_t>(byte[k]);
            if (tile_r == last_r && tr > 0 && tile_r + tr < a.qt_sld)
                a.qts[static_cast<int64_t>(c0 + k) * a.qt_sld + tile_r + tr] = kUnitScale;
        }
    }
    if (a.tile_scale) {
        if (t == 0) a.qts[tile_c * a.qt_sld + tile_r] = static_cast<uint8_t>(tile_byte);
        if (tile_r == last_r && t > 0 && tile_r + t < a.qt_sld) a.qts[tile_c * a.qt_sld + tile_r + t] = kUnitScale;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c = 32 * i + (t >> 3), part = t & 7;      // a column's 128 bytes by eight lanes
        const int64_t col = static_cast<int64_t>(tile_c) * 128 + c;
        const int from = c >> 3;                            // the column's tc
        const u32x4 v = *reinterpret_cast<const u32x4*>(codes + (c ^ (from & 1)) * 128 + 16 * (part ^ (from >> 1)));
        if (col < a.d)
            *reinterpret_cast<u32x4*>(a.qt + col * a.qt_ld + tile_r * 128 + 16 * part) = from & 1 ? u32x4{v[2], v[3], v[0], v[1]} : v;
    }
}

// ---------------------------------------------------------------------------
// Launch shapes.

// Forward.  Many rows of up to 5 chunks: a wavefront takes a whole row and
// needs no barrier (2560 columns, us, whole rows / shared rows: 4096 rows 13.9
// / 16.7, 2048 rows 8.5 / 10.2, 1024 rows 6.7 / 5.9, 256 rows 5.1 / 3.2; 1032
// columns: the same at 2048 rows, 12.2 / 13.9 at 8192).  Few rows and wide ones:
// one chunk per wavefront up to 16, so that a row's loads are spread over as
// many wavefronts as it has chunks (8192 x 8192: 84.1 against 86.4 with four,
// before streaming stores).
struct RowShape {
    int chunks;     // per wavefront
    int waves;      // per workgroup
    bool wide;
    int64_t grid;   // of the gradient, whose workgroups walk over the rows
};

RowShape row_shape(int64_t n, int d) {
    const int total = (d + kSlice - 1) / kSlice;
    RowShape s;
    s.wide = n < 2048 || total > 5;
    if (!s.wide) {
        s.chunks = total;
        s.waves = 4;
    } else {
        s.waves = std::min(kMaxWaves, total);
        s.chunks = (total + s.waves - 1) / s.waves;
        s.waves = (total + s.chunks - 1) / s.chunks;
    }
    return s;
}

// Gradient.  A row by a workgroup, one chunk per wavefront up to 16: when the
// shape was chosen, at 32768 x 2560 119 us with the column sums against 128
// with two chunks and 132 with a wavefront to a row (fewer registers, more
// wavefronts); 116 now.  512 workgroups walk over the rows (1024: 132 us then:
// more partial sums; 256: slower in every shape).
// One launch or two, us: 1 x 2560 2.5 / 4.4, 512 x 2560 5.9 / 10.0, 777 x 520
// (fp32) 5.5 / 7.6, 1024 x 2560 10.4 / 11.5, 512 x 8192 (fp32) 14.1 / 16.6; but
// 1024 x 8192 21.9 / 19.4, 1500 x 2560 13.7 / 12.7, 1500 x 520 8.7 / 9.0, 2048 x
// 136 9.3 / 8.0.
bool few_rows(int64_t n, int d) { return n <= 1024 && n * d <= 1 << 22; }


RowShape grad_shape(int64_t n, int d) {
    const int total = (d + kSlice - 1) / kSlice;
    RowShape s;
    s.wide = true;
    s.waves = std::min(kMaxWaves, total);
    s.chunks = (total + s.waves - 1) / s.waves;
    s.waves = (total + s.chunks - 1) / s.chunks;
    s.grid = std::max<int64_t>(1, std::min<int64_t>(n, kPartialRows));   // no rows: one workgroup writes a row of zeros
    return s;
}

// Rows that a workgroup of the gradient takes at once: narrow rows alone would
// leave too few wavefronts to the chip.  One row / several, us: 200,000 x 136
// 357 / 57, 32768 x 512 70 / 29, 32768 x 1024 81 / 51, 6024 x 120 14.9 / 7.9, 4000 x
// 1032 (fp32) 16.1 / 13.8 (two rows; five 15.9), 32768 x 2048 101 / 98, 8192 x
// 2048 (fp32) 34.0 / 35.1; at 2560 columns three rows take 128 us for one's 116.
int grad_slots(int64_t n, const RowShape& s) {
    const int most = s.waves <= 2 ? kMaxWaves / s.waves : s.waves <= 4 ? 2 : 1;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, (n + s.grid - 1) / s.grid)));
}

template <bool F32, bool WIDE, bool STREAM>
void launch_norm(int chunks, dim3 grid, dim3 block, hipStream_t st, const NormArgs& a) {
#define NG8_CASE(C) case C: hipLaunchKernelGGL((add_norm_kernel<C, F32, WIDE, STREAM>), grid, block, 0, st, a); break
    switch (chunks) { NG8_CASE(1); NG8_CASE(2); NG8_CASE(3); NG8_CASE(4); NG8_CASE(5); default:
        if constexpr (WIDE) switch (chunks) { NG8_CASE(6); NG8_CASE(7); default: NG8_CASE(8); } }
#undef NG8_CASE
}

template <bool F32>
void launch_norm_grad(int chunks, dim3 grid, dim3 block, hipStream_t st, const NormGradArgs& a) {
#define NG8_CASE(C) case C: hipLaunchKernelGGL((add_norm_grad_kernel<C, F32, false>), grid, block, 0, st, a); break
    if (static_cast<int>(block.x) > 64 * a.waves) hipLaunchKernelGGL((add_norm_grad_kernel<1, F32, true>), grid, block, 0, st, a);
    else switch (chunks) { NG8_CASE(1); NG8_CASE(2); NG8_CASE(3); NG8_CASE(4); NG8_CASE(5); NG8_CASE(6); NG8_CASE(7); default: NG8_CASE(8); }
#undef NG8_CASE
}

int check_rows(int64_t n, int32_t d) {
    if (n < 0) return fail(NGRAM_EINVAL, "n=%lld is negative", (long long)n);
    if (d <= 0 || d % kVec != 0) return fail(NGRAM_EINVAL, "d=%d must be a positive multiple of %d", d, kVec);
    if (d > NGRAM_MAX_D) return fail(NGRAM_ERANGE, "d=%d above %d", d, NGRAM_MAX_D);
    if (n > NGRAM_FP8_MAX) return fail(NGRAM_ERANGE, "n=%lld above %lld", (long long)n, (long long)NGRAM_FP8_MAX);
    return NGRAM_OK;
}

int check_value(int dtype, const char* what) {
    if (dtype != NGRAM_F32 && dtype != NGRAM_BF16) return fail(NGRAM_EINVAL, "%s=%d is not an ngram_value", what, dtype);
    return NGRAM_OK;
}


}  // namespace
}  // namespace ng8

using namespace ng8;

extern "C" {

int64_t ngram_fp8_code_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > NGRAM_FP8_MAX || cols > NGRAM_FP8_MAX) return -1;
    return rows * code_ld(cols);
}

int64_t ngram_fp8_scale_bytes(int64_t rows, int64_t cols, int32_t block_rows) {
    if (rows < 0 || cols < 0 || rows > NGRAM_FP8_MAX || cols > NGRAM_FP8_MAX) return -1;
    if (block_rows != 1 && block_rows != kBlock) return -1;
    return (block_rows == 1 ? rows : blocks_of(rows)) * scale_ld(cols);
}

int ngram_add_norm(const void* x, int32_t x_dtype, const uint16_t* residual, int64_t n, int32_t d, const float* gamma,
                   float eps, uint16_t* sum_out, uint16_t* y_out, const ngram_fp8* q_out, float* r_out,
                   ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    int rc = check_rows(n, d);
    if (rc) return rc;
    if ((rc = check_value(x_dtype, "x_dtype"))) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps)) return fail(NGRAM_EINVAL, "eps must be finite and not negative");
    if (q_out) {
        if ((rc = check_fp8(q_out, "q_out"))) return rc;
        if (q_out->rows != n || q_out->cols != d || q_out->block_rows != 1)
            return fail(NGRAM_EINVAL, "q_out must be %lld x %d with block_rows 1", (long long)n, d);
    }
    if (!gamma) return fail(NGRAM_EINVAL, "gamma is NULL");
    if (n == 0) return NGRAM_OK;
    if (!x) return fail(NGRAM_EINVAL, "x is NULL");
    if (!sum_out && !y_out && !q_out && !r_out) return fail(NGRAM_EINVAL, "no output is asked for");
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(sum_out, 16) || !aligned(y_out, 16))
        return fail(NGRAM_EALIGN, "x, residual, gamma, sum_out and y_out must be 16-byte aligned");
    if (!aligned(r_out, 4)) return fail(NGRAM_EALIGN, "r_out must be 4-byte aligned");
    NormArgs a;
    a.gamma = gamma; a.d = d;
    a.ld = static_cast<int32_t>(code_ld(d));
    a.sld = static_cast<int32_t>(scale_ld(d));
    a.eps = eps;
    a.inv_d = 1.0f / static_cast<float>(d);
    const RowShape s = row_shape(n, d);
    const dim3 block(64 * s.waves);
    const int per = s.wide ? 1 : s.waves;                       // rows of a workgroup
    const int64_t most = most_groups(64 * s.waves) * per;       // and of a launch
    const bool f32 = x_dtype == NGRAM_F32;
    for (int64_t row = 0; row < n; row += most) {
        a.n = std::min(most, n - row);
        a.x = static_cast<const uint8_t*>(x) + row * d * value_bytes(x_dtype);
        a.residual = residual ? residual + row * d : nullptr;
        a.sum_out = sum_out ? sum_out + row * d : nullptr;
        a.y_out = y_out ? y_out + row * d : nullptr;
        a.codes = q_out ? q_out->codes + row * a.ld : nullptr;
        a.scales = q_out ? q_out->scales + row * a.sld : nullptr;
        a.r_out = r_out ? r_out + row : nullptr;
        const dim3 grid(static_cast<unsigned>((a.n + per - 1) / per));
        if (!s.wide) {
            if (f32) launch_norm<true, false, true>(s.chunks, grid, block, stream, a);
            else launch_norm<false, false, true>(s.chunks, grid, block, stream, a);
        } else if (n * d >= 1 << 20) {      // see put()
            if (f32) launch_norm<true, true, true>(s.chunks, grid, block, stream, a);
            else launch_norm<false, true, true>(s.chunks, grid, block, stream, a);
        } else {
            if (f32) launch_norm<true, true, false>(s.chunks, grid, block, stream, a);
            else launch_norm<false, true, false>(s.chunks, grid, block, stream, a);
        }
        if ((rc = hip_status("ngram_add_norm launch"))) return rc;
    }
    return NGRAM_OK;
}

int64_t ngram_add_norm_grad_workspace_bytes(int64_t n, int32_t d) {
    if (n < 0 || n > NGRAM_FP8_MAX || d <= 0 || d % kVec != 0 || d > NGRAM_MAX_D) return -1;
    return grad_shape(n, d).grid * d * 4;
}

int ngram_add_norm_grad(const void* dy, int32_t dy_dtype, const uint16_t* sum, const float* r, const float* gamma,
                        const uint16_t* dsum, int64_t n, int32_t d, uint16_t* dx_out, float* dgamma_out,
                        void* workspace, int64_t workspace_bytes, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    int rc = check_rows(n, d);
    if (rc) return rc;
    if ((rc = check_value(dy_dtype, "dy_dtype"))) return rc;
    if (!gamma || !dgamma_out) return fail(NGRAM_EINVAL, "gamma or dgamma_out is NULL");
    if (n > 0 && (!dy || !sum || !r || !dx_out)) return fail(NGRAM_EINVAL, "dy, sum, r or dx_out is NULL");
    if (!aligned(dy, 16) || !aligned(sum, 16) || !aligned(gamma, 16) || !aligned(dsum, 16) || !aligned(dx_out, 16) ||
        !aligned(dgamma_out, 4) || !aligned(r, 4))
        return fail(NGRAM_EALIGN, "dy, sum, gamma, dsum and dx_out must be 16-byte aligned, r and dgamma_out 4-byte");
    const int64_t need = ngram_add_norm_grad_workspace_bytes(n, d);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return fail(NGRAM_EINVAL, "workspace must hold %lld bytes, 16-byte aligned", (long long)need);
    NormGradArgs a;
    a.waves = 0;
    a.dy = dy; a.sum = sum; a.r = r; a.gamma = gamma; a.dsum = dsum; a.dx = dx_out;
    a.partial = static_cast<float*>(workspace);
    a.n = n; a.d = d;
    a.inv_d = 1.0f / static_cast<float>(d);
    const RowShape s = grad_shape(n, d);
    if (few_rows(n, d) && s.chunks == 1 && dx_out != dy) {
        const int slots = kMaxWaves / s.waves;
        const NormGradFewArgs f{a, dgamma_out, (d + 31) / 32, s.waves};
        const dim3 few(static_cast<unsigned>(f.column_groups + (n + slots - 1) / slots)), threads(64 * kMaxWaves);
        if (dy_dtype == NGRAM_F32) hipLaunchKernelGGL((add_norm_grad_few_kernel<true>), few, threads, 0, stream, f);
        else hipLaunchKernelGGL((add_norm_grad_few_kernel<false>), few, threads, 0, stream, f);
        return hip_status("ngram_add_norm_grad launch");
    }
    const dim3 grid(static_cast<unsigned>(s.grid)), block(64 * s.waves * grad_slots(n, s));
    a.waves = s.waves;
    if (dy_dtype == NGRAM_F32) launch_norm_grad<true>(s.chunks, grid, block, stream, a);
    else launch_norm_grad<false>(s.chunks, grid, block, stream, a);
    hipLaunchKernelGGL(column_sum_kernel, dim3((d + 63) / 64), dim3(1024), 0, stream, a.partial,
                       static_cast<int>(s.grid), d, dgamma_out);
    return hip_status("ngram_add_norm_grad launch");
}

int ngram_quant_fp8(const void* x, int32_t x_dtype, int64_t n, int32_t d, const ngram_fp8* q, const ngram_fp8* qt,
                    ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    int rc = check_rows(n, d);
    if (rc) return rc;
    if ((rc = check_value(x_dtype, "x_dtype"))) return rc;
    if (!q && !qt) return fail(NGRAM_EINVAL, "q and qt are both NULL");
    if (q) {
        if ((rc = check_fp8(q, "q"))) return rc;
        if (q->rows != n || q->cols != d) return fail(NGRAM_EINVAL, "q must be %lld x %d", (long long)n, d);
    }
    if (qt) {
        if ((rc = check_fp8(qt, "qt"))) return rc;
        if (qt->rows != d || qt->cols != n) return fail(NGRAM_EINVAL, "qt must be %d x %lld", d, (long long)n);
    }
    if (q && qt && q->block_rows != qt->block_rows)
        return fail(NGRAM_EINVAL, "q and qt must have the same block_rows");
    if (n == 0) return NGRAM_OK;
    if (!x) return fail(NGRAM_EINVAL, "x is NULL");
    if (!aligned(x, 16)) return fail(NGRAM_EALIGN, "x must be 16-byte aligned");
    QuantArgs a;
    a.x = x;
    a.q = q ? q->codes : nullptr;
    a.qs = q ? q->scales : nullptr;
    a.qt = qt ? qt->codes : nullptr;
    a.qts = qt ? qt->scales : nullptr;
    a.n = n; a.d = d;
    a.q_ld = code_ld(d); a.q_sld = scale_ld(d);
    a.qt_ld = code_ld(n); a.qt_sld = scale_ld(n);
    a.tiles_d = static_cast<int32_t>(blocks_of(d));
    a.tile_scale = (q ? q : qt)->block_rows == kBlock;
    const int64_t tiles = blocks_of(n) * a.tiles_d;
    if (tiles > most_groups(256)) return fail(NGRAM_ERANGE, "n=%lld too large for one launch", (long long)n);
    if (x_dtype == NGRAM_F32)
        hipLaunchKernelGGL((quant_kernel<true>), dim3(static_cast<unsigned>(tiles)), dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((quant_kernel<false>), dim3(static_cast<unsigned>(tiles)), dim3(256), 0, stream, a);
    return hip_status("ngram_quant_fp8 launch");
}

}  // extern "C"
