// Matrix product of 8-bit operands with a scale per block of 128 for MI355X
// (gfx950): ngram_project_fp8.  C[i][o] = sum over the 128-column blocks b of
// 2^(ea[i][b] + eb[o][b]) * sum over j in b of A[i][j] B[o][j].
//
// The scales are powers of two, so v_mfma_scale_f32_16x16x128_f8f6f4 applies
// them itself: one instruction multiplies a 16 x 128 by a 128 x 16 tile,
// scales each row's (column's) products by its E8M0 bytes and adds to fp32
// accumulators, which therefore run over all of K with no rescaling pass.
// The instruction takes one byte per 32 columns; a block of 128 gives all
// four groups of lanes the same byte, and since both operands use the same
// order of the 128 columns over the lanes, that order does not matter.
//
// Precision.  The 8-bit instructions (this one and the unscaled ones alike)
// align the products of a group to its largest and keep about 12 bits below
// it: measured on random operands, errors of 3e-5 to 5e-5 of the result's
// norm, whatever K.  That is far below the rounding of a bf16 result (2e-3), but
// not below fp32's.  So bf16 results use the 8-bit instruction, and fp32
// results the bf16 one (v_mfma_f32_16x16x32_bf16, half the rate), whose
// products and sums are exact to fp32's rounding: a code times its scale is
// exactly a bf16 value, and the operands are widened in registers.
#include "common8.h"

#include <algorithm>

namespace ng8 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kStep = 128;      // columns of K per step: one scale block, 128 bytes a row

struct ProjArgs {
    const uint8_t* a;       // [M][ld]
    const uint8_t* as;      // [M >> ash][sld]
    const uint8_t* b;       // [N][ld]
    const uint8_t* bs;      // [N >> bsh][sld]
    void* c;                // [M][N]
    float* partial;         // [splits][M][N] where splits > 1
    int64_t m;
    int64_t n;
    int64_t ld;
    int64_t sld;
    int32_t ash, bsh;       // 0: a scale row per row, 7: per 128 rows
    int32_t steps;          // all of K
    int32_t split_steps;    // of one split: a multiple of 4
    int32_t splits;
    int32_t ntiles_n;
    int32_t ntiles;
};

__device__ __forceinline__ f32x4 mfma_scaled(i32x8 x, i32x8 y, f32x4 acc, uint32_t xs, uint32_t ys) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, static_cast<int>(xs), 0, static_cast<int>(ys));
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi) {
    return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
                 static_cast<int>(hi[0]), static_cast<int>(hi[1]), static_cast<int>(hi[2]), static_cast<int>(hi[3])};
}

// A lane's 32 codes of one row times their scale, as the operands of four
// bf16 instructions.  Exact for values from bf16's smallest normal number on.
struct Wide {
    bf16x8 q[4];
};
__device__ __forceinline__ Wide widen(i32x8 c, uint32_t scale_byte) {
    const float s = scale_value(scale_byte & 0xFFu);
    Wide w;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], s, true);
        w.q[i >> 1][4 * (i & 1)] = lo[0];
        w.q[i >> 1][4 * (i & 1) + 1] = lo[1];
        w.q[i >> 1][4 * (i & 1) + 2] = hi[0];
        w.q[i >> 1][4 * (i & 1) + 3] = hi[1];
    }
    return w;
}
__device__ __forceinline__ f32x4 mfma_wide(const Wide& x, const Wide& y, f32x4 acc) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.q[i], y.q[i], acc, 0, 0, 0);
    return acc;
}

// Four consecutive outputs of row i from column o (o % 4 == 0, N % 8 == 0:
// all four are inside the row or none is).
template <bool F32>
__device__ __forceinline__ void store4(void* c, int64_t at, f32x4 v) {
    if (F32) *reinterpret_cast<f32x4*>(static_cast<float*>(c) + at) = v;
    else *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(c) + at) = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}

// ---------------------------------------------------------------------------
// Tiled kernel: a workgroup of WM x WN wavefronts owns a tile of 16 TM WM rows
// of A by 16 TN WN rows of B and walks K in steps of 128 through two LDS
// buffers, filled straight from global memory.
//
// LDS rows are 128 bytes (eight 16-byte chunks); chunk c of row r sits at
// position c ^ ((r >> 1) & 7), so the 16 rows that a group of 16 lanes reads
// fall on 16 different 16-byte bank groups.  A load instruction fills 8 rows.
// Scale words (four steps' bytes of a row) go through LDS too.
__device__ __forceinline__ uint32_t chunk_pos(int row, int c) {
    return static_cast<uint32_t>(row) * kStep + (static_cast<uint32_t>(c ^ ((row >> 1) & 7)) << 4);
}

template <int TM, int TN, int WM, int WN>
struct Tile {
    static constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, Waves = WM * WN, Threads = 64 * Waves;
    static constexpr int Stage = (BM + BN) * kStep;             // bytes of one operand buffer
    static constexpr int ScaleStage = (BM + BN) * 4;            // bytes of one scale buffer
    static constexpr int Lds = 2 * Stage + 2 * ScaleStage;
    static constexpr int Groups = (BM + BN) / 8 / Waves;        // load instructions per wavefront and step
    static constexpr int ScaleLoads = (BM + BN) / 64;           // wavefronts that load scales
    static_assert(BM % 64 == 0 && BN % 64 == 0 && (BM / 8) % Groups == 0 && ScaleLoads <= Waves, "tile shape");
};

// XCD-aware tile order: workgroup b runs on XCD b mod 8, and the tiles of an
// XCD are a contiguous run of the row-tile-major order, so that one row tile's
// A stays in that XCD's L2; a run of whole tile rows is walked column by
// column, so that its concurrent tiles share one B tile.
__device__ __forceinline__ bool tile_of(int b, int ntiles, int ntiles_n, int* mt, int* nt) {
    const int per = (ntiles + 7) / 8, xcd = b & 7, slot = b >> 3;
    const int full = ntiles - 8 * (per - 1);
    const int count = xcd < full ? per : per - 1;
    if (slot >= count) return false;
    const int base = xcd < full ? xcd * per : full * per + (xcd - full) * (per - 1);
    if (base % ntiles_n == 0 && count % ntiles_n == 0) {
        const int rows_x = count / ntiles_n;
        *nt = slot / rows_x;
        *mt = base / ntiles_n + (slot - *nt * rows_x);
    } else {
        const int tile = base + slot;
        *mt = tile / ntiles_n;
        *nt = tile - *mt * ntiles_n;
    }
    return true;
}

template <int TM, int TN, int WM, int WN, bool F32>
__global__ void __launch_bounds__(64 * WM * WN, 1) project_fp8_kernel(const ProjArgs a) {
    using T = Tile<TM, TN, WM, WN>;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.y;
    int mt, nt;
    if (!tile_of(blockIdx.x, a.ntiles, a.ntiles_n, &mt, &nt)) return;
    const int64_t m0 = static_cast<int64_t>(mt) * T::BM, n0 = static_cast<int64_t>(nt) * T::BN;
    const int wm = (wave / WN) * 16 * TM, wn = (wave % WN) * 16 * TN;
    const int k_begin = split * a.split_steps;
    const int k_end = min(k_begin + a.split_steps, a.steps);

    // Operand loads: wavefront w fills row groups w Groups .. of [A tile | B
    // tile].  Rows past M or N are clamped: their results are never stored.
    const bool of_a = wave * T::Groups < T::BM / 8;
    const int64_t tile0 = of_a ? m0 : n0, last = (of_a ? a.m : a.n) - 1;
    const uint8_t* src = (of_a ? a.a : a.b) + tile0 * a.ld + static_cast<int64_t>(k_begin) * kStep;
    uint32_t off[T::Groups];
#pragma unroll
    for (int q = 0; q < T::Groups; ++q) {
        const int r = 8 * (wave * T::Groups + q - (of_a ? 0 : T::BM / 8)) + (lane >> 3);
        const int rr = static_cast<int>(min(tile0 + r, last) - tile0);
        off[q] = static_cast<uint32_t>(rr) * static_cast<uint32_t>(a.ld) + 16 * ((lane & 7) ^ ((r >> 1) & 7));
    }
    // Scale loads: wavefront w < ScaleLoads fills 64 rows of [A | B].
    const uint8_t* ssrc = a.as;
    if (wave < T::ScaleLoads) {
        const bool sa = wave * 64 < T::BM;
        const int64_t row = sa ? min(m0 + wave * 64 + lane, a.m - 1) : min(n0 + wave * 64 - T::BM + lane, a.n - 1);
        ssrc = (sa ? a.as : a.bs) + (row >> (sa ? a.ash : a.bsh)) * a.sld + k_begin;
    }
    auto issue = [&](int i) {       // step k_begin + i into buffer i & 1
        uint8_t* const buf = lds + (i & 1) * T::Stage;
#pragma unroll
        for (int q = 0; q < T::Groups; ++q)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + static_cast<int64_t>(i) * kStep + off[q]),
                                             (__attribute__((address_space(3))) void*)(buf + (wave * T::Groups + q) * 1024), 16, 0, 0);
        if ((i & 3) == 0 && wave < T::ScaleLoads)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(ssrc + i),
                                             (__attribute__((address_space(3))) void*)(lds + 2 * T::Stage + ((i >> 2) & 1) * T::ScaleStage + wave * 256), 4, 0, 0);
    };

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t sa[TM], sb[TN];
    const int steps = k_end - k_begin;
    const int lr = lane & 15, lc = (lane >> 4) * 2;
    issue(0);
    for (int i = 0; i < steps; ++i) {
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (i + 1 < steps) issue(i + 1);
        const uint8_t* const at = lds + (i & 1) * T::Stage;
        const uint8_t* const bt = at + T::BM * kStep;
        if ((i & 3) == 0) {
            const uint32_t* const sc = reinterpret_cast<const uint32_t*>(lds + 2 * T::Stage + ((i >> 2) & 1) * T::ScaleStage);
#pragma unroll
            for (int s = 0; s < TM; ++s) sa[s] = sc[wm + 16 * s + lr];
#pragma unroll
            for (int s = 0; s < TN; ++s) sb[s] = sc[T::BM + wn + 16 * s + lr];
        }
        const auto frag = [&](const uint8_t* base, int r) {
            return join(*reinterpret_cast<const u32x4*>(base + chunk_pos(r, lc)), *reinterpret_cast<const u32x4*>(base + chunk_pos(r, lc + 1)));
        };
        if constexpr (F32) {
            Wide fb[TN];
#pragma unroll
            for (int s = 0; s < TN; ++s) fb[s] = widen(frag(bt, wn + 16 * s + lr), sb[s]);
#pragma unroll
            for (int s = 0; s < TM; ++s) {
                const Wide fa = widen(frag(at, wm + 16 * s + lr), sa[s]);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[s][j] = mfma_wide(fb[j], fa, acc[s][j]);
            }
        } else {
            i32x8 fb[TN];
#pragma unroll
            for (int s = 0; s < TN; ++s) fb[s] = frag(bt, wn + 16 * s + lr);
#pragma unroll
            for (int s = 0; s < TM; ++s) {
                const i32x8 fa = frag(at, wm + 16 * s + lr);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[s][j] = mfma_scaled(fb[j], fa, acc[s][j], sb[j], sa[s]);
            }
        }
#pragma unroll
        for (int s = 0; s < TM; ++s) sa[s] >>= 8;
#pragma unroll
        for (int s = 0; s < TN; ++s) sb[s] >>= 8;
    }
    // The B fragment is the instruction's row operand, so lane l holds, of
    // each 16 x 16 tile, row l & 15 of A and four consecutive rows
    // 4 (l >> 4) .. +3 of B: four consecutive outputs.
#pragma unroll
    for (int s = 0; s < TM; ++s) {
        const int64_t row = m0 + wm + 16 * s + lr;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t col = n0 + wn + 16 * j + 4 * (lane >> 4);
            if (row < a.m && col < a.n) {
                if (a.splits > 1) store4<true>(a.partial, (split * a.m + row) * a.n + col, acc[s][j]);
                else store4<F32>(a.c, row * a.n + col, acc[s][j]);
            }
        }
    }
}

// The sum of the splits' partial products, in their order.
template <bool F32>
__global__ void __launch_bounds__(256) split_sum_kernel(const float* __restrict__ partial, int splits, int64_t count, void* c) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= count) return;
    f32x4 t = *reinterpret_cast<const f32x4*>(partial + i);
    for (int s = 1; s < splits; ++s) t += *reinterpret_cast<const f32x4*>(partial + s * count + i);
    store4<F32>(c, i, t);
}

// ---------------------------------------------------------------------------
// Few rows of A (decode): bound by the one read of B.  A workgroup owns 16
// rows of B; its eight wavefronts take every eighth step of K with operands
// straight from global memory (B is read once, A stays in L2), and join their
// accumulators in LDS.  The matrix cores have time to spare here, so both
// result types take the exact instruction.
template <int MT, bool F32>
__global__ void __launch_bounds__(512) project_fp8_rows_kernel(const ProjArgs a) {
    __shared__ f32x4 part[8][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (16 * MT);
    const int64_t br = min(n0 + lr, a.n - 1);
    const uint8_t* const bp = a.b + br * a.ld + 32 * (lane >> 4);
    const uint8_t* const bsp = a.bs + (br >> a.bsh) * a.sld;
    const uint8_t* ap[MT];
    const uint8_t* asp[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t ar = min(m0 + 16 * t + lr, a.m - 1);
        ap[t] = a.a + ar * a.ld + 32 * (lane >> 4);
        asp[t] = a.as + (ar >> a.ash) * a.sld;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int kb = wave; kb < a.steps; kb += 8) {
        const u32x4* const p = reinterpret_cast<const u32x4*>(bp + static_cast<int64_t>(kb) * kStep);
        const Wide fb = widen(join(p[0], p[1]), bsp[kb]);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const u32x4* const q = reinterpret_cast<const u32x4*>(ap[t] + static_cast<int64_t>(kb) * kStep);
            acc[t] = mfma_wide(fb, widen(join(q[0], q[1]), asp[t][kb]), acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < MT; t += 8) {
        f32x4 v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < 8; ++w) v += part[w][t][lane];
        const int64_t row = m0 + 16 * t + lr, col = n0 + 4 * (lane >> 4);
        if (row < a.m && col < a.n) store4<F32>(a.c, row * a.n + col, v);
    }
}

// ---------------------------------------------------------------------------
// Which kernel, tile and split.
struct Plan {
    int kind;           // 0: few rows; 1: 64 x 64; 2: 128 x 128; 3: 256 x 256
    int splits;
    int split_steps;
};

constexpr int kUnits = 256;     // compute units

Plan plan_of(int64_t m, int64_t n, int64_t k) {
    const int steps = static_cast<int>(blocks_of(k));
    Plan p{0, 1, (steps + 3) / 4 * 4};
    if (m <= 64) return p;
    const auto tiles = [&](int64_t t) { return ((m + t - 1) / t) * ((n + t - 1) / t); };
    p.kind = tiles(256) >= kUnits ? 3 : tiles(128) >= kUnits ? 2 : 1;
    // long K over few tiles (the weight gradient): larger tiles, K split
    if (p.kind < 3 && steps >= 32) p.kind = tiles(256) >= 32 ? 3 : 2;
    const int64_t have = tiles(p.kind == 3 ? 256 : p.kind == 2 ? 128 : 64);
    const int64_t want = (p.kind == 3 ? 1 : 2) * kUnits;
    int64_t splits = std::min<int64_t>(std::max<int64_t>(1, want / std::max<int64_t>(1, have)), std::max(1, steps / 16));
    p.split_steps = static_cast<int>(((steps + splits - 1) / splits + 3) / 4 * 4);
    p.splits = (steps + p.split_steps - 1) / p.split_steps;
    return p;
}

template <int TM, int TN, int WM, int WN>
int launch_tile(ProjArgs& a, bool f32, hipStream_t st) {
    using T = Tile<TM, TN, WM, WN>;
    const int64_t mt = (a.m + T::BM - 1) / T::BM, nt = (a.n + T::BN - 1) / T::BN;
    if (mt * nt > INT32_MAX / 16) return fail(NGRAM_ERANGE, "%lld x %lld too large for one launch", (long long)a.m, (long long)a.n);
    a.ntiles_n = static_cast<int32_t>(nt);
    a.ntiles = static_cast<int32_t>(mt * nt);
    const dim3 grid(8 * ((a.ntiles + 7) / 8), a.splits), block(T::Threads);
    if (f32) hipLaunchKernelGGL((project_fp8_kernel<TM, TN, WM, WN, true>), grid, block, T::Lds, st, a);
    else hipLaunchKernelGGL((project_fp8_kernel<TM, TN, WM, WN, false>), grid, block, T::Lds, st, a);
    return NGRAM_OK;
}

template <int MT>
void launch_rows(const ProjArgs& a, bool f32, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>((a.n + 15) / 16), static_cast<unsigned>((a.m + 16 * MT - 1) / (16 * MT))), block(512);
    if (f32) hipLaunchKernelGGL((project_fp8_rows_kernel<MT, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((project_fp8_rows_kernel<MT, false>), grid, block, 0, st, a);
}

// m rows by n columns over k columns of K; the tile kernels address a tile's
// operand rows with 32-bit offsets, hence the limit on k.
constexpr int64_t kMaxK = int64_t{1} << 23;

bool sizes_ok(int64_t m, int64_t n, int64_t k) {
    return m >= 0 && n > 0 && k > 0 && m <= NGRAM_FP8_MAX && n <= NGRAM_FP8_MAX && k <= kMaxK && n % kVec == 0;
}

}  // namespace
}  // namespace ng8

using namespace ng8;

extern "C" {

int64_t ngram_project_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k) {
    if (!sizes_ok(m, n, k)) return -1;
    const Plan p = plan_of(m, n, k);
    return p.splits > 1 ? 4 * p.splits * m * n : 0;
}

int ngram_project_fp8(const ngram_fp8* A, const ngram_fp8* B, void* C, int32_t c_dtype, void* workspace,
                      int64_t workspace_bytes, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    int rc = check_fp8(A, "A");
    if (rc) return rc;
    if ((rc = check_fp8(B, "B"))) return rc;
    if (c_dtype != NGRAM_F32 && c_dtype != NGRAM_BF16) return fail(NGRAM_EINVAL, "c_dtype=%d is not an ngram_value", c_dtype);
    if (A->cols != B->cols) return fail(NGRAM_EINVAL, "A has %lld columns and B %lld", (long long)A->cols, (long long)B->cols);
    if (A->cols < 1 || B->rows < 1 || B->rows % kVec != 0)
        return fail(NGRAM_EINVAL, "columns=%lld must be positive and B's rows=%lld a positive multiple of %d", (long long)A->cols,
                    (long long)B->rows, kVec);
    if (!sizes_ok(A->rows, B->rows, A->cols)) return fail(NGRAM_ERANGE, "columns=%lld above %lld", (long long)A->cols, (long long)kMaxK);
    if (A->rows == 0) return NGRAM_OK;
    if (!C) return fail(NGRAM_EINVAL, "C is NULL");
    if (!aligned(C, 16)) return fail(NGRAM_EALIGN, "C must be 16-byte aligned");
    const Plan p = plan_of(A->rows, B->rows, A->cols);
    const int64_t need = ngram_project_fp8_workspace_bytes(A->rows, B->rows, A->cols);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return fail(NGRAM_EINVAL, "workspace must hold %lld bytes, 16-byte aligned", (long long)need);
    ProjArgs a;
    a.a = A->codes; a.as = A->scales; a.b = B->codes; a.bs = B->scales; a.c = C;
    a.partial = static_cast<float*>(workspace);
    a.m = A->rows; a.n = B->rows; a.ld = code_ld(A->cols); a.sld = scale_ld(A->cols);
    a.ash = A->block_rows == kBlock ? 7 : 0;
    a.bsh = B->block_rows == kBlock ? 7 : 0;
    a.steps = static_cast<int32_t>(blocks_of(A->cols));
    a.split_steps = p.split_steps; a.splits = p.splits;
    a.ntiles_n = a.ntiles = 0;
    const bool f32 = c_dtype == NGRAM_F32;
    rc = NGRAM_OK;
    if (p.kind == 0) {
        if ((a.n + 15) / 16 > INT32_MAX) return fail(NGRAM_ERANGE, "B too large for one launch");
        if (a.m <= 16) launch_rows<1>(a, f32, stream);
        else if (a.m <= 32) launch_rows<2>(a, f32, stream);
        else launch_rows<4>(a, f32, stream);
    } else if (p.kind == 1) {
        rc = launch_tile<2, 2, 2, 2>(a, f32, stream);
    } else if (p.kind == 2) {
        rc = launch_tile<4, 4, 2, 2>(a, f32, stream);
    } else {
        rc = launch_tile<8, 4, 2, 4>(a, f32, stream);
    }
    if (rc) return rc;
    if (a.splits > 1) {
        const int64_t count = a.m * a.n, groups = (count / 4 + 255) / 256;
        if (groups > INT32_MAX) return fail(NGRAM_ERANGE, "C too large for one launch");
        if (f32) hipLaunchKernelGGL((split_sum_kernel<true>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, stream, a.partial, a.splits, count, C);
        else hipLaunchKernelGGL((split_sum_kernel<false>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, stream, a.partial, a.splits, count, C);
    }
    return hip_status("ngram_project_fp8 launch");
}

}  // extern "C"
