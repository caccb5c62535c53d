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
// Precision.  The 8-bit instruction takes the products of eight consecutive
// columns as multiples of 2^(E - 13), cut towards zero, where E is the largest
// sum of two codes' exponents among the eight (-6 for a subnormal code), and
// adds in fp32 from there on (found with chosen codes; the unscaled 8-bit
// instructions do the same).  A group is off by less than 2^(E - 10).  On random
// operands that is 3e-5 to 5e-5 of the result's norm, whatever K, far below
// the rounding of a bf16 result (1.66e-3 of the norm with and without it, also
// with columns 1000 times the others), though about one bf16 value in 80 goes to
// its neighbour, and an output whose large products cancel loses more.  It is
// not below fp32's rounding.  So bf16 results use the 8-bit instruction, which
// is twice as fast, and fp32 results the bf16 one (v_mfma_f32_16x16x32_bf16),
// whose products and sums are exact to fp32's rounding: a code times its scale
// is exactly a bf16 value, and the operands are widened in registers.
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
    int32_t band;           // tile rows walked together
    int32_t stride;         // items from one of a workgroup to its next
    int32_t first;          // the launch's first item, a multiple of 8 (few rows: 16 rows of B; not of the large tiles)
};

// acc + x y, each scaled by the lowest byte of its word.
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
// of A by 16 TN WN rows of B and walks K in steps of 128 through NS LDS
// buffers, filled straight from global memory (no registers on the way).
//
// LDS rows are 128 bytes (eight 16-byte chunks); chunk c of row r sits at
// position c ^ ((r >> 1) & 7).  A fragment read takes chunks g and g + 4 in
// lane group g = lane >> 4: the LDS serves 16 lanes at a time, 0-3 with 12-15 and
// 20-27 and so on, and in this order they fall on 16 different 16-byte bank
// groups (no conflicts counted; chunks 2 g and 2 g + 1 had one for every read).
// A load instruction fills 8 rows.
//
// Scales go through LDS as well: a row's word of four steps' bytes with the
// first of the four, and a byte read for each fragment and step.
//
// Measured: bf16 results 32768 x 2560 x 2560 181 us, 2.4 PFLOP/s, and 8192 x
// 2560 x 2560 49 to 53 us, 2.0 to 2.2 (256 x 320 tiles); 8192 x 8192 x 8192
// 440 us, 2.5 PFLOP/s (256 x 256).  Products alone, on random codes, stop at 3.9
// to 4.0 PFLOP/s: the card holds about 2.0 GHz under this load.  A step is bound
// by LDS and the matrix cores together: 256 x 256 reads 192 KB of fragments
// and has 64 KB brought in, 2000 cycles at 128 bytes a cycle, beside 2048 of
// products, and takes about 3400 (without the products 2500).  Hence the
// largest tile a wavefront can hold, 128 x 80: 13 fragments for 40 products,
// where 128 x 64 has 12 for 32.  A round's stores, 128 or 160 KB a unit, all
// at once, take 10 to 15%.
// fp32 results (256 x 128 tiles) 2560 x 2560 x 8192 97 to 110 us, 1.0 to 1.1
// PFLOP/s of the 1.3 that a large bf16 product reaches: 200 tiles for 256
// compute units.
template <int TM_, int TN_, int WM_, int WN_, int NS_, bool F32_>
struct Tile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, NS = NS_;
    static constexpr bool F32 = F32_;
    static constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, Waves = WM * WN, Threads = 64 * Waves;
    static constexpr int Rows = BM + BN;
    static constexpr int Stage = Rows * kStep;                  // bytes of one operand buffer
    static constexpr int ScaleLoads = (Rows + Threads - 1) / Threads;       // instructions per wavefront and four steps
    static constexpr int ScaleStage = (Rows + 63) / 64 * 256;         // bytes of one scale buffer: four steps
    static constexpr int ScaleBuffers = 4;      // a step and the NS that are loaded ahead of it touch no more groups of four
    static constexpr int Lds = NS * Stage + ScaleBuffers * ScaleStage;
    static constexpr int Tail = TN > 4 ? 1 : 2;     // rows of fragments multiplied after a step's barrier (no registers for two with TN = 5)
    // load instructions per wavefront and step, 8 rows each; B's last may be some wavefronts' only
    static constexpr int LoadsA = BM / 8 / Waves, LoadsB = (BN / 8 + Waves - 1) / Waves, Loads = LoadsA + LoadsB;
    static_assert(BM % (8 * Waves) == 0 && Waves % 2 == 0 && TM >= 4 && TM % 2 == 0, "tile shape");
    static_assert(NS >= 2 && NS <= 4 && Lds <= 160 * 1024, "buffers");
    static_assert(NS == 2 || BN % (8 * Waves) == 0, "counted waits need every wavefront's loads alike");
};

// Work item w of the launch's order: workgroup b runs on XCD b mod 8 and takes
// items b, b + stride, ... (the stride is a multiple of 8), and the items of an XCD
// are a contiguous run of the order: split by split, and in a split bands of `band` tile
// rows, each walked column by column.  The tiles that an XCD has in flight
// then share `band` tiles of A and some of B at the same place of K, which its
// L2 holds: 2 + 16 tiles for 32 workgroups of a large tile, 8 + 4 for a small
// one, where whole columns would want 32 + 1.  (Bands of 1, 3, 4 and 8 of the large
// tiles: within 3% at 32768 x 2560 x 2560, 2 the fastest there.)
struct Item {
    int32_t mt, nt, split, valid;
};
__device__ __forceinline__ Item item_of(int w, const ProjArgs& a) {
    const int total = a.ntiles * a.splits;
    const int per = (total + 7) / 8, xcd = w & 7, slot = w >> 3;
    const int full = total - 8 * (per - 1);
    const int count = xcd < full ? per : per - 1;
    const int idx = (xcd < full ? xcd * per : full * per + (xcd - full) * (per - 1)) + slot;
    const int split = idx / a.ntiles, tile = idx - split * a.ntiles;
    const int first = tile / (a.band * a.ntiles_n) * a.band;             // the band's first row
    const int rows = min(a.band, a.ntiles / a.ntiles_n - first);
    const int r = tile - first * a.ntiles_n, nt = r / max(rows, 1);
    return Item{__builtin_amdgcn_readfirstlane(first + r - nt * rows), __builtin_amdgcn_readfirstlane(nt),
                __builtin_amdgcn_readfirstlane(split), __builtin_amdgcn_readfirstlane(slot < count ? 1 : 0)};
}

// Keeps the products of a group where they are written: the compiler would
// otherwise gather all of a step's reads in front of the barrier and all its
// products behind it.
template <int N>
__device__ __forceinline__ void pin(f32x4* acc) {
#pragma unroll
    for (int j = 0; j < N; ++j) __asm__ volatile("" : "+v"(acc[j]));
    __builtin_amdgcn_sched_barrier(0);
}

// The B fragment is the instruction's row operand, so lane l holds, of each
// 16 x 16 tile, row l & 15 of A and four consecutive rows 4 (l >> 4) .. +3 of
// B: four consecutive outputs, 16 bytes of fp32.  In bf16 that is 8, so two
// neighbouring tiles' values are exchanged between lane groups 0 and 1, 2 and
// 3: then a lane has eight consecutive outputs of one of the two, and a store
// writes 64 consecutive bytes of 16 rows (32-byte pieces took 8% more time for
// the whole product at 32768 x 2560 x 2560).  An odd last tile is exchanged with
// the one of the next 16 rows.
template <int TM, int TN, bool F32>
__device__ __forceinline__ void store_tile(const ProjArgs& a, const f32x4 (&acc)[TM][TN], int m0, int n0, int split, int lane) {
    const int m = static_cast<int>(a.m), n = static_cast<int>(a.n);     // at most 2^30
    const int lr = lane & 15, g = lane >> 4;
#pragma unroll
    for (int s = 0; s < TM; ++s) {
        const int row = m0 + 16 * s + lr;
        const int64_t at = static_cast<int64_t>(row) * a.n;
        if (F32 || a.splits > 1) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int col = n0 + 16 * j + 4 * g;
                if (row < m && col < n) {
                    if (a.splits > 1) store4<true>(a.partial, split * a.m * a.n + at + col, acc[s][j]);
                    else store4<F32>(a.c, at + col, acc[s][j]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j + 1 < TN; j += 2) {
                const f32x4 x = acc[s][j], y = acc[s][j + 1];
                const auto p = __builtin_amdgcn_permlane16_swap(bf16_pair(x[0], x[1]), bf16_pair(y[0], y[1]), false, false);
                const auto q = __builtin_amdgcn_permlane16_swap(bf16_pair(x[2], x[3]), bf16_pair(y[2], y[3]), false, false);
                const int col = n0 + 16 * j + 16 * (g & 1) + 8 * (g >> 1);
                if (row < m && col < n)
                    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.c) + at + col) = u32x4{p[0], q[0], p[1], q[1]};
            }
            if (TN % 2 == 1 && s % 2 == 1) {
                const f32x4 x = acc[s - 1][TN - 1], y = acc[s][TN - 1];
                const auto p = __builtin_amdgcn_permlane16_swap(bf16_pair(x[0], x[1]), bf16_pair(y[0], y[1]), false, false);
                const auto q = __builtin_amdgcn_permlane16_swap(bf16_pair(x[2], x[3]), bf16_pair(y[2], y[3]), false, false);
                const int r = row - 16 * (1 - (g & 1)), col = n0 + 16 * (TN - 1) + 8 * (g >> 1);
                if (r < m && col < n)
                    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.c) + static_cast<int64_t>(r) * a.n + col) = u32x4{p[0], q[0], p[1], q[1]};
            }
        }
    }
}

template <class T>
__global__ void __launch_bounds__(T::Threads, 1) project_fp8_kernel(const ProjArgs a) {
    constexpr int TM = T::TM, TN = T::TN, NS = T::NS;
    constexpr bool F32 = T::F32, Two = NS == 2;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = (wave / T::WN) * 16 * TM, wn = (wave % T::WN) * 16 * TN;
    int w = blockIdx.x, lw = w;
    Item now = item_of(w, a);
    if (!now.valid) return;

    // Loads run ahead of the products, through the end of an item into the next.
    //
    // Operands: wavefront v fills row groups v, v + Waves, .. of the A tile
    // and of the B tile, 8 rows an instruction; every other group has the
    // same swizzle, so all of a wavefront's do.  Rows past M or N are clamped to the last row (their
    // results are never stored): the limit is that row's offset.  Scales:
    // thread t < Rows brings the word of row t of [A tile | B tile].
    const uint32_t ld = static_cast<uint32_t>(a.ld);
    const uint32_t chunk = 16u * ((lane & 7) ^ (lane >> 4) ^ 4 * (wave & 1));
    const uint32_t off = (8 * wave + (lane >> 3)) * ld + chunk;
    uint8_t* const sbuf = lds + NS * T::Stage;
    const uint8_t *pa, *pb, *ps[T::ScaleLoads];     // the load step's first rows, the first of its scale bytes
    uint32_t soff[T::ScaleLoads];                   // from there to the thread's
    uint32_t last_a, last_b;            // offsets of the tiles' last rows
    int ahead, left;                    // the load step in its item, steps left with it
    int put_to = -1;                    // the scale buffer loaded last
    const auto steps_of = [&](const Item& it) { return min(a.split_steps, a.steps - it.split * a.split_steps); };
    const auto load_from = [&](const Item& it) {
        const int64_t m0 = static_cast<int64_t>(it.mt) * T::BM, n0 = static_cast<int64_t>(it.nt) * T::BN;
        const int64_t k0 = static_cast<int64_t>(it.split) * a.split_steps;
        last_a = (static_cast<uint32_t>(min(a.m - m0, static_cast<int64_t>(T::BM))) - 1) * ld;
        last_b = (static_cast<uint32_t>(min(a.n - n0, static_cast<int64_t>(T::BN))) - 1) * ld;
        pa = a.a + m0 * a.ld + k0 * kStep;
        pb = a.b + n0 * a.ld + k0 * kStep;
#pragma unroll
        for (int q = 0; q < T::ScaleLoads; ++q) {
            const bool sa = (q * T::Waves + wave) * 64 < T::BM;
            const int64_t first = sa ? m0 : n0, row = min(first + t + q * T::Threads - (sa ? 0 : T::BM), (sa ? a.m : a.n) - 1);
            const int shift = sa ? a.ash : a.bsh;
            ps[q] = (sa ? a.as : a.bs) + (first >> shift) * a.sld + k0;
            soff[q] = static_cast<uint32_t>((row >> shift) - (first >> shift)) * static_cast<uint32_t>(a.sld);
        }
        ahead = 0;
        left = steps_of(it);
    };
    const auto step_on = [&] {          // after a step's loads
        if (--left > 0) {
            pa += kStep;
            pb += kStep;
#pragma unroll
            for (int q = 0; q < T::ScaleLoads; ++q) ps[q] += 1;
            ++ahead;
            return;
        }
        lw += a.stride;
        const Item it = item_of(lw, a);
        if (it.valid) {
            load_from(it);
        } else {                        // nothing follows: the last step again, never read
            lw -= a.stride;
            left = 1;
        }
    };
    const auto load = [&](const uint8_t* s, uint32_t last, uint8_t* to, int q) {
        const uint32_t at = min(off + 8 * T::Waves * q * ld, last + chunk);
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(s + at),
                                         (__attribute__((address_space(3))) void*)(to + (q * T::Waves + wave) * 1024), 16, 0, 0);
    };
    const auto load_a = [&](int buffer, int q) { load(pa, last_a, lds + buffer * T::Stage, q); };
    const auto load_b = [&](int buffer, int q) {
        if ((q + 1) * T::Waves <= T::BN / 8 || q * T::Waves + wave < T::BN / 8)
            load(pb, last_b, lds + buffer * T::Stage + T::BM * kStep, q);
    };
    const auto load_scales = [&] {      // ahead of a step's other loads
        if ((ahead & 3) != 0) return;
        put_to = (put_to + 1) & (T::ScaleBuffers - 1);
#pragma unroll
        for (int q = 0; q < T::ScaleLoads; ++q)
            if ((q * T::Waves + wave) * 64 < T::Rows)
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(ps[q] + soff[q]),
                                                 (__attribute__((address_space(3))) void*)(sbuf + put_to * T::ScaleStage + (q * T::Waves + wave) * 256), 4, 0, 0);
    };

    // A lane reads chunks g and g + 4 (g = lane >> 4) of its fragment rows.
    // Rows 16 s + lr of a fragment share the swizzle of lr, so one lane
    // offset per chunk serves them all.
    const int lr = lane & 15, g = lane >> 4;
    const uint32_t lo = lr * kStep + ((g ^ ((lr >> 1) & 7)) << 4), hi = lo ^ 64u;
    const auto frag = [&](const uint8_t* rows, int s) {
        return join(*reinterpret_cast<const u32x4*>(rows + s * 16 * kStep + lo), *reinterpret_cast<const u32x4*>(rows + s * 16 * kStep + hi));
    };
    const uint32_t a_row = wm * kStep, b_row = (T::BM + wn) * kStep;
    uint32_t sa[TM], sb[TN];
    const auto scales = [&](int i, int buffer) { return sbuf + buffer * T::ScaleStage + (i & 3) + lr * 4; };  // step i's
    const uint8_t* sp = scales(0, 0);
    const auto a_scale = [&](int s) -> uint32_t { return sp[(wm + 16 * s) * 4]; };
    const auto b_scale = [&](int j) -> uint32_t { return sp[(T::BM + wn + 16 * j) * 4]; };
    f32x4 acc[TM][TN];
    const auto clear = [&] {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    i32x8 fb[TN], fa, next;     // codes; the bf16 instruction's operands are widened from them when they are used
    Wide wb[F32 ? TN : 1];
    const auto times = [&](int s, int j, const i32x8& x, const Wide& xw, uint32_t xs, uint32_t ys) {
        if constexpr (F32) acc[s][j] = mfma_wide(wb[j], xw, acc[s][j]);
        else acc[s][j] = mfma_scaled(fb[j], x, acc[s][j], ys, xs);
    };
    const auto wide = [&](const i32x8& x, uint32_t scale) {
        Wide v{};
        if constexpr (F32) v = widen(x, scale);
        return v;
    };
    // Before the loop: step 0, and the loads of the steps after it (with two
    // buffers, A's of step 1).
    load_from(now);
#pragma unroll
    for (int s = 0; s < (Two ? 1 : NS); ++s) {
        load_scales();
#pragma unroll
        for (int q = 0; q < T::LoadsA; ++q) load_a(s, q);
#pragma unroll
        for (int q = 0; q < T::LoadsB; ++q) load_b(s, q);
        step_on();
    }
    __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(Two ? 0 : (NS - 1) * T::Loads) : "memory");
    __syncthreads();
    if (Two) {
        load_scales();
#pragma unroll
        for (int q = 0; q < T::LoadsA; ++q) load_a(1, q);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        sb[j] = b_scale(j);
        fb[j] = frag(lds + b_row, j);
    }
    sa[0] = a_scale(0);
    sa[1] = a_scale(1);
    fa = frag(lds + a_row, 0);
    clear();
    int i = 0, steps = steps_of(now), read_from = 0;
    for (int buffer = 0;;) {
        const int after = buffer + 1 == NS ? 0 : buffer + 1;
        const uint8_t* const at = lds + buffer * T::Stage + a_row;
        if constexpr (F32)
#pragma unroll
            for (int j = 0; j < TN; ++j) wb[j] = widen(fb[j], sb[j]);
        // Rows 0 .. TM - Tail - 1.  A load instruction takes the wavefront's turn
        // for as long as the CU's one load path needs for it (16 cycles or
        // more), so the large tile's loads are spread: A's over the tail of
        // the step that frees the buffer, B's over the head of the next.
        i32x8 over = {};        // the last row's, where two are multiplied after the barrier
#pragma unroll
        for (int s = 0; s < TM - T::Tail; ++s) {
            next = frag(at, s + 1);
            if (T::Tail == 2 && s == TM - 3) over = frag(at, TM - 1);
            if (s + 2 < TM) sa[s + 2] = a_scale(s + 2);
            const Wide xw = wide(fa, sa[s]);
#pragma unroll
            for (int j = 0; j < TN; ++j) times(s, j, fa, xw, sa[s], sb[j]);
            fa = next;
            // the first product waits for this group's reads; the next
            // group's are issued behind it
            if (!F32) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (s == TM - 3) __builtin_amdgcn_sched_group_barrier(0x100, T::Tail == 2 ? 5 : 3, 0);
                else __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, TN - 1, 0);
            }
            pin<TN>(acc[s]);
            if (Two && s < 2)
#pragma unroll
                for (int q = s * T::LoadsB / 2; q < (s + 1) * T::LoadsB / 2; ++q) load_b(after, q);
        }
        if (Two) step_on();
        // the next step's loads have landed: NS - 2 later steps' may be in flight
        __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((NS - 2) * T::Loads) : "memory");
        __builtin_amdgcn_s_barrier();
        __asm__ volatile("" ::: "memory");
        const int to = ++i < steps ? i : 0;
        if ((to & 3) == 0) read_from = (read_from + 1) & (T::ScaleBuffers - 1);
        sp = scales(to, read_from);
        // A step's last row fragments (fa, over) are multiplied after the
        // barrier that ends its reads, while the next step's first fragments
        // are on their way.  A B fragment and its scale are read again only
        // behind their last product: no registers for both.
        const uint8_t* const nt = lds + after * T::Stage;
        const i32x8 first = frag(nt + a_row, 0);
        const Wide xw = wide(fa, sa[TM - T::Tail]), yw = wide(over, sa[TM - 1]);
        uint32_t s0, s1;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            times(TM - T::Tail, j, fa, xw, sa[TM - T::Tail], sb[j]);
            if (T::Tail == 2) times(TM - 1, j, over, yw, sa[TM - 1], sb[j]);
            pin<1>(&acc[TM - T::Tail][j]);
            if (T::Tail == 2) pin<1>(&acc[TM - 1][j]);
            fb[j] = frag(nt + b_row, j);
            sb[j] = b_scale(j);
            if (j == 0) {
                s0 = a_scale(0);
                s1 = a_scale(1);
            }
            if (j == 0) load_scales();
#pragma unroll
            for (int q = j * T::LoadsA / TN; q < (j + 1) * T::LoadsA / TN; ++q) load_a(buffer, q);
            if (!Two)
#pragma unroll
                for (int q = j * T::LoadsB / TN; q < (j + 1) * T::LoadsB / TN; ++q) load_b(buffer, q);
        }
        if (!Two) step_on();
        fa = first;
        sa[0] = s0;
        sa[1] = s1;
        buffer = after;
        if (i < steps) continue;
        store_tile<TM, TN, F32>(a, acc, now.mt * T::BM + wm, now.nt * T::BN + wn, now.split, lane);
        w += a.stride;
        now = item_of(w, a);
        if (!now.valid) break;
        i = 0;
        steps = steps_of(now);
        clear();
    }
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");        // loads into LDS end before the workgroup does
}

// Small results, where a step is over long before the next one's loads have
// landed: a workgroup's G groups of WM x WN wavefronts each take every G-th
// step of K of one tile, so that G steps' loads are in flight and the chain of
// waits is G times shorter, and join their accumulators in LDS at the end.
// Same LDS layout and fragments as above; a scale word is loaded with every
// G steps.
//
// Bound by a round's chain of load, barrier, fragment reads and products, not
// by a unit: 777 x 4104 over 1032 columns in fp32, 14.7 us (231 tiles, five
// rounds of about 1.6 us, launch and first loads 5, stores 3.5); one group of
// 8 or 4 wavefronts with four steps' loads ahead took 17 to 20, 64 x 64 tiles
// 17.6.  128 x 128 tiles have 4 x 4 fragments a wavefront, not 4 x 2
// (14.7 against 15.4 us): a widened fragment then serves four products, not
// two, and widening is 16 vector instructions.  A bf16 result has nothing to
// widen and takes the same time either way (1024 x 2560 x 2560: 16.5 us).
template <int TM_, int TN_, int WM_, int WN_, int G_, bool F32_>
struct SmallTile {
    static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, G = G_;
    static constexpr bool F32 = F32_;
    static constexpr int BM = 16 * TM * WM, BN = 16 * TN * WN, Waves = WM * WN, Threads = 64 * Waves * G;
    static constexpr int Rows = BM + BN;
    static constexpr int Part = Rows * kStep;                   // bytes of one group's operand buffer
    static constexpr int Stage = G * Part + Rows * 4;           // of a stage: the groups' operands, then the scale words
    static constexpr int Lds = 2 * Stage;
    static constexpr int LoadsA = BM / 8 / Waves, LoadsB = BN / 8 / Waves;
    static_assert(BM % 64 == 0 && BN % 64 == 0 && LoadsA % 2 == 0 && LoadsB % 2 == 0 && Rows / 64 <= Waves * G, "tile shape");
    static_assert(4 % G == 0 && TM % 2 == 0 && TN % 2 == 0 && Lds <= 160 * 1024 && (G - 1) * BM * BN * 4 <= Lds, "groups");
};

template <class T>
__global__ void __launch_bounds__(T::Threads, 1) project_fp8_small_kernel(const ProjArgs a) {
    constexpr int TM = T::TM, TN = T::TN, G = T::G;
    constexpr bool F32 = T::F32;
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const int t = threadIdx.x, lane = t & 63;
    const int all = __builtin_amdgcn_readfirstlane(t >> 6), group = all / T::Waves, wave = all % T::Waves;
    const int wm = (wave / T::WN) * 16 * TM, wn = (wave % T::WN) * 16 * TN;
    const Item it = item_of(a.first + static_cast<int>(blockIdx.x), a);
    if (!it.valid) return;
    const int64_t m0 = static_cast<int64_t>(it.mt) * T::BM, n0 = static_cast<int64_t>(it.nt) * T::BN;
    const int k0 = it.split * a.split_steps, k1 = min(k0 + a.split_steps, a.steps);
    const int rounds = (k1 - k0 + G - 1) / G;

    const uint32_t ld = static_cast<uint32_t>(a.ld);
    const uint32_t chunk0 = 16u * ((lane & 7) ^ (lane >> 4)), flip = (chunk0 ^ 64u) - chunk0;
    const uint32_t off_a = (8 * wave * T::LoadsA + (lane >> 3)) * ld + chunk0, off_b = (8 * wave * T::LoadsB + (lane >> 3)) * ld + chunk0;
    const uint32_t last_a = (static_cast<uint32_t>(min(a.m - m0, static_cast<int64_t>(T::BM))) - 1) * ld + chunk0;
    const uint32_t last_b = (static_cast<uint32_t>(min(a.n - n0, static_cast<int64_t>(T::BN))) - 1) * ld + chunk0;
    const uint8_t* const pa = a.a + m0 * a.ld;
    const uint8_t* const pb = a.b + n0 * a.ld;
    const bool sa_row = t < T::BM;
    const int64_t srow = sa_row ? min(m0 + t, a.m - 1) : min(n0 + t - T::BM, a.n - 1);
    const uint8_t* const ps = (sa_row ? a.as : a.bs) + (srow >> (sa_row ? a.ash : a.bsh)) * a.sld;
    const auto issue = [&](int r) {     // round r: this group's step, the last one again where there is none
        uint8_t* const stage = lds + (r & 1) * T::Stage;
        uint8_t* const to = stage + group * T::Part;
        const int64_t k = static_cast<int64_t>(min(k0 + r * G + group, k1 - 1)) * kStep;
        if (all < T::Rows / 64)
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(ps + ((k0 + r * G) & ~3)),
                                             (__attribute__((address_space(3))) void*)(stage + G * T::Part + all * 256), 4, 0, 0);
#pragma unroll
        for (int q = 0; q < T::LoadsA; ++q) {
            const uint32_t at = min(off_a + 8 * q * ld, last_a) + (q & 1 ? flip : 0u);      // modulo 2^32: flip may be -64
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(pa + k + at),
                                             (__attribute__((address_space(3))) void*)(to + (wave * T::LoadsA + q) * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < T::LoadsB; ++q) {
            const uint32_t at = min(off_b + 8 * q * ld, last_b) + (q & 1 ? flip : 0u);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(pb + k + at),
                                             (__attribute__((address_space(3))) void*)(to + T::BM * kStep + (wave * T::LoadsB + q) * 1024), 16, 0, 0);
        }
    };
    const int lr = lane & 15, g = lane >> 4;
    const uint32_t lo = lr * kStep + ((g ^ ((lr >> 1) & 7)) << 4), hi = lo ^ 64u;
    f32x4 acc[TM][TN];
#pragma unroll
    for (int s = 0; s < TM; ++s)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[s][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    issue(0);
    for (int r = 0; r < rounds; ++r) {
        __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __asm__ volatile("" ::: "memory");
        if (r + 1 < rounds) issue(r + 1);
        const int step = k0 + r * G + group;
        if (step >= k1) continue;       // the whole wavefront; it comes back to the barrier
        const uint8_t* const stage = lds + (r & 1) * T::Stage;
        const uint8_t* const at = stage + group * T::Part + wm * kStep;
        const uint8_t* const bt = stage + group * T::Part + (T::BM + wn) * kStep;
        const uint8_t* const sc = stage + G * T::Part + (step & 3) + lr * 4;
        uint32_t sa[TM], sb[TN];
        i32x8 fa[TM], fb[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            sb[j] = sc[(T::BM + wn + 16 * j) * 4];
            fb[j] = join(*reinterpret_cast<const u32x4*>(bt + j * 16 * kStep + lo), *reinterpret_cast<const u32x4*>(bt + j * 16 * kStep + hi));
        }
#pragma unroll
        for (int s = 0; s < TM; ++s) {
            sa[s] = sc[(wm + 16 * s) * 4];
            fa[s] = join(*reinterpret_cast<const u32x4*>(at + s * 16 * kStep + lo), *reinterpret_cast<const u32x4*>(at + s * 16 * kStep + hi));
        }
        if constexpr (F32) {
            Wide wb[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) wb[j] = widen(fb[j], sb[j]);
#pragma unroll
            for (int s = 0; s < TM; ++s) {
                const Wide wa = widen(fa[s], sa[s]);
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[s][j] = mfma_wide(wb[j], wa, acc[s][j]);
                pin<TN>(acc[s]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < TM; ++s)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[s][j] = mfma_scaled(fb[j], fa[s], acc[s][j], sb[j], sa[s]);
        }
    }
    if (G > 1) {
        __syncthreads();                // every read of the operands is done
        f32x4* const part = reinterpret_cast<f32x4*>(lds);
        constexpr int PerWave = TM * TN * 64;
        if (group > 0) {
#pragma unroll
            for (int s = 0; s < TM; ++s)
#pragma unroll
                for (int j = 0; j < TN; ++j) part[((group - 1) * T::Waves + wave) * PerWave + (s * TN + j) * 64 + lane] = acc[s][j];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int o = 0; o < G - 1; ++o)
#pragma unroll
            for (int s = 0; s < TM; ++s)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[s][j] += part[(o * T::Waves + wave) * PerWave + (s * TN + j) * 64 + lane];
    }
    store_tile<TM, TN, F32>(a, acc, it.mt * T::BM + wm, it.nt * T::BN + wn, it.split, lane);
}

// The sum of the splits' partial products, in their order: bound by memory,
// 4 (splits + 1) bytes an element for fp32.
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
// rows of B; its 16 wavefronts take every 16th step of K with operands
// straight from global memory (B is read once, A stays in L2), and join their
// accumulators in LDS.  The matrix cores have time to spare here, so both
// result types take the exact instruction.  4 x 2560 x 2560: 4.0 us (8
// wavefronts 4.9; four steps' loads ahead 5.0, for want of wavefronts), of
// which an empty launch is about 2.5; 8 x 8192 x 8192: 16.5 us, 4.1 TB/s.
constexpr int kRowWaves = 16;

template <int MT, bool F32>
__global__ void __launch_bounds__(64 * kRowWaves) project_fp8_rows_kernel(const ProjArgs a) {
    __shared__ f32x4 part[kRowWaves][MT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lr = lane & 15;
    const int64_t n0 = (a.first + static_cast<int64_t>(blockIdx.x)) * 16;
    const int64_t br = min(n0 + lr, a.n - 1);
    const uint8_t* const bp = a.b + br * a.ld + 32 * (lane >> 4);
    const uint8_t* const bsp = a.bs + (br >> a.bsh) * a.sld;
    const uint8_t* ap[MT];
    const uint8_t* asp[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t ar = min(static_cast<int64_t>(16 * t + lr), a.m - 1);
        ap[t] = a.a + ar * a.ld + 32 * (lane >> 4);
        asp[t] = a.as + (ar >> a.ash) * a.sld;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int kb = wave; kb < a.steps; kb += kRowWaves) {
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
    for (int t = wave; t < MT; t += kRowWaves) {
        f32x4 v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < kRowWaves; ++w) v += part[w][t][lane];
        const int64_t row = 16 * t + lr, col = n0 + 4 * (lane >> 4);
        if (row < a.m && col < a.n) store4<F32>(a.c, row * a.n + col, v);
    }
}

// ---------------------------------------------------------------------------
// Which kernel, tile and split.
struct Plan {
    int kind;           // 0: few rows; 1: 64 x 64; 2: 128 x 128; 3: 256 x 256 (fp32: 256 x 128); 4: 256 x 320 (bf16 only)
    int splits;
    int split_steps;    // a multiple of 4
};

constexpr int kUnits = 256;     // compute units
constexpr int64_t kRows = 32;   // most rows of A for the few-rows kernel (64 rows: 8.6 us against the small tile's 7.3)

// The tile kernels run one workgroup per compute unit, so a product takes
// ceil(items / 256) rounds of one item's time, and an item's time is nearly a fixed
// part plus a part per step.  Measured on MI355X at 16 to 32768 rows (us, bf16 /
// fp32 result): 64 x 64: 3 + 0.23 / 0.32 a step; 128 x 128: 4 + 0.53 / 0.9;
// the large tiles 8 + 1.5 (256 x 256), 12 + 1.75 (256 x 320), fp32 8 + 1.5.  At 2560 x
// 2560 the large tiles win from about 4000 rows (36 against 45 us), 128 x 128
// from about 600 (1024 rows: 16 against 24).  256 x 320 has the better rate where
// it fills its rounds: 8192 x 2560 x 2560 is one round of 256 tiles, 52 us, or
// 320 tiles of 256 x 256 in two rounds, 69; 32768 rows are four rounds, 181 us,
// or five, 190; but 8192 x 8192 x 8192 is 832 in four rounds, 472 us, or 1024
// in four, 440.  Splitting K pays where tiles are few
// and K is long; it costs a second launch and the partial sums' way through memory.
Plan plan_of(int64_t m, int64_t n, int64_t k, bool f32) {
    const int steps = static_cast<int>(blocks_of(k));
    Plan best{0, 1, (steps + 3) / 4 * 4};
    if (m <= kRows) return best;
    const double fixed[4] = {3, 4, 8, 12}, step16[4] = {0.23, 0.53, 1.5, 1.75}, step32[4] = {0.32, 0.9, 1.5, 0};
    const int64_t rows[4] = {64, 128, 256, 256}, cols[4] = {64, 128, f32 ? 128 : 256, 320};
    double least = 0;
    for (int kind = 1; kind <= (f32 ? 3 : 4); ++kind) {
        const int64_t tiles = ((m + rows[kind - 1] - 1) / rows[kind - 1]) * ((n + cols[kind - 1] - 1) / cols[kind - 1]);
        int before = 0;
        for (int want = 1; want <= 32; ++want) {
            const int per = ((steps + want - 1) / want + 3) / 4 * 4, splits = (steps + per - 1) / per;
            if (splits == before || (splits > 1 && per < 16)) continue;
            before = splits;
            const double rounds = static_cast<double>((tiles * splits + kUnits - 1) / kUnits);
            double us = rounds * (fixed[kind - 1] + (f32 ? step32 : step16)[kind - 1] * std::min(per, steps));
            if (splits > 1) us += 4 + 8e-6 * static_cast<double>(splits) * static_cast<double>(m) * static_cast<double>(n) / 4;
            if (best.kind == 0 || us < least) {
                least = us;
                best = Plan{kind, splits, per};
            }
        }
    }
    return best;
}

// Launches `groups` workgroups, `step` of them a unit, as many at once as a
// launch takes; a.first tells each launch where it begins.
template <class F>
void in_parts(ProjArgs& a, int64_t groups, int threads, int64_t step, F launch) {
    const int64_t most = most_groups(threads) / step * step;
    for (int64_t at = 0; at < groups; at += most) {
        a.first = static_cast<int32_t>(at);
        launch(dim3(static_cast<unsigned>(std::min(most, groups - at))));
    }
}

template <class T>
int launch_tile(ProjArgs& a, hipStream_t st) {
    const int64_t mt = (a.m + T::BM - 1) / T::BM, nt = (a.n + T::BN - 1) / T::BN, items = mt * nt * a.splits;
    if (items > INT32_MAX / 2) return fail(NGRAM_ERANGE, "%lld x %lld too large for one launch", (long long)a.m, (long long)a.n);
    a.ntiles_n = static_cast<int32_t>(nt);
    a.ntiles = static_cast<int32_t>(mt * nt);
    a.band = T::BM >= 256 ? 2 : 8;
    // as many workgroups as the chip holds at once, each with every stride-th
    // item; where an item has fewer steps than there are buffers, an item each
    const int64_t room = kUnits * std::max(1, 160 * 1024 / T::Lds);
    const int64_t least = std::min<int64_t>(a.split_steps, a.steps - (a.splits - 1) * a.split_steps);     // the last split's steps
    const dim3 grid(static_cast<unsigned>(least < 4 ? (items + 7) / 8 * 8 : std::min((items + 7) / 8 * 8, room))), block(T::Threads);
    if (grid.x > most_groups(T::Threads)) return fail(NGRAM_ERANGE, "%lld x %lld too large for one launch", (long long)a.m, (long long)a.n);
    a.stride = static_cast<int32_t>(grid.x);
    hipLaunchKernelGGL((project_fp8_kernel<T>), grid, block, T::Lds, st, a);
    return NGRAM_OK;
}

template <class T>
int launch_small(ProjArgs& a, hipStream_t st) {
    const int64_t mt = (a.m + T::BM - 1) / T::BM, nt = (a.n + T::BN - 1) / T::BN, items = mt * nt * a.splits;
    if (items > INT32_MAX / 2) return fail(NGRAM_ERANGE, "%lld x %lld too large for one launch", (long long)a.m, (long long)a.n);
    a.ntiles_n = static_cast<int32_t>(nt);
    a.ntiles = static_cast<int32_t>(mt * nt);
    a.band = 8;
    in_parts(a, (items + 7) / 8 * 8, T::Threads, 8, [&](dim3 grid) {
        hipLaunchKernelGGL((project_fp8_small_kernel<T>), grid, dim3(T::Threads), T::Lds, st, a);
    });
    return NGRAM_OK;
}

template <int MT>
void launch_rows(ProjArgs& a, bool f32, hipStream_t st) {
    const dim3 block(64 * kRowWaves);
    in_parts(a, (a.n + 15) / 16, 64 * kRowWaves, 1, [&](dim3 grid) {
        if (f32) hipLaunchKernelGGL((project_fp8_rows_kernel<MT, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((project_fp8_rows_kernel<MT, false>), grid, block, 0, st, a);
    });
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

int64_t ngram_project_fp8_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t c_dtype) {
    if (!sizes_ok(m, n, k) || (c_dtype != NGRAM_F32 && c_dtype != NGRAM_BF16)) return -1;
    const Plan p = plan_of(m, n, k, c_dtype == NGRAM_F32);
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
    const bool f32 = c_dtype == NGRAM_F32;
    const Plan p = plan_of(A->rows, B->rows, A->cols, f32);
    const int64_t need = p.splits > 1 ? 4 * p.splits * A->rows * B->rows : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return fail(NGRAM_EINVAL, "workspace must hold %lld bytes, 16-byte aligned", (long long)need);
    const int64_t count = A->rows * B->rows, groups = (count / 4 + 255) / 256;      // of the splits' sum
    if (p.splits > 1 && groups > most_groups(256)) return fail(NGRAM_ERANGE, "C too large for a split of K");
    ProjArgs a;
    a.a = A->codes; a.as = A->scales; a.b = B->codes; a.bs = B->scales; a.c = C;
    a.partial = static_cast<float*>(workspace);
    a.m = A->rows; a.n = B->rows; a.ld = code_ld(A->cols); a.sld = scale_ld(A->cols);
    a.ash = A->block_rows == kBlock ? 7 : 0;
    a.bsh = B->block_rows == kBlock ? 7 : 0;
    a.steps = static_cast<int32_t>(blocks_of(A->cols));
    a.split_steps = p.split_steps; a.splits = p.splits;
    a.ntiles_n = a.ntiles = a.band = a.stride = a.first = 0;
    rc = NGRAM_OK;
    if (p.kind == 0) {
        if (a.m <= 16) launch_rows<1>(a, f32, stream);
        else launch_rows<2>(a, f32, stream);
    } else if (p.kind == 1) {
        rc = f32 ? launch_small<SmallTile<2, 2, 2, 2, 4, true>>(a, stream) : launch_small<SmallTile<2, 2, 2, 2, 4, false>>(a, stream);
    } else if (p.kind == 2) {
        rc = f32 ? launch_small<SmallTile<4, 4, 2, 2, 2, true>>(a, stream) : launch_small<SmallTile<4, 4, 2, 2, 2, false>>(a, stream);
    } else if (p.kind == 3) {
        rc = f32 ? launch_tile<Tile<4, 4, 4, 2, 3, true>>(a, stream) : launch_tile<Tile<8, 4, 2, 4, 2, false>>(a, stream);
    } else {
        rc = launch_tile<Tile<8, 5, 2, 4, 2, false>>(a, stream);
    }
    if (rc) return rc;
    if (a.splits > 1) {
        if (f32) hipLaunchKernelGGL((split_sum_kernel<true>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, stream, a.partial, a.splits, count, C);
        else hipLaunchKernelGGL((split_sum_kernel<false>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, stream, a.partial, a.splits, count, C);
    }
    return hip_status("ngram_project_fp8 launch");
}

}  // extern "C"
