// Distillation from a teacher's top logits for MI355X (gfx950): ngram_distill
// and ngram_distill_grad.  The formulas are in include/ngram.h.  Times in comments are on the
// card: of one kernel, or of a call replayed in a graph.
#include "rows8.h"

#include <algorithm>
#include <cmath>

namespace ng8 {
namespace {

constexpr int kMaxK = NGRAM_DISTILL_MAX_K;
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kBitVectors = 16384;      // vectors of a chunk at most: 16 KB of marks
constexpr int kScan = 128;              // places of a short list
// Gradients above this size are stored past the caches' usual keeping (1021 x 32003 fp32, forward and
// backward: 84 us against 97; 4096 x 151936 bf16 498 against 523); smaller ones are read next where they lie.
constexpr int64_t kStreamFrom = int64_t{64} << 20;

struct RowSums;

struct DistillArgs {
    const void* z;
    const void* t;
    const int32_t* ids;
    const float* teacher_lse;
    float* loss;
    float* stats;           // written by the forward, read by the gradient
    const float* weight;
    void* dz;
    RowSums* part;          // [n][chunks], or NULL: statistics are given
    int64_t n, v, ld, dld;
    float* z_at;            // [n][k]: listed tokens' logits for a loss that is written beside the gradient, or NULL
    int64_t first;          // the launch's first row
    int32_t k, t32;
    int32_t chunks;         // workgroups a row
    int32_t per;            // vectors of a chunk
    float scale;            // of the gradient, without the row's weight and T
    float c;                // log2(e) / T
    float floor;            // -2^20 / c
    double inv_t, t2;       // 1 / T, T^2
};

__device__ __forceinline__ float teacher_at(const DistillArgs& a, int64_t i) {
    return a.t32 ? static_cast<const float*>(a.t)[i]
                 : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.t)[i]) << 16);
}

__device__ __forceinline__ double wave_sum_f64(double x) {
#pragma unroll
    for (int s = 1; s < 64; s *= 2) x += __shfl_xor(x, s);
    return x;
}

// ---------------------------------------------------------------------------
// Sums of exp.  With c = log2(e) / T a set of logits is (m, s): m its largest
// and s the sum of 2^((x - m) c).
//
// A pass over a row holds s as the sum of 2^(x c - R), R = m c rounded to fp32: one
// fused multiply-add and one exp2 an element, each rounded relative to its own size, and 2^(R - m c)
// at the end takes R's rounding off (settled).  That rounding is an exponent of the
// largest element, so m c has to stay small: a thread starts at m = -2^20 / c (the
// floor), so that |m c| is at most 2^20 and the rounding 2^-4 in every thread of a row whose
// largest logit lies within 2^19 / c; a logit below the floor (a masked one of -1e9, say) adds
// exactly 0 to such a row.  Other rows (logits of hundreds of thousands and more
// times T, masked throughout among them) are summed once more by (x - m) c: 4096 x 151936 bf16 with the
// gradient and the rest 521 us, 826 where all rows are.  Without the floor a thread whose
// first vector is masked by -1e10 would hold infinity, to be multiplied with 0 later.
//
// With the teacher's rest the pass leaves listed tokens out and takes the unlisted ones'
// sum about their own largest logit, however far that lies below the row's (in a sum about
// the row's they would be 0 from 87 T on, and log Q -infinity); the listed tokens, a few, are added afterwards.
struct Sums {
    float m, s;
};
struct RowSums {
    Sums all, off;                      // of all tokens; of the unlisted ones, with the rest
};

__device__ __forceinline__ bool usual(float m, float floor) { return fabsf(m) <= -0.5f * floor; }
// What a sum at `from` is multiplied with to be one at `to`; USUAL: at its R.
template <bool USUAL>
__device__ __forceinline__ float rescale(float from, float to, float c) { return USUAL ? exp2_fast(from * c - to * c) : exp2_fast((from - to) * c); }
template <bool USUAL>
__device__ __forceinline__ Sums join(const Sums& x, const Sums& y, float c) {
    const float m = fmaxf(x.m, y.m), f = rescale<USUAL>(x.m, m, c), g = rescale<USUAL>(y.m, m, c);
    return {m, x.s * f + y.s * g};
}
template <bool USUAL>
__device__ __forceinline__ Sums join_wave(const Sums& x, float c) {
    const float m = wave_max(x.m), f = rescale<USUAL>(x.m, m, c);
    return {m, wave_sum(x.s * f)};
}
__device__ __forceinline__ Sums settled(const Sums& t, float c) {
    return {t.m, t.s * exp2_fast(__builtin_fmaf(-t.m, c, t.m * c))};
}

// Adds the elements of G vectors, with REST but for those that have a bit in `listed`.  USUAL:
// x c - R, else (x - m) c.  One rescaling for all of them, and sums by pairs, so
// that few of the instructions wait for each other.
template <bool F32, bool REST, bool USUAL, int G>
__device__ __forceinline__ void add_vectors(Sums& t, const u32x4 (&v)[G], const uint32_t (&listed)[G], float c) {
    constexpr int E = Row<F32>::E;
    float x[G * E];
    float top = t.m;
#pragma unroll
    for (int k = 0; k < G * E; ++k) {
        x[k] = Row<F32>::at(v[k / E], k % E);
        if (REST) x[k] = listed[k / E] & (1u << (k % E)) ? kNegInf : x[k];
        top = fmaxf(top, x[k]);
    }
    const float R = top * c, f = USUAL ? exp2_fast(t.m * c - R) : exp2_fast((t.m - top) * c);
    t.m = top;
#pragma unroll
    for (int k = 0; k < G * E; ++k) x[k] = USUAL ? exp2_fast(__builtin_fmaf(x[k], c, -R)) : exp2_fast((x[k] - top) * c);
#pragma unroll
    for (int n = G * E / 2; n > 0; n /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k) x[k] += x[k + n];
    t.s = __builtin_fmaf(t.s, f, x[0]);
}
template <bool F32, bool REST, bool USUAL>
__device__ __forceinline__ void add_vector(Sums& t, const u32x4& v, uint32_t listed, float c) {
    add_vectors<F32, REST, USUAL, 1>(t, {v}, {listed}, c);
}

// A workgroup's sums joined, in every thread.
template <int WAVES, bool USUAL>
__device__ __forceinline__ Sums join_group(const Sums& x, Sums* room, int lane, int wave, float c) {
    const Sums w = join_wave<USUAL>(x, c);
    if (lane == 0) room[wave] = w;
    __syncthreads();
    Sums t = room[0];
#pragma unroll
    for (int h = 1; h < WAVES; ++h) t = join<USUAL>(t, room[h], c);
    return t;
}
// A row's (or its part's) sums, in every thread: t from the pass over its vectors, or again() of a second
// pass by differences; with REST `on` has this thread's listed tokens (listed_sums).
template <int WAVES, bool REST, typename Again>
__device__ __forceinline__ RowSums finish_sums(const DistillArgs& a, Sums t, Sums on, bool twice, Sums (*room)[WAVES], int lane, int wave, Again again) {
    if (REST) {
        const Sums w = join_wave<false>(on, a.c);
        if (lane == 0) room[2][wave] = w;
    }
    t = join_group<WAVES, true>(t, room[0], lane, wave, a.c);
    if (usual(t.m, a.floor)) t = settled(t, a.c);
    else t = join_group<WAVES, false>(again(), room[1], lane, wave, a.c);
    if (!REST) return {t, {kLowest, 0.0f}};
    on = room[2][0];
    const int holding = twice ? WAVES : min(WAVES, (a.k + 63) / 64);        // wavefronts that hold listed tokens
    for (int h = 1; h < holding; ++h) on = join<false>(on, room[2][h], a.c);
    return {join<false>(on, t, a.c), t};
}

// This thread's vectors of from .. to - 1, kAhead loads at a time in flight;
// the first are asked for before anything else is done.
constexpr int kAhead = 4;
template <bool F32, int THREADS = kThreads>
struct Vectors {
    const Row<F32>& r;
    int i, to, whole;
    u32x4 v[kAhead];
    __device__ __forceinline__ Vectors(const Row<F32>& row, int from, int end)
        : r(row), i(from + static_cast<int>(threadIdx.x)), to(end), whole(min(end, static_cast<int>(row.v / Row<F32>::E))) {
        fetch(i);
    }
    __device__ __forceinline__ void fetch(int at) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (at + u * THREADS < whole) v[u] = r.load_whole(at + u * THREADS);
    }
    // f(vector, its number)
    template <typename F>
    __device__ __forceinline__ void each(F f) {
        while (i < whole) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (i + u * THREADS < whole) f(v[u], i + u * THREADS);
            i += kAhead * THREADS;
            fetch(i);
        }
        if (whole < to && threadIdx.x == THREADS - 1) f(r.load(whole), whole);
    }
};

// ---------------------------------------------------------------------------
// The teacher of a row, by one wavefront: log p = (t - m) / T - log_sum.  m is
// the largest listed logit (0 with a given log sum); log_sum is +inf where
// nothing is listed, so that every p is 0.  t(j) and on(j): place j's logit, and
// whether it names a token.
struct Teacher {
    double m, log_sum;
    __device__ __forceinline__ double log_p(double inv_t, float t) const { return (t - m) * inv_t - log_sum; }
};
template <typename T, typename On>
__device__ __forceinline__ Teacher teacher_of(const DistillArgs& a, int64_t row, int lane, T t, On on) {
    if (a.teacher_lse) return {0, a.teacher_lse[row]};
    float m = kNegInf;
    for (int j = lane; j < a.k; j += 64)
        if (on(j)) m = t(j) == t(j) && m == m ? fmaxf(m, t(j)) : __builtin_nanf("");
    const float top = wave_max(m);
    if (__ballot(m != m)) return {0, __builtin_nan("")};
    if (top == kNegInf) return {0, __builtin_inf()};
    double s = 0;
    for (int j = lane; j < a.k; j += 64)
        if (on(j)) s += exp((static_cast<double>(t(j)) - top) * a.inv_t);
    return {top, log(wave_sum_f64(s))};
}

// Loss and statistics of a row, by one wavefront.  z(j): the student's logit of place j.
template <typename T, typename On, typename Z>
__device__ __forceinline__ void write_loss(const DistillArgs& a, int64_t row, const RowSums& sums, const Teacher& teacher, int lane, T t, On on, Z z) {
    const Sums s = sums.all, off = sums.off;
    const double log_s = log(static_cast<double>(s.s));         // log q = (z - m) / T - log_s
    double sum = 0, mass = 0, log_rest = 0;
    for (int j = lane; j < a.k; j += 64) {
        if (!on(j)) continue;
        const double log_p = teacher.log_p(a.inv_t, t(j)), p = exp(log_p);
        mass += p;
        if (!(p == 0)) sum += p * (log_p - ((static_cast<double>(z(j)) - s.m) * a.inv_t - log_s));
    }
    sum = wave_sum_f64(sum);
    if (a.teacher_lse) {
        const double rest = 1 - wave_sum_f64(mass);
        log_rest = (static_cast<double>(off.m) - s.m) * a.inv_t + (log(static_cast<double>(off.s)) - log_s);
        if (!(rest <= 0)) sum += rest * (log(rest) - log_rest);
    }
    if (lane == 0) {
        // a student that is not a distribution has no loss, also where nothing is listed
        if (a.loss) a.loss[row] = static_cast<float>(log_s - log_s == 0 ? sum * a.t2 : __builtin_nan(""));
        if (a.stats) {
            a.stats[3 * row] = s.s == 0.0f ? kNegInf : s.m;
            a.stats[3 * row + 1] = static_cast<float>(log_s);
            a.stats[3 * row + 2] = static_cast<float>(log_rest);
        }
    }
}
template <bool F32>
__device__ void write_loss_of(const DistillArgs& a, int64_t row, const RowSums& s, int lane) {
    const Row<F32> r(a.z, row * a.ld, a.v);
    const int32_t* const ids = a.ids + row * a.k;
    const auto t = [&](int j) { return teacher_at(a, row * a.k + j); };
    const auto on = [&](int j) { return ids[j] >= 0 && ids[j] < a.v; };
    const Teacher teacher = teacher_of(a, row, lane, t, on);
    write_loss(a, row, s, teacher, lane, t, on, [&](int j) { return r.element(ids[j]); });
}

// Marks of the listed tokens among vectors from .. to - 1 of a row, E bits a
// vector, and whether one of them is listed twice.
template <int E>
__device__ __forceinline__ void mark_listed(const DistillArgs& a, int64_t row, int from, int to, uint32_t* marks, int* twice) {
    const int words = (max(0, to - from) * E + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kThreads) marks[i] = 0;
    if (threadIdx.x == 0) *twice = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += kThreads) {
        const int id = a.ids[row * a.k + j];
        if (id >= 0 && id < a.v && id / E >= from && id / E < to) {
            const uint32_t bit = static_cast<uint32_t>(id - from * E), mask = 1u << (bit & 31);
            if (atomicOr(&marks[bit >> 5], mask) & mask) *twice = 1;
        }
    }
    __syncthreads();
}
template <int E>
__device__ __forceinline__ uint32_t marks_of(const uint32_t* marks, int vector) { return marks[(vector * E) >> 5] >> ((vector * E) & 31); }

// This thread's share of the listed tokens' sum.  Places hold a token each and z(j) is that of
// place j; where some token has several, marked tokens are taken in their order, each once.
template <bool F32, typename On, typename Z>
__device__ __forceinline__ Sums listed_sums(const DistillArgs& a, const Row<F32>& r, const uint32_t* marks, int words, int first, bool twice, On on, Z z) {
    Sums t{kLowest, 0.0f};
    if (!twice) {
        for (int j = threadIdx.x; j < a.k; j += blockDim.x)
            if (on(j)) t = join<false>(t, {z(j), 1.0f}, a.c);
        return t;
    }
    for (int i = threadIdx.x; i < words; i += blockDim.x)
        for (uint32_t bits = marks[i]; bits != 0; bits &= bits - 1) t = join<false>(t, {r.element(first + 32 * i + __builtin_ctz(bits)), 1.0f}, a.c);
    return t;
}

// The sums of a chunk of a row; the row's loss where it is one chunk.  1021 x
// 32003 fp32 with the rest: 28 us, 4.6 TB/s, bound by memory and the marks in LDS.
template <bool F32, bool REST>
__global__ void __launch_bounds__(kThreads) distill_stats_kernel(const DistillArgs a) {
    constexpr int E = Row<F32>::E;
    __shared__ Sums room[3][kWaves];
    __shared__ uint32_t marks[REST ? kBitVectors * E / 32 : 1];
    __shared__ float z_of[REST ? kMaxK : 1];
    __shared__ int twice;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = a.first + blockIdx.x / a.chunks;
    const int chunk = static_cast<int>(blockIdx.x % a.chunks);
    const Row<F32> r(a.z, row * a.ld, a.v);
    const int from = chunk * a.per, to = min(r.vectors(), from + a.per);
    Vectors<F32> mine(r, from, to);
    if (REST) mark_listed<E>(a, row, from, to, marks, &twice);
    const int32_t* const ids = a.ids + row * a.k;
    const auto on = [&](int j) { return ids[j] >= 0 && ids[j] < a.v; };
    const auto here = [&](int j) { return on(j) && ids[j] / E >= from && ids[j] / E < to; };
    Sums t{a.floor, 0.0f}, listed{kLowest, 0.0f};
    mine.each([&](const u32x4& v, int i) { add_vector<F32, REST, true>(t, v, REST ? marks_of<E>(marks, i - from) : 0, a.c); });
    if (REST || a.z_at) {               // behind the loop: the caches have them now.  z_at: the gradient may take the logits' place
        for (int j = threadIdx.x; j < a.k; j += kThreads) {
            if (!here(j)) continue;
            const float z = r.element(ids[j]);
            if (a.z_at) a.z_at[row * a.k + j] = z;
            if (REST) z_of[j] = z;
        }
    }
    if (REST) listed = listed_sums(a, r, marks, ((to - from) * E + 31) / 32, from * E, twice, here, [&](int j) { return z_of[j]; });
    const RowSums sums = finish_sums<kWaves, REST>(a, t, listed, REST && twice, room, lane, wave, [&] {
        Sums u{kLowest, 0.0f};
        Vectors<F32> again(r, from, to);
        again.each([&](const u32x4& v, int i) { add_vector<F32, REST, false>(u, v, REST ? marks_of<E>(marks, i - from) : 0, a.c); });
        return u;
    });
    if (wave != 0) return;
    if (a.chunks > 1) {
        if (lane == 0) a.part[row * a.chunks + chunk] = sums;
    } else if (REST) {
        const auto t_at = [&](int j) { return teacher_at(a, row * a.k + j); };
        write_loss(a, row, sums, teacher_of(a, row, lane, t_at, on), lane, t_at, on, [&](int j) { return z_of[j]; });
    } else {
        write_loss_of<F32>(a, row, sums, lane);
    }
}

template <bool REST>
__device__ __forceinline__ RowSums join_chunks(const DistillArgs& a, int64_t row, int lane) {
    RowSums t{{kLowest, 0.0f}, {kLowest, 0.0f}};
    for (int c = lane; c < a.chunks; c += 64) {
        const RowSums p = a.part[row * a.chunks + c];
        t.all = join<false>(t.all, p.all, a.c);
        if (REST) t.off = join<false>(t.off, p.off, a.c);
    }
    t.all = join_wave<false>(t.all, a.c);
    if (REST) t.off = join_wave<false>(t.off, a.c);
    return t;
}

template <bool F32>
__global__ void __launch_bounds__(256) distill_finish_kernel(const DistillArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = a.first + static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row < a.n) write_loss_of<F32>(a, row, a.teacher_lse ? join_chunks<true>(a, row, lane) : join_chunks<false>(a, row, lane), lane);
}

// ---------------------------------------------------------------------------
// The gradient: gs (a q - p), gs the row's factor.  q = 2^((x - m) c - L), L = log2
// of the sum.  For bf16, whose result rounds by 2^-9, as 2^(x c - K) where |K| < 2^12: K = m c + L as one
// fp32 number, which takes the factor too, and whose rounding of 2^-13 at most is 2^-13.5
// of the result (at 2^16 it would be more than bf16's).
//
// Off the list with the teacher's rest a = 1 - P / Q (1 where P or Q is 0), and a q is (Q - P) times the
// unlisted tokens' own softmax, which stands where Q is too small for a number.
struct Slope {
    float m, L;                     // L = log2 of the sum of 2^((x - m) c)
    float gs, on;                   // the row's factor; a of listed tokens
    float off_m, off_L, factor;     // of other tokens: factor 2^((x - off_m) c - off_L)
};

template <bool F32>
struct Gradient {
    float m, c, L, K, factor;
    uint32_t sign;
    bool zero, wide;
    __device__ __forceinline__ Gradient(const Slope& s, float c_) : m(s.off_m), c(c_), L(s.off_L), factor(s.factor) {
        K = __builtin_fmaf(m, c, L - __builtin_amdgcn_logf(fabsf(factor)));
        // the logarithm of a factor that is neither finite nor positive is no exponent
        wide = F32 || !(fabsf(K) < 4096.0f) || !(fabsf(factor) > 1e-30f && fabsf(factor) < 1e30f);
        sign = factor < 0.0f ? 0x80008000u : 0;
        zero = s.gs == 0.0f;
    }
    __device__ __forceinline__ float q(float x) const { return exp2_fast(__builtin_fmaf(x - m, c, -L)); }
    __device__ __forceinline__ u32x4 of_wide(const u32x4& v) const {
        constexpr int E = Row<F32>::E;
        u32x4 out;
#pragma unroll
        for (int k = 0; k < E; k += 2) {
            const float g0 = q(Row<F32>::at(v, k)) * factor, g1 = q(Row<F32>::at(v, k + 1)) * factor;
            if (F32) {
                out[k & 3] = __float_as_uint(g0);
                out[(k + 1) & 3] = __float_as_uint(g1);
            } else {
                out[(k >> 1) & 3] = bf16_pair(g0, g1);
            }
        }
        return zero ? u32x4{0, 0, 0, 0} : out;
    }
    // where not `wide`
    __device__ __forceinline__ u32x4 of_usual(const u32x4& v) const {
        u32x4 out;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            out[k] = sign ^ bf16_pair(exp2_fast(__builtin_fmaf(Row<F32>::at(v, 2 * k), c, -K)),
                                      exp2_fast(__builtin_fmaf(Row<F32>::at(v, 2 * k + 1), c, -K)));
        return out;
    }
    __device__ __forceinline__ u32x4 of(const u32x4& v) const {
        if (F32) return of_wide(v);
        return wide ? of_wide(v) : of_usual(v);
    }
};

__device__ __forceinline__ float row_factor(const DistillArgs& a, int64_t row) { return (a.weight ? a.weight[row] : 1.0f) * a.scale; }

// Writes a listed token's gradient over what stands there.
template <bool F32>
__device__ __forceinline__ void put_listed(const Row<F32>& w, const Slope& s, float c, int id, float p, float z) {
    const float g = (exp2_fast(__builtin_fmaf(z - s.m, c, -s.L)) * s.on - p) * s.gs;
    char* const at = w.base + static_cast<int64_t>(id) * (F32 ? 4 : 2);
    if (F32) *reinterpret_cast<float*>(at) = g;
    else *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(bf16_pair(g, g));
}
// The same for place j of a list that may name a token twice.
template <bool F32>
__device__ __forceinline__ void write_listed(const Row<F32>& w, const Slope& s, float c, const int32_t* id_of, const float* p_of, int j, int k, int twice,
                                             float z) {
    const int id = id_of[j];
    float p = p_of[j];
    if (twice) {
        double sum = 0;
        for (int e = 0; e < k; ++e) {
            if (id_of[e] != id) continue;
            if (e < j) return;              // the token's first place writes
            sum += p_of[e];
        }
        p = static_cast<float>(sum);
    }
    put_listed<F32>(w, s, c, id, p, z);
}

// Q - P, or Q where there is nothing to share out: no rest, or nobody to take it.
__device__ __forceinline__ float share(float q, double rest, bool nobody) { return rest <= 0 || nobody ? q : static_cast<float>(q - rest); }

// From a row's sums; mass = sum of p.
template <bool REST>
__device__ __forceinline__ Slope slope_of(const DistillArgs& a, float gs, const RowSums& t, double mass) {
    Slope s{t.all.m, __builtin_amdgcn_logf(t.all.s), gs, static_cast<float>(mass), 0, 0, 0};
    s.off_m = s.m;
    s.off_L = s.L;
    s.factor = gs * s.on;
    if (REST) {
        const bool nobody = t.off.s == 0.0f;
        s.on = 1.0f;
        s.off_m = t.off.m;
        s.off_L = nobody ? 0.0f : __builtin_amdgcn_logf(t.off.s);
        s.factor = gs * share(t.off.s / t.all.s * rescale<false>(t.off.m, t.all.m, a.c), 1 - mass, nobody);
    }
    return s;
}
// From the forward's statistics: the unlisted tokens' softmax about the row's largest logit, which loses log Q's
// rounding and its own, as much as log Q is large; from kFar on the row is summed once more, by one
// workgroup (1021 x 32003 fp32 70 us against 44, 24 x 151936 bf16 39 against 8).
constexpr float kFar = -64.0f;
__device__ __forceinline__ bool far_rest(float log_q) { return log_q < kFar && log_q > kNegInf; }
template <bool REST>
__device__ __forceinline__ Slope slope_given(float m, float log_s, float log_q, float q, float gs, double mass) {
    Slope s{m, log_s * kLog2e, gs, static_cast<float>(mass), m, 0, 0};
    s.off_L = s.L;
    s.factor = gs * s.on;
    if (REST) {
        const bool nobody = log_q == kNegInf;
        s.on = 1.0f;
        s.off_L = nobody ? 0.0f : static_cast<float>((static_cast<double>(log_s) + log_q) * 1.4426950408889634074);
        s.factor = gs * share(q, 1 - mass, nobody);
    }
    return s;
}

// The gradient of a chunk of a row, from the forward's statistics or from the
// chunks' sums (then the row's first workgroup writes its loss): a q
// everywhere, then the listed tokens once more.  Their logits are read before anything is
// written, since dz may be z.  1021 x 32003 fp32 with the rest: 47 to 53 us, 5.2 TB/s,
// bound by memory; of few rows (24 x 151936 bf16, 8 us) by the teacher's fp64 side,
// which every chunk computes.
template <bool F32, bool REST, bool STREAM>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const DistillArgs a) {
    constexpr int E = Row<F32>::E;
    __shared__ uint32_t marks[kBitVectors * E / 32];
    __shared__ int32_t id_of[kMaxK];
    __shared__ float p_of[kMaxK];
    __shared__ int twice;
    __shared__ Teacher teacher_;
    __shared__ double mass_;
    __shared__ RowSums sums_;
    __shared__ float stats_[4];                 // with Q
    __shared__ Sums room[kWaves];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = a.first + blockIdx.x / a.chunks;
    const int chunk = static_cast<int>(blockIdx.x % a.chunks);
    const Row<F32> r(a.z, row * a.ld, a.v), w(a.dz, row * a.dld, a.v);
    int from = chunk * a.per, to = min(w.vectors(), from + a.per);
    Vectors<F32> mine(r, from, to);
    const int32_t* const ids = a.ids + row * a.k;
    const auto t_at = [&](int j) { return teacher_at(a, row * a.k + j); };
    const auto on = [&](int j) { return ids[j] >= 0 && ids[j] < a.v; };
    if (wave == 0) {
        const Teacher teacher = teacher_of(a, row, lane, t_at, on);
        double mass = 0;
        for (int j = lane; j < a.k; j += 64)
            if (on(j)) mass += exp(teacher.log_p(a.inv_t, t_at(j)));
        mass = wave_sum_f64(mass);
        if (lane == 0) {
            teacher_ = teacher;
            mass_ = mass;
        }
    } else if (wave == 1) {
        if (a.part) {
            const RowSums sums = join_chunks<REST>(a, row, lane);
            if (lane == 0) sums_ = sums;
        } else if (lane < 3) {
            const float x = a.stats[3 * row + lane];
            stats_[lane] = x;
            if (REST && lane == 2) stats_[3] = static_cast<float>(exp(static_cast<double>(x)));
        }
    }
    if (a.k > kScan) {
        mark_listed<E>(a, row, from, to, marks, &twice);
    } else {
        if (threadIdx.x == 0) twice = 0;
        __syncthreads();
    }
    const float gs = row_factor(a, row);
    Slope s = a.part ? slope_of<REST>(a, gs, sums_, mass_) : slope_given<REST>(stats_[0], stats_[1], stats_[2], stats_[3], gs, mass_);
    const bool far = REST && !a.part && far_rest(stats_[2]);
    if (far) {                                  // the row is its first workgroup's: others must not write what that one reads
        if (chunk != 0) return;
        from = 0;
        to = w.vectors();
    }
    const Teacher teacher = teacher_;
    // this thread's listed tokens
    constexpr int PER = kMaxK / kThreads;
    float listed[PER];
    bool write[PER];
#pragma unroll
    for (int h = 0; h < PER; ++h) {
        const int j = threadIdx.x + h * kThreads;
        write[h] = false;
        if (j >= a.k) continue;
        const int id = ids[j];
        const bool here = id >= 0 && id < a.v && id / E >= from && id / E < to && s.gs != 0.0f;
        id_of[j] = here ? id : -1;
        p_of[j] = here ? static_cast<float>(exp(teacher.log_p(a.inv_t, t_at(j)))) : 0.0f;
        write[h] = here;
        if (here) listed[h] = r.element(id);
    }
    __syncthreads();
    if (a.k <= kScan && write[0]) {             // a short list is compared place by place
        for (int e = 0; e < static_cast<int>(threadIdx.x); ++e)
            if (id_of[e] == id_of[threadIdx.x]) twice = 1;
    }
    if (far) {
        Sums t{kLowest, 0.0f};
        for (int at = 0; at < to; at += kBitVectors) {
            const int end = min(to, at + kBitVectors);
            __syncthreads();                    // marks and `twice` of before are read
            mark_listed<E>(a, row, at, end, marks, &twice);
            for (int i = at + static_cast<int>(threadIdx.x); i < end; i += kThreads)
                add_vector<F32, true, false>(t, r.load(i), marks_of<E>(marks, i - at), a.c);
        }
        t = join_group<kWaves, false>(t, room, lane, wave, a.c);
        s.off_m = t.m;
        s.off_L = __builtin_amdgcn_logf(t.s);
        if (threadIdx.x == 0) twice = 1;        // in one of the ranges or not
        const Gradient<F32> g(s, a.c);
        Vectors<F32> all(r, from, to);
        all.each([&](const u32x4& v, int i) { w.template put<STREAM>(i, g.of(v)); });
    } else {
        const Gradient<F32> g(s, a.c);
        mine.each([&](const u32x4& v, int i) { w.template put<STREAM>(i, g.of(v)); });
    }
    // what was stored above has arrived before it is written over
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < PER; ++h)
        if (write[h]) write_listed<F32>(w, s, a.c, id_of, p_of, threadIdx.x + h * kThreads, a.k, twice, listed[h]);
    if (a.part && chunk == 0 && wave == kWaves - 1)
        write_loss(a, row, sums_, teacher, lane, t_at, on, [&](int j) { return a.z_at[row * a.k + j]; });
}

// ---------------------------------------------------------------------------
// Loss and gradient in one pass over memory: a row's vectors stay in registers
// (NV a thread) between its sums and its gradient.
// A row in registers between both would read memory once, but leaves eight
// wavefronts a compute unit: 4096 x 151936 bf16 took 546 us with all of a row in
// registers (512 threads, 38 vectors each), 560 as one stream that asks for the next row as it stores this
// one, 586 with nothing kept (read twice, from the last-level cache the second time); 1024 threads with 14
// vectors each and the rest read again 496.  Rows of up to 6144 vectors fit whole: 512 threads, two or three
// workgroups a unit (4096 x 32003 bf16 140 us, with 1024 threads 198); up to 2048 with a third of the registers
// (4096 x 5003 bf16 43 us, 61 with all).
constexpr int kRowMarks = 1 << 18;      // tokens of a row at most

// The teacher's side is one wavefront's work while the row's loads are on
// their way.  Vectors beyond those in registers are read again.
template <bool F32, bool REST, bool STREAM, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS) distill_row_kernel(const DistillArgs a) {
    constexpr int E = Row<F32>::E;
    extern __shared__ uint32_t marks[];                 // v / 32 + 1
    __shared__ Sums room[3][THREADS / 64];
    __shared__ int32_t id_of[kMaxK];
    __shared__ float t_of[kMaxK], z_of[kMaxK], p_of[kMaxK];
    __shared__ int twice;
    __shared__ Teacher teacher_;
    __shared__ double mass_;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row = a.first + blockIdx.x;
    const Row<F32> r(a.z, row * a.ld, a.v), w(a.dz, row * a.dld, a.v);
    const int whole = static_cast<int>(a.v) / E, vectors = r.vectors();
    u32x4 raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (tid < whole - j * THREADS) raw[j] = r.load_whole(tid + j * THREADS);
    for (int i = tid; i < static_cast<int>(a.v) / 32 + 1; i += THREADS) marks[i] = 0;
    if (tid == 0) twice = 0;
    for (int j = tid; j < a.k; j += THREADS) {
        const int id = a.ids[row * a.k + j];
        const bool on = id >= 0 && id < a.v;
        id_of[j] = on ? id : -1;
        t_of[j] = teacher_at(a, row * a.k + j);
        z_of[j] = on ? r.element(id) : 0.0f;
    }
    __syncthreads();
    for (int j = tid; j < a.k; j += THREADS) {
        const int id = id_of[j];
        if (id < 0) continue;
        const uint32_t mask = 1u << (id & 31);
        if (atomicOr(&marks[id >> 5], mask) & mask) twice = 1;
    }
    if (REST) __syncthreads();
    const auto t_at = [&](int j) { return t_of[j]; };
    const auto on = [&](int j) { return id_of[j] >= 0; };
    if (wave == 0) {
        const Teacher teacher = teacher_of(a, row, lane, t_at, on);
        double mass = 0;
        for (int j = lane; j < a.k; j += 64) {
            const double p = on(j) ? exp(teacher.log_p(a.inv_t, t_of[j])) : 0;
            mass += p;
            p_of[j] = static_cast<float>(p);
        }
        mass = wave_sum_f64(mass);
        if (lane == 0) {
            teacher_ = teacher;
            mass_ = mass;
        }
    }
    Sums t{a.floor, 0.0f}, listed{kLowest, 0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (tid < whole - j * THREADS) add_vector<F32, REST, true>(t, raw[j], REST ? marks_of<E>(marks, tid + j * THREADS) : 0, a.c);
    Vectors<F32, THREADS> beyond(r, NV * THREADS, vectors);
    beyond.each([&](const u32x4& v, int i) { add_vector<F32, REST, true>(t, v, REST ? marks_of<E>(marks, i) : 0, a.c); });
    if (REST) listed = listed_sums(a, r, marks, static_cast<int>(a.v) / 32 + 1, 0, twice, on, [&](int j) { return z_of[j]; });
    const RowSums sums = finish_sums<THREADS / 64, REST>(a, t, listed, REST && twice, room, lane, wave, [&] {
        Sums u{kLowest, 0.0f};
        for (int i = tid; i < vectors; i += THREADS) add_vector<F32, REST, false>(u, r.load(i), REST ? marks_of<E>(marks, i) : 0, a.c);
        return u;
    });
    if (wave == 0) write_loss(a, row, sums, teacher_, lane, t_at, on, [&](int j) { return z_of[j]; });
    const Slope s = slope_of<REST>(a, row_factor(a, row), sums, mass_);
    const Gradient<F32> g(s, a.c);
    if (!F32 && g.wide) {                               // rare, and short
        for (int i = tid; i < min(whole, NV * THREADS); i += THREADS) w.store_whole(i, g.of_wide(r.load_whole(i)));
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (tid < whole - j * THREADS) w.template put<STREAM>(tid + j * THREADS, F32 ? g.of_wide(raw[j]) : g.of_usual(raw[j]));
    }
    Vectors<F32, THREADS> again(r, NV * THREADS, vectors);
    again.each([&](const u32x4& v, int i) { w.template put<STREAM>(i, g.of(v)); });
    if (s.gs == 0.0f) return;
    // what was stored above has arrived before it is written over
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int j = tid; j < a.k; j += THREADS)
        if (id_of[j] >= 0) write_listed<F32>(w, s, a.c, id_of, p_of, j, a.k, twice, z_of[j]);
}

// Workgroups a row: one where rows fill the card; few rows are cut into parts
// of 512 vectors and more, for 512 workgroups.  (24 x 151936 bf16 with the gradient, 15.1 us now, was 15.7, for 1024 workgroups 20.0,
// for 256 15.2; 96 rows 24, 29 and 26.  Parts of 256 vectors: 16 rows 16.4 against 14.2.)
int chunks_of(int64_t n, int64_t v, int dtype) {
    const int64_t e = dtype == NGRAM_F32 ? 4 : 8, vectors = (v + e - 1) / e;
    const int64_t want = 512 / std::max<int64_t>(n, 1);
    return static_cast<int>(std::max<int64_t>((vectors + kBitVectors - 1) / kBitVectors, std::min<int64_t>(want, vectors / 512)));
}

int check_args(const ngram_distill_args* p) {
    if (!p) return fail(NGRAM_EINVAL, "the arguments are NULL");
    if (p->n < 0 || p->k < 1) return fail(NGRAM_EINVAL, "n=%lld must not be negative and k=%d at least 1", (long long)p->n, p->k);
    if ((p->dtype != NGRAM_F32 && p->dtype != NGRAM_BF16) || (p->teacher_dtype != NGRAM_F32 && p->teacher_dtype != NGRAM_BF16))
        return fail(NGRAM_EINVAL, "dtype=%d or teacher_dtype=%d is not an ngram_value", p->dtype, p->teacher_dtype);
    if (p->k > NGRAM_DISTILL_MAX_K || p->V < 1 || p->V > NGRAM_FP8_MAX || p->n > NGRAM_FP8_MAX)
        return fail(NGRAM_ERANGE, "k=%d (to %d), V=%lld or n=%lld (to 2^30) out of range", p->k, NGRAM_DISTILL_MAX_K, (long long)p->V, (long long)p->n);
    if (p->ld < p->V) return fail(NGRAM_EINVAL, "ld=%lld is below V=%lld", (long long)p->ld, (long long)p->V);
    if (!(p->temperature >= 0x1p-120f) || std::isinf(p->temperature))
        return fail(NGRAM_EINVAL, "temperature=%g must be finite and at least 2^-120", p->temperature);
    if (p->n == 0) return NGRAM_OK;
    if (!p->logits || !p->teacher || !p->ids) return fail(NGRAM_EINVAL, "logits, teacher or ids is NULL");
    const uintptr_t ze = p->dtype == NGRAM_F32 ? 4 : 2, te = p->teacher_dtype == NGRAM_F32 ? 4 : 2;
    if (!aligned(p->logits, ze) || !aligned(p->teacher, te) || !aligned(p->ids, 4) || !aligned(p->teacher_lse, 4))
        return fail(NGRAM_EALIGN, "an argument is not aligned to its elements");
    return NGRAM_OK;
}

// Whether rows of dz share bytes with rows of z: two ranges that meet share some unless their rows lie as far apart, each
// in the gaps of the other's.
bool overlap(const ngram_distill_args* p, const void* dz, int64_t dld) {
    const __int128 e = p->dtype == NGRAM_F32 ? 4 : 2, row = p->V * e, ld = p->ld * e, dl = dld * e, n = p->n;
    const __int128 off = static_cast<__int128>(reinterpret_cast<uintptr_t>(dz)) - static_cast<__int128>(reinterpret_cast<uintptr_t>(p->logits));
    if (off >= (n - 1) * ld + row || -off >= (n - 1) * dl + row) return false;
    if (n == 1 || ld != dl) return true;
    const __int128 at = (off % ld + ld) % ld;
    return at < row || ld - at < row;
}

int check_grad(const ngram_distill_args* p, const float* weight, float scale, const void* dz, int64_t dld) {
    if (dld < p->V) return fail(NGRAM_EINVAL, "dld=%lld is below V=%lld", (long long)dld, (long long)p->V);
    if (dz && dz == p->logits && dld != p->ld) return fail(NGRAM_EINVAL, "dlogits_out takes logits' place, but dld=%lld is not ld=%lld", (long long)dld, (long long)p->ld);
    if (!std::isfinite(scale)) return fail(NGRAM_EINVAL, "scale=%g must be finite", scale);
    if (!aligned(dz, p->dtype == NGRAM_F32 ? 4 : 2) || !aligned(weight, 4)) return fail(NGRAM_EALIGN, "dlogits_out or weight is not aligned to its elements");
    // workgroups read a row while others write theirs
    if (p->n > 0 && dz && dz != p->logits && overlap(p, dz, dld)) return fail(NGRAM_EINVAL, "dlogits_out overlaps logits without being logits");
    return NGRAM_OK;
}

DistillArgs device_args(const ngram_distill_args* p) {
    DistillArgs a = {};
    a.z = p->logits; a.t = p->teacher; a.ids = p->ids; a.teacher_lse = p->teacher_lse;
    a.n = p->n; a.v = p->V; a.ld = p->ld; a.k = p->k; a.t32 = p->teacher_dtype == NGRAM_F32;
    a.inv_t = 1.0 / p->temperature;
    a.t2 = static_cast<double>(p->temperature) * p->temperature;
    a.c = static_cast<float>(1.4426950408889634074 * a.inv_t);
    a.floor = static_cast<float>(-std::min(0x1p20 / a.c, static_cast<double>(kLowest) * -1));
    a.chunks = chunks_of(p->n, p->V, p->dtype);
    const int64_t e = p->dtype == NGRAM_F32 ? 4 : 8, vectors = (p->V + e - 1) / e;
    a.per = static_cast<int32_t>((vectors + a.chunks - 1) / a.chunks);
    a.per = (a.per + 7) / 8 * 8;                                            // whole words of marks
    a.chunks = static_cast<int32_t>((vectors + a.per - 1) / a.per);         // which may leave fewer: a row's last chunk has its last vector
    return a;
}

// Launches over all units of `rows_a_unit` rows, `per_row` workgroups each.
template <typename L>
void over_rows(DistillArgs a, int64_t units, int64_t per_row, int threads, int64_t rows_a_unit, L launch) {
    const int64_t most = std::max<int64_t>(1, most_groups(threads) / per_row);
    for (int64_t u = 0; u < units; u += most) {
        a.first = u * rows_a_unit;
        launch(a, dim3(static_cast<uint32_t>(std::min(most, units - u) * per_row)));
    }
}

bool streams(const DistillArgs& a, bool f32) { return a.n * a.v * (f32 ? 4 : 2) > kStreamFrom; }

template <bool F32, bool REST>
void launch_grad_of(const DistillArgs& a, hipStream_t st) {
    over_rows(a, a.n, a.chunks, kThreads, 1, [&](const DistillArgs& b, dim3 grid) {
        if (streams(a, F32)) hipLaunchKernelGGL((distill_grad_kernel<F32, REST, true>), grid, dim3(kThreads), 0, st, b);
        else hipLaunchKernelGGL((distill_grad_kernel<F32, REST, false>), grid, dim3(kThreads), 0, st, b);
    });
}
void launch_grad(const DistillArgs& a, bool f32, hipStream_t st) {
    if (f32 && a.teacher_lse) launch_grad_of<true, true>(a, st);
    else if (f32) launch_grad_of<true, false>(a, st);
    else if (a.teacher_lse) launch_grad_of<false, true>(a, st);
    else launch_grad_of<false, false>(a, st);
}

// Rows in one workgroup each, loss and gradient in one launch: short ones, or enough of them to fill the card, and
// short enough for the marks.  us, so and apart: 1 x 1001 bf16 6.2 and 13.3, 1 x 32003 fp32 9.2 and 11.9, 256 x 32003
// bf16 14.0 and 27, 200 x 151936 bf16 36 and 46, 128 x 151936 fp32 37, 120 of them apart 41; but 24 x 151936 bf16 22
// and 15, 96 of them 27 and 23.
bool whole_rows(const DistillArgs& a, int64_t e) { return a.v <= kRowMarks && (a.v <= 8192 * e || a.n >= 128); }

template <bool F32, bool REST, bool STREAM, int THREADS, int NV>
void launch_row(const DistillArgs& a, hipStream_t st) {
    const uint32_t lds = static_cast<uint32_t>((a.v / 32 + 1) * 4);
    over_rows(a, a.n, 1, THREADS, 1, [&](const DistillArgs& b, dim3 grid) {
        hipLaunchKernelGGL((distill_row_kernel<F32, REST, STREAM, THREADS, NV>), grid, dim3(THREADS), lds, st, b);
    });
}
template <bool F32, bool REST, bool STREAM>
void launch_rows_of(const DistillArgs& a, hipStream_t st) {
    const int64_t vectors = a.v / Row<F32>::E;
    if (vectors <= 4 * 512) launch_row<F32, REST, STREAM, 512, 4>(a, st);
    else if (vectors <= 12 * 512) launch_row<F32, REST, STREAM, 512, 12>(a, st);
    else launch_row<F32, REST, STREAM, 1024, 14>(a, st);
}
template <bool F32, bool REST>
void launch_rows(const DistillArgs& a, hipStream_t st) {
    if (streams(a, F32)) launch_rows_of<F32, REST, true>(a, st);
    else launch_rows_of<F32, REST, false>(a, st);
}

// Bytes of a workspace: the chunks' sums, statistics that the caller does not
// ask for, and the listed tokens' logits.
struct Room {
    int64_t part, stats, z_at, total;
};
Room room_of(int64_t n, int64_t v, int64_t k, int dtype) {
    DistillArgs a = {};
    a.n = n;
    a.v = v;
    Room r;
    const auto round = [](int64_t b) { return (b + 15) / 16 * 16; };
    const int64_t chunks = chunks_of(n, v, dtype);
    r.part = 0;
    r.stats = chunks > 1 ? round(n * chunks * static_cast<int64_t>(sizeof(RowSums))) : 0;
    r.z_at = r.stats + round(n * 12);
    r.total = r.z_at + (chunks > 1 ? round(n * k * 4) : 0);
    return r;
}

}  // namespace
}  // namespace ng8

using namespace ng8;

extern "C" {

int64_t ngram_distill_workspace_bytes(int64_t n, int64_t V, int32_t k, int32_t dtype) {
    if (n < 0 || n > NGRAM_FP8_MAX || V < 1 || V > NGRAM_FP8_MAX || k < 1 || k > NGRAM_DISTILL_MAX_K || (dtype != NGRAM_F32 && dtype != NGRAM_BF16))
        return -1;
    return room_of(n, V, k, dtype).total;
}

int ngram_distill(const ngram_distill_args* p, float* loss_out, float* stats_out, const float* weight, float scale,
                  void* dlogits_out, int64_t dld, void* workspace, int64_t workspace_bytes, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    int rc = check_args(p);
    if (rc) return rc;
    if (p->n > 0 && !loss_out && !stats_out && !dlogits_out) return fail(NGRAM_EINVAL, "loss_out, stats_out and dlogits_out are NULL");
    if (!aligned(loss_out, 4) || !aligned(stats_out, 4)) return fail(NGRAM_EALIGN, "loss_out and stats_out must be 4-byte aligned");
    if (dlogits_out && (rc = check_grad(p, weight, scale, dlogits_out, dld))) return rc;
    if (p->n == 0) return NGRAM_OK;
    DistillArgs a = device_args(p);
    const Room room = room_of(a.n, a.v, a.k, p->dtype);
    if (!workspace || workspace_bytes < room.total || !aligned(workspace, 16))
        return fail(NGRAM_EINVAL, "workspace must hold %lld bytes, 16-byte aligned", (long long)room.total);
    char* const at = static_cast<char*>(workspace);
    a.loss = loss_out;
    a.part = reinterpret_cast<RowSums*>(at + room.part);
    a.stats = stats_out ? stats_out : reinterpret_cast<float*>(at + room.stats);
    a.weight = weight; a.scale = static_cast<float>(static_cast<double>(scale) * p->temperature); a.dz = dlogits_out; a.dld = dld;
    const bool f32 = p->dtype == NGRAM_F32;
    if (dlogits_out && whole_rows(a, f32 ? 4 : 8)) {
        if (f32 && a.teacher_lse) launch_rows<true, true>(a, stream);
        else if (f32) launch_rows<true, false>(a, stream);
        else if (a.teacher_lse) launch_rows<false, true>(a, stream);
        else launch_rows<false, false>(a, stream);
        return hip_status("ngram_distill");
    }
    if (dlogits_out && a.chunks > 1) a.z_at = reinterpret_cast<float*>(at + room.z_at);
    over_rows(a, a.n, a.chunks, kThreads, 1, [&](const DistillArgs& b, dim3 grid) {
        const dim3 block(kThreads);
        if (f32 && b.teacher_lse) hipLaunchKernelGGL((distill_stats_kernel<true, true>), grid, block, 0, stream, b);
        else if (f32) hipLaunchKernelGGL((distill_stats_kernel<true, false>), grid, block, 0, stream, b);
        else if (b.teacher_lse) hipLaunchKernelGGL((distill_stats_kernel<false, true>), grid, block, 0, stream, b);
        else hipLaunchKernelGGL((distill_stats_kernel<false, false>), grid, block, 0, stream, b);
    });
    if (a.chunks > 1 && !dlogits_out) over_rows(a, (a.n + 3) / 4, 1, 256, 4, [&](const DistillArgs& b, dim3 grid) {
        if (f32) hipLaunchKernelGGL(distill_finish_kernel<true>, grid, dim3(256), 0, stream, b);
        else hipLaunchKernelGGL(distill_finish_kernel<false>, grid, dim3(256), 0, stream, b);
    });
    if (dlogits_out) {
        if (a.chunks == 1) a.part = nullptr;        // the loss and the statistics are there
        launch_grad(a, f32, stream);
    }
    return hip_status("ngram_distill");
}

int ngram_distill_grad(const ngram_distill_args* p, const float* stats, const float* weight, float scale, void* dlogits_out,
                       int64_t dld, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    int rc = check_args(p);
    if (rc) return rc;
    if ((rc = check_grad(p, weight, scale, dlogits_out, dld))) return rc;
    if (p->n == 0) return NGRAM_OK;
    if (!stats || !dlogits_out) return fail(NGRAM_EINVAL, "stats or dlogits_out is NULL");
    if (!aligned(stats, 4)) return fail(NGRAM_EALIGN, "stats must be 4-byte aligned");
    DistillArgs a = device_args(p);
    a.stats = const_cast<float*>(stats);
    a.weight = weight; a.scale = static_cast<float>(static_cast<double>(scale) * p->temperature); a.dz = dlogits_out; a.dld = dld;
    launch_grad(a, p->dtype == NGRAM_F32, stream);
    return hip_status("ngram_distill_grad");
}

}  // extern "C"
