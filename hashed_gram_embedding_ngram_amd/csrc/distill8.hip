// Distillation from a teacher's top logits for MI355X (gfx950): ngram_distill
// and ngram_distill_grad.  The formulas are in include/ngram.h.
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

struct DistillArgs {
    const void* z;
    const void* t;
    const int32_t* ids;
    const float* teacher_lse;
    float* loss;
    float* stats;           // written by the forward, read by the gradient
    const float* weight;
    void* dz;
    Soft* part;             // [n][chunks][2]: the whole row's, and the unlisted tokens'
    int64_t n, v, ld, dld;
    int64_t first;          // the launch's first row
    int32_t k, t32;
    int32_t chunks;         // workgroups a row
    int32_t per;            // vectors of a chunk
    float scale;            // of the gradient, without the row's weight and T
    float c;                // log2(e) / T
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

// The teacher of a row, by one wavefront: log p = (t - m) / T - log_sum.  m is
// the largest listed logit (0 with a given log sum); log_sum +inf where nothing
// is listed (every p is 0).
struct Teacher {
    double m, log_sum;
    __device__ __forceinline__ double log_p(const DistillArgs& a, int64_t i) const { return (teacher_at(a, i) - m) * a.inv_t - log_sum; }
};
__device__ Teacher teacher_of(const DistillArgs& a, int64_t row, int lane) {
    if (a.teacher_lse) return {0, a.teacher_lse[row]};
    float m = kNegInf;
    for (int j = lane; j < a.k; j += 64) {
        const int id = a.ids[row * a.k + j];
        const float t = teacher_at(a, row * a.k + j);
        if (id >= 0 && id < a.v) m = t == t && m == m ? fmaxf(m, t) : __builtin_nanf("");
    }
    const float top = wave_max(m);
    if (__ballot(m != m)) return {0, __builtin_nan("")};
    if (top == kNegInf) return {0, __builtin_inf()};
    double s = 0;
    for (int j = lane; j < a.k; j += 64) {
        const int id = a.ids[row * a.k + j];
        if (id >= 0 && id < a.v) s += exp((static_cast<double>(teacher_at(a, row * a.k + j)) - top) * a.inv_t);
    }
    return {top, log(wave_sum_f64(s))};
}

// Marks of the listed tokens among vectors from .. to - 1 of a row, E bits a
// vector, and whether one of them is listed twice.
template <int E>
__device__ __forceinline__ void mark_listed(const DistillArgs& a, int64_t row, int from, int to, uint32_t* marks, int* twice) {
    const int words = (max(0, to - from) * E + 31) / 32;
    for (int i = threadIdx.x; i < words; i += blockDim.x) marks[i] = 0;
    if (threadIdx.x == 0) *twice = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < a.k; j += blockDim.x) {
        const int id = a.ids[row * a.k + j];
        if (id >= 0 && id < a.v && id / E >= from && id / E < to) {
            const uint32_t bit = static_cast<uint32_t>(id - from * E), mask = 1u << (bit & 31);
            if (atomicOr(&marks[bit >> 5], mask) & mask) *twice = 1;
        }
    }
    __syncthreads();
}

// Maximum and sum of a chunk of a row, and, with the teacher's rest, the same
// of the tokens that are not listed.
template <bool F32, bool REST>
__global__ void __launch_bounds__(kThreads) distill_stats_kernel(const DistillArgs a) {
    constexpr int E = Row<F32>::E;
    __shared__ Soft joined[2][kWaves];
    __shared__ uint32_t marks[REST ? kBitVectors * E / 32 : 1];
    __shared__ int twice;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = a.first + blockIdx.x / a.chunks;
    const int chunk = static_cast<int>(blockIdx.x % a.chunks);
    const Row<F32> r(a.z, row * a.ld, a.v);
    const int from = chunk * a.per, to = min(r.vectors(), from + a.per);
    if (REST) mark_listed<E>(a, row, from, to, marks, &twice);
    Soft all{kLowest, 0.0f};
    float off = 0.0f;                   // the unlisted tokens' part of the sum, at the same maximum
    for (int i = from + static_cast<int>(threadIdx.x); i < to; i += kThreads) {
        const u32x4 raw = r.load(i);
        float x[E];
        float top = kNegInf;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            x[k] = Row<F32>::at(raw, k);
            top = fmaxf(top, x[k]);
        }
        const float m = fmaxf(all.m, top);
        const float f = exp2_fast((all.m - m) * a.c);
        all.s *= f;
        off *= f;
        all.m = m;
        if (!REST) {
#pragma unroll
            for (int k = 0; k < E; ++k) all.s += exp2_fast((x[k] - m) * a.c);
        } else {
            const int b = (i - from) * E;
            const uint32_t listed = marks[b >> 5] >> (b & 31);
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float e = exp2_fast((x[k] - m) * a.c);
                all.s += e;
                off += listed & (1u << k) ? 0.0f : e;
            }
        }
    }
    const float m = wave_max(all.m), f = exp2_fast((all.m - m) * a.c);
    all.s = wave_sum(all.s * f);
    if (REST) off = wave_sum(off * f);
    if (lane == 0) {
        joined[0][wave] = {m, all.s};
        joined[1][wave] = {m, off};
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        Soft* const out = a.part + (row * a.chunks + chunk) * 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Soft s = joined[h][0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) s = soft_join(s, joined[h][w], a.c);
            out[h] = s;
        }
    }
}

// Loss and statistics of a row, by one wavefront.
template <bool F32>
__device__ void finish_row(const DistillArgs& a, int64_t row, Soft all, Soft off, int lane) {
    const double log_s = log(static_cast<double>(all.s));       // log q = (z - all.m) / T - log_s
    const Teacher t = teacher_of(a, row, lane);
    const Row<F32> r(a.z, row * a.ld, a.v);
    double sum = 0, mass = 0;
    for (int j = lane; j < a.k; j += 64) {
        const int id = a.ids[row * a.k + j];
        if (id < 0 || id >= a.v) continue;
        const double log_p = t.log_p(a, row * a.k + j), p = exp(log_p);
        mass += p;
        if (!(p == 0)) sum += p * (log_p - ((static_cast<double>(r.element(id)) - all.m) * a.inv_t - log_s));
    }
    sum = wave_sum_f64(sum);
    double log_rest = 0;
    if (a.teacher_lse) {
        const double rest = 1 - wave_sum_f64(mass);
        log_rest = (static_cast<double>(off.m) - all.m) * a.inv_t + log(static_cast<double>(off.s)) - log_s;
        if (!(rest <= 0)) sum += rest * (log(rest) - log_rest);
    }
    if (lane == 0) {
        // a student that is not a distribution has no loss, also where nothing is listed
        if (a.loss) a.loss[row] = static_cast<float>(log_s - log_s == 0 ? sum * a.t2 : __builtin_nan(""));
        if (a.stats) {
            a.stats[3 * row] = all.s == 0.0f ? kNegInf : all.m;
            a.stats[3 * row + 1] = static_cast<float>(log_s);
            a.stats[3 * row + 2] = static_cast<float>(log_rest);
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(256) distill_finish_kernel(const DistillArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t row = a.first + static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= a.n) return;
    Soft all{kLowest, 0.0f}, off{kLowest, 0.0f};
    for (int c = lane; c < a.chunks; c += 64) {
        const Soft* const p = a.part + (row * a.chunks + c) * 2;
        all = soft_join(all, p[0], a.c);
        off = soft_join(off, p[1], a.c);
    }
    all = soft_wave(all, a.c);
    off = soft_wave(off, a.c);
    finish_row<F32>(a, row, all, off, lane);
}

// The gradient of a chunk of a row: a q everywhere, then the listed tokens
// once more.  Their logits are read before anything is written, since dz may be z.
template <bool F32, bool REST>
__global__ void __launch_bounds__(kThreads) distill_grad_kernel(const DistillArgs a) {
    constexpr int E = Row<F32>::E;
    __shared__ uint32_t marks[kBitVectors * E / 32];
    __shared__ int32_t id_of[kMaxK];
    __shared__ float p_of[kMaxK];
    __shared__ int twice;
    __shared__ Teacher teacher;
    __shared__ double mass_;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = a.first + blockIdx.x / a.chunks;
    const int chunk = static_cast<int>(blockIdx.x % a.chunks);
    const Row<F32> r(a.z, row * a.ld, a.v), w(a.dz, row * a.dld, a.v);
    const float gs = (a.weight ? a.weight[row] : 1.0f) * a.scale;
    const int from = chunk * a.per, to = min(w.vectors(), from + a.per);
    if (gs == 0.0f) {
        for (int i = from + static_cast<int>(threadIdx.x); i < to; i += kThreads) w.store(i, u32x4{0, 0, 0, 0});
        return;
    }
    if (wave == 0) {
        const Teacher t = teacher_of(a, row, lane);
        double mass = 0;
        for (int j = lane; j < a.k; j += 64) {
            const int id = a.ids[row * a.k + j];
            if (id >= 0 && id < a.v) mass += exp(t.log_p(a, row * a.k + j));
        }
        mass = wave_sum_f64(mass);
        if (lane == 0) {
            teacher = t;
            mass_ = mass;
        }
    }
    mark_listed<E>(a, row, from, to, marks, &twice);
    const double mass = mass_, rest = 1 - mass;
    const float m = a.stats[3 * row], log_s = a.stats[3 * row + 1];
    float on_f = static_cast<float>(mass), off_f = on_f;
    if (REST) {
        on_f = 1.0f;
        const double log_rest = a.stats[3 * row + 2];
        off_f = rest > 0 && log_rest > -__builtin_inf() ? static_cast<float>(1 - exp(log(rest) - log_rest)) : 1.0f;
    }
    const float L = log_s * kLog2e;
    const auto q_of = [&](float x) { return exp2_fast(__builtin_fmaf(x - m, a.c, -L)); };
    // this thread's listed tokens
    constexpr int PER = kMaxK / kThreads;
    float listed[PER];
    bool mine[PER];
#pragma unroll
    for (int h = 0; h < PER; ++h) {
        const int j = threadIdx.x + h * kThreads;
        mine[h] = false;
        if (j >= a.k) continue;
        const int id = a.ids[row * a.k + j];
        const bool on = id >= 0 && id < a.v && id / E >= from && id / E < to;
        const float p = on ? static_cast<float>(exp(teacher.log_p(a, row * a.k + j))) : 0.0f;
        id_of[j] = on ? id : -1;
        p_of[j] = p;
        mine[h] = on;
        if (on) listed[h] = r.element(id);
    }
    __syncthreads();
    const float gq = gs * off_f;
    for (int i = from + static_cast<int>(threadIdx.x); i < to; i += kThreads) {
        const u32x4 raw = r.load(i);
        u32x4 out;
#pragma unroll
        for (int k = 0; k < E; k += 2) {
            const float g0 = q_of(Row<F32>::at(raw, k)) * gq, g1 = q_of(Row<F32>::at(raw, k + 1)) * gq;
            if (F32) {
                out[k & 3] = __float_as_uint(g0);
                out[(k + 1) & 3] = __float_as_uint(g1);
            } else {
                out[(k >> 1) & 3] = bf16_pair(g0, g1);
            }
        }
        w.store(i, out);
    }
    // what was stored above has arrived before it is written over
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
#pragma unroll
    for (int h = 0; h < PER; ++h) {
        if (!mine[h]) continue;
        const int j = threadIdx.x + h * kThreads, id = id_of[j];
        float p = p_of[j];
        bool first = true;
        if (twice) {
            double sum = 0;
            for (int e = 0; e < a.k; ++e) {
                if (id_of[e] != id) continue;
                if (e < j) first = false;
                sum += p_of[e];
            }
            p = static_cast<float>(sum);
        }
        if (!first) continue;
        const float g = (q_of(listed[h]) * on_f - p) * gs;
        char* const at = w.base + static_cast<int64_t>(id) * (F32 ? 4 : 2);
        if (F32) *reinterpret_cast<float*>(at) = g;
        else *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(bf16_pair(g, g));
    }
}

// Loss and gradient of a row in one pass over memory: the row's vectors stay in
// registers (NV a thread) between the sums and the gradient; what goes beyond them is
// read again.  The teacher's side is one wavefront's work while the row's loads
// are on their way.
constexpr int kRowMarks = 1 << 18;      // tokens of a row at most

template <bool F32, bool REST, int NV>
__global__ void __launch_bounds__(kThreads) distill_row_kernel(const DistillArgs a) {
    constexpr int E = Row<F32>::E;
    extern __shared__ uint32_t marks[];                 // (v + 31) / 32
    __shared__ Soft joined[2][kWaves];
    __shared__ int32_t id_of[kMaxK];
    __shared__ float t_of[kMaxK], z_of[kMaxK], p_of[kMaxK];
    __shared__ int twice;
    __shared__ Teacher teacher;
    __shared__ double mass_;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t row = a.first + blockIdx.x;
    const Row<F32> r(a.z, row * a.ld, a.v), w(a.dz, row * a.dld, a.v);
    const float gs = (a.weight ? a.weight[row] : 1.0f) * a.scale;
    const int whole = static_cast<int>(a.v) / E, all_vectors = r.vectors();
    u32x4 raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = tid + j * kThreads;
        if (i < whole) raw[j] = *reinterpret_cast<const Loose*>(r.base + static_cast<int64_t>(i) * 16);
    }
    for (int i = tid; i < (static_cast<int>(a.v) + 31) / 32; i += kThreads) marks[i] = 0;
    if (tid == 0) twice = 0;
    for (int j = tid; j < a.k; j += kThreads) {
        const int id = a.ids[row * a.k + j];
        const bool on = id >= 0 && id < a.v;
        id_of[j] = on ? id : -1;
        t_of[j] = teacher_at(a, row * a.k + j);
        z_of[j] = on ? r.element(id) : 0.0f;
    }
    __syncthreads();
    for (int j = tid; j < a.k; j += kThreads) {
        const int id = id_of[j];
        if (id < 0) continue;
        const uint32_t mask = 1u << (id & 31);
        if (atomicOr(&marks[id >> 5], mask) & mask) twice = 1;
    }
    if (REST) __syncthreads();
    if (wave == 0) {
        Teacher t{0, 0};
        if (a.teacher_lse) {
            t.log_sum = a.teacher_lse[row];
        } else {
            float m = kNegInf;
            for (int j = lane; j < a.k; j += 64)
                if (id_of[j] >= 0) m = t_of[j] == t_of[j] && m == m ? fmaxf(m, t_of[j]) : __builtin_nanf("");
            const float top = wave_max(m);
            const bool nan = __ballot(m != m) != 0;
            double s = 0;
            for (int j = lane; j < a.k; j += 64)
                if (id_of[j] >= 0) s += exp((static_cast<double>(t_of[j]) - top) * a.inv_t);
            s = wave_sum_f64(s);
            if (nan) t.log_sum = __builtin_nan("");
            else if (top == kNegInf) t.log_sum = __builtin_inf();
            else t = {top, log(s)};
        }
        double mass = 0;
        for (int j = lane; j < a.k; j += 64) {
            const double p = id_of[j] >= 0 ? exp((t_of[j] - t.m) * a.inv_t - t.log_sum) : 0;
            mass += p;
            p_of[j] = static_cast<float>(p);
        }
        mass = wave_sum_f64(mass);
        if (lane == 0) {
            teacher = t;
            mass_ = mass;
        }
    }
    Soft all{kLowest, 0.0f};
    float off = 0.0f;
    const auto add = [&](const u32x4& v, int i) {
        float x[E];
        float top = kNegInf;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            x[k] = Row<F32>::at(v, k);
            top = fmaxf(top, x[k]);
        }
        const float m = fmaxf(all.m, top);
        const float f = exp2_fast((all.m - m) * a.c);
        all.s *= f;
        off *= f;
        all.m = m;
        const uint32_t listed = REST ? marks[(i * E) >> 5] >> ((i * E) & 31) : 0;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const float e = exp2_fast((x[k] - m) * a.c);
            all.s += e;
            if (REST) off += listed & (1u << k) ? 0.0f : e;
        }
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (tid + j * kThreads < whole) add(raw[j], tid + j * kThreads);
    for (int i = tid + NV * kThreads; i < whole; i += kThreads) add(r.load(i), i);
    if (whole < all_vectors && tid == kThreads - 1) add(r.load(whole), whole);
    {
        const float m = wave_max(all.m), f = exp2_fast((all.m - m) * a.c);
        all.s = wave_sum(all.s * f);
        if (REST) off = wave_sum(off * f);
        if (lane == 0) {
            joined[0][wave] = {m, all.s};
            joined[1][wave] = {m, off};
        }
    }
    __syncthreads();
    Soft o = joined[1][0];
    all = joined[0][0];
#pragma unroll
    for (int h = 1; h < kWaves; ++h) {
        all = soft_join(all, joined[0][h], a.c);
        if (REST) o = soft_join(o, joined[1][h], a.c);
    }
    if (wave == 0) {
        const double log_s = log(static_cast<double>(all.s));
        double sum = 0, log_rest = 0;
        for (int j = lane; j < a.k; j += 64) {
            if (id_of[j] < 0) continue;
            const double log_p = (t_of[j] - teacher.m) * a.inv_t - teacher.log_sum, p = exp(log_p);
            if (!(p == 0)) sum += p * (log_p - ((static_cast<double>(z_of[j]) - all.m) * a.inv_t - log_s));
        }
        sum = wave_sum_f64(sum);
        if (REST) {
            const double rest = 1 - mass_;
            log_rest = (static_cast<double>(o.m) - all.m) * a.inv_t + log(static_cast<double>(o.s)) - log_s;
            if (!(rest <= 0)) sum += rest * (log(rest) - log_rest);
        }
        if (lane == 0) {
            if (a.loss) a.loss[row] = static_cast<float>(log_s - log_s == 0 ? sum * a.t2 : __builtin_nan(""));
            a.stats[3 * row] = all.s == 0.0f ? kNegInf : all.m;
            a.stats[3 * row + 1] = static_cast<float>(log_s);
            a.stats[3 * row + 2] = static_cast<float>(log_rest);
        }
    }
    float on_f = static_cast<float>(mass_), off_f = on_f;
    if (REST) {
        on_f = 1.0f;
        const float rest = static_cast<float>(1 - mass_);
        off_f = rest > 0.0f && o.s > 0.0f ? 1.0f - rest * (all.s / o.s) * exp2_fast((all.m - o.m) * a.c) : 1.0f;
    }
    const float L = __builtin_amdgcn_logf(all.s), m = all.m, gq = gs * off_f;
    const auto q_of = [&](float x) { return exp2_fast(__builtin_fmaf(x - m, a.c, -L)); };
    const auto grad = [&](const u32x4& v) {
        u32x4 out;
#pragma unroll
        for (int k = 0; k < E; k += 2) {
            const float g0 = q_of(Row<F32>::at(v, k)) * gq, g1 = q_of(Row<F32>::at(v, k + 1)) * gq;
            if (F32) {
                out[k & 3] = __float_as_uint(g0);
                out[(k + 1) & 3] = __float_as_uint(g1);
            } else {
                out[(k >> 1) & 3] = bf16_pair(g0, g1);
            }
        }
        return gs == 0.0f ? u32x4{0, 0, 0, 0} : out;
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = tid + j * kThreads;
        if (i < whole) *reinterpret_cast<Loose*>(w.base + static_cast<int64_t>(i) * 16) = grad(raw[j]);
    }
    for (int i = tid + NV * kThreads; i < whole; i += kThreads) w.store(i, grad(r.load(i)));
    if (whole < all_vectors && tid == kThreads - 1) w.store(whole, grad(r.load(whole)));
    if (gs == 0.0f) return;
    // what was stored above has arrived before it is written over
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int j = tid; j < a.k; j += kThreads) {
        const int id = id_of[j];
        if (id < 0) continue;
        float p = p_of[j];
        bool first = true;
        if (twice) {
            double sum = 0;
            for (int e = 0; e < a.k; ++e) {
                if (id_of[e] != id) continue;
                if (e < j) first = false;
                sum += p_of[e];
            }
            p = static_cast<float>(sum);
        }
        if (!first) continue;
        const float g = (q_of(z_of[j]) * on_f - p) * gs;
        char* const at = w.base + static_cast<int64_t>(id) * (F32 ? 4 : 2);
        if (F32) *reinterpret_cast<float*>(at) = g;
        else *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(bf16_pair(g, g));
    }
}

// Workgroups a row: one where rows fill the card; few rows are cut into parts
// of 512 vectors and more.
int chunks_of(int64_t n, int64_t v, int dtype) {
    const int64_t e = dtype == NGRAM_F32 ? 4 : 8, vectors = (v + e - 1) / e;
    const int64_t want = (1024 + n - 1) / std::max<int64_t>(n, 1);
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
    if (!(p->temperature > 0.0f) || std::isinf(p->temperature)) return fail(NGRAM_EINVAL, "temperature=%g must be positive and finite", p->temperature);
    if (p->n == 0) return NGRAM_OK;
    if (!p->logits || !p->teacher || !p->ids) return fail(NGRAM_EINVAL, "logits, teacher or ids is NULL");
    const uintptr_t ze = p->dtype == NGRAM_F32 ? 4 : 2, te = p->teacher_dtype == NGRAM_F32 ? 4 : 2;
    if (!aligned(p->logits, ze) || !aligned(p->teacher, te) || !aligned(p->ids, 4) || !aligned(p->teacher_lse, 4))
        return fail(NGRAM_EALIGN, "an argument is not aligned to its elements");
    return NGRAM_OK;
}

int check_grad(const ngram_distill_args* p, const float* weight, float scale, const void* dz, int64_t dld) {
    if (dld < p->V) return fail(NGRAM_EINVAL, "dld=%lld is below V=%lld", (long long)dld, (long long)p->V);
    if (dz && dz == p->logits && dld != p->ld) return fail(NGRAM_EINVAL, "dlogits_out takes logits' place, but dld=%lld is not ld=%lld", (long long)dld, (long long)p->ld);
    if (!std::isfinite(scale)) return fail(NGRAM_EINVAL, "scale=%g must be finite", scale);
    if (!aligned(dz, p->dtype == NGRAM_F32 ? 4 : 2) || !aligned(weight, 4)) return fail(NGRAM_EALIGN, "dlogits_out or weight is not aligned to its elements");
    return NGRAM_OK;
}

DistillArgs device_args(const ngram_distill_args* p) {
    DistillArgs a = {};
    a.z = p->logits; a.t = p->teacher; a.ids = p->ids; a.teacher_lse = p->teacher_lse;
    a.n = p->n; a.v = p->V; a.ld = p->ld; a.k = p->k; a.t32 = p->teacher_dtype == NGRAM_F32;
    a.inv_t = 1.0 / p->temperature;
    a.t2 = static_cast<double>(p->temperature) * p->temperature;
    a.c = static_cast<float>(1.4426950408889634074 * a.inv_t);
    a.chunks = chunks_of(p->n, p->V, p->dtype);
    const int64_t e = p->dtype == NGRAM_F32 ? 4 : 8, vectors = (p->V + e - 1) / e;
    a.per = static_cast<int32_t>((vectors + a.chunks - 1) / a.chunks);
    a.per = (a.per + 7) / 8 * 8;                                            // whole words of marks
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

void launch_grad(const DistillArgs& a, bool f32, hipStream_t st) {
    over_rows(a, a.n, a.chunks, kThreads, 1, [&](const DistillArgs& b, dim3 grid) {
        const dim3 block(kThreads);
        if (f32 && b.teacher_lse) hipLaunchKernelGGL((distill_grad_kernel<true, true>), grid, block, 0, st, b);
        else if (f32) hipLaunchKernelGGL((distill_grad_kernel<true, false>), grid, block, 0, st, b);
        else if (b.teacher_lse) hipLaunchKernelGGL((distill_grad_kernel<false, true>), grid, block, 0, st, b);
        else hipLaunchKernelGGL((distill_grad_kernel<false, false>), grid, block, 0, st, b);
    });
}

// Rows in one workgroup each: enough of them to fill the card, short enough for the marks.
bool whole_rows(const DistillArgs& a) { return a.n >= 256 && a.v <= kRowMarks; }

template <bool F32, bool REST, int NV>
void launch_rows_of(const DistillArgs& a, hipStream_t st) {
    const uint32_t lds = static_cast<uint32_t>((a.v + 31) / 32 * 4);
    over_rows(a, a.n, 1, kThreads, 1, [&](const DistillArgs& b, dim3 grid) {
        hipLaunchKernelGGL((distill_row_kernel<F32, REST, NV>), grid, dim3(kThreads), lds, st, b);
    });
}
template <bool F32, bool REST>
void launch_rows(const DistillArgs& a, hipStream_t st) {
    const int64_t vectors = a.v / Row<F32>::E;
    if (vectors <= 4 * kThreads) launch_rows_of<F32, REST, 4>(a, st);
    else if (vectors <= 12 * kThreads) launch_rows_of<F32, REST, 12>(a, st);
    else if (vectors <= 24 * kThreads) launch_rows_of<F32, REST, 24>(a, st);
    else launch_rows_of<F32, REST, 38>(a, st);
}

}  // namespace
}  // namespace ng8

using namespace ng8;

extern "C" {

int64_t ngram_distill_workspace_bytes(int64_t n, int64_t V, int32_t dtype) {
    if (n < 0 || n > NGRAM_FP8_MAX || V < 1 || V > NGRAM_FP8_MAX || (dtype != NGRAM_F32 && dtype != NGRAM_BF16)) return -1;
    return n * chunks_of(n, V, dtype) * 2 * static_cast<int64_t>(sizeof(Soft)) + n * 12;
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
    const int64_t parts = a.n * a.chunks * 2 * static_cast<int64_t>(sizeof(Soft)), need = parts + a.n * 12;
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return fail(NGRAM_EINVAL, "workspace must hold %lld bytes, 16-byte aligned", (long long)need);
    a.loss = loss_out;
    a.part = static_cast<Soft*>(workspace);
    a.stats = stats_out ? stats_out : reinterpret_cast<float*>(static_cast<char*>(workspace) + parts);
    a.weight = weight; a.scale = static_cast<float>(static_cast<double>(scale) * p->temperature); a.dz = dlogits_out; a.dld = dld;
    const bool f32 = p->dtype == NGRAM_F32;
    if (dlogits_out && whole_rows(a)) {
        if (f32 && a.teacher_lse) launch_rows<true, true>(a, stream);
        else if (f32) launch_rows<true, false>(a, stream);
        else if (a.teacher_lse) launch_rows<false, true>(a, stream);
        else launch_rows<false, false>(a, stream);
        return hip_status("ngram_distill");
    }
    over_rows(a, a.n, a.chunks, kThreads, 1, [&](const DistillArgs& b, dim3 grid) {
        const dim3 block(kThreads);
        if (f32 && b.teacher_lse) hipLaunchKernelGGL((distill_stats_kernel<true, true>), grid, block, 0, stream, b);
        else if (f32) hipLaunchKernelGGL((distill_stats_kernel<true, false>), grid, block, 0, stream, b);
        else if (b.teacher_lse) hipLaunchKernelGGL((distill_stats_kernel<false, true>), grid, block, 0, stream, b);
        else hipLaunchKernelGGL((distill_stats_kernel<false, false>), grid, block, 0, stream, b);
    });
    over_rows(a, (a.n + 3) / 4, 1, 256, 4, [&](const DistillArgs& b, dim3 grid) {
        if (f32) hipLaunchKernelGGL(distill_finish_kernel<true>, grid, dim3(256), 0, stream, b);
        else hipLaunchKernelGGL(distill_finish_kernel<false>, grid, dim3(256), 0, stream, b);
    });
    if (dlogits_out) launch_grad(a, f32, stream);
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
