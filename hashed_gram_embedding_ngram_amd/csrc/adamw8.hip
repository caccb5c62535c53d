// AdamW for MI355X (gfx950): ngram_adamw over many tensors at once and
// ngram_adamw_rows over the touched rows of a table, with moments in fp32 or
// in 8 bits.  The formulas are in include/ngram.h.  Both are bound by HBM
// bandwidth: 10 bytes an element for bf16 parameters and gradients with 8-bit
// moments, 28 for everything in fp32.  A lane has eight consecutive elements:
// every access of a wavefront is 512 to 2048 consecutive bytes, and a scale
// block of 128 is a group of 16 lanes, which finds its largest value by lane
// moves.  Everything is read and written once, so all of it goes past the
// caches' usual keeping (260,000 rows of 2560: 1670-1700 us with plain
// accesses, 1400-1450 so).  Measured: 200M bf16 parameters with 8-bit moments
// 325 us, 6.2 TB/s; 60M of everything in fp32 322 us, 5.2 TB/s; those rows 5.5
// TB/s.  A large copy reaches 5.5 TB/s.
#include "common8.h"

#include <algorithm>
#include <cmath>

namespace ng8 {
namespace {

struct StepConst {
    float beta1, om_beta1, beta2, om_beta2;
    float decay;        // 1 - lr * weight_decay
    float rate;         // lr / (1 - beta1^step)
    float root;         // 1 / sqrt(1 - beta2^step)
    float eps;
    float grad_scale;
    uint64_t key;
};

// splitmix64's first output from state x.
__host__ __device__ inline uint64_t mix64(uint64_t x) {
    uint64_t z = x + 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// bf16 of x, rounded away from zero with the probability that r16 gives.
__device__ __forceinline__ uint32_t bf16_up_bits(float x, uint32_t r16) {     // in the high half
    return __float_as_uint(x) + (__builtin_isfinite(x) ? r16 : 0u);
}

// Code K (0..3) of a word: x rounded to E4M3 up or down at random.  The
// instruction adds the high 20 bits of `seed` below the kept bits and
// truncates, subnormal codes included: x goes to the upper of its two
// neighbours in proportion to its distance from the lower.  |x| <= 448 stays
// <= 448 (448 has no bits below the kept ones); infinities and NaN give the
// NaN code.
template <int K>
__device__ __forceinline__ uint32_t code_up(float x, uint32_t seed, uint32_t word) {
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_sr_fp8_f32(x, static_cast<int>(seed), static_cast<int>(word), K));
}
__device__ __forceinline__ uint32_t codes4_up(const float* x, const uint32_t* seed, float inv) {
    uint32_t w = code_up<0>(x[0] * inv, seed[0], 0u);
    w = code_up<1>(x[1] * inv, seed[1], w);
    w = code_up<2>(x[2] * inv, seed[2], w);
    return code_up<3>(x[3] * inv, seed[3], w);
}
// Bytes that are zero where `x` is above zero become 1, the smallest code.
__device__ __forceinline__ uint32_t keep_positive4(uint32_t w, const float* x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w |= ((w >> (8 * k)) & 0xFFu) == 0u && x[k] > 0.0f ? 1u << (8 * k) : 0u;
    return w;
}

// Everything one lane holds of eight consecutive elements.
template <bool P32, bool G32, bool S8>
struct Eight {
    Raw8<P32> p;
    Raw8<G32> g;
    Raw8<true> m, v;        // fp32 moments
    u32x2 mc, vc;           // or their codes
    uint32_t ms, vs;        // and scale bytes
};

// The hardware's root of a v below 2^-126 is zero.  Beside an eps of 2^24 times
// the largest root that this drops (2^-63 c.root) the quotient stays what it
// is; with a smaller eps the step would become m / eps, and SMALL kernels take
// the root of 2^64 v there.  (A test of the values in every call, or of a flag,
// took 1.2 to 1.7% of the time with 8-bit moments.)
inline bool needs_small(const StepConst& c) { return c.eps < 0x1p-39f * c.root; }

// One step on eight elements; `index` is the first one's place in the random
// sequence.  All 16 lanes of a block of 128 take part (those past the end with
// zeros).  In 8 bits v holds the square root of the second moment, which
// needs half the exponent range, and keeps it above zero where it was above
// zero: a zero would make the next step divide by eps alone.
template <bool SMALL, bool P32, bool G32, bool S8>
__device__ __forceinline__ void step8(Eight<P32, G32, S8>& e, const StepConst& c, uint64_t index) {
    float p[8], g[8], m[8], v[8];
    e.p.get(p);
    e.g.get(g);
    if (S8) {
        const float sm = scale_value(e.ms), sv = scale_value(e.vs);
        codes8_to_f32(e.mc, m);
        codes8_to_f32(e.vc, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m[k] *= sm;
            v[k] *= sv;
            v[k] *= v[k];
        }
    } else {
        e.m.get(m);
        e.v.get(v);
    }
    uint32_t word[8];
    if (S8 || !P32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t z = mix64(c.key + (index >> 1) + k);
            word[2 * k] = static_cast<uint32_t>(z);
            word[2 * k + 1] = static_cast<uint32_t>(z >> 32);
        }
    }
    float root[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float gk = g[k] * c.grad_scale;
        m[k] = c.beta1 * m[k] + c.om_beta1 * gk;
        v[k] = c.beta2 * v[k] + c.om_beta2 * (gk * gk);
        // hardware root and reciprocal: one unit in the last place each
        // (correctly rounded ones are 18 instructions more, and 8-bit moments
        // leave about 65 an element before arithmetic and not memory sets
        // the time)
        root[k] = __builtin_amdgcn_sqrtf(v[k]);
        if (SMALL) root[k] = v[k] < 0x1p-126f ? __builtin_amdgcn_sqrtf(v[k] * 0x1p64f) * 0x1p-32f : root[k];
        p[k] = p[k] * c.decay - c.rate * (m[k] * __builtin_amdgcn_rcpf(root[k] * c.root + c.eps));
    }
    if (P32) {
        e.p.a = u32x4{__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]), __float_as_uint(p[3])};
        e.p.b = u32x4{__float_as_uint(p[4]), __float_as_uint(p[5]), __float_as_uint(p[6]), __float_as_uint(p[7])};
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            e.p.a[k] = __builtin_amdgcn_perm(bf16_up_bits(p[2 * k + 1], (word[2 * k + 1] >> 8) & 0xFFFFu),
                                             bf16_up_bits(p[2 * k], (word[2 * k] >> 8) & 0xFFFFu), 0x07060302u);
    }
    if (S8) {
        e.ms = block_scale16(m);
        e.vs = block_scale16(root);
        const float im = inverse_scale(e.ms), iv = inverse_scale(e.vs);
        uint32_t low[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) low[k] = word[k] << 12;
        e.mc = u32x2{codes4_up(m, low, im), codes4_up(m + 4, low + 4, im)};
        e.vc = u32x2{keep_positive4(codes4_up(root, word, iv), root), keep_positive4(codes4_up(root + 4, word + 4, iv), root + 4)};
    } else {
        e.m.a = u32x4{__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]), __float_as_uint(m[3])};
        e.m.b = u32x4{__float_as_uint(m[4]), __float_as_uint(m[5]), __float_as_uint(m[6]), __float_as_uint(m[7])};
        e.v.a = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        e.v.b = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const Raw8<F32>& x) {
    if (F32) {
        u32x4* const d = reinterpret_cast<u32x4*>(static_cast<float*>(p) + i);
        __builtin_nontemporal_store(x.a, d);
        __builtin_nontemporal_store(x.b, d + 1);
    } else {
        __builtin_nontemporal_store(x.a, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i));
    }
}

// The first `live` (1 .. 7) of eight elements, zeros behind them: one load for
// each element, the last one's again past it, so that all are in flight at once.
template <typename V>
__device__ __forceinline__ void load_each(uint32_t u[8], const void* p, int64_t i, int live) {
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = static_cast<const V*>(p)[i + min(k, live - 1)];
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = k < live ? u[k] : 0u;
}
template <bool F32>
__device__ __forceinline__ void load_some(Raw8<F32>& x, const void* p, int64_t i, int live) {
    uint32_t u[8];
    if (F32) {
        load_each<uint32_t>(u, p, i, live);
        x.a = u32x4{u[0], u[1], u[2], u[3]};
        x.b = u32x4{u[4], u[5], u[6], u[7]};
    } else {
        load_each<uint16_t>(u, p, i, live);
        x.a = u32x4{u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16};
    }
}
__device__ __forceinline__ u32x2 codes_some(const void* p, int64_t i, int live) {
    uint32_t u[8];
    load_each<uint8_t>(u, p, i, live);
    return u32x2{u[0] | u[1] << 8 | u[2] << 16 | u[3] << 24, u[4] | u[5] << 8 | u[6] << 16 | u[7] << 24};
}
template <bool F32>
__device__ __forceinline__ void store_some(void* p, int64_t i, const Raw8<F32>& x, int live) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k >= live) break;
        if (F32) static_cast<uint32_t*>(p)[i + k] = k < 4 ? x.a[k & 3] : x.b[k & 3];
        else static_cast<uint16_t*>(p)[i + k] = static_cast<uint16_t>(x.a[k >> 1] >> (16 * (k & 1)));
    }
}

struct TensorArg {
    void* p;
    const void* g;
    void* m;
    void* v;
    uint8_t* ms;
    uint8_t* vs;
    int64_t numel;
    uint64_t offset;
};

// A launch takes up to 48 tensors of one kind by value (3.5 KB of kernel
// arguments): no descriptor has to reach the device ahead of the call, so
// nothing is allocated or copied and the call can be captured in a graph.
constexpr int kTensorsPerLaunch = 48;
// Elements per workgroup: one round of 256 lanes x 8.  Measured on 200M bf16
// parameters with 8-bit moments, before the streaming accesses: 367 us against
// 387 with two rounds and 402 with four; on 300,000 fp32 elements 3.6 us
// against 4.2 and 6.1 (3.3 now: a tensor's odd last elements are loaded at once).
constexpr int kChunk = 2048;

struct AdamArgs {
    TensorArg t[kTensorsPerLaunch];
    uint32_t end[kTensorsPerLaunch];    // workgroups of tensors 0 .. i
    StepConst c;
    int32_t count;
};

template <bool SMALL, bool P32, bool G32, bool S8>
__global__ void __launch_bounds__(256) adamw_kernel(const AdamArgs a) {
    const int lane = threadIdx.x & 63;
    // the tensor of this workgroup: the number of tensors that end at or
    // before it, counted over the lanes
    const uint32_t end = lane < a.count ? a.end[lane] : 0xFFFFFFFFu;
    const int which = __builtin_popcountll(__ballot(end <= blockIdx.x));
    const uint32_t first = which == 0 ? 0u : a.end[which - 1];
    const TensorArg t = a.t[which];
    const int64_t i = static_cast<int64_t>(blockIdx.x - first) * kChunk + threadIdx.x * kVec;
    if (i >= (t.numel + 127) / 128 * 128) return;       // whole groups of 16 lanes
    Eight<P32, G32, S8> e;
    const int64_t left = t.numel - i;
    const int live = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
    if (live == 8) {
        e.p.load_stream(t.p, i);
        e.g.load_stream(t.g, i);
        if (S8) {
            e.mc = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(t.m) + i));
            e.vc = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(t.v) + i));
        } else {
            e.m.load_stream(t.m, i);
            e.v.load_stream(t.v, i);
        }
    } else if (live > 0) {
        load_some(e.p, t.p, i, live);
        load_some(e.g, t.g, i, live);
        if (S8) {
            e.mc = codes_some(t.m, i, live);
            e.vc = codes_some(t.v, i, live);
        } else {
            load_some(e.m, t.m, i, live);
            load_some(e.v, t.v, i, live);
        }
    } else {
        e.p.zero();
        e.g.zero();
        e.m.zero();
        e.v.zero();
        e.mc = u32x2{0, 0};
        e.vc = u32x2{0, 0};
    }
    if (S8) {
        e.ms = t.ms[i >> 7];
        e.vs = t.vs[i >> 7];
    }
    step8<SMALL>(e, a.c, t.offset + static_cast<uint64_t>(i));
    if (live == 8) {
        store8(t.p, i, e.p);
        if (S8) {
            __builtin_nontemporal_store(e.mc, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(t.m) + i));
            __builtin_nontemporal_store(e.vc, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(t.v) + i));
        } else {
            store8(t.m, i, e.m);
            store8(t.v, i, e.v);
        }
    } else {
        store_some(t.p, i, e.p, live);
        if (S8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= live) break;
                static_cast<uint8_t*>(t.m)[i + k] = static_cast<uint8_t>(e.mc[k >> 2] >> (8 * (k & 3)));
                static_cast<uint8_t*>(t.v)[i + k] = static_cast<uint8_t>(e.vc[k >> 2] >> (8 * (k & 3)));
            }
        } else {
            store_some(t.m, i, e.m, live);
            store_some(t.v, i, e.v, live);
        }
    }
    if (S8 && (lane & 15) == 0) {
        t.ms[i >> 7] = static_cast<uint8_t>(e.ms);
        t.vs[i >> 7] = static_cast<uint8_t>(e.vs);
    }
}

// The step on rows rows[0 .. *count) of a [R][d] table from their gradients
// g[u][d].  16 lanes own a block of 128 columns of one row; the launch covers
// max_rows rows and the lanes past *count leave at once, so the count stays on
// the device.
struct RowsArgs {
    void* p;
    void* m;
    void* v;
    uint8_t* ms;
    uint8_t* vs;
    const int32_t* rows;
    const void* g;
    const int64_t* count;
    int64_t first;      // rows and gradient rows of earlier launches, which `rows` and `g` are already past
    int64_t max_rows;   // of this launch
    int64_t R;
    int32_t d;
    int32_t nb;         // blocks of 128 columns in a row
    StepConst c;
};

template <bool SMALL, bool P32, bool G32, bool S8>
__global__ void __launch_bounds__(256) adamw_rows_kernel(const RowsArgs a) {
    const uint32_t unit = blockIdx.x * 16 + (threadIdx.x >> 4), nb = static_cast<uint32_t>(a.nb);
    const uint32_t u = unit / nb;
    const int64_t count = a.count ? min(*a.count - a.first, a.max_rows) : a.max_rows;
    if (u >= count) return;
    const int64_t row = a.rows[u];
    if (row < 0 || row >= a.R) return;
    const int col = static_cast<int>(unit - u * nb) * kBlock + static_cast<int>(threadIdx.x & 15) * kVec;
    const bool live = col < a.d;
    const int64_t at = row * a.d + col;
    Eight<P32, G32, S8> e;
    if (live) {
        e.g.load_stream(a.g, static_cast<int64_t>(u) * a.d + col);
        e.p.load_stream(a.p, at);
        if (S8) {
            e.mc = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.m) + at));
            e.vc = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(a.v) + at));
            e.ms = a.ms[row * a.nb + (col >> 7)];
            e.vs = a.vs[row * a.nb + (col >> 7)];
        } else {
            e.m.load_stream(a.m, at);
            e.v.load_stream(a.v, at);
        }
    } else {
        e.g.zero();
        e.p.zero();
        e.m.zero();
        e.v.zero();
        e.mc = u32x2{0, 0};
        e.vc = u32x2{0, 0};
        e.ms = e.vs = kUnitScale;
    }
    step8<SMALL>(e, a.c, static_cast<uint64_t>(at));
    if (!live) return;
    store8(a.p, at, e.p);
    if (S8) {
        __builtin_nontemporal_store(e.mc, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.m) + at));
        __builtin_nontemporal_store(e.vc, reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.v) + at));
        if ((threadIdx.x & 15) == 0) {
            a.ms[row * a.nb + (col >> 7)] = static_cast<uint8_t>(e.ms);
            a.vs[row * a.nb + (col >> 7)] = static_cast<uint8_t>(e.vs);
        }
    } else {
        store8(a.m, at, e.m);
        store8(a.v, at, e.v);
    }
}

int step_const(const ngram_adamw_step* h, StepConst* c) {
    if (!h) return fail(NGRAM_EINVAL, "the step's constants are NULL");
    if (h->step < 1) return fail(NGRAM_EINVAL, "step=%lld must be at least 1", (long long)h->step);
    if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0))
        return fail(NGRAM_EINVAL, "beta1 and beta2 must lie in [0, 1)");
    if (!(h->eps > 0.0) || !std::isfinite(h->eps) || !std::isfinite(h->lr) || !std::isfinite(h->weight_decay) ||
        !std::isfinite(h->grad_scale))
        return fail(NGRAM_EINVAL, "eps must be positive, and lr, eps, weight_decay and grad_scale finite");
    // evaluated in float64 and rounded once each
    c->beta1 = static_cast<float>(h->beta1);
    c->om_beta1 = static_cast<float>(1.0 - h->beta1);
    c->beta2 = static_cast<float>(h->beta2);
    c->om_beta2 = static_cast<float>(1.0 - h->beta2);
    c->decay = static_cast<float>(1.0 - h->lr * h->weight_decay);
    c->rate = static_cast<float>(h->lr / (1.0 - std::pow(h->beta1, static_cast<double>(h->step))));
    c->root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h->beta2, static_cast<double>(h->step))));
    c->eps = static_cast<float>(h->eps);
    if (c->eps < 0x1p-126f) return fail(NGRAM_EINVAL, "eps=%g below fp32's smallest normal number", h->eps);
    c->grad_scale = static_cast<float>(h->grad_scale);
    c->key = mix64(mix64(h->seed) + static_cast<uint64_t>(h->step));
    return NGRAM_OK;
}

int check_kind(int p_dtype, int g_dtype, int state) {
    if ((p_dtype != NGRAM_F32 && p_dtype != NGRAM_BF16) || (g_dtype != NGRAM_F32 && g_dtype != NGRAM_BF16))
        return fail(NGRAM_EINVAL, "p_dtype=%d or g_dtype=%d is not an ngram_value", p_dtype, g_dtype);
    if (state != NGRAM_STATE_F32 && state != NGRAM_STATE_FP8)
        return fail(NGRAM_EINVAL, "state=%d is not an ngram_state", state);
    return NGRAM_OK;
}

int kind_of(int p_dtype, int g_dtype, int state) {
    return (p_dtype == NGRAM_F32 ? 4 : 0) | (g_dtype == NGRAM_F32 ? 2 : 0) | (state == NGRAM_STATE_FP8 ? 1 : 0);
}

// Elements from .. from + take - 1 of a tensor; `from` is a multiple of kChunk.
TensorArg part_of(const ngram_adamw_tensor& t, int64_t from, int64_t take) {
    const size_t pb = value_bytes(t.p_dtype), gb = value_bytes(t.g_dtype), sb = t.state == NGRAM_STATE_FP8 ? 1 : 4;
    return TensorArg{static_cast<uint8_t*>(t.p) + from * pb, static_cast<const uint8_t*>(t.g) + from * gb,
                     static_cast<uint8_t*>(t.m) + from * sb, static_cast<uint8_t*>(t.v) + from * sb,
                     t.m_scale ? t.m_scale + from / kBlock : nullptr, t.v_scale ? t.v_scale + from / kBlock : nullptr,
                     take, static_cast<uint64_t>(t.rng_offset) + static_cast<uint64_t>(from)};
}

#define NG8_BY_KIND(kind, CALL)                      \
    switch (kind) {                                  \
        case 0: CALL(false, false, false); break;    \
        case 1: CALL(false, false, true); break;     \
        case 2: CALL(false, true, false); break;     \
        case 3: CALL(false, true, true); break;      \
        case 4: CALL(true, false, false); break;     \
        case 5: CALL(true, false, true); break;      \
        case 6: CALL(true, true, false); break;      \
        default: CALL(true, true, true); break;      \
    }

}  // namespace
}  // namespace ng8

using namespace ng8;

extern "C" {

int ngram_adamw(const ngram_adamw_tensor* tensors, int32_t count, const ngram_adamw_step* step, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    AdamArgs a;
    int rc = step_const(step, &a.c);
    if (rc) return rc;
    if (count < 0) return fail(NGRAM_EINVAL, "count=%d is negative", count);
    if (count > 0 && !tensors) return fail(NGRAM_EINVAL, "tensors is NULL");
    for (int32_t i = 0; i < count; ++i) {
        const ngram_adamw_tensor& t = tensors[i];
        if ((rc = check_kind(t.p_dtype, t.g_dtype, t.state))) return rc;
        if (t.numel < 0) return fail(NGRAM_EINVAL, "tensor %d: numel=%lld is negative", i, (long long)t.numel);
        if (t.numel > (int64_t{1} << 41)) return fail(NGRAM_ERANGE, "tensor %d: numel=%lld too large", i, (long long)t.numel);
        if (t.rng_offset < 0 || t.rng_offset % kVec != 0)
            return fail(NGRAM_EINVAL, "tensor %d: rng_offset must be a multiple of %d, not negative", i, kVec);
        if (t.numel == 0) continue;
        const bool s8 = t.state == NGRAM_STATE_FP8;
        if (!t.p || !t.g || !t.m || !t.v || (s8 && (!t.m_scale || !t.v_scale)))
            return fail(NGRAM_EINVAL, "tensor %d: a pointer is NULL", i);
        if (!aligned(t.p, 16) || !aligned(t.g, 16) || !aligned(t.m, s8 ? 8 : 16) || !aligned(t.v, s8 ? 8 : 16))
            return fail(NGRAM_EALIGN, "tensor %d: p, g and fp32 moments must be 16-byte aligned, 8-bit moments 8-byte", i);
    }
    const bool small = needs_small(a.c);
    // one launch for each kind that occurs and each 48 tensors of it, or each
    // 2^35 elements: a tensor is cut there, and goes on in the next launch
    for (int kind = 0; kind < 8; ++kind) {
        int32_t i = 0;
        int64_t from = 0;       // tensor i's elements that earlier launches have
        while (i < count) {
            a.count = 0;
            int64_t groups = 0;
            const int64_t most = most_groups(256);
            while (i < count && a.count < kTensorsPerLaunch && groups < most) {
                const ngram_adamw_tensor& t = tensors[i];
                if (t.numel == 0 || kind_of(t.p_dtype, t.g_dtype, t.state) != kind) {
                    ++i;
                    continue;
                }
                const int64_t take = std::min(t.numel - from, (most - groups) * kChunk);
                a.t[a.count] = part_of(t, from, take);
                groups += (take + kChunk - 1) / kChunk;
                a.end[a.count++] = static_cast<uint32_t>(groups);
                from += take;
                if (from == t.numel) {
                    ++i;
                    from = 0;
                }
            }
            if (a.count == 0) break;
            const dim3 grid(static_cast<unsigned>(groups)), block(256);
#define NG8_ADAM(P, G, S)                                                                           \
    if (small) hipLaunchKernelGGL((adamw_kernel<true, P, G, S>), grid, block, 0, stream, a);        \
    else hipLaunchKernelGGL((adamw_kernel<false, P, G, S>), grid, block, 0, stream, a)
            NG8_BY_KIND(kind, NG8_ADAM)
#undef NG8_ADAM
            if ((rc = hip_status("ngram_adamw launch"))) return rc;
        }
    }
    return NGRAM_OK;
}

int ngram_adamw_rows(const ngram_adamw_tensor* table, int64_t R, int32_t d, const int32_t* rows, int64_t max_rows,
                     const int64_t* n_rows, const ngram_adamw_step* step, ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    RowsArgs a;
    int rc = step_const(step, &a.c);
    if (rc) return rc;
    if (!table) return fail(NGRAM_EINVAL, "table is NULL");
    if ((rc = check_kind(table->p_dtype, table->g_dtype, table->state))) return rc;
    if (R < 1 || R > NGRAM_MAX_ROWS) return fail(NGRAM_ERANGE, "R=%lld outside [1, 2^31 - 1]", (long long)R);
    if (d <= 0 || d % kVec != 0) return fail(NGRAM_EINVAL, "d=%d must be a positive multiple of %d", d, kVec);
    if (d > NGRAM_MAX_D) return fail(NGRAM_ERANGE, "d=%d above %d", d, NGRAM_MAX_D);
    if (table->numel != R * d) return fail(NGRAM_EINVAL, "table: numel=%lld is not R * d", (long long)table->numel);
    if (table->rng_offset != 0) return fail(NGRAM_EINVAL, "table: rng_offset must be 0");
    if (max_rows < 0) return fail(NGRAM_EINVAL, "max_rows=%lld is negative", (long long)max_rows);
    if (max_rows > NGRAM_MAX_ROWS) return fail(NGRAM_ERANGE, "max_rows=%lld above 2^31 - 1", (long long)max_rows);
    if (max_rows == 0) return NGRAM_OK;
    const bool s8 = table->state == NGRAM_STATE_FP8;
    if (!rows || !table->p || !table->g || !table->m || !table->v || (s8 && (!table->m_scale || !table->v_scale)))
        return fail(NGRAM_EINVAL, "rows or a pointer of the table is NULL");
    if (!aligned(table->p, 16) || !aligned(table->g, 16) || !aligned(table->m, s8 ? 8 : 16) ||
        !aligned(table->v, s8 ? 8 : 16) || !aligned(rows, 4) || !aligned(n_rows, 8))
        return fail(NGRAM_EALIGN, "p, g and fp32 moments must be 16-byte aligned, 8-bit moments and n_rows 8-byte, rows 4-byte");
    a.p = table->p; a.m = table->m; a.v = table->v; a.ms = table->m_scale; a.vs = table->v_scale;
    a.count = n_rows; a.R = R; a.d = d;
    a.nb = static_cast<int32_t>(blocks_of(d));
    const int64_t most = most_groups(256) * 16 / a.nb;      // rows of a launch: 16 blocks a workgroup
    const bool small = needs_small(a.c);
    for (a.first = 0; a.first < max_rows; a.first += most) {
        a.rows = rows + a.first;
        a.g = static_cast<const uint8_t*>(table->g) + a.first * d * value_bytes(table->g_dtype);
        a.max_rows = std::min(most, max_rows - a.first);
        const dim3 grid(static_cast<unsigned>((a.max_rows * a.nb + 15) / 16)), block(256);
#define NG8_ROWS(P, G, S)                                                                           \
        if (small) hipLaunchKernelGGL((adamw_rows_kernel<true, P, G, S>), grid, block, 0, stream, a);   \
        else hipLaunchKernelGGL((adamw_rows_kernel<false, P, G, S>), grid, block, 0, stream, a)
        NG8_BY_KIND(kind_of(table->p_dtype, table->g_dtype, table->state), NG8_ROWS)
#undef NG8_ROWS
        if ((rc = hip_status("ngram_adamw_rows launch"))) return rc;
    }
    return NGRAM_OK;
}

}  // extern "C"
