// Beam search for MI355X (gfx950): ngram_beam_step, ngram_beam_reorder.  The
// formulas are in include/ngram.h.  Times in comments are on the
// card: of one kernel, or of a call replayed in a graph.
#include "rows8.h"

#include <algorithm>

namespace ng8 {
namespace {

// A logit and its token in one number that orders candidates of a beam: a
// larger logit first, then a lower token.  0 is no candidate.
__device__ __forceinline__ uint64_t key_of(float x, int token) {
    uint32_t u = __float_as_uint(x + 0.0f);                         // -0 becomes 0
    u = u & 0x80000000u ? ~u : u | 0x80000000u;
    return static_cast<uint64_t>(u) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(token));
}
__device__ __forceinline__ float key_logit(uint64_t k) {
    const uint32_t u = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int key_token(uint64_t k) { return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k)); }

// The value of lane ^ X.  Within 16 lanes by lane moves; 16 and 32 by the
// exchange of rows, whose two results hold each pair's even and odd row.
template <int X>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
    if constexpr (X == 1) return dpp<0xB1>(x);
    else if constexpr (X == 2) return dpp<0x4E>(x);
    else if constexpr (X == 3) return dpp<0x1B>(x);
    else if constexpr (X == 7) return dpp<0x141>(x);
    else if constexpr (X == 8) return dpp<0x128>(x);
    else if constexpr (X == 15) return dpp<0x140>(x);
    else if constexpr (X == 4) return lane_xor<3>(lane_xor<7>(x));
    else if constexpr (X == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        return threadIdx.x & 16 ? r[0] : r[1];
    } else if constexpr (X == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return threadIdx.x & 32 ? r[0] : r[1];
    } else if constexpr (X == 31) return lane_xor<16>(lane_xor<15>(x));
    else return lane_xor<32>(lane_xor<31>(x));          // 63
}
template <int X>
__device__ __forceinline__ uint64_t lane_xor64(uint64_t x) {
    return static_cast<uint64_t>(lane_xor<X>(static_cast<uint32_t>(x >> 32))) << 32 | lane_xor<X>(static_cast<uint32_t>(x));
}
__device__ __forceinline__ uint64_t lane64(uint64_t x, int lane) {
    return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x >> 32), lane))) << 32 |
           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(x)), lane));
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t x) {
    x = max(x, lane_xor64<1>(x));
    x = max(x, lane_xor64<2>(x));
    x = max(x, lane_xor64<7>(x));
    x = max(x, lane_xor64<15>(x));
    x = max(x, lane_xor64<16>(x));
    return max(x, lane_xor64<32>(x));
}

// One step of a sorting network, falling: of lanes i and i ^ X the one without BIT
// keeps the larger.
template <int X, int BIT>
__device__ __forceinline__ void exchange(uint64_t& k) {
    const uint64_t other = lane_xor64<X>(k);
    if ((other > k) == ((threadIdx.x & BIT) == 0)) k = other;
}
template <int X, int BIT>
__device__ __forceinline__ void exchange(float& x) {
    const float other = __uint_as_float(lane_xor<X>(__float_as_uint(x)));
    x = threadIdx.x & BIT ? fminf(x, other) : fmaxf(x, other);
}
// 64 values that rise and fall at most once, by halving distances.
template <typename T>
__device__ __forceinline__ void merge64(T& k) {
    exchange<32, 32>(k);
    exchange<16, 16>(k);
    exchange<8, 8>(k);
    exchange<4, 4>(k);
    exchange<2, 2>(k);
    exchange<1, 1>(k);
}
// 64 values in any order: sorted runs of 2, 4, .. 64, each the merge of two of
// half its length, the second taken backwards.
template <typename T>
__device__ __forceinline__ void sort64(T& k) {
    exchange<1, 1>(k);
    exchange<3, 2>(k);
    exchange<1, 1>(k);
    exchange<7, 4>(k);
    exchange<2, 2>(k);
    exchange<1, 1>(k);
    exchange<15, 8>(k);
    exchange<4, 4>(k);
    exchange<2, 2>(k);
    exchange<1, 1>(k);
    exchange<31, 16>(k);
    exchange<8, 8>(k);
    exchange<4, 4>(k);
    exchange<2, 2>(k);
    exchange<1, 1>(k);
    exchange<63, 32>(k);
    exchange<16, 16>(k);
    exchange<8, 8>(k);
    exchange<4, 4>(k);
    exchange<2, 2>(k);
    exchange<1, 1>(k);
}

struct StepArgs {
    const void* logits;
    const float* scores;
    const int32_t* tokens;
    const int32_t* history;
    const uint8_t* finished;
    float* scores_out;
    int32_t* tokens_out;
    int32_t* parents_out;
    int32_t* history_out;
    uint8_t* finished_out;
    uint64_t* keys;         // [rows][lists][beams], each list falling, 0 past its end
    Soft* soft;             // [rows][lists]
    int64_t ld;
    int64_t first;          // the launch's first row (scan) or sequence (join)
    int32_t v, beams, end;
    int32_t chunks;         // workgroups a row
    int32_t lists;          // wavefronts a row: 4 chunks
};

__device__ __forceinline__ bool alive(const StepArgs& a, int64_t row) { return a.scores[row] > kNegInf; }

constexpr int kScanWaves = 4;
constexpr int kAhead = 4;           // vectors of a lane at a time
constexpr int kRoom = 640;          // keys of a wavefront's buffer: below 64 kept plus 512 of one vector

// The 64 largest keys of buf[0 .. count), lane l the l-th; 0 past the last.
__device__ __forceinline__ uint64_t largest(const uint64_t* buf, int count, int lane) {
    uint64_t best = lane < count ? buf[lane] : 0;
    sort64(best);
    for (int i = 64; i < count; i += 64) {
        uint64_t more = i + lane < count ? buf[i + lane] : 0;
        sort64(more);
        best = max(best, lane_xor64<63>(more));         // the 64 largest of both, falling and rising once
        merge64(best);
    }
    return best;
}
// The `keep` largest keys of buf[0 .. count) to buf[0 .. keep).
__device__ __forceinline__ void compress(uint64_t* buf, int count, int keep, int lane) {
    const uint64_t best = largest(buf, count, lane);
    __builtin_amdgcn_wave_barrier();
    if (lane < keep) buf[lane] = best;
    __builtin_amdgcn_wave_barrier();
}

// One pass over the logits: a wavefront takes a run of a row's vectors, keeps
// the running maximum and sum of the softmax in each lane, and the `beams`
// largest logits in a buffer in LDS: an element above the threshold (the
// smallest kept so far) is appended, and the buffer is cut to the largest when
// it fills, which raises the threshold.  A wavefront's steps go upwards, so an
// element equal to the threshold has a higher token than those kept; within a step
// vectors go upwards too.
//
// Bound by memory where rows are many: 512 rows of 151936 fp32 take 60 us, 5.2
// TB/s.  Cutting by sorts of 64 keys:
// rounds of maxima, one for each beam, took 41 us against 23 for 176 rows of 109117 bf16
// with 16 beams.  Four rows of 151936 bf16: 8.4 us of loads that wait, sorts and the launch.
template <bool F32>
__global__ void __launch_bounds__(64 * kScanWaves) beam_scan_kernel(const StepArgs a) {
    constexpr int E = Row<F32>::E;
    constexpr float c = 1.44269504088896340736f;
    __shared__ uint64_t room[kScanWaves][kRoom];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = a.first + blockIdx.x / a.chunks;
    const int list = static_cast<int>(blockIdx.x % a.chunks) * kScanWaves + wave;
    if (!alive(a, row) || (a.finished && a.finished[row])) return;
    uint64_t* const buf = room[wave];
    const Row<F32> r(a.logits, row * a.ld, a.v);
    const int vectors = r.vectors();
    const int groups = (vectors + 63) / 64, per = (groups + a.lists - 1) / a.lists;
    const int from = list * per * 64, to = min(vectors, from + per * 64);
    Soft soft{kLowest, 0.0f};
    float thr = kNegInf;
    float low = kNegInf;                // of this step's elements, those below are not among the largest
    int count = 0;
    constexpr uint32_t kNothing = F32 ? 0xFF800000u : 0xFF80FF80u;
    u32x4 ahead[kAhead];
    const auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int i = i0 + 64 * u + lane;
            ahead[u] = u32x4{kNothing, kNothing, kNothing, kNothing};
            if (i < to) ahead[u] = r.load(i);
        }
    };
    fetch(from);
    for (int i0 = from; i0 < to; i0 += 64 * kAhead) {
        u32x4 raw[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) raw[u] = ahead[u];
        fetch(i0 + 64 * kAhead);
        float top = kNegInf;
#pragma unroll
        for (int k = 0; k < kAhead * E; ++k) top = fmaxf(top, Row<F32>::at(raw[k / E], k % E));
        const float m = fmaxf(soft.m, top);
        soft.s *= exp2_fast((soft.m - m) * c);
        soft.m = m;
        float e[kAhead * E];
#pragma unroll
        for (int k = 0; k < kAhead * E; ++k) e[k] = exp2_fast((Row<F32>::at(raw[k / E], k % E) - m) * c);
#pragma unroll
        for (int n = kAhead * E / 2; n > 0; n /= 2)
#pragma unroll
            for (int k = 0; k < n; ++k) e[k] += e[k + n];
        soft.s += e[0];
        if (__ballot(top > thr) == 0) continue;
        if (thr == kNegInf) {
            // nothing kept yet: the `beams` largest lane maxima bound the threshold from below
            float t = top;
            sort64(t);
            low = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(t), a.beams - 1));
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float x = Row<F32>::at(raw[u], k);
                const bool in = x > thr && x >= low;
                const uint64_t hit = __ballot(in);
                if (in) {
                    const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(hit >> 32),
                                                                 __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(hit), 0));
                    buf[count + before] = key_of(x, (i0 + 64 * u + lane) * E + k);
                }
                count += __popcll(hit);
            }
            if (count >= 64) {
                __builtin_amdgcn_wave_barrier();
                compress(buf, count, a.beams, lane);
                count = min(count, a.beams);
                if (count == a.beams) thr = key_logit(buf[count - 1]);
            }
        }
        // `beams` or more elements of this step reach `low`, and a later one equal to it has a higher token
        thr = fmaxf(thr, low);
        low = kNegInf;
    }
    __builtin_amdgcn_wave_barrier();
    const uint64_t best = largest(buf, count, lane);
    const int64_t at = row * a.lists + list;
    if (lane < a.beams) a.keys[at * a.beams + lane] = best;
    soft = soft_wave(soft, c);
    if (lane == 0) a.soft[at] = soft;
}

// A sequence's lists joined.  A wavefront a beam: the `beams`th largest of its
// lists' heads bounds its largest keys from below, so `beams` lists at most hold
// keys that reach it; those are gathered and sorted.  Then one wavefront merges the
// beams by score, each lane at the next place of one beam's list.  One sequence of
// four beams 5.6 us, 11 of 16 beams 11, 64 of eight 8: bound by dependent steps (loads,
// sorts, an fp64 logarithm, a maximum over lanes for each place).
constexpr int kJoinWaves = 16;

__global__ void __launch_bounds__(64 * kJoinWaves) beam_join_kernel(const StepArgs a) {
    extern __shared__ uint64_t gathered[];          // min(lists, beams) lists' keys, for each wavefront
    __shared__ uint64_t best[NGRAM_MAX_BEAMS][NGRAM_MAX_BEAMS], order_of[NGRAM_MAX_BEAMS][NGRAM_MAX_BEAMS];
    __shared__ int done[NGRAM_MAX_BEAMS];
    __shared__ int last[NGRAM_MAX_BEAMS][2];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row0 = (a.first + blockIdx.x) * a.beams;
    for (int b = wave; b < a.beams; b += static_cast<int>(blockDim.x >> 6)) {
        const int64_t row = row0 + b;
        const bool fin = a.finished && a.finished[row];
        double log_s = 0, m = 0;
        uint64_t out = 0;
        if (!alive(a, row)) {
            ;                                               // no candidate
        } else if (fin) {
            if (lane == 0) out = key_of(0.0f, a.end);       // its score and no more
        } else {
            // lists of this row: at most 64
            const uint64_t* const keys = a.keys + row * a.lists * a.beams;
            Soft s{kLowest, 0.0f};
            uint64_t head = 0;
            if (lane < a.lists) {
                s = a.soft[row * a.lists + lane];
                head = keys[lane * a.beams];
            }
            s = soft_wave(s, 1.44269504088896340736f);
            m = s.m;
            log_s = log(static_cast<double>(s.s));
            if (log_s == log_s) {                           // no NaN or +inf in the row
                sort64(head);
                const uint64_t least = lane64(head, a.beams - 1);
                uint64_t* const buf = gathered + static_cast<int64_t>(wave) * min(a.lists, a.beams) * a.beams;
                int count = 0;
                for (int i = 0; i < a.lists * a.beams; i += 64) {
                    const uint64_t k = i + lane < a.lists * a.beams ? keys[i + lane] : 0;
                    const uint64_t hit = __ballot(k != 0 && k >= least);
                    const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(hit >> 32),
                                                                 __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(hit), 0));
                    if (k != 0 && k >= least) buf[count + before] = k;
                    count += __popcll(hit);
                }
                __builtin_amdgcn_wave_barrier();
                out = largest(buf, count, lane);
                __builtin_amdgcn_wave_barrier();
            }
        }
        if (lane < a.beams) {
            // score + ((logit - max) - log sum exp(logits - max)), in an order that keeps the differences of
            // huge logits, as a number that orders candidates; 0 for none
            const double score = a.scores[row] + ((key_logit(out) - m) - log_s) + 0.0;
            const uint64_t u = __builtin_bit_cast(uint64_t, score);
            best[b][lane] = out;
            order_of[b][lane] = out && score > -__builtin_inf() ? u >> 63 ? ~u : u | (UINT64_C(1) << 63) : 0;
        }
        if (lane == 0) {
            done[b] = fin;
            if (a.history) {
                last[b][0] = a.history[2 * row + 1];
                last[b][1] = a.tokens[row];
            }
        }
    }
    __syncthreads();
    if (wave != 0) return;
    int taken = 0, from = -1, place = 0;                    // from, place: lane r's candidate
    uint64_t order = lane < a.beams ? order_of[lane][0] : 0, won = 0;
    for (int r = 0; r < a.beams; ++r) {
        const uint64_t top = wave_max64(order);
        if (top == 0) break;
        const int who = __builtin_ctzll(__ballot(order == top));            // ties to the lowest beam
        const int at = __builtin_amdgcn_readlane(taken, who);
        if (lane == r) {
            from = who;
            place = at;
            won = top;
        }
        if (lane == who) order = ++taken < a.beams ? order_of[lane][taken] : 0;
    }
    int token = -1, marked = 0, h0 = -1, h1 = -1;
    float score = kNegInf;
    if (lane >= a.beams) return;
    const int64_t to = row0 + lane;
    if (from >= 0) {
        token = key_token(best[from][place]);
        score = static_cast<float>(__builtin_bit_cast(double, won >> 63 ? won & ~(UINT64_C(1) << 63) : ~won));
        marked = done[from] || token == a.end;
        h0 = last[from][0];
        h1 = last[from][1];
    }
    a.scores_out[to] = score;
    if (a.tokens_out) a.tokens_out[to] = token;
    a.parents_out[to] = from;
    if (a.finished_out) a.finished_out[to] = static_cast<uint8_t>(marked);
    if (a.history_out) {
        a.history_out[2 * to] = h0;
        a.history_out[2 * to + 1] = h1;
    }
}

// Workgroups a row: enough rows fill the card with one each; few rows are cut,
// to 16 parts at most (64 lists, one a lane of the join) of 4096 elements and more.
// 1024 workgroups and more: 64 x 8 x 151936 fp32 70 us (512: 92), 11 x 16 x 109117 bf16 37 (42).  4096 elements:
// 8 x 4 x 50257 11.7 us (8192: 12.5), 1 x 8 x 5003 11.8 (13.2); 2048 changes nothing.
int chunks_of(int64_t rows, int64_t v) {
    const int64_t want = (1024 + rows - 1) / std::max<int64_t>(rows, 1);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, 16, (v + 4095) / 4096})));
}

bool step_sizes_ok(int64_t batch, int32_t beams, int64_t v, int32_t dtype) {
    return batch >= 0 && batch <= NGRAM_FP8_MAX && beams >= 1 && beams <= NGRAM_MAX_BEAMS && v >= 1 && v < NGRAM_PAD_ID &&
           (dtype == NGRAM_F32 || dtype == NGRAM_BF16);
}
int64_t step_bytes(int64_t rows, int lists, int beams) { return rows * lists * (8 * static_cast<int64_t>(beams) + sizeof(Soft)); }

// ---------------------------------------------------------------------------
// Reordering.  A thread owns one column of 16, 4 or 1 bytes of a sequence's
// rows: it reads what every row that changes takes, then writes those
// rows, so nothing is read after it was overwritten and rows that stay move
// no bytes.  24 states of 128 rows of 256 KB: 237 us, a copy's rate (5.0 TB/s); with
// addresses in registers of each lane instead of uniform ones 378.
constexpr int kStates = 64;

struct ReorderArgs {
    const int32_t* parents;
    int32_t beams;
    int32_t count;
    int64_t first;                      // the launch's first workgroup
    int64_t start[kStates + 1];         // the first workgroup of each state
    ngram_beam_state state[kStates];
};

template <int B, typename T>
__device__ __forceinline__ void reorder_columns(char* base, int64_t stride, bool on, const int* parent) {
    const uint32_t at = threadIdx.x * static_cast<uint32_t>(sizeof(T));
    T v[B];
    if (!on) return;
#pragma unroll
    for (int b = 0; b < B; ++b)
        if (parent[b] >= 0) v[b] = *reinterpret_cast<const T*>(base + parent[b] * stride + at);
#pragma unroll
    for (int b = 0; b < B; ++b)
        if (parent[b] >= 0) *reinterpret_cast<T*>(base + b * stride + at) = v[b];
}

inline __host__ __device__ int unit_of(const ngram_beam_state& s) {
    const uint64_t u = reinterpret_cast<uint64_t>(s.data) | static_cast<uint64_t>(s.row_bytes) | static_cast<uint64_t>(s.stride);
    return u % 16 == 0 ? 16 : u % 4 == 0 ? 4 : 1;
}

template <int B>
__global__ void __launch_bounds__(256) beam_reorder_kernel(const ReorderArgs a) {
    const int64_t wg = a.first + blockIdx.x;
    int s = 0;
    while (s + 1 < a.count && wg >= a.start[s + 1]) ++s;
    const ngram_beam_state st = a.state[s];
    const int unit = unit_of(st);
    const int64_t columns = st.row_bytes / unit;
    const uint32_t blocks = static_cast<uint32_t>((columns + 255) / 256), at = static_cast<uint32_t>(wg - a.start[s]);
    const uint32_t seq = at / blocks, block = at - seq * blocks;
    // the parent of each row that changes, or -1; addresses are uniform but for the thread's distance
    int parent[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        parent[b] = -1;
        if (b < a.beams) {
            const int p = __builtin_amdgcn_readfirstlane(a.parents[static_cast<int64_t>(seq) * a.beams + b]);
            if (p >= 0 && p < a.beams && p != b) parent[b] = p;
        }
    }
    char* const base = static_cast<char*>(st.data) + static_cast<int64_t>(seq) * a.beams * st.stride + static_cast<int64_t>(block) * 256 * unit;
    const bool on = static_cast<int64_t>(block) * 256 + threadIdx.x < columns;
    if (unit == 16) reorder_columns<B, u32x4>(base, st.stride, on, parent);
    else if (unit == 4) reorder_columns<B, uint32_t>(base, st.stride, on, parent);
    else reorder_columns<B, uint8_t>(base, st.stride, on, parent);
}

}  // namespace
}  // namespace ng8

using namespace ng8;

extern "C" {

int64_t ngram_beam_step_workspace_bytes(int64_t batch, int32_t beams, int64_t V, int32_t dtype) {
    if (!step_sizes_ok(batch, beams, V, dtype)) return -1;
    return step_bytes(batch * beams, kScanWaves * chunks_of(batch * beams, V), beams);
}

int ngram_beam_step(const void* logits, int32_t dtype, int64_t batch, int32_t beams, int64_t V, int64_t ld,
                    const float* scores, const int32_t* tokens, const int32_t* history, const uint8_t* finished,
                    int32_t end_token, float* scores_out, int32_t* tokens_out, int32_t* parents_out,
                    int32_t* history_out, uint8_t* finished_out, void* workspace, int64_t workspace_bytes,
                    ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    if (batch < 0) return fail(NGRAM_EINVAL, "batch=%lld is negative", (long long)batch);
    if (dtype != NGRAM_F32 && dtype != NGRAM_BF16) return fail(NGRAM_EINVAL, "dtype=%d is not an ngram_value", dtype);
    if (!step_sizes_ok(batch, beams, V, dtype))
        return fail(NGRAM_ERANGE, "batch=%lld, beams=%d (1 to %d) or V=%lld (1 to %d) out of range", (long long)batch, beams, NGRAM_MAX_BEAMS,
                    (long long)V, NGRAM_PAD_ID - 1);
    if (ld < V) return fail(NGRAM_EINVAL, "ld=%lld is below V=%lld", (long long)ld, (long long)V);
    if (end_token < -1 || end_token >= V) return fail(NGRAM_EINVAL, "end_token=%d is neither -1 nor a token", end_token);
    if (finished && end_token < 0) return fail(NGRAM_EINVAL, "finished beams need an end_token");
    if ((history != nullptr) != (history_out != nullptr) || (history && !tokens))
        return fail(NGRAM_EINVAL, "history, tokens and history_out go together");
    if (batch == 0) return NGRAM_OK;
    if (!logits || !scores || !scores_out || !parents_out) return fail(NGRAM_EINVAL, "logits, scores, scores_out or parents_out is NULL");
    if (!aligned(logits, dtype == NGRAM_F32 ? 4 : 2) || !aligned(scores, 4) || !aligned(tokens, 4) || !aligned(history, 4) ||
        !aligned(scores_out, 4) || !aligned(tokens_out, 4) || !aligned(parents_out, 4) || !aligned(history_out, 4))
        return fail(NGRAM_EALIGN, "an argument is not aligned to its elements");
    StepArgs a = {};
    const int64_t rows = batch * beams;
    a.logits = logits; a.scores = scores; a.tokens = tokens; a.history = history; a.finished = finished;
    a.scores_out = scores_out; a.tokens_out = tokens_out; a.parents_out = parents_out; a.history_out = history_out; a.finished_out = finished_out;
    a.ld = ld; a.v = static_cast<int32_t>(V); a.beams = beams; a.end = end_token;
    a.chunks = chunks_of(rows, V); a.lists = kScanWaves * a.chunks;
    const int64_t need = step_bytes(rows, a.lists, beams);
    if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
        return fail(NGRAM_EINVAL, "workspace must hold %lld bytes, 16-byte aligned", (long long)need);
    a.keys = static_cast<uint64_t*>(workspace);
    a.soft = reinterpret_cast<Soft*>(a.keys + rows * a.lists * beams);
    const int64_t most = most_groups(64 * kScanWaves) / a.chunks;
    for (a.first = 0; a.first < rows; a.first += most) {
        const dim3 grid(static_cast<uint32_t>(std::min(most, rows - a.first) * a.chunks));
        if (dtype == NGRAM_F32) hipLaunchKernelGGL(beam_scan_kernel<true>, grid, dim3(64 * kScanWaves), 0, stream, a);
        else hipLaunchKernelGGL(beam_scan_kernel<false>, grid, dim3(64 * kScanWaves), 0, stream, a);
    }
    const int row_room = std::min(a.lists, beams) * beams * 8, waves = std::min(beams, kJoinWaves), room = waves * row_room;
    for (a.first = 0; a.first < batch; a.first += most_groups(64 * waves))
        hipLaunchKernelGGL(beam_join_kernel, dim3(static_cast<uint32_t>(std::min(most_groups(64 * waves), batch - a.first))),
                           dim3(64 * waves), room, stream, a);
    return hip_status("ngram_beam_step");
}

int ngram_beam_reorder(const ngram_beam_state* states, int32_t count, const int32_t* parents, int64_t batch, int32_t beams,
                       ngram_stream_t stream) {
    fail(NGRAM_OK, "%s", "");
    if (count < 0 || batch < 0) return fail(NGRAM_EINVAL, "count=%d or batch=%lld is negative", count, (long long)batch);
    if (beams < 1 || beams > NGRAM_MAX_BEAMS || batch > NGRAM_FP8_MAX)
        return fail(NGRAM_ERANGE, "beams=%d (1 to %d) or batch=%lld out of range", beams, NGRAM_MAX_BEAMS, (long long)batch);
    if (count > 0 && !states) return fail(NGRAM_EINVAL, "states is NULL");
    for (int i = 0; i < count; ++i) {
        const ngram_beam_state& s = states[i];
        if (s.row_bytes < 0 || s.stride < s.row_bytes)
            return fail(NGRAM_EINVAL, "state %d: row_bytes=%lld must not be negative nor above stride=%lld", i, (long long)s.row_bytes, (long long)s.stride);
        // a state's workgroups are counted in 32 bits
        if (s.row_bytes > (INT64_C(1) << 40) || (s.row_bytes / unit_of(s) / 256 + 1) * std::max<int64_t>(batch, 1) > INT64_C(0x7FFFFFFF))
            return fail(NGRAM_ERANGE, "state %d: row_bytes=%lld for %lld sequences is out of range", i, (long long)s.row_bytes, (long long)batch);
        if (s.row_bytes > 0 && batch > 0 && !s.data) return fail(NGRAM_EINVAL, "state %d: data is NULL", i);
    }
    if (batch == 0 || count == 0) return NGRAM_OK;
    if (!parents) return fail(NGRAM_EINVAL, "parents is NULL");
    if (!aligned(parents, 4)) return fail(NGRAM_EALIGN, "parents must be 4-byte aligned");
    for (int at = 0; at < count; at += kStates) {
        ReorderArgs a = {};
        a.parents = parents;
        a.beams = beams;
        int64_t total = 0;
        for (int i = at; i < std::min(count, at + kStates); ++i) {
            if (states[i].row_bytes == 0) continue;
            const int64_t blocks = (states[i].row_bytes / unit_of(states[i]) + 255) / 256;
            a.start[a.count] = total;
            a.state[a.count++] = states[i];
            total += batch * blocks;
        }
        a.start[a.count] = total;
        for (a.first = 0; a.first < total; a.first += most_groups(256)) {
            const dim3 grid(static_cast<uint32_t>(std::min(most_groups(256), total - a.first))), block(256);
            if (beams <= 4) hipLaunchKernelGGL(beam_reorder_kernel<4>, grid, block, 0, stream, a);
            else if (beams <= 16) hipLaunchKernelGGL(beam_reorder_kernel<16>, grid, block, 0, stream, a);
            else hipLaunchKernelGGL(beam_reorder_kernel<32>, grid, block, 0, stream, a);
        }
    }
    return hip_status("ngram_beam_reorder");
}

}  // extern "C"
