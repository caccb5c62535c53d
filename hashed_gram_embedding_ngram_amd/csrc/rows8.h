// Rows of logits for the kernels that walk a vocabulary: rows of any length at
// any element-aligned address, read and written in vectors of 16 bytes.
#ifndef NGRAM_ROWS8_H
#define NGRAM_ROWS8_H

#include "common8.h"

namespace ng8 {

constexpr float kNegInf = -__builtin_inff();

typedef u32x4 Loose __attribute__((aligned(2)));        // 16 bytes at any element

// A row of V elements; vector i has elements E i .. E i + E - 1, whatever the
// row's alignment (the hardware reads and writes 16 bytes at any element's
// address), so sums of equal rows run in the same order wherever they lie.
template <bool F32>
struct Row {
    static constexpr int E = F32 ? 4 : 8;
    char* base;
    int64_t v;

    __device__ __forceinline__ Row(const void* p, int64_t at, int64_t len)
        : base(const_cast<char*>(static_cast<const char*>(p)) + at * (F32 ? 4 : 2)), v(len) {}
    __device__ __forceinline__ int vectors() const { return static_cast<int>((v + E - 1) / E); }
    __device__ __forceinline__ bool whole(int i) const { return static_cast<int64_t>(i + 1) * E <= v; }
    __device__ __forceinline__ float element(int64_t j) const {      // 0 <= j < v
        const char* const p = base + j * (F32 ? 4 : 2);
        return F32 ? *reinterpret_cast<const float*>(p)
                   : __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
    }
    __device__ __forceinline__ u32x4 load_whole(int i) const { return *reinterpret_cast<const Loose*>(base + static_cast<int64_t>(i) * 16); }
    __device__ __forceinline__ void store_whole(int i, const u32x4& x) const { *reinterpret_cast<Loose*>(base + static_cast<int64_t>(i) * 16) = x; }
    // past the caches' usual keeping
    __device__ __forceinline__ void store_stream(int i, const u32x4& x) const {
        __builtin_nontemporal_store(x, reinterpret_cast<Loose*>(base + static_cast<int64_t>(i) * 16));
    }
    // The 16 bytes of vector i; places past the row are -inf, and no byte past
    // it is read.
    __device__ __forceinline__ u32x4 load(int i) const {
        if (whole(i)) return load_whole(i);
        u32x4 r;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t j = static_cast<int64_t>(i) * E + k * (E / 4);
            if (F32) {
                r[k] = j < v ? __float_as_uint(element(j)) : 0xFF800000u;
            } else {
                const uint32_t lo = j < v ? __float_as_uint(element(j)) >> 16 : 0xFF80u;
                const uint32_t hi = j + 1 < v ? __float_as_uint(element(j + 1)) : 0xFF800000u;
                r[k] = lo | (hi & 0xFFFF0000u);
            }
        }
        return r;
    }
    __device__ __forceinline__ void store(int i, const u32x4& x) const {
        if (whole(i)) {
            store_whole(i, x);
            return;
        }
#pragma unroll
        for (int k = 0; k < E; ++k) {
            const int64_t j = static_cast<int64_t>(i) * E + k;
            if (j >= v) continue;
            if (F32) reinterpret_cast<uint32_t*>(base)[j] = x[k & 3];
            else reinterpret_cast<uint16_t*>(base)[j] = static_cast<uint16_t>(x[(k >> 1) & 3] >> (16 * (k & 1)));
        }
    }
    template <bool STREAM>
    __device__ __forceinline__ void put(int i, const u32x4& x) const {
        if (!whole(i)) store(i, x);
        else if (STREAM) store_stream(i, x);
        else store_whole(i, x);
    }
    static __device__ __forceinline__ float at(const u32x4& r, int k) {      // k a constant once unrolled
        if (F32) return __uint_as_float(r[k & 3]);
        return k & 1 ? bf16_hi(r[k >> 1]) : bf16_lo(r[k >> 1]);
    }
};

// The largest of a value over the wavefront, in all lanes (NaN left out).
__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, __uint_as_float(dpp<0xB1>(__float_as_uint(x))));
    x = fmaxf(x, __uint_as_float(dpp<0x4E>(__float_as_uint(x))));
    x = fmaxf(x, __uint_as_float(dpp<0x141>(__float_as_uint(x))));
    x = fmaxf(x, __uint_as_float(dpp<0x140>(__float_as_uint(x))));
    const int i = static_cast<int>(__float_as_uint(x));
    const float a = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 0)));
    const float b = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 16)));
    const float c = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 32)));
    const float d = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 48)));
    return fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// Running maximum and sum of exp((z - m) c'), c' = log2(e) / temperature, of a
// set of logits.  The empty set is (lowest, 0), so that no difference of two
// infinities is formed; a NaN or +inf makes the sum NaN.
constexpr float kLowest = -3.4028234663852886e38f;

struct Soft {
    float m, s;
};
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ Soft soft_join(Soft a, Soft b, float c) {
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * exp2_fast((a.m - m) * c) + b.s * exp2_fast((b.m - m) * c)};
}
__device__ __forceinline__ Soft soft_wave(Soft x, float c) {
    const float m = wave_max(x.m);
    return {m, wave_sum(x.s * exp2_fast((x.m - m) * c))};
}

}  // namespace ng8
#endif
