// What the 8-bit sources share: host-side checks and errors, lane
// reductions, and the E4M3 / E8M0 block format.
#ifndef NGRAM_COMMON8_H
#define NGRAM_COMMON8_H

#include <hip/hip_runtime.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "ngram.h"

namespace ng8 {

constexpr int kBlock = NGRAM_FP8_BLOCK;         // columns per scale
constexpr int kVec = 8;                         // elements per lane
constexpr int kSlice = 64 * kVec;               // columns per wavefront chunk: four scale blocks
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kUnitScale = 127;            // the E8M0 byte of 1

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Host side.

// Formats this thread's message (the 512-byte buffer that ngram_last_error()
// returns and the library's first source file owns; empty for OK).
int fail(int status, const char* fmt, ...);
int hip_status(const char* what);
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t blocks_of(int64_t cols) { return (cols + kBlock - 1) / kBlock; }
inline int64_t code_ld(int64_t cols) { return blocks_of(cols) * kBlock; }
inline int64_t scale_ld(int64_t cols) { return (blocks_of(cols) + 3) / 4 * 4; }
inline size_t value_bytes(int dtype) { return dtype == NGRAM_F32 ? 4 : 2; }
// The most workgroups of a launch: 2^32 and more work items in a dimension are
// not run in full, and no error tells.  Larger work goes in several launches.
inline int64_t most_groups(int threads) { return INT64_C(0xFFFFFFFF) / threads; }
// Checks a caller's 8-bit matrix; `what` names it in the message.
int check_fp8(const ngram_fp8* q, const char* what);

// ---------------------------------------------------------------------------
// Device side: moves between the 16 lanes of a row, and sums over the 64.

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xF, 0xF, false));
}

// The largest x of the lane's group of 16, in all 16 lanes.
__device__ __forceinline__ uint32_t max16(uint32_t x) {
    x = max(x, dpp<0xB1>(x));       // quad_perm [1,0,3,2]
    x = max(x, dpp<0x4E>(x));       // quad_perm [2,3,0,1]
    x = max(x, dpp<0x141>(x));      // row_half_mirror
    return max(x, dpp<0x140>(x));   // row_mirror
}

// The sum of x over the wavefront, in all lanes; the order of the additions
// is fixed and the same for every lane.
__device__ __forceinline__ float wave_sum(float x) {
    x = x + __uint_as_float(dpp<0xB1>(__float_as_uint(x)));
    x = x + __uint_as_float(dpp<0x4E>(__float_as_uint(x)));
    x = x + __uint_as_float(dpp<0x141>(__float_as_uint(x)));
    x = x + __uint_as_float(dpp<0x140>(__float_as_uint(x)));
    const int i = static_cast<int>(__float_as_uint(x));
    const float a = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 0)));
    const float b = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 16)));
    const float c = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 32)));
    const float d = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(i, 48)));
    return (a + b) + (c + d);
}

// Two fp32 values to bf16, nearest, ties to even, in one instruction (for all
// 2^32 values the same bits as rounding by hand; a NaN stays a NaN).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}
__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Eight consecutive elements from p + i, which is 16-byte aligned (bf16) or
// 32-byte aligned within a 16-byte aligned fp32 array.
template <bool F32>
struct Raw8 {
    u32x4 a, b;
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        if (F32) {
            const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
            a = s[0];
            b = s[1];
        } else {
            a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
        }
    }
    // the same past the caches' usual keeping: read once, by one lane
    __device__ __forceinline__ void load_stream(const void* p, int64_t i) {
        if (F32) {
            const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + i);
            a = __builtin_nontemporal_load(s);
            b = __builtin_nontemporal_load(s + 1);
        } else {
            a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i));
        }
    }
    __device__ __forceinline__ void zero() { a = u32x4{0, 0, 0, 0}; b = u32x4{0, 0, 0, 0}; }
    __device__ __forceinline__ float at(int k) const {      // k a constant once unrolled
        if (F32) return __uint_as_float(k < 4 ? a[k & 3] : b[k & 3]);
        return k & 1 ? bf16_hi(a[k >> 1]) : bf16_lo(a[k >> 1]);
    }
    __device__ __forceinline__ void get(float v[8]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (F32) {
                v[k] = __uint_as_float(a[k]);
                v[4 + k] = __uint_as_float(b[k]);
            } else {
                v[2 * k] = bf16_lo(a[k]);
                v[2 * k + 1] = bf16_hi(a[k]);
            }
        }
    }
};

// ---------------------------------------------------------------------------
// Block format: codes are E4M3 (largest finite value 448 = 1.75 * 2^8), the
// scale of a block is 2^e with the smallest e >= -126 for which no finite
// value of the block exceeds 448 * 2^e, stored as the byte e + 127; a block
// without a finite nonzero value has e = 0.  Infinities and NaN become the
// NaN code and do not count for e.

// The largest |x| of x[0..7], NaN left out, as bits (v_max_f32 returns its
// other operand where one is NaN).
__device__ __forceinline__ uint32_t amax_bits(const float x[8]) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
    return __float_as_uint(m);
}
// The same over finite values only.
__device__ __forceinline__ uint32_t finite_amax_bits(const float x[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t u = __float_as_uint(x[k]) & 0x7FFFFFFFu;
        m = max(m, u < kInfBits ? u : 0u);
    }
    return m;
}
// The scale byte of a block whose largest finite magnitude has these bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int e = static_cast<int>(amax >> 23) - 135 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return amax == 0 ? kUnitScale : static_cast<uint32_t>(max(e, -126) + 127);
}
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }     // 2^e, e >= -126
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254 - byte) << 23); }   // 2^-e
// The scale byte of the lane's block of 128 (its group of 16 lanes, eight
// elements each).  A block that holds an infinity takes a second look at
// its finite values; the wavefront branches only where one does.
__device__ __forceinline__ uint32_t block_scale16(const float x[8]) {
    uint32_t m = max16(amax_bits(x));
    if (__builtin_expect(__ballot(m >= kInfBits) != 0, 0)) m = max16(finite_amax_bits(x));
    return scale_byte(m);
}
// Four codes: E4M3 nearest-even of x * inv (exact scaling: inv is a power of
// two).  Callers pass |x * inv| <= 448 for finite x; the conversion gives the
// NaN code for infinities and NaN.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv) {
    const int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true));
}
__device__ __forceinline__ void codes8_to_f32(u32x2 c, float v[8]) {
    typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[k]), false);
        const f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(c[k]), true);
        v[4 * k] = lo[0];
        v[4 * k + 1] = lo[1];
        v[4 * k + 2] = hi[0];
        v[4 * k + 3] = hi[1];
    }
}

}  // namespace ng8
#endif
