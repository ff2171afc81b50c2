// qar_kv8_device.h -- what the kernels of the 8-bit cache share: its elements,
// and the arithmetic of attention over it.
#pragma once

#include <float.h>
#include <hip/hip_runtime.h>

#include "qar_device.h"
#include "qar_launch.h"
#include "qar_serve.h"

namespace qar {

typedef _Float16 kv_half8 __attribute__((ext_vector_type(8)));
typedef _Float16 kv_half2 __attribute__((ext_vector_type(2)));
typedef float kv_f32x4 __attribute__((ext_vector_type(4)));
typedef float kv_f32x16 __attribute__((ext_vector_type(16)));

constexpr int kPage = 64;

// ---------------------------------------------------------------------------
// small pieces

__device__ __forceinline__ int32_t valid_page(int32_t id, uint32_t pages) { return (uint32_t)id < pages ? id : -1; }

__device__ __forceinline__ int32_t clamp_length(int32_t n, uint32_t top) {
    return n < 0 ? 0 : (uint32_t)n > top ? (int32_t)top : n;
}

// Elements e .. e + 3 (a multiple of 4, aligned) as binary32.
template <int IN>
__device__ __forceinline__ kv_f32x4 load4(const void* x, size_t e) {
    if constexpr (IN == kInBF16) {
        const uint2 q = *reinterpret_cast<const uint2*>((const uint16_t*)x + e);
        return kv_f32x4{bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
    } else {
        return *reinterpret_cast<const kv_f32x4*>((const float*)x + e);
    }
}

// Elements e .. e + 7, each read once by the caller.
template <int IN>
__device__ __forceinline__ void load8(const void* x, size_t e, kv_f32x4 (&v)[2]) {
    if constexpr (IN == kInBF16) {
        const uint4 q = load_b128((const uint16_t*)x + e);
        v[0] = kv_f32x4{bf16_lo(q.x), bf16_hi(q.x), bf16_lo(q.y), bf16_hi(q.y)};
        v[1] = kv_f32x4{bf16_lo(q.z), bf16_hi(q.z), bf16_lo(q.w), bf16_hi(q.w)};
    } else {
        v[0] = __builtin_bit_cast(kv_f32x4, load_b128((const float*)x + e));
        v[1] = __builtin_bit_cast(kv_f32x4, load_b128((const float*)x + e + 4));
    }
}

template <int OUT>
__device__ __forceinline__ void store4(void* x, size_t e, kv_f32x4 v) {
    if constexpr (OUT == kOutBF16)
        store_b64((uint16_t*)x + e, make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
    else
        store_b128((float*)x + e, __builtin_bit_cast(uint4, v));
}

// The same for stores that fill a line piece by piece: these wait in the
// cache for the rest of it.
template <int OUT>
__device__ __forceinline__ void merge4(void* x, size_t e, kv_f32x4 v) {
    if constexpr (OUT == kOutBF16)
        *reinterpret_cast<uint2*>((uint16_t*)x + e) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    else
        *reinterpret_cast<kv_f32x4*>((float*)x + e) = v;
}

__device__ __forceinline__ kv_f32x4 values4(uint32_t w, float s) {
    return kv_f32x4{code_f32(w, 0) * s, code_f32(w, 1) * s, code_f32(w, 2) * s, code_f32(w, 3) * s};
}

__device__ __forceinline__ float absmax4(kv_f32x4 v, float m) {
    return fmaxf(fmaxf(fmaxf(m, fabsf(v[0])), fmaxf(fabsf(v[1]), fabsf(v[2]))), fabsf(v[3]));
}

// 4 x 4 bytes: word i of the result holds byte i of each of the four words.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);
    const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
    w[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
    w[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
    w[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
    w[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// ---------------------------------------------------------------------------
// attention's arithmetic
//
// Codes are exact in binary16, so the cache enters the products without
// rounding.  A query row enters multiplied by the power of two that brings
// its largest magnitude into [2^14, 2^15): bfloat16's 8 bits are then exact
// for all but elements 2^29 times smaller than the row's largest; binary32
// queries are split in two binary16 terms (an error of 2^-23 of an element, or
// of 2^-39 of the row's largest where that is more).  The softmax's numerators
// enter the second product multiplied by 2^14, in one term (an error of at most
// 2^-11 of each, for outputs that are rounded to 2^-8) or, for binary32, two.
// Sums, maxima and outputs are binary32.
//
// A page's value scale enters with the numerators, as its ratio to the largest
// scale so far (`Unit`), so that the second product adds to the outputs
// directly; these are in that largest scale's units.  The ratio is at most 1
// and costs nothing (its logarithm is part of the exponent); numerators times
// ratio below 2^-28 of the row's largest are binary16 subnormals, off by up
// to 2^-39 of the largest scale's values.
constexpr float kLift = 14.0f;          // log2 of the numerators' factor

struct Unit {
    float unit = 0.0f;   // outputs are in units of this scale
    float lift = kLift;  // log2 of the numerators' factor for this page ...
    float drop = 1.0f;   // ... and what undoes the ratio in it
    // The next page's scale; returns what the outputs so far are multiplied by.
    __device__ __forceinline__ float next(float scale) {
        float shrink = 1.0f;
        if (scale > unit) {
            shrink = unit / scale;
            unit = scale;
        }
        // a ratio below 2^-60 leaves nothing of the page, but its numerators still count;
        // hardware reciprocals and logarithms are good to a unit in the last place
        const float ratio = unit > 0.0f ? fminf(fmaxf(scale * __builtin_amdgcn_rcpf(unit), 0x1p-60f), 1.0f) : 1.0f;
        lift = kLift + __builtin_amdgcn_logf(ratio);
        drop = __builtin_amdgcn_rcpf(ratio);
        return shrink;
    }
};

// One instruction, which the compiler forms itself: it counts the wait states
// between a matrix instruction and a vector instruction that reads its result,
// but not for inline assembly.
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// The maximum and the sum over lanes i, i + 32 and over lanes i, i + 16, ...:
// each exchange swaps half the rows of two copies of v, so that a lane has its
// own value in one and its partner's in the other.
struct Pair {
    float a, b;
};
__device__ __forceinline__ Pair with_lane_32(float v) {
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    const uint32_t a = r[0], b = r[1];
    return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ Pair with_lane_16(float v) {
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    const uint32_t a = r[0], b = r[1];
    return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ __forceinline__ float max_over_32(float v) {
    const Pair p = with_lane_32(v);
    return fmaxf(p.a, p.b);
}
__device__ __forceinline__ float max_over_16(float v) {
    const Pair p = with_lane_16(v);
    return max_over_32(fmaxf(p.a, p.b));
}
__device__ __forceinline__ float sum_over_32(float v) {
    const Pair p = with_lane_32(v);
    return p.a + p.b;
}
__device__ __forceinline__ float sum_over_16(float v) {
    const Pair p = with_lane_16(v);
    return sum_over_32(p.a + p.b);
}

// Eight codes as binary16: the byte of code + 128 under the high byte 0x64
// is 1024 + 128 + code, from which 1152 is taken exactly.
__device__ __forceinline__ kv_half8 half_codes(uint32_t lo, uint32_t hi) {
    const kv_half2 bias = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    uint32_t w[4];
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    w[0] = __builtin_amdgcn_perm(0x64646464u, lo, 0x04010400u);
    w[1] = __builtin_amdgcn_perm(0x64646464u, lo, 0x04030402u);
    w[2] = __builtin_amdgcn_perm(0x64646464u, hi, 0x04010400u);
    w[3] = __builtin_amdgcn_perm(0x64646464u, hi, 0x04030402u);
    uint4 q;
    q.x = __builtin_bit_cast(uint32_t, __builtin_bit_cast(kv_half2, w[0]) + bias);
    q.y = __builtin_bit_cast(uint32_t, __builtin_bit_cast(kv_half2, w[1]) + bias);
    q.z = __builtin_bit_cast(uint32_t, __builtin_bit_cast(kv_half2, w[2]) + bias);
    q.w = __builtin_bit_cast(uint32_t, __builtin_bit_cast(kv_half2, w[3]) + bias);
    return __builtin_bit_cast(kv_half8, q);
}

// Eight binary32 values as T binary16 terms.
template <int T>
__device__ __forceinline__ void half_terms(const float (&x)[8], kv_half8 (&out)[T]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[0][i] = (_Float16)x[i];
    if constexpr (T == 2) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[1][i] = (_Float16)(x[i] - (float)out[0][i]);
    }
}

// A lane's share of a query row: runs of RUN channels from channel `first`,
// one every STEP.  Loading and converting are apart so that the cache's loads
// can be issued between them.  OVER: the lanes that hold the row's other
// channels.
template <int IN, int DIM, int RUN, int STEP>
struct Query {
    static constexpr int N = DIM / STEP * (RUN / 8);
    kv_f32x4 x[N][2];
    __device__ __forceinline__ void load(const void* q, size_t row, int first, bool there) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const size_t e = row * DIM + i / (RUN / 8) * STEP + first + i % (RUN / 8) * 8;
            x[i][0] = x[i][1] = kv_f32x4{};
            if (there) {
                x[i][0] = load4<IN>(q, e);
                x[i][1] = load4<IN>(q, e + 4);
            }
        }
    }
    // binary16 fragments of eight; returns what undoes the row's factor
    template <int OVER, int T>
    __device__ __forceinline__ float convert(bool negative, kv_half8 (&out)[N][T]) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) m = absmax4(x[i][1], absmax4(x[i][0], m));
        m = OVER == 16 ? max_over_16(m) : max_over_32(m);
        const int e = min(268 - (int)(__builtin_bit_cast(uint32_t, m) >> 23), 253);
        const float f = __builtin_bit_cast(float, (uint32_t)e << 23 | (negative ? 0x80000000u : 0u));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = x[i][k / 4][k % 4] * f;
            half_terms<T>(y, out[i]);
        }
        return __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
    }
};

template <int OUT>
__device__ __forceinline__ void store1(void* x, size_t e, float v) {
    if constexpr (OUT == kOutBF16)
        ((uint16_t*)x)[e] = (uint16_t)pack_bf16x2(v, 0.0f);
    else
        ((float*)x)[e] = v;
}

__device__ __forceinline__ uint32_t exchange_bits_2_3(uint32_t v) {
    return (v & ~12u) | (v & 4u) << 1 | (v & 8u) >> 1;
}

// A barrier for LDS alone: __syncthreads would also wait for the loads from
// memory that are under way.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// 16 bytes for each lane to LDS, the lanes' one behind the other from `to`,
// which is the wave's.
__device__ __forceinline__ void to_lds(const void* from, void* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

} // namespace qar
