// qar_mx4.hip -- microscaled 4-bit floating point on gfx950: quantize,
// dequantize, and the product of 4-bit weights with activations that are
// quantized on the way.
//
// A block is 32 consecutive elements of a row: 32 E2M1 codes (16 bytes, the
// even element in the low nibble) and one byte e that stands for 2^(e-127).
// With the block's largest magnitude in [2^p, 2^(p+1)) the scale is 2^(p-2):
// that maps it into [4, 8), and what lies above 6 becomes 6.  Codes are the
// nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, the even code where two are as near,
// the sign kept; the hardware's scaled conversions do exactly that
// (tests/test_gpu_mx4.py compares them with the definition).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qar_device.h"
#include "qar_launch.h"
#include "qar_serve.h"

namespace qar {
namespace {

typedef int mx_i32x8 __attribute__((ext_vector_type(8)));
typedef int mx_i32x4 __attribute__((ext_vector_type(4)));
typedef float mx_f32x4 __attribute__((ext_vector_type(4)));
typedef float mx_f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned short mx_u16x2 __attribute__((ext_vector_type(2)));

constexpr int kE2M1 = 4;                // the matrix instructions' format code
constexpr uint32_t kScaleOfZero = 124;  // an all-zero block: exponent 0 - 3

// The scale byte of a block from the bits of its largest magnitude (binary32;
// bf16 values enter with their bits shifted up).
__device__ __forceinline__ uint32_t scale_byte(uint32_t peak) {
    const int e = (int)(peak >> 23) - 2;
    return peak == 0 ? kScaleOfZero : (uint32_t)min(max(e, 1), 252);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
    // 2^-127 is a subnormal; the quantizer never makes it, a caller's weights may
    return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

// Eight elements as they lie in memory: bf16 pairs or binary32.
template <int IN>
struct Eight {
    uint32_t w[IN == kInBF16 ? 4 : 8];
};

template <int IN>
__device__ __forceinline__ Eight<IN> load8(const void* x, size_t e) {
    Eight<IN> v;
    if constexpr (IN == kInBF16) {
        const uint4 q = *reinterpret_cast<const uint4*>((const uint16_t*)x + e);
        v.w[0] = q.x, v.w[1] = q.y, v.w[2] = q.z, v.w[3] = q.w;
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>((const float*)x + e);
        const uint4 b = *reinterpret_cast<const uint4*>((const float*)x + e + 4);
        v.w[0] = a.x, v.w[1] = a.y, v.w[2] = a.z, v.w[3] = a.w;
        v.w[4] = b.x, v.w[5] = b.y, v.w[6] = b.z, v.w[7] = b.w;
    }
    return v;
}

// The first `count` of eight elements, zero for the others.  Eight come in one
// load wherever they lie: vector memory instructions take any address (element
// by element, quantizing bf16 [3863, 2922] and back took 33.6 us instead of 14.5).
template <int IN>
__device__ __forceinline__ Eight<IN> load8_some(const void* x, size_t e, int count) {
    Eight<IN> v = {};
    if (count == 8) {
        __builtin_memcpy(v.w, (const char*)x + e * (IN == kInBF16 ? 2 : 4), sizeof v.w);
        return v;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < count) {
            if constexpr (IN == kInBF16)
                v.w[i / 2] |= (uint32_t)((const uint16_t*)x)[e + i] << (16 * (i % 2));
            else
                v.w[i] = ((const uint32_t*)x)[e + i];
        }
    return v;
}

// Largest magnitude, as binary32 bits (for bf16 the two halves' maxima are
// joined by peak_of).
template <int IN>
__device__ __forceinline__ uint32_t abs_max(const Eight<IN>& v, uint32_t m) {
    if constexpr (IN == kInBF16) {
        mx_u16x2 t = __builtin_bit_cast(mx_u16x2, m);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t = __builtin_elementwise_max(t, __builtin_bit_cast(mx_u16x2, v.w[i] & 0x7FFF7FFFu));
        return __builtin_bit_cast(uint32_t, t);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, v.w[i] & 0x7FFFFFFFu);
        return m;
    }
}

template <int IN>
__device__ __forceinline__ uint32_t peak_of(uint32_t m) {
    if constexpr (IN == kInBF16) return max(m & 0xFFFF0000u, m << 16);
    return m;
}

// The eight codes, four bytes.
template <int IN>
__device__ __forceinline__ uint32_t codes8(const Eight<IN>& v, float scale) {
    uint32_t c = 0;
    if constexpr (IN == kInBF16) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(qar_bf16x2, v.w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(qar_bf16x2, v.w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(qar_bf16x2, v.w[2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(qar_bf16x2, v.w[3]), scale, 3);
    } else {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __builtin_bit_cast(float, v.w[i]);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[4], f[5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[6], f[7], scale, 3);
    }
    return c;
}

// The maximum over a block's four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppSwapAdjacent, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, kDppSwapPairs, 0xF, 0xF, false));
    return m;
}

// ---------------------------------------------------------------------------
// quantize.  A lane owns eight elements, four lanes a block.  Three places for
// the result: as the caller's rows of codes, as the fragments that the
// few-row product reads, and as the padded rows of the tiled product.

enum : int { kRows = 0, kFragments = 1, kTiles = 2 };

struct QuantizeArgs {
    const void* x;
    uint8_t *codes, *scales;
    size_t rows, cols;
    uint32_t blocks;      // of a row
    uint32_t padded;      // blocks that are written of each row (those behind the last are zero)
    const uint8_t* w_scales;   // kTiles: weight scales that are laid out in the same launch
    uint8_t* w_tiles;
    size_t w_rows;
    uint32_t quantize_groups;
};

// Byte address of a scale in the tiled product's order: for 32 rows and eight
// blocks, a 32-bit word for each lane (row % 32, block % 2), its bytes the
// four steps of the matrix instruction.
__device__ __forceinline__ size_t tile_scale_at(size_t row, uint32_t block, uint32_t padded) {
    return ((row / 32) * (padded / 8) + block / 8) * 256 + ((block % 2) * 32 + row % 32) * 4 + block % 8 / 2;
}

template <int IN, int PLACE, bool FAST>
__global__ __launch_bounds__(kThreads) void mx4_quantize_kernel(QuantizeArgs a) {
    constexpr int U = 4;
    if constexpr (PLACE == kTiles) {
        if (blockIdx.x >= a.quantize_groups) {
            // weight scales: a thread gathers one word
            const size_t chunks = a.padded / 8, words = (a.w_rows + 31) / 32 * chunks * 64;
            const size_t i = (size_t)(blockIdx.x - a.quantize_groups) * kThreads + threadIdx.x;
            if (i >= words) return;
            const uint32_t lane = i % 64;
            const size_t chunk = i / 64 % chunks, row = i / 64 / chunks * 32 + lane % 32;
            uint32_t word = 0;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const size_t block = chunk * 8 + 2 * s + lane / 32;
                const uint32_t byte = row < a.w_rows && block < a.blocks ? a.w_scales[row * a.blocks + block] : 127u;
                word |= byte << (8 * s);
            }
            reinterpret_cast<uint32_t*>(a.w_tiles)[i] = word;
            return;
        }
    }
    const uint32_t per_row = a.padded * 4;
    const size_t total = a.rows * per_row;
    const size_t first = (size_t)blockIdx.x * (U * kThreads) + threadIdx.x;
    Eight<IN> v[U];
    size_t row[U];
    uint32_t part[U];                              // eighth of a row, its block * 4 + lane of the block
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t i = first + (size_t)u * kThreads;
        v[u] = Eight<IN>{};
        if (i >= total) continue;
        if constexpr (FAST && PLACE == kRows) {
            // rows of whole blocks: the tensor is one row
            v[u] = load8<IN>(a.x, i * 8);
        } else {
            if (total >> 32) {
                row[u] = i / per_row;
                part[u] = (uint32_t)(i % per_row);
            } else {
                row[u] = (uint32_t)i / per_row;
                part[u] = (uint32_t)i % per_row;
            }
            const size_t e = (size_t)part[u] * 8;
            if (FAST) {
                if (e < a.cols) v[u] = load8<IN>(a.x, row[u] * a.cols + e);
            } else if (e < a.cols) {
                v[u] = load8_some<IN>(a.x, row[u] * a.cols + e, (int)min((size_t)8, a.cols - e));
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t i = first + (size_t)u * kThreads;
        const uint32_t byte = scale_byte(quad_max(peak_of<IN>(abs_max<IN>(v[u], 0))));
        if (i >= total) continue;                 // whole blocks, and whole chunks where they matter
        const uint32_t c = codes8<IN>(v[u], scale_value(byte));
        const bool leads = threadIdx.x % 4 == 0;
        if constexpr (PLACE == kRows) {
            store_b32(a.codes + i * 4, c);
            if (leads) a.scales[i / 4] = (uint8_t)byte;
        } else {
            const uint32_t block = part[u] / 4, quarter = part[u] % 4;
            const size_t at = PLACE == kFragments
                                  ? (((row[u] / 16) * (a.padded / 8) + block / 8) * 2 + block % 2) * 64 + block % 8 / 2 * 16 + row[u] % 16
                                  : row[u] * a.padded + block;
            *reinterpret_cast<uint32_t*>(a.codes + at * 16 + quarter * 4) = c;
            if constexpr (PLACE == kFragments) {
                if (leads) a.scales[at] = (uint8_t)byte;
            } else {
                // 32 lanes have a row's chunk of eight blocks: every other block's byte makes a word
                uint32_t word = byte << (block % 8 / 2 * 8);
                word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, kDppRowRotate8, 0xF, 0xF, false);
                word |= (uint32_t)__shfl_xor((int)word, 16);
                if (leads && block % 8 < 2)
                    *reinterpret_cast<uint32_t*>(a.scales + tile_scale_at(row[u], block, a.padded)) = word;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// dequantize.  A lane writes 16 bytes: eight bf16 or four binary32.  A code
// has two significant bits, so its product with a power of two is exact in
// both types.

__device__ __forceinline__ float e2m1_value(uint32_t code) {
    // 0, .5, 1, 1.5 | 2, 3, 4, 6 as the high halves of binary32 values
    const uint32_t lo = code & 4 ? 0x40404000u : 0x3F000000u, hi = code & 4 ? 0x40C04080u : 0x3FC03F80u;
    const uint32_t pair = code & 2 ? hi : lo;
    const uint32_t half = code & 1 ? pair >> 16 : pair & 0xFFFFu;
    return __builtin_bit_cast(float, (half << 16) | (code & 8) << 28);
}

// P values.  The hardware's conversion takes two at a time; scales near the
// ends of the exponent's range, whose products are subnormal or overflow, are
// multiplied out.
template <int P>
__device__ __forceinline__ void values_of(uint32_t c, uint32_t byte, float (&y)[P]) {
    const float s = scale_value(byte);
    if (byte - 4u < 244u) {
        qar_float2 v[4];
        v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
        v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
        v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
        v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = v[k / 2][k % 2];
    } else {
#pragma unroll
        for (int k = 0; k < P; ++k) y[k] = e2m1_value(c >> (4 * k)) * s;
    }
}

template <int OUT, bool FAST>
__global__ __launch_bounds__(kThreads) void mx4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, size_t rows,
                                                                 size_t cols, uint32_t blocks, void* out) {
    constexpr int P = OUT == kOutBF16 ? 8 : 4, U = 4;
    const uint32_t per_row = blocks * (32 / P);
    const size_t total = rows * per_row;
    const size_t first = (size_t)blockIdx.x * (U * kThreads) + threadIdx.x;
    uint32_t c[U] = {}, byte[U] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t i = first + (size_t)u * kThreads;
        if (i >= total) continue;
        c[u] = P == 8 ? load_b32(codes + i * 4) : load_b16(codes + i * 2);
        byte[u] = scales[i * P / 32];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const size_t i = first + (size_t)u * kThreads;
        if (i >= total) continue;
        float y[P];
        values_of<P>(c[u], byte[u], y);
        size_t at = i * P;
        int count = P;
        if constexpr (!FAST) {
            const size_t row = total >> 32 ? i / per_row : (uint32_t)i / per_row;
            const size_t e = (i - row * per_row) * P;
            if (e >= cols) continue;
            at = row * cols + e;
            count = (int)min((size_t)P, cols - e);
        }
        if constexpr (OUT == kOutBF16) {
            const uint4 q = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                       pack_bf16x2(y[6], y[7]));
            if constexpr (FAST) {
                store_b128((uint16_t*)out + at, q);
            } else if (count == P) {
                __builtin_memcpy((uint16_t*)out + at, &q, 16);
            } else {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < P; ++k)
                    if (k < count) ((uint16_t*)out)[at + k] = (uint16_t)(w[k / 2] >> (16 * (k % 2)));
            }
        } else {
            if constexpr (FAST) {
                store_b128((float*)out + at, make_uint4(__builtin_bit_cast(uint32_t, y[0]), __builtin_bit_cast(uint32_t, y[1]),
                                                        __builtin_bit_cast(uint32_t, y[2]), __builtin_bit_cast(uint32_t, y[3])));
            } else if (count == P) {
                __builtin_memcpy((float*)out + at, y, 16);
            } else {
#pragma unroll
                for (int k = 0; k < P; ++k)
                    if (k < count) ((float*)out)[at + k] = y[k];
            }
        }
    }
}

// ---------------------------------------------------------------------------
// activations.  EXACT: for binary32 results, to a few units of 2^-24; otherwise
// for results that are rounded to bf16's 2^-9, to 2^-16.

// e^(x + low), low far below x (to 2^-22, or 2^-16 for |x| < 90)
template <bool EXACT>
__device__ __forceinline__ float exp_of(float x, float low = 0.0f) {
    constexpr float kLog2E = 1.44269504088896340736f;
    const float t = x * kLog2E, e = __builtin_amdgcn_exp2f(t);
    if constexpr (!EXACT) return e;
    // the product's rounding, and what log2 e is more than its binary32 value
    const float rest = __builtin_fmaf(x, 1.92596299112661746887e-8f, __builtin_fmaf(x, kLog2E, -t));
    return e > 0.0f && e < INFINITY ? __builtin_fmaf(e, __builtin_fmaf(rest, 0.693147180559945309f, low), e) : e;
}

// -2 sqrt(2 / pi) (v + 0.044715 v^3).  An exponent of 80 has to be known to 2^-28
// of itself: with EXACT every rounding and the constants' own go into `low`.
template <bool EXACT>
__device__ __forceinline__ float tanh_exponent(float v, float& low) {
    constexpr double k1 = -1.59576912160573071176, k3 = k1 * 0.044715;
    constexpr float c1 = (float)k1, c3 = (float)k3;
    const float square = v * v;
    if constexpr (!EXACT) return v * __builtin_fmaf(c3, square, c1);
    const float cube = c3 * square, p = cube + c1, back = p - c1;
    const float lost = __builtin_fmaf(c3, square, -cube) + c3 * __builtin_fmaf(v, v, -square) + (float)(k3 - c3) * square +
                       (float)(k1 - c1) + ((cube - back) + (c1 - (p - back)));
    const float u = v * p;
    low = __builtin_fmaf(v, lost, __builtin_fmaf(v, p, -u));
    return u;
}

// Half the complementary error function of a / sqrt 2, a >= 0: e^(-a^2 / 2)
// times t Q(t), t = 1 / (1 + k a).  Q was fitted to the scaled function for the
// smallest relative error over 0 .. 14 (2^-23.6 with the coefficients as they are
// rounded here, or 2^-16.9); behind that the exponential leaves nothing.
template <bool EXACT>
__device__ __forceinline__ float half_erfc(float a) {
    const float square = a * a;
    float t, q, e;
    if constexpr (EXACT) {
        constexpr float c[9] = {0.139621407f, 0.139861897f, 0.119832717f, 0.105508596f, -0.0231112316f,
                                0.159176186f, -0.255716026f, 0.143972546f, -0.0291461032f};
        t = 1.0f / __builtin_fmaf(0.35f, a, 1.0f);
        q = c[8];
#pragma unroll
        for (int i = 7; i >= 0; --i) q = __builtin_fmaf(q, t, c[i]);
        e = exp_of<true>(-0.5f * square, -0.5f * __builtin_fmaf(a, a, -square));
    } else {
        constexpr float c[6] = {0.120074235f, 0.11374189f, 0.14419657f, -0.0169485137f, 0.216037527f,
                                -0.0770976022f};
        t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, a, 1.0f));
        q = c[5];
#pragma unroll
        for (int i = 4; i >= 0; --i) q = __builtin_fmaf(q, t, c[i]);
        e = exp_of<false>(-0.5f * square);
    }
    return e * (t * q);
}

// N elements of a row from column `col` as binary32, zeros behind its end.
template <int N, class T>
__device__ __forceinline__ void row_values(const T* x, size_t row_at, size_t col, size_t cols, float (&y)[N]) {
    const T* p = x + row_at + col;
    T w[N] = {};
    if (col + N <= cols)
        __builtin_memcpy(w, p, sizeof w);
    else
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (col + k < cols) w[k] = p[k];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (sizeof(T) == 2)
            y[k] = bf16_lo(w[k]);
        else
            y[k] = w[k];
    }
}

// The elements of 16 bytes.
template <class T>
__device__ __forceinline__ void values_of_16(uint4 q, float (&y)[16 / sizeof(T)]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2)
            y[2 * i] = bf16_lo(w[i]), y[2 * i + 1] = bf16_hi(w[i]);
        else
            y[i] = __builtin_bit_cast(float, w[i]);
    }
}

// The activation of N values: which one is decided once for all.
template <bool EXACT, int N>
__device__ __forceinline__ void activate(float (&y)[N], int activation) {
    const auto over = [](float n, float d) { return EXACT ? n / d : n * __builtin_amdgcn_rcpf(d); };
    const auto all = [&](auto f) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = f(y[i]);
    };
    switch (activation) {
    case kActRelu: all([](float v) { return v < 0.0f ? 0.0f : v; }); break;
    case kActSilu: all([&](float v) { return over(v, 1.0f + exp_of<EXACT>(-v)); }); break;
    case kActGelu:
        // v (1 - h) above 0, v h below.  From 64 on h is 0, which an infinity must not meet.
        all([](float v) {
            const float a = fminf(fabsf(v), 64.0f);
            return __builtin_fmaf(-a, half_erfc<EXACT>(a), v < 0.0f ? 0.0f : v);
        });
        break;
    case kActGeluTanh:
        // (1 + tanh u) / 2 = 1 / (1 + e^(-2 u))
        all([&](float v) {
            float low = 0.0f;
            const float u = tanh_exponent<EXACT>(v, low);
            return over(v, 1.0f + exp_of<EXACT>(u, low));
        });
        break;
    default: break;
    }
}

// ---------------------------------------------------------------------------
// the product, few rows of x: out[r][c] = sum over k of x[r][k] w[c][k].
//
// Bound by reading the weights, so these go from memory to registers once and
// no tile of them waits in LDS: a wave takes 16 CT weight rows ("columns" of
// the output) and a run of the k axis, and the waves' sums meet in LDS at the
// end.  16x16x128 matrix instructions: lane l = 16 g + r holds one block of
// row r, 16 contiguous bytes of codes and one scale.  The two instructions of
// a chunk of eight blocks (128 bytes of a row, a line) take blocks 2 g and
// 2 g + 1 of lane group g, so that a lane's two loads are neighbours and one
// 16-bit load brings both scales.
//   FUSED: the waves quantize x themselves, each its run of k.
struct LinearArgs {
    const void* x;
    const uint8_t *codes, *scales;     // weights
    const uint8_t *x_codes, *x_scales; // quantized x, in fragments (FUSED: unused) or tiles
    const uint8_t* w_tiles;            // the tiled product's weight scales
    void* out;
    size_t rows, inner, cols;
    uint32_t blocks;                   // of a weight row
    uint32_t padded;
    uint32_t row_tiles, col_tiles;     // of the tiled product
    int out_kind;
    const void *bias, *residual;       // of out's type, may be null
    int activation;
};

__device__ __forceinline__ mx_i32x8 operand(uint4 q) {
    return mx_i32x8{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

template <int IN>
__device__ __forceinline__ void quantize_block(const Eight<IN> (&v)[4], uint4& codes, uint32_t& byte) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = abs_max<IN>(v[i], m);
    byte = scale_byte(peak_of<IN>(m));
    const float s = scale_value(byte);
    codes = make_uint4(codes8<IN>(v[0], s), codes8<IN>(v[1], s), codes8<IN>(v[2], s), codes8<IN>(v[3], s));
}

// Scale bytes of blocks b and b + 1 of a row, in the low bytes (of the last
// block alone in the lowest).
__device__ __forceinline__ uint32_t scale_pair(const uint8_t* scales, uint32_t b, uint32_t blocks) {
    if (blocks == 1) return scales[0];
    uint16_t pair;
    __builtin_memcpy(&pair, scales + min(b, blocks - 2), 2);
    return b == blocks - 1 ? pair >> 8 : pair;
}

// A wave quantizes 256 k of up to 16 rows of x into its own part of LDS: 32
// lanes read 256 k of a row (whole lines, and no line twice), four neighbours
// make a block's codes.  Rows behind the last are left out: what their lanes
// then read from LDS reaches only sums that are not stored.
template <int IN>
struct RowsOfX {
    Eight<IN> raw[8];
    __device__ __forceinline__ void load(const LinearArgs& a, uint32_t chunk, uint32_t lane) {
        const size_t k = (size_t)min(chunk * 8 + lane % 32 / 4, a.blocks - 1) * 32 + lane % 4 * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (2u * i >= a.rows) break;
            raw[i] = load8<IN>(a.x, min((size_t)(2 * i + lane / 32), a.rows - 1) * a.inner + k);
        }
    }
    __device__ __forceinline__ void quantize(const LinearArgs& a, uint32_t lane, uint32_t (&codes)[8][16][4],
                                             uint8_t (&scales)[8][16]) const {
        const uint32_t block = lane % 32 / 4;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (2u * i >= a.rows) break;
            const uint32_t byte = scale_byte(quad_max(peak_of<IN>(abs_max<IN>(raw[i], 0))));
            codes[block][2 * i + lane / 32][lane % 4] = codes8<IN>(raw[i], scale_value(byte));
            if (lane % 4 == 0) scales[block][2 * i + lane / 32] = (uint8_t)byte;
        }
        // one wave writes and reads: its own order suffices
        __builtin_amdgcn_wave_barrier();
    }
};

template <int IN, int MT, int CT, int NW, bool FUSED, bool EPILOGUE>
__global__ __launch_bounds__(NW * 64) void mx4_few_rows_kernel(LinearArgs a) {
    static_assert(!FUSED || MT == 1, "rows of one tile");
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, r = lane % 16, g = lane / 16;
    const size_t c0 = (size_t)blockIdx.x * (16 * CT);
    const size_t row_bytes = (size_t)a.blocks * 16;
    const uint8_t* wp[CT];
    const uint8_t* sp[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        const size_t c = min(c0 + t * 16 + r, a.cols - 1);
        wp[t] = a.codes + c * row_bytes;
        sp[t] = a.scales + c * a.blocks;
    }
    const uint32_t chunks = a.padded / 8, run = (chunks + NW - 1) / NW;
    const uint32_t first = wave * run, last = min(first + run, chunks);
    mx_f32x4 acc[MT][CT] = {};

    // the waves' sums, and before that the wave's own codes and scales of x
    __shared__ union {
        mx_f32x4 sums[NW][MT * CT][64];
        struct {
            uint32_t codes[8][16][4];
            uint8_t scales[8][16];
        } x[FUSED ? NW : 1];
    } lds;

    // the next chunk's loads are under way while this one's are used
    RowsOfX<IN> raw;
    uint4 w[CT][2], xq[FUSED ? 1 : MT][2];
    uint32_t ws[CT], xs[FUSED ? 1 : MT][2];
    auto load = [&](uint32_t c) {
        if constexpr (FUSED) {
            raw.load(a, c, lane);
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const size_t at = (((size_t)m * chunks + c) * 2 + e) * 64 + lane;
                    xq[m][e] = *reinterpret_cast<const uint4*>(a.x_codes + at * 16);
                    xs[m][e] = a.x_scales[at];
                }
        }
        // behind the row's end its last blocks again, against zeros of x
        const uint32_t b0 = min(c * 8 + 2 * g, a.blocks - 1), b1 = min(b0 + 1, a.blocks - 1);
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            w[t][0] = *reinterpret_cast<const uint4*>(wp[t] + (size_t)b0 * 16);
            w[t][1] = *reinterpret_cast<const uint4*>(wp[t] + (size_t)b1 * 16);
            ws[t] = scale_pair(sp[t], b0, a.blocks);
        }
    };
    if (first < last) load(first);
    for (uint32_t c = first; c < last; ++c) {
        if constexpr (FUSED) raw.quantize(a, lane, lds.x[wave].codes, lds.x[wave].scales);
        uint4 wc[CT][2], xc[MT][2];
        uint32_t wsc[CT], xsc[MT][2];
#pragma unroll
        for (int t = 0; t < CT; ++t) wc[t][0] = w[t][0], wc[t][1] = w[t][1], wsc[t] = ws[t];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if constexpr (FUSED) {
                    xc[m][e] = *reinterpret_cast<const uint4*>(lds.x[wave].codes[2 * g + e][r]);
                    xsc[m][e] = lds.x[wave].scales[2 * g + e][r];
                } else {
                    xc[m][e] = xq[m][e];
                    xsc[m][e] = xs[m][e];
                }
                if (c * 8 + 2 * g + e >= a.blocks) xc[m][e] = make_uint4(0, 0, 0, 0);
            }
        if (c + 1 < last) load(c + 1);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    acc[m][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        operand(wc[t][e]), operand(xc[m][e]), acc[m][t], kE2M1, kE2M1, 0, (int)(wsc[t] >> (8 * e)), 0,
                        (int)xsc[m][e]);
    }
    if (FUSED) __syncthreads();

    // lane l holds x row l % 16 and columns 4 (l / 16) .. + 3 of each 16 x 16 tile
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < CT; ++t) lds.sums[wave][m * CT + t][lane] = acc[m][t];
    __syncthreads();
    // a thread adds up four columns of a row, in wave order
    for (uint32_t i = threadIdx.x; i < MT * CT * 64; i += NW * 64) {
        // neighbouring threads take neighbouring columns
        const uint32_t m = i / (CT * 64), rest = i % (CT * 64), row16 = rest / (CT * 4), quad = rest % (CT * 4);
        const uint32_t t = quad / 4, src = quad % 4 * 16 + row16;
        mx_f32x4 y = lds.sums[0][m * CT + t][src];
#pragma unroll
        for (int v = 1; v < NW; ++v) y += lds.sums[v][m * CT + t][src];
        const size_t row = m * 16 + row16, col = c0 + quad * 4;
        if (row >= a.rows) continue;
        const size_t at = row * a.cols + col;
        if constexpr (EPILOGUE) {
            float v[4] = {y[0], y[1], y[2], y[3]}, bias[4] = {}, add[4] = {};
            if (a.out_kind == kOutBF16) {
                if (a.bias) row_values<4>((const uint16_t*)a.bias, 0, col, a.cols, bias);
                if (a.residual) row_values<4>((const uint16_t*)a.residual, row * a.cols, col, a.cols, add);
            } else {
                if (a.bias) row_values<4>((const float*)a.bias, 0, col, a.cols, bias);
                if (a.residual) row_values<4>((const float*)a.residual, row * a.cols, col, a.cols, add);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] += bias[k];
            if (a.out_kind == kOutBF16)
                activate<false>(v, a.activation);
            else
                activate<true>(v, a.activation);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = v[k] + add[k];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (col + k >= a.cols) break;
            if (a.out_kind == kOutBF16)
                ((uint16_t*)a.out)[at + k] = (uint16_t)pack_bf16x2(y[k], 0.0f);
            else
                ((float*)a.out)[at + k] = y[k];
        }
    }
}

// ---------------------------------------------------------------------------
// the product, many rows: tiles of BM rows of x and BN weight rows, 256 k at a
// time through LDS in two buffers.  128 bytes of a row are eight blocks; they
// arrive by direct loads to LDS, whose lanes write 16 bytes each one behind the
// other, so the order in LDS is chosen by the addresses that the lanes read:
// block b of row r lies in slot b ^ (r / 2 % 8), and the sixteen lanes that a
// 16-byte read serves at once lie in sixteen different groups of four banks
// (with r % 8 half of the reads' cycles were bank conflicts).
// 32x32x64 matrix instructions: lane l holds block l / 32 of the step for row
// l % 32.

// N elements (16 bytes) of an output row from column `col`, as far as the row
// goes; whole ones in one store, aligned or not.
template <int N, class T>
__device__ __forceinline__ void store_row(T* out, size_t row_at, size_t col, size_t cols, uint4 v) {
    if (col >= cols) return;
    T* p = out + row_at + col;
    if (col + N <= cols) {
        __builtin_memcpy(p, &v, 16);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (col + k >= cols) break;
        if constexpr (sizeof(T) == 2)
            p[k] = (T)(w[k / 2] >> (16 * (k % 2)));
        else
            p[k] = __builtin_bit_cast(T, w[k]);
    }
}

// Waits until at most N of the wave's loads are under way (and no LDS read
// is), then for the workgroup.  __syncthreads would wait for all of them.
template <int N>
__device__ __forceinline__ void arrive() {
    static_assert(N < 64, "vmcnt");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 7 << 4);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int OUT, int BM, int BN, int WM, int WN, bool EPILOGUE, bool DEEP>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void mx4_tiled_kernel(LinearArgs a) {
    static_assert(BM == BN, "one size of buffer");
    constexpr int NT = (BM / WM) * (BN / WN) * 64;
    constexpr int TM = WM / 32, TN = WN / 32, LOADS = BM * 8 / NT;
    static_assert(!DEEP || BM == 64, "eight buffers, loads that arrive() can count");
    __shared__ uint4 s0[BM * 8], s1[BM * 8], s2[BM * 8], s3[BM * 8], s4[BM * 8];
    __shared__ uint4 s5[DEEP ? BM * 8 : 1], s6[DEEP ? BM * 8 : 1], s7[DEEP ? BM * 8 : 1];
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const uint32_t wm = wave / (BN / WN), wn = wave % (BN / WN);

    // XCD x takes a contiguous range of tiles; within it bands of 8 row tiles,
    // column tile by column tile, so that what runs at once shares both operands
    const uint32_t tiles = a.row_tiles * a.col_tiles;
    const uint32_t t = xcd_tile(blockIdx.x, tiles);
    const uint32_t band = t / (8 * a.col_tiles), in_band = t % (8 * a.col_tiles);
    const uint32_t height = min(8u, a.row_tiles - band * 8);
    const size_t m0 = (size_t)(band * 8 + in_band % height) * BM, n0 = (size_t)(in_band / height) * BN;

    const uint32_t chunks = a.padded / 8;
    const uint32_t slot_row = tid / 8, block = tid % 8 ^ slot_row / 2 % 8;
    // offsets from the tile's first rows: 256 rows of 2^24 k at most are 2^31 bytes
    const uint8_t *x_base = a.x_codes + m0 * a.padded * 16, *w_base = a.codes + n0 * a.blocks * 16;
    uint32_t x_at[LOADS], w_at[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const uint32_t row = i * (NT / 8) + slot_row;
        x_at[i] = (uint32_t)min((size_t)row, a.rows - 1 - m0) * a.padded * 16 + block * 16;
        w_at[i] = (uint32_t)min((size_t)row, a.cols - 1 - n0) * a.blocks * 16;
    }
    // load i of the thread's LOADS
    auto fetch_x = [&](uint32_t c, uint4* to, int i) {
        const uint8_t* base = x_base + (size_t)min(c, chunks - 1) * 128;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(base + x_at[i]),
                                         (__attribute__((address_space(3))) void*)(to + i * NT + wave * 64), 16, 0, 0);
    };
    auto fetch_w = [&](uint32_t c, uint4* to, int i) {
        // behind a row's last block x is padded with zeros, so any block of the weights will do there
        const uint32_t at = min(c * 8 + block, a.blocks - 1) * 16;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(w_base + (w_at[i] + at)),
                                         (__attribute__((address_space(3))) void*)(to + i * NT + wave * 64), 16, 0, 0);
    };
    const uint32_t* as_tile = reinterpret_cast<const uint32_t*>(a.x_scales) + (m0 + wm * WM) / 32 * chunks * 64 + lane;
    const uint32_t* bs_tile = reinterpret_cast<const uint32_t*>(a.w_tiles) + (n0 + wn * WN) / 32 * chunks * 64 + lane;
    int sa[TM], sb[TN];
    auto fetch_scales = [&](uint32_t chunk, int (&sa)[TM], int (&sb)[TN]) {
        const uint32_t c = min(chunk, chunks - 1);
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = (int)as_tile[((size_t)i * chunks + c) * 64];
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = (int)bs_tile[((size_t)j * chunks + c) * 64];
    };

    mx_f32x16 acc[TM][TN] = {};
    const uint32_t fr = lane % 32, half = lane / 32;
    // byte offset of a fragment for step 0; step s differs in bits 5 and 6 only
    const uint32_t fx0 = (wm * WM + fr) * 128 + (half ^ fr / 2 % 8) * 16, fw0 = (wn * WN + fr) * 128 + (half ^ fr / 2 % 8) * 16;
    auto step = [&](auto S, const uint4* xs, const uint4* ws, uint32_t fx, uint32_t fw, const int (&ca)[TM],
                    const int (&cb)[TN], auto loads) {
        constexpr int s = decltype(S)::value;
        mx_i32x8 fa[TM], fb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            fa[i] = operand(*reinterpret_cast<const uint4*>((const char*)xs + (fx ^ (32 * s)) + i * 32 * 128));
#pragma unroll
        for (int j = 0; j < TN; ++j)
            fb[j] = operand(*reinterpret_cast<const uint4*>((const char*)ws + (fw ^ (32 * s)) + j * 32 * 128));
        loads();
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], kE2M1, kE2M1, s, cb[j],
                                                                           s, ca[i]);
    };
    // Chunk c's x lies in buffer 2 c % 5 and its weights in (2 c + 1) % 5.
    // When chunk c begins, the buffers of chunk c - 1 are free: the weights of
    // chunk c + 1 and then x of chunk c + 2 are asked for, spread over the
    // steps, because waves that all issue their loads first wait for the
    // address units with the matrix units idle.  Behind the last chunk the
    // last is asked for again, which keeps the counts.
    auto chunk = [&](uint32_t c, uint4* xs, uint4* ws, uint4* w_next, uint4* x_after) {
        arrive<LOADS>();                            // all but x of chunk c + 1
        int ca[TM], cb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) ca[i] = sa[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) cb[j] = sb[j];
        // the five buffers' fragment addresses would not fit the registers
        uint32_t fx = fx0, fw = fw0;
        asm volatile("" : "+v"(fx), "+v"(fw));
        step(std::integral_constant<int, 0>{}, xs, ws, fx, fw, ca, cb, [&] {
#pragma unroll
            for (int i = 0; i < LOADS / 2; ++i) fetch_w(c + 1, w_next, i);
        });
        step(std::integral_constant<int, 1>{}, xs, ws, fx, fw, ca, cb, [&] {
#pragma unroll
            for (int i = LOADS / 2; i < LOADS; ++i) fetch_w(c + 1, w_next, i);
            fetch_scales(c + 1, sa, sb);
            asm volatile("" ::: "memory");          // x last: what arrive() lets pass
        });
        step(std::integral_constant<int, 2>{}, xs, ws, fx, fw, ca, cb, [&] {
#pragma unroll
            for (int i = 0; i < LOADS / 2; ++i) fetch_x(c + 2, x_after, i);
        });
        step(std::integral_constant<int, 3>{}, xs, ws, fx, fw, ca, cb, [&] {
#pragma unroll
            for (int i = LOADS / 2; i < LOADS; ++i) fetch_x(c + 2, x_after, i);
        });
    };
    using T = std::conditional_t<OUT == kOutBF16, uint16_t, float>;
    using S = std::conditional_t<EPILOGUE, float, T>;
    // A buffer to a wave, or half of one: all are read out, and none is being written.
    constexpr int ROW = WN * sizeof(S), SHARE = NT / 64 > 4 ? 2 : 1, STRIP = BM * 128 / SHARE;
    constexpr int NOW = std::min(STRIP / (32 * ROW), TM);
    static_assert(NOW > 0 && TM % NOW == 0 && NT / 64 <= 8 && ROW % 128 == 0, "strips");
    constexpr int N = 16 / sizeof(T), PER = WN / N;  // columns of a lane, lanes to a row
    constexpr int STORES = NOW * 32 * PER / 64, ALL = STORES * (TM / NOW);
    const size_t col = n0 + wn * WN + lane % PER * N;
    // A tile inside a bf16 output's columns asks for all of its residual before it
    // waits for the last loads to LDS (8192 x 5376 x 21504 with bias and GELU: the
    // call 693 -> 633 to 650 us); binary32, twice the registers, four stores' worth at a time.  Small
    // tiles, one wave to a SIMD, have registers enough to ask before their first
    // chunk (300 x 5760 x 2880, binary32: 17.8 -> 17.1 us).
    constexpr bool EARLY = EPILOGUE && (sizeof(T) == 2 || DEEP);
    constexpr int AT_ONCE = EPILOGUE && !EARLY ? 4 : STORES;
    [[maybe_unused]] uint4 residual[EARLY ? ALL : 1];
    const bool early = EARLY && a.residual && n0 + BN <= a.cols;
    const auto row_of = [&](int k) {                // of store k
        return m0 + wm * WM + k / STORES * (NOW * 32) + k % STORES * (64 / PER) + lane / PER;
    };
    const auto ask_for_residual = [&] {
#pragma unroll
        for (int k = 0; k < ALL; ++k)
            if constexpr (EARLY)                     // for rows behind the last, the last: it goes nowhere
                __builtin_memcpy(&residual[k], (const T*)a.residual + std::min(row_of(k), a.rows - 1) * a.cols + col, 16);
    };

    if constexpr (DEEP) {
        // A small tile's products of a chunk are over long before memory answers:
        // three chunks are under way, in four pairs of buffers.  The sums are
        // formed in the same order.
        int da[4][TM], db[4][TN];
        auto fetch = [&](uint32_t c, uint4* xs, uint4* ws, int (&ca)[TM], int (&cb)[TN]) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) fetch_x(c, xs, i);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) fetch_w(c, ws, i);
            fetch_scales(c, ca, cb);
            asm volatile("" ::: "memory");          // whole chunks: what arrive() counts
        };
        constexpr int PER = 2 * LOADS + TM + TN;
        auto products = [&](auto P, const uint4* xs, const uint4* ws) {
            constexpr int p = decltype(P)::value;
            step(std::integral_constant<int, 0>{}, xs, ws, fx0, fw0, da[p], db[p], [] {});
            step(std::integral_constant<int, 1>{}, xs, ws, fx0, fw0, da[p], db[p], [] {});
            step(std::integral_constant<int, 2>{}, xs, ws, fx0, fw0, da[p], db[p], [] {});
            step(std::integral_constant<int, 3>{}, xs, ws, fx0, fw0, da[p], db[p], [] {});
        };
        auto deep_chunk = [&](auto P, uint32_t c, uint4* xs, uint4* ws, uint4* x_next, uint4* w_next) {
            constexpr int before = (decltype(P)::value + 3) % 4;
            arrive<2 * PER>();                      // all but chunks c + 1 and c + 2
            fetch(c + 3, x_next, w_next, da[before], db[before]);
            products(P, xs, ws);
        };
        if (early) ask_for_residual();
        asm volatile("" ::: "memory");
        fetch(0, s0, s1, da[0], db[0]);
        fetch(1, s2, s3, da[1], db[1]);
        fetch(2, s4, s5, da[2], db[2]);
        constexpr std::integral_constant<int, 0> P0{};
        constexpr std::integral_constant<int, 1> P1{};
        constexpr std::integral_constant<int, 2> P2{};
        constexpr std::integral_constant<int, 3> P3{};
        uint32_t c = 0;
        for (; c + 4 <= chunks; c += 4) {
            deep_chunk(P0, c, s0, s1, s6, s7);
            deep_chunk(P1, c + 1, s2, s3, s0, s1);
            deep_chunk(P2, c + 2, s4, s5, s2, s3);
            deep_chunk(P3, c + 3, s6, s7, s4, s5);
        }
        if (c < chunks) {
            arrive<2 * PER>();
            products(P0, s0, s1);
            if (c + 1 < chunks) {
                arrive<PER>();
                products(P1, s2, s3);
                if (c + 2 < chunks) {
                    arrive<0>();
                    products(P2, s4, s5);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) fetch_x(0, s0, i);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) fetch_w(0, s1, i);
        fetch_scales(0, sa, sb);
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < LOADS; ++i) fetch_x(1, s2, i);
        // Whole rounds of the buffers and then the rest, nested: where paths meet
        // on which different loads are the last, the compiler would wait for all.
        uint32_t c = 0;
        for (; c + 5 <= chunks; c += 5) {
            chunk(c, s0, s1, s3, s4);
            chunk(c + 1, s2, s3, s0, s1);
            chunk(c + 2, s4, s0, s2, s3);
            chunk(c + 3, s1, s2, s4, s0);
            chunk(c + 4, s3, s4, s1, s2);
        }
        if (c < chunks) {
            chunk(c, s0, s1, s3, s4);
            if (c + 1 < chunks) {
                chunk(c + 1, s2, s3, s0, s1);
                if (c + 2 < chunks) {
                    chunk(c + 2, s4, s0, s2, s3);
                    if (c + 3 < chunks) chunk(c + 3, s1, s2, s4, s0);
                }
            }
        }
    }
    // The weights are the first operand, so lane l = 32 h + r holds row r of a
    // subtile and its columns 8 q + 4 h .. + 3 in registers 4 q .. + 3.  They
    // pass through the wave's own stretch of LDS, a few subtiles of rows at a
    // time, so that a store writes whole lines: eight lanes a row of 128 bytes
    // (straight from the registers a store touches 32 rows with 32 bytes each).
    // 16-byte slot c of row r lies at c ^ (r % 8) of its group of eight.
    // With an epilogue they pass as binary32: bias, activation and residual come
    // on the way out, where a lane's columns are the same for all of its rows and
    // the residual is read in whole lines, and the result is rounded once.
    if (!DEEP && early) {
        ask_for_residual();
        arrive<ALL>();
    } else {
        arrive<0>();                                // nothing may write to LDS that is no longer this workgroup's
    }
    const uint32_t home = wave / SHARE;
    char* strip = reinterpret_cast<char*>(home == 0 ? s0 : home == 1 ? s1 : home == 2 ? s2 : s3) + wave % SHARE * STRIP;
    [[maybe_unused]] float bias[N] = {};
    if constexpr (EPILOGUE)
        if (a.bias) row_values<N>((const T*)a.bias, 0, col, a.cols, bias);
#pragma unroll
    for (int i0 = 0; i0 < TM; i0 += NOW) {
#pragma unroll
        for (int i = 0; i < NOW; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t row = i * 32 + fr, at = (j * 32 + 8 * q + 4 * half) * sizeof(S);
                    char* to = strip + row * ROW + (at & ~127u) + ((at / 16 % 8 ^ row % 8) * 16) + at % 16;
                    const float y0 = acc[i0 + i][j][4 * q], y1 = acc[i0 + i][j][4 * q + 1], y2 = acc[i0 + i][j][4 * q + 2],
                                y3 = acc[i0 + i][j][4 * q + 3];
                    if constexpr (sizeof(S) == 2)
                        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(y0, y1), pack_bf16x2(y2, y3));
                    else
                        *reinterpret_cast<mx_f32x4*>(to) = mx_f32x4{y0, y1, y2, y3};
                }
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int k0 = 0; k0 < STORES; k0 += AT_ONCE) {
            [[maybe_unused]] float add[EPILOGUE ? AT_ONCE : 1][N] = {};
            if constexpr (EPILOGUE)
                if (a.residual && !early)
#pragma unroll
                    for (int k = 0; k < AT_ONCE; ++k)
                        if (row_of(i0 / NOW * STORES + k0 + k) < a.rows)
                            row_values<N>((const T*)a.residual, row_of(i0 / NOW * STORES + k0 + k) * a.cols, col, a.cols, add[k]);
#pragma unroll
            for (int k = 0; k < AT_ONCE; ++k) {
                const uint32_t row = (k0 + k) * (64 / PER) + lane / PER;
                const size_t r = row_of(i0 / NOW * STORES + k0 + k);
                const auto slot = [&](uint32_t c) {
                    return *reinterpret_cast<const uint4*>(strip + row * ROW + (c & ~7u) * 16 + ((c % 8 ^ row % 8) * 16));
                };
                uint4 v;
                if constexpr (!EPILOGUE) {
                    v = slot(lane % PER);
                } else {
                    if constexpr (EARLY)
                        if (early) values_of_16<T>(residual[i0 / NOW * STORES + k], add[k]);
                    float y[N];
#pragma unroll
                    for (int e = 0; e < N; e += 4) {
                        const uint4 w = slot((lane % PER * N + e) / 4);
                        y[e] = __builtin_bit_cast(float, w.x) + bias[e], y[e + 1] = __builtin_bit_cast(float, w.y) + bias[e + 1];
                        y[e + 2] = __builtin_bit_cast(float, w.z) + bias[e + 2], y[e + 3] = __builtin_bit_cast(float, w.w) + bias[e + 3];
                    }
                    activate<sizeof(T) == 4>(y, a.activation);
#pragma unroll
                    for (int e = 0; e < N; ++e) y[e] += add[k][e];
                    if constexpr (sizeof(T) == 2)
                        v = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                       pack_bf16x2(y[6], y[7]));
                    else
                        v = make_uint4(__builtin_bit_cast(uint32_t, y[0]), __builtin_bit_cast(uint32_t, y[1]),
                                       __builtin_bit_cast(uint32_t, y[2]), __builtin_bit_cast(uint32_t, y[3]));
                }
                if (r < a.rows) store_row<N>((T*)a.out, r * a.cols, col, a.cols, v);
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

uint32_t groups_for(size_t items, size_t per_group) { return (uint32_t)((items + per_group - 1) / per_group); }

uint32_t round_up(uint32_t v, uint32_t to) { return (v + to - 1) / to * to; }

template <int IN, int PLACE>
hipError_t quantize_into(const QuantizeArgs& a, uint32_t extra_groups, hipStream_t st) {
    const uint32_t groups = a.quantize_groups + extra_groups;
    // whole 16-byte loads: rows start aligned; one flat range: rows of whole blocks
    const bool fast = PLACE == kRows ? a.cols % 32 == 0 : a.cols % 8 == 0;
    return launch_threads(fast ? mx4_quantize_kernel<IN, PLACE, true> : mx4_quantize_kernel<IN, PLACE, false>, groups,
                          kThreads, st, a);
}

template <int PLACE>
hipError_t quantize_call(QuantizeArgs a, int kind, hipStream_t st) {
    a.quantize_groups = groups_for(a.rows * a.padded * 4, 4 * kThreads);
    const uint32_t extra =
        PLACE == kTiles ? groups_for((a.w_rows + 31) / 32 * (a.padded / 8) * 64, kThreads) : 0;
    return kind == kInBF16 ? quantize_into<kInBF16, PLACE>(a, extra, st) : quantize_into<kInF32, PLACE>(a, extra, st);
}

// Two tiles of columns to a workgroup halve the reading of x, one gives twice
// the workgroups.  Measured, two tiles against one: [5, 3840] x [3840, 15360]
// 10.3 against 13.4 us, [1, 5376] x [5376, 5376] 8.9 against 7.4; for 32 rows
// [32, 5376] x [5376, 5376] 12.5 against 14.2, [50, 8000] x [8000, 2880] 17.6
// against 13.7.  Four tiles and four or sixteen waves were slower than the
// better of these everywhere but once (2%).
template <int IN, int MT, bool FUSED, bool EPILOGUE>
hipError_t few_rows(const LinearArgs& a, hipStream_t st) {
    constexpr int NW = 8;
    if (groups_for(a.cols, 32) >= (MT == 1 ? 256u : 160u))
        return launch_threads(mx4_few_rows_kernel<IN, MT, 2, NW, FUSED, EPILOGUE>, groups_for(a.cols, 32), NW * 64, st, a);
    return launch_threads(mx4_few_rows_kernel<IN, MT, 1, NW, FUSED, EPILOGUE>, groups_for(a.cols, 16), NW * 64, st, a);
}

template <int OUT, int BM, int BN, int WM, int WN, bool EPILOGUE, bool DEEP = false>
hipError_t tiled(LinearArgs& a, hipStream_t st) {
    a.row_tiles = groups_for(a.rows, BM);
    a.col_tiles = groups_for(a.cols, BN);
    return launch_threads(mx4_tiled_kernel<OUT, BM, BN, WM, WN, EPILOGUE, DEEP>, a.row_tiles * a.col_tiles,
                          (BM / WM) * (BN / WN) * 64, st, a);
}

// The few-row kernel, which reads x again for every 16 or 32 columns, against
// tiles of 64: for 40 rows of 5376 x 5376 13.1 against 16.6 us, for 64 rows of
// 1152 x 1152 6.9 against 7.7, of 3840 x 15360 19.4 against 16.0 to 19.0.
constexpr size_t kFewRows = 64;

// Tiles of 16 rows that the few-row kernel is built for.  It reads the
// fragments of all of them, so the workspace holds as many: what lies in those
// without a row reaches only sums that are not stored.
uint32_t few_tiles(size_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

// Blocks of x in fragments.
size_t few_fragments(size_t rows, uint32_t padded) { return (size_t)few_tiles(rows) * 16 * padded; }

// One tile of rows of whole blocks is quantized inside the product.
bool fused(size_t rows, size_t inner) { return rows <= 16 && inner % 32 == 0; }

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

} // namespace

hipError_t launch_mx4_quantize(const void* x, int kind, size_t rows, size_t cols, uint8_t* codes, uint8_t* scales,
                               hipStream_t st) {
    QuantizeArgs a = {};
    a.x = x, a.codes = codes, a.scales = scales, a.rows = rows, a.cols = cols;
    a.blocks = a.padded = groups_for(cols, 32);
    return quantize_call<kRows>(a, kind, st);
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, size_t rows, size_t cols, void* out, int kind,
                                 hipStream_t st) {
    const uint32_t blocks = groups_for(cols, 32);
    const bool fast = cols % 32 == 0;
    const auto go = [&](auto OUT, uint32_t lanes) {
        constexpr int O = decltype(OUT)::value;
        return launch_threads(fast ? mx4_dequantize_kernel<O, true> : mx4_dequantize_kernel<O, false>,
                              groups_for(rows * blocks * lanes, 4 * kThreads), kThreads, st, codes, scales, rows, cols, blocks,
                              out);
    };
    return kind == kOutBF16 ? go(std::integral_constant<int, kOutBF16>{}, 4) : go(std::integral_constant<int, kOutF32>{}, 8);
}

size_t mx4_linear_workspace(size_t rows, size_t inner, size_t cols) {
    const uint32_t blocks = groups_for(inner, 32);
    if (fused(rows, inner)) return 0;
    if (rows <= kFewRows) {
        const size_t fragments = few_fragments(rows, round_up(blocks, 8));
        return align256(fragments * 16) + align256(fragments);
    }
    const size_t padded = round_up(blocks, 8);
    return align256(rows * padded * 16) + align256((rows + 255) / 256 * 256 * padded) +
           align256((cols + 255) / 256 * 256 * padded);
}

namespace {

template <bool EPILOGUE>
hipError_t linear(LinearArgs a, int kind, const uint8_t* w_scales, void* workspace, hipStream_t st) {
    const size_t rows = a.rows, inner = a.inner, cols = a.cols;
    if (fused(rows, inner)) {
        a.padded = round_up(a.blocks, 8);
        return kind == kInBF16 ? few_rows<kInBF16, 1, true, EPILOGUE>(a, st) : few_rows<kInF32, 1, true, EPILOGUE>(a, st);
    }
    QuantizeArgs q = {};
    q.x = a.x, q.rows = rows, q.cols = inner, q.blocks = a.blocks;
    q.codes = (uint8_t*)workspace;
    a.x_codes = q.codes;
    if (rows <= kFewRows) {
        q.padded = a.padded = round_up(a.blocks, 8);
        q.scales = q.codes + align256(few_fragments(rows, a.padded) * 16);
        a.x_scales = q.scales;
        const hipError_t e = quantize_call<kFragments>(q, kind, st);
        if (e != hipSuccess) return e;
        // fragments are the same for both types of x: one kernel serves them
        if (few_tiles(rows) == 1) return few_rows<kInBF16, 1, false, EPILOGUE>(a, st);
        if (few_tiles(rows) == 2) return few_rows<kInBF16, 2, false, EPILOGUE>(a, st);
        return few_rows<kInBF16, 4, false, EPILOGUE>(a, st);
    }
    q.padded = a.padded = round_up(a.blocks, 8);
    q.scales = q.codes + align256(rows * q.padded * 16);
    q.w_tiles = q.scales + align256((rows + 255) / 256 * 256 * (size_t)q.padded);
    q.w_scales = w_scales;
    q.w_rows = cols;
    a.x_scales = q.scales;
    a.w_tiles = q.w_tiles;
    const hipError_t e = quantize_call<kTiles>(q, kind, st);
    if (e != hipSuccess) return e;
    // The largest tile that gives every CU one.  Tiles of 64 against 128: 500
    // rows of 3840 x 3840 15.2 against 17.5 us, 1000 of 2880 x 9000 37.1 against
    // 33.5; 128 against 256: 2000 rows of 5376 x 5376 48.9 against 51.4, 8192 of
    // 5376 x 21504 1.3 times the time.
    const auto tiles = [&](size_t size) { return (size_t)groups_for(rows, size) * groups_for(cols, size); };
    const auto go = [&](auto OUT) {
        constexpr int out = decltype(OUT)::value;
        if (tiles(256) >= 256) return tiled<out, 256, 256, 128, 64, EPILOGUE>(a, st);
        if (tiles(128) >= 256) return tiled<out, 128, 128, 64, 64, EPILOGUE>(a, st);
        // with more than two tiles to a CU, others on it fill the waits, as long as
        // their buffers fit.  Three chunks under way against one to two: 300 rows of
        // 5760 x 2880 (225 tiles) 15.8 against 18.1 us, 128 of 21504 x 5376 (168) 40
        // against 50, 500 of 3840 x 3840 (480) 14.2 against 15.1, but 100 of
        // 5376 x 21504 (672) 27.5 against 24.5.
        if (tiles(64) <= 512) return tiled<out, 64, 64, 32, 64, EPILOGUE, true>(a, st);
        return tiled<out, 64, 64, 32, 64, EPILOGUE>(a, st);
    };
    return a.out_kind == kOutBF16 ? go(std::integral_constant<int, kOutBF16>{}) : go(std::integral_constant<int, kOutF32>{});
}

} // namespace

hipError_t launch_mx4_linear(const void* x, int kind, size_t rows, size_t inner, const uint8_t* codes, const uint8_t* scales,
                             size_t cols, const Epilogue& epilogue, void* out, int out_kind, void* workspace, hipStream_t st) {
    LinearArgs a = {};
    a.x = x, a.codes = codes, a.scales = scales, a.out = out, a.out_kind = out_kind;
    a.rows = rows, a.inner = inner, a.cols = cols;
    a.blocks = groups_for(inner, 32);
    a.bias = epilogue.bias, a.residual = epilogue.residual, a.activation = epilogue.activation;
    return a.bias || a.residual || a.activation != kActNone ? linear<true>(a, kind, scales, workspace, st)
                                                            : linear<false>(a, kind, scales, workspace, st);
}

} // namespace qar
