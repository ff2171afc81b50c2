// qar_kv8.hip -- a paged cache of keys and values held in 8 bits on gfx950:
// tokens enter it, are read back, attended to, and evicted by weight.
//
// A page holds 64 tokens of every head: keys as [64][dim], values as
// [dim][64] codes (each the layout whose contiguous bytes run along the sum
// of its matrix product), and one binary32 scale for each page and head of
// either.  value = code * scale; scale = absmax / 127, codes as everywhere
// in this library.
//
// Entries of the page table outside [0, pages) stand for pages that are not
// there: nothing is written to them, they read as zeros and attention sees
// none of their keys.
#include <float.h>
#include <hip/hip_runtime.h>

#include "qar_device.h"
#include "qar_launch.h"
#include "qar_serve.h"

namespace qar {
namespace {

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

// Calls f with the function that gives four values' codes, packed, for a scale
// that the workgroup shares: how a scale is divided by (exactly either way) is
// decided once, and its reciprocal formed once, for all that f encodes.
template <class F>
__device__ __forceinline__ void with_codes(float s, F f) {
    if (s >= kFastQuotientMinScale) {
        const float r = 1.0f / s;
        f([&](kv_f32x4 v) {
            return pack4(code_bits_of(fast_quotient(v[0], s, r)), code_bits_of(fast_quotient(v[1], s, r)),
                         code_bits_of(fast_quotient(v[2], s, r)), code_bits_of(fast_quotient(v[3], s, r)));
        });
    } else if (s != 0.0f) {
        f([&](kv_f32x4 v) {
            return pack4(clamped_code_bits_of(v[0] / s), clamped_code_bits_of(v[1] / s), clamped_code_bits_of(v[2] / s),
                         clamped_code_bits_of(v[3] / s));
        });
    } else {
        f([](kv_f32x4) { return 0u; });
    }
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

// The maximum over a workgroup of kThreads; every thread gets it.
__device__ __forceinline__ float group_max(float m, float (&shared)[kThreads / 64]) {
    m = lanes_max<64>(m);
    if (threadIdx.x % 64 == 0) shared[threadIdx.x / 64] = m;
    __syncthreads();
    return fmaxf(fmaxf(shared[0], shared[1]), fmaxf(shared[2], shared[3]));
}

// ---------------------------------------------------------------------------
// append.  A workgroup takes one page of one head, keys or values.  It holds
// the page's new values in registers between the maximum and the codes, so
// they are read once.  Old tokens of the page (its first new token need not
// be its first) keep their codes unless the new ones raise the page's scale;
// then their values are quantized again with it.

struct AppendArgs {
    Kv8 c;
    const int32_t* starts;
    const void *k_new, *v_new;
    uint32_t tokens, touched;      // pages that `tokens` tokens can touch
};

template <int DIM, int IN>
__global__ __launch_bounds__(kThreads) void kv8_append_kernel(AppendArgs a) {
    constexpr int Q = DIM / 4, E = DIM / 8;  // groups of four and of eight channels
    constexpr int U = kPage * E / kThreads;  // of the latter for each thread
    __shared__ float shared[kThreads / 64];
    __shared__ uint32_t tile[Q][kPage + 1];  // values: word (channels / 4, token)
    const uint32_t which = blockIdx.x % 2, h = blockIdx.x / 2 % a.c.heads;
    const uint32_t rest = blockIdx.x / 2 / a.c.heads, b = rest / a.touched;
    const int64_t start = a.starts[b];
    if (start < 0) return;
    const int64_t page = start / kPage + rest % a.touched, p0 = page * kPage;
    const int64_t lo = start > p0 ? start : p0;
    const int64_t hi = start + a.tokens < p0 + kPage ? start + a.tokens : p0 + kPage;
    if (lo >= hi || page >= a.c.width) return;
    const int32_t id = valid_page(a.c.table[(size_t)b * a.c.width + page], a.c.pages);
    if (id < 0) return;
    const int old = (int)(lo - p0), fresh = (int)(hi - lo);
    const size_t at = (size_t)id * a.c.heads + h;
    const void* x = which ? a.v_new : a.k_new;
    float* scale_at = (which ? a.c.v_scales : a.c.k_scales) + at;
    int8_t* codes = (which ? a.c.v : a.c.k) + at * (kPage * DIM);
    const float before = old ? *scale_at : 0.0f;

    kv_f32x4 v[U][2];
    float m = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + threadIdx.x, t = i / E, e = i % E;
        v[u][0] = v[u][1] = kv_f32x4{};
        if (t < fresh)
            load8<IN>(x, (((size_t)b * a.tokens + (size_t)(lo - start) + t) * a.c.heads + h) * DIM + e * 8, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) m = absmax4(v[u][1], absmax4(v[u][0], m));
    const float scale = fmaxf(before, group_max(m, shared) / 127.0f);   // waits until all have read `before`
    const bool grown = scale > before;
    if (threadIdx.x == 0) *scale_at = scale;

    with_codes(scale, [&](auto codes4) {
        if (which == 0) {
            if (grown)
                for (int i = threadIdx.x; i < old * Q; i += kThreads) {
                    uint32_t* w = reinterpret_cast<uint32_t*>(codes) + i;
                    *w = codes4(values4(*w, before));
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = u * kThreads + threadIdx.x;
                if (i / E < fresh)
                    reinterpret_cast<uint2*>(codes)[old * E + i] = make_uint2(codes4(v[u][0]), codes4(v[u][1]));
            }
            return;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * kThreads + threadIdx.x, t = i / E, e = i % E;
            if (t >= fresh) break;
            tile[2 * e][old + t] = codes4(v[u][0]);
            tile[2 * e + 1][old + t] = codes4(v[u][1]);
        }
        __syncthreads();
        // four channels by four tokens at a time
        for (int i = threadIdx.x; i < Q * (kPage / 4); i += kThreads) {
            const int q = i / (kPage / 4), t = i % (kPage / 4) * 4;
            if (t >= old + fresh || (t + 4 <= old && !grown)) continue;
            uint32_t w[4], keep[4] = {};
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = t + k >= old && t + k < old + fresh ? tile[q][t + k] : 0;
            transpose4(w);
            uint32_t* row = reinterpret_cast<uint32_t*>(codes + (size_t)q * 4 * kPage + t);
            if (t < old) {
                const uint32_t mask = old - t >= 4 ? ~0u : (1u << (8 * (old - t))) - 1u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    keep[k] = row[k * (kPage / 4)];
                    if (grown) keep[k] = codes4(values4(keep[k], before));
                    keep[k] &= mask;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) row[k * (kPage / 4)] = w[k] | keep[k];
        }
    });
}

// ---------------------------------------------------------------------------
// read.  The same workgroups; the values' codes change from [dim][token] to
// [token][dim] by 4 x 4 byte transposes on the way into LDS.

struct ReadArgs {
    Kv8 c;
    const int32_t* starts;
    void *k_out, *v_out;
    uint32_t tokens, touched;
};

template <int DIM, int OUT>
__global__ __launch_bounds__(kThreads) void kv8_read_kernel(ReadArgs a) {
    constexpr int Q = DIM / 4;
    constexpr int U = kPage * Q / kThreads;
    __shared__ uint32_t tile[kPage][Q + 1];
    const uint32_t which = blockIdx.x % 2, h = blockIdx.x / 2 % a.c.heads;
    const uint32_t rest = blockIdx.x / 2 / a.c.heads, b = rest / a.touched;
    const int64_t start = a.starts[b] < 0 ? 0 : a.starts[b];
    const int64_t page = start / kPage + rest % a.touched, p0 = page * kPage;
    const int64_t lo = start > p0 ? start : p0;
    const int64_t hi = start + a.tokens < p0 + kPage ? start + a.tokens : p0 + kPage;
    if (lo >= hi) return;
    const int32_t n = clamp_length(a.c.lengths[b], a.c.width * kPage);
    const int skip = (int)(lo - p0), count = (int)(hi - lo);
    int there = n > lo && a.starts[b] >= 0 ? (int)(n - lo < count ? n - lo : count) : 0;    // tokens of this page that the cache holds
    const int32_t id = there ? valid_page(a.c.table[(size_t)b * a.c.width + page], a.c.pages) : -1;
    if (id < 0) there = 0;
    const size_t at = id < 0 ? 0 : (size_t)id * a.c.heads + h;
    const float s = there ? (which ? a.c.v_scales : a.c.k_scales)[at] : 0.0f;
    const int8_t* codes = (which ? a.c.v : a.c.k) + at * (kPage * DIM);
    void* out = which ? a.v_out : a.k_out;
    const size_t first = (size_t)b * a.tokens + (size_t)(lo - start);

    if (which && there) {
#pragma unroll
        for (int u = 0; u < U / 4; ++u) {
            const int i = u * kThreads + threadIdx.x, q = i / (kPage / 4), t = i % (kPage / 4);
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = reinterpret_cast<const uint32_t*>(codes)[(q * 4 + k) * (kPage / 4) + t];
            transpose4(w);
#pragma unroll
            for (int k = 0; k < 4; ++k) tile[t * 4 + k][q] = w[k];
        }
    }
    if (which) __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + threadIdx.x, t = i / Q, q = i % Q;
        if (t >= count) break;
        uint32_t w = 0;
        if (t < there) w = which ? tile[skip + t][q] : reinterpret_cast<const uint32_t*>(codes)[skip * Q + i];
        store4<OUT>(out, ((first + t) * a.c.heads + h) * DIM + q * 4, values4(w, s));
    }
}

// ---------------------------------------------------------------------------
// attention.
//
// Scores are formed transposed, S^T = K Q^T, and so is the output, O^T = V^T
// P^T: a lane's accumulators then hold many keys (or channels) of ONE row, so
// the softmax needs one exchange between lanes for a whole page, its factors
// multiply accumulators without being broadcast, and the scores leave the
// first product in the registers in which the second wants them.  That last
// step works by the order in which keys are given to the rows of the first
// product; see the two kernels.
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

struct AttendArgs {
    Kv8 c;
    const void* q;
    const int32_t* q_lens;              // may be null: every sequence has `queries`
    void* out;
    float *part, *stats;                // of the splits
    float* lse;                         // log2 of each row's sum, for the weights; may be null
    float* weights;
    uint32_t queries, heads, group, rows, splits, pages_per_split, tiles;
    float scale;                        // of the scores, times log2(e), without its sign
    bool negative;                      // its sign, which the queries take
};

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

// A sequence's numbers.  Row r of a kv head is query r / group with head
// r % group of its group; it sees the keys below limit(r).
struct Sequence {
    int32_t n, m;
    uint32_t group, rows;
    __device__ __forceinline__ Sequence(const AttendArgs& a, uint32_t b)
        : n(clamp_length(a.c.lengths[b], a.c.width * kPage)),
          m(a.q_lens ? clamp_length(a.q_lens[b], a.queries) : (int32_t)a.queries), group(a.group), rows(a.rows) {}
    __device__ __forceinline__ bool counts(uint32_t r) const { return r < rows && (int32_t)(r / group) < m; }
    __device__ __forceinline__ int32_t limit(uint32_t r) const { return n - m + (int32_t)(r / group) + 1; }
};

// Row of the queries' and outputs' [batch, queries, heads] for row r.
__device__ __forceinline__ size_t query_row(const AttendArgs& a, uint32_t b, uint32_t h, uint32_t r) {
    return ((size_t)b * a.queries + r / a.group) * a.heads + h * a.group + r % a.group;
}

template <int OUT>
__device__ __forceinline__ void store1(void* x, size_t e, float v) {
    if constexpr (OUT == kOutBF16)
        ((uint16_t*)x)[e] = (uint16_t)pack_bf16x2(v, 0.0f);
    else
        ((float*)x)[e] = v;
}

// --- few rows (16 MT at most): bound by reading the cache.  Every wave takes
// a page at a time, straight from memory to registers, the next page's keys
// on their way while this page's are used and the values likewise; no wave
// waits for another until the end.
//
// 16x16x32 products: lane l = 16 g + r gives row r (a key, a channel) eight
// elements of the sum and receives, for row r of the queries, the keys 4 g ..
// 4 g + 3 of a tile of 16.  Row r of tile t is given key 16 (r / 4) + 4 t +
// r % 4: then lane group g receives keys 16 g .. 16 g + 15 over the four
// tiles, which are the 16 contiguous bytes that it loads of each channel of
// the values.

// Two waves to a SIMD where the registers allow: the compiler then keeps the
// products' results where the softmax can use them without a move.
template <int DIM, int MT, int IN, int NW>
__global__ __launch_bounds__(NW * 64, DIM == 256 || MT == 2 ? 1 : 2) void kv8_attend_few_kernel(AttendArgs a) {
    constexpr int T = IN == kInBF16 ? 1 : 2;
    constexpr int KC = DIM / 64, VC = DIM / 16;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, r = lane % 16, g = lane / 16;
    const uint32_t split = blockIdx.x % a.splits, bh = blockIdx.x / a.splits, h = bh % a.c.heads, b = bh / a.c.heads;
    // The wave's first 64 pages are looked up at once, one in each lane, while
    // the sequence's length is on its way: entries behind it are not used.
    const uint32_t first = split * a.pages_per_split, limit_page = min(first + a.pages_per_split, a.c.width);
    int32_t my_id;
    float my_ks, my_vs;
    auto look_up = [&](uint32_t page) {
        my_id = -1, my_ks = my_vs = 0.0f;
        if (page < limit_page) {
            my_id = valid_page(a.c.table[(size_t)b * a.c.width + page], a.c.pages);
            if (my_id >= 0) {
                my_ks = a.c.k_scales[(size_t)my_id * a.c.heads + h];
                my_vs = a.c.v_scales[(size_t)my_id * a.c.heads + h];
            }
        }
    };
    look_up(first + wave + lane * NW);
    const Sequence seq(a, b);
    const uint32_t pages = (uint32_t)(seq.n + kPage - 1) / kPage, last = min(limit_page, pages);
    if (first >= last && split) return;

    Query<IN, DIM, 16, 64> raw[MT];
    int32_t limit[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const uint32_t row = i * 16 + r;
        const bool there = seq.counts(row);
        raw[i].load(a.q, there ? query_row(a, b, h, row) : 0, g * 16, there);
        limit[i] = there ? seq.limit(row) : INT32_MAX;       // rows that are not there are not stored
    }
    kv_half8 q[MT][DIM / 32][T];
    float undo[MT];
    const int32_t all_see = seq.n - seq.m + 1;               // every row sees the keys below

    kv_f32x4 o[MT][VC] = {};
    Unit unit;
    float top[MT], total[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) top[i] = -FLT_MAX, total[i] = 0.0f;

    const size_t head_bytes = (size_t)kPage * DIM;
    // values are read once, keys once more where weights are wanted: these may
    // stay in the caches (125 against 130 us for 64 sequences of 8,000 tokens)
    const uint32_t k_at = (r / 4 * 16 + r % 4) * DIM + g * 16, v_at = r * kPage + g * 16;
    uint4 kr[4][KC], vr[VC];
    auto load_k = [&](int32_t id) {
        const int8_t* p = a.c.k + ((size_t)max(id, 0) * a.c.heads + h) * head_bytes + k_at;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int c = 0; c < KC; ++c) kr[t][c] = *reinterpret_cast<const uint4*>(p + t * 4 * DIM + c * 64);
    };
    auto load_v = [&](int32_t id) {
        const int8_t* p = a.c.v + ((size_t)max(id, 0) * a.c.heads + h) * head_bytes + v_at;
#pragma unroll
        for (int c = 0; c < VC; ++c) vr[c] = load_b128(p + c * 16 * kPage);
    };

    for (uint32_t base = first + wave; base < last; base += 64 * NW) {
        if (base != first + wave) look_up(base + lane * NW);
        const uint32_t count = min(64u, (last - base + NW - 1) / NW);
        int32_t id = __builtin_amdgcn_readlane(my_id, 0);
        load_k(id);
        load_v(id);
        if (base == first + wave) {
#pragma unroll
            for (int i = 0; i < MT; ++i) undo[i] = raw[i].template convert<16, T>(a.negative, q[i]) * a.scale;
        }
        for (uint32_t i = 0; i < count; ++i) {
            const int32_t next = __builtin_amdgcn_readlane(my_id, min(i + 1, count - 1));
            const float ks = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_ks), i));
            const float vs = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_vs), i));
            const int32_t key0 = (int32_t)((base + i * NW) * kPage);

            kv_f32x4 s[MT][4] = {};
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    kv_half8 k[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        k[t] = u ? half_codes(kr[t][c].z, kr[t][c].w) : half_codes(kr[t][c].x, kr[t][c].y);
#pragma unroll
                    for (int j = 0; j < MT; ++j)
#pragma unroll
                        for (int e = 0; e < T; ++e)
#pragma unroll
                            for (int t = 0; t < 4; ++t)
                                s[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[t], q[j][2 * c + u][e], s[j][t], 0, 0, 0);
                }
            if (i + 1 < count) load_k(next);

            const float shrink_all = unit.next(vs);
            if (shrink_all != 1.0f)
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int c = 0; c < VC; ++c) o[j][c] *= shrink_all;
            kv_half8 p[MT][2][T];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                float factor = ks * undo[j];
                if (key0 + kPage > all_see || id < 0) {
                    const int32_t sees = (id < 0 ? 0 : limit[j]) - key0 - (int32_t)g * 16;
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int k = 0; k < 4; ++k) s[j][t][k] = 4 * t + k < sees ? s[j][t][k] * factor : -INFINITY;
                    factor = 1.0f;
                }
                float m = max3(s[j][0][0], s[j][0][1], s[j][0][2]);
#pragma unroll
                for (int k = 3; k < 15; k += 2) m = max3(m, s[j][k / 4][k % 4], s[j][(k + 1) / 4][(k + 1) % 4]);
                m = fmaxf(max_over_16(fmaxf(m, s[j][3][3])) * factor, top[j]);
                if (__any(m > top[j])) {
                    const float shrink = __builtin_amdgcn_exp2f(top[j] - m);
                    total[j] *= shrink;
#pragma unroll
                    for (int c = 0; c < VC; ++c) o[j][c] *= shrink;
                    top[j] = m;
                }
                const float off = unit.lift - m;
                float sum = 0.0f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        x[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[j][2 * u + k / 4][k % 4], factor, off));
                    sum += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
                    half_terms<T>(x, p[j][u]);
                }
                total[j] = __builtin_fmaf(sum, unit.drop, total[j]);
            }
            // two tiles at a time, so that neighbouring products add to different ones
#pragma unroll
            for (int c = 0; c < VC; c += 2) {
                const kv_half8 v[2][2] = {{half_codes(vr[c].x, vr[c].y), half_codes(vr[c + 1].x, vr[c + 1].y)},
                                          {half_codes(vr[c].z, vr[c].w), half_codes(vr[c + 1].z, vr[c + 1].w)}};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < T; ++e)
#pragma unroll
                        for (int j = 0; j < MT; ++j)
#pragma unroll
                            for (int d = 0; d < 2; ++d)
                                o[j][c + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[u][d], p[j][u][e], o[j][c + d], 0, 0, 0);
            }
            if (i + 1 < count) load_v(next);
            id = next;
        }
    }

    // the waves' results meet in LDS, 16 rows at a time
    __shared__ float os[NW][16][DIM + 4];
    __shared__ float tops[NW][16], totals[NW][16];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        if (j) __syncthreads();
        if (j * 16u < a.rows) {
            total[j] = sum_over_16(total[j]);
            if (g == 0) tops[wave][r] = top[j], totals[wave][r] = total[j];
#pragma unroll
            for (int c = 0; c < VC; ++c) *reinterpret_cast<kv_f32x4*>(&os[wave][r][c * 16 + g * 4]) = o[j][c] * unit.unit;
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < 16 * DIM; i += NW * 64) {
            const uint32_t row16 = i / DIM, d = i % DIM, row = j * 16 + row16;
            if (row >= a.rows) break;
            float m = tops[0][row16], l = 0.0f, y = 0.0f;
#pragma unroll
            for (int w = 1; w < NW; ++w) m = fmaxf(m, tops[w][row16]);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float f = __builtin_amdgcn_exp2f(tops[w][row16] - m);
                l = __builtin_fmaf(totals[w][row16], f, l);
                y = __builtin_fmaf(os[w][row16][d], f, y);
            }
            if (a.splits == 1) {
                const bool seen = seq.counts(row) && l != 0.0f;
                store1<IN>(a.out, query_row(a, b, h, row) * DIM + d, seen ? y / l : 0.0f);
                if (a.lse && d == 0) a.lse[(size_t)bh * a.rows + row] = seen ? m - kLift + __builtin_amdgcn_logf(l) : INFINITY;
            } else {
                const size_t at = ((size_t)bh * a.splits + split) * a.rows + row;
                a.part[at * DIM + d] = y;
                if (d == 0) a.stats[at * 2] = m, a.stats[at * 2 + 1] = l;
            }
        }
    }
}

// The splits' results joined: DIM / 4 lanes with four channels each take a row,
// or GROUPS times as many, each time some of its splits.  Few rows with many
// splits want many groups, or they wait for one load after another (one group:
// 16.0 us, eight: 5.7 for 256 rows of 32 splits); many rows with few splits one, or
// most groups have nothing to read (eight: 22.7 us, one: 7.5 for 23,580 rows of 3
// splits).
constexpr int kJoinRows = 8;                // rows times groups of a workgroup

template <int DIM, int OUT, int GROUPS>
__global__ __launch_bounds__(kJoinRows * DIM / 4) void kv8_join_kernel(AttendArgs a) {
    constexpr int Q = DIM / 4, ROWS = kJoinRows / GROUPS;
    __shared__ kv_f32x4 ys[ROWS][GROUPS][Q];
    __shared__ float tops[ROWS][GROUPS], totals[ROWS][GROUPS];
    const uint32_t q = threadIdx.x % Q, group = threadIdx.x / Q % GROUPS;
    const uint32_t mine = ROWS > 1 ? threadIdx.x / Q / GROUPS : 0;
    const uint32_t rows = a.c.batch * a.c.heads * a.rows, item = blockIdx.x * ROWS + mine;
    const bool inside = item < rows;
    const uint32_t row = item % a.rows, bh = min(item, rows - 1) / a.rows, h = bh % a.c.heads, b = bh / a.c.heads;
    const Sequence seq(a, b);
    // the splits that hold keys which this row may see
    const int32_t seen_keys = inside && seq.counts(row) ? min(seq.limit(row), seq.n) : 0;
    const uint32_t pages = seen_keys > 0 ? (uint32_t)(seen_keys + kPage - 1) / kPage : 0;
    const uint32_t used = (pages + a.pages_per_split - 1) / a.pages_per_split;
    float m = -FLT_MAX, l = 0.0f;
    kv_f32x4 y = {};
#pragma unroll 4
    for (uint32_t s = group; s < used; s += GROUPS) {
        const size_t at = ((size_t)bh * a.splits + s) * a.rows + row;
        const float2 stat = *reinterpret_cast<const float2*>(a.stats + at * 2);
        const kv_f32x4 x = *reinterpret_cast<const kv_f32x4*>(a.part + at * DIM + q * 4);
        const float top = fmaxf(m, stat.x), f = __builtin_amdgcn_exp2f(m - top), e = __builtin_amdgcn_exp2f(stat.x - top);
        m = top;
        l = __builtin_fmaf(stat.y, e, l * f);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = __builtin_fmaf(x[k], e, y[k] * f);
    }
    if constexpr (GROUPS > 1) {
        ys[mine][group][q] = y;
        if (q == 0) tops[mine][group] = m, totals[mine][group] = l;
        __syncthreads();
        if (group) return;
        m = tops[mine][0];
#pragma unroll
        for (int s = 1; s < GROUPS; ++s) m = fmaxf(m, tops[mine][s]);
        l = 0.0f;
        y = kv_f32x4{};
#pragma unroll
        for (int s = 0; s < GROUPS; ++s) {
            const float f = __builtin_amdgcn_exp2f(tops[mine][s] - m);
            l = __builtin_fmaf(totals[mine][s], f, l);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __builtin_fmaf(ys[mine][s][q][k], f, y[k]);
        }
    }
    if (!inside) return;
    const bool seen = l != 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = seen ? y[k] / l : 0.0f;
    store4<OUT>(a.out, query_row(a, b, h, row) * DIM + q * 4, y);
    if (a.lse && q == 0) a.lse[item] = seen ? m - kLift + __builtin_amdgcn_logf(l) : INFINITY;
}

// --- many rows: four waves of 32 rows share a page in LDS, converted to
// binary16 once for all of them; the next page's codes are on their way to LDS
// meanwhile, so that no registers wait for them and one more workgroup fits a
// CU (1,000 queries x 64 heads of 64 channels 100 -> 92 us, 16 heads of 256
// channels 126 -> 121; with 128 channels within 2% of two buffers of tiles and
// codes in registers).
//
// Bound by vector and matrix instructions together: for 4 x 1,024 queries x 32
// heads over 4,096 keys (0.8 PFLOP/s) the matrix units are busy in 35% of the
// cycles and vector instructions issue in 52%, at 2.0 GHz, to which the chip
// lowers its clock (2.4 GHz) for both.  Causal prompts wait for their longest
// tiles as well.  Measured and left out, each within 4% or slower: the next
// page's scores formed beside this page's exponentials, LDS reads 4 to 10
// products ahead, eight waves with half the keys each, raised priorities for
// the longest tiles, for matrix instructions or for one of the workgroups of a
// CU; 64 rows to a wave took 1.45 times the time, the longest tiles cut over the
// keys 1.3 to 1.6 times.
//
// 32x32x16 products: lane l = 32 g + r.  Row m of a tile of 32 keys is given
// the key with bits 2 and 3 of m exchanged: lane half g then receives keys 16
// a + 8 g .. + 7, the eight contiguous keys of the values' fragment for step
// a.  LDS rows are eight 16-byte slots (128 bytes) or a multiple; slot c of
// row r lies at c ^ (r / 2 % 8), in longer rows at c ^ (r % 16), so that the
// sixteen lanes that a 16-byte read serves at once lie in different banks.

constexpr int kTileRows = 128;

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

template <int DIM, int IN>
__global__ __launch_bounds__(kThreads, (DIM == 256 ? 1 : DIM == 128 ? 2 : 3) + (IN == kInBF16 && DIM < 256))
    void kv8_attend_many_kernel(AttendArgs a) {
    constexpr int T = IN == kInBF16 ? 1 : 2;
    constexpr int U = DIM / 64;                        // 16-byte loads of a thread, keys and values each
    constexpr int KR = DIM / 8;                        // slots of a row of keys
    const auto k_swizzle = [](uint32_t row) { return DIM == 64 ? row / 2 % 8 : row % 16; };
    __shared__ kv_half8 k_tile[kPage * KR], v_tile[DIM * 8];
    __shared__ uint4 k_codes[U * kThreads], v_codes[U * kThreads];
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), r = lane % 32,
                   g = lane / 32;
    // the last tiles see the most keys: first
    const uint32_t split = blockIdx.x % a.splits, rest = blockIdx.x / a.splits;
    const uint32_t heads = a.c.heads * a.c.batch, turn = rest / heads, tile = a.tiles - 1 - turn;
    // A CU's workgroups are 256 apart or a multiple: sequences are turned every
    // 256, or a long one would have all of its tiles on the same CUs (two
    // prompts of up to 2,048 tokens 105 -> 97 us; within 2% for other batches).
    const uint32_t h = rest % a.c.heads, b = (rest % heads / a.c.heads + (uint32_t)((size_t)turn * heads / 256)) % a.c.batch;
    const uint32_t bh = b * a.c.heads + h;
    const uint32_t first_row = tile * kTileRows + wave * 32, row = first_row + r;

    // Loads that depend on no other come first: a row of queries whatever the
    // sequence's length, and the first pages, which are used if they count.
    Query<IN, DIM, 8, 16> raw;
    raw.load(a.q, query_row(a, b, h, min(row, a.rows - 1)), g * 8, true);
    const int32_t* table = a.c.table + (size_t)b * a.c.width;
    const uint32_t first = split * a.pages_per_split, limit_page = min(first + a.pages_per_split, a.c.width);
    // The pages' numbers and scales come 64 at a time, one in each lane: looked
    // up one by one, every page would wait for a scalar load, and with it for
    // the wave's LDS reads.  Asked for in ascending order; pages behind
    // `limit_page` are read as the one before it and not used.
    struct Page {
        int32_t id;
        float ks, vs;          // 0 for a page that is not there: what page 0 holds must not matter
    };
    uint32_t base = first;
    int32_t my_id;
    float my_ks, my_vs;
    auto look_up = [&] {
        my_id = valid_page(table[min(base + lane, limit_page - 1)], a.c.pages);
        const size_t at = (size_t)max(my_id, 0) * a.c.heads + h;
        my_ks = my_id < 0 ? 0.0f : a.c.k_scales[at];
        my_vs = my_id < 0 ? 0.0f : a.c.v_scales[at];
    };
    auto page_at = [&](uint32_t page) {
        if (page - base >= 64) {
            base = page;
            look_up();
        }
        const uint32_t i = page - base;
        return Page{__builtin_amdgcn_readlane(my_id, i),
                    __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_ks), i)),
                    __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_vs), i))};
    };
    // A page's codes go straight to LDS; each lane later reads what it asked
    // for itself.
    auto fetch = [&](int32_t id) {
        const size_t at = ((size_t)max(id, 0) * a.c.heads + h) * (kPage * DIM) + tid * 16;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to_lds(a.c.k + at + u * kThreads * 16, k_codes + u * kThreads + wave * 64);
            to_lds(a.c.v + at + u * kThreads * 16, v_codes + u * kThreads + wave * 64);
        }
    };
    look_up();
    Page now = page_at(first), next = page_at(first + 1);
    fetch(now.id);

    const Sequence seq(a, b);
    const bool there = seq.counts(row);
    // pages that the tile's last row and the wave's last row see
    const auto pages_of = [&](uint32_t last_row) {
        const int32_t i = min((int32_t)(min(last_row, seq.rows - 1) / seq.group), seq.m - 1);
        const int32_t keys = seq.m > 0 && (int32_t)(tile * kTileRows / seq.group) < seq.m ? seq.n - seq.m + i + 1 : 0;
        return keys > 0 ? (uint32_t)(keys + kPage - 1) / kPage : 0u;
    };
    const uint32_t last = min(limit_page, pages_of(tile * kTileRows + kTileRows - 1));
    const uint32_t my_last = first_row < seq.rows ? min(last, pages_of(first_row + 31)) : 0;
    const int32_t limit = there ? seq.limit(row) : INT32_MAX;
    // every row of the wave sees the keys below (rows without a query see all)
    const int32_t all_see = seq.n - seq.m + (int32_t)(first_row / seq.group) + 1;

    kv_half8 q[DIM / 16][T];
    const float undo = raw.template convert<32, T>(a.negative, q) * a.scale;

    kv_f32x16 o[DIM / 32] = {};
    Unit unit;
    float top = -FLT_MAX, total = 0.0f;
    // byte offsets of the first fragments; the others differ by an exclusive or
    // or a constant
    const uint32_t k_first = r * (KR * 16) + (g ^ k_swizzle(r)) * 16, v_first = r * 128 + (g ^ r / 2 % 8) * 16;
    for (uint32_t page = first; page < last; ++page) {
        loads_done();
        uint4 kr[U], vr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) kr[u] = k_codes[u * kThreads + tid], vr[u] = v_codes[u * kThreads + tid];
        lds_barrier();                               // all waves are done with the page before
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = u * kThreads + tid;
            const uint32_t key = i / (DIM / 16), lr = exchange_bits_2_3(key), c = i % (DIM / 16) * 2;
            k_tile[lr * KR + (c ^ k_swizzle(lr))] = half_codes(kr[u].x, kr[u].y);
            k_tile[lr * KR + ((c + 1) ^ k_swizzle(lr))] = half_codes(kr[u].z, kr[u].w);
            const uint32_t d = i / 4, e = i % 4 * 2;
            v_tile[d * 8 + (e ^ d / 2 % 8)] = half_codes(vr[u].x, vr[u].y);
            v_tile[d * 8 + ((e + 1) ^ d / 2 % 8)] = half_codes(vr[u].z, vr[u].w);
        }
        const Page after = page_at(page + 2);
        if (page + 1 < last) fetch(next.id);
        lds_barrier();
        // kept in registers, all the fragments' addresses would take thirteen
        uint32_t k_at = k_first, v_at = v_first;
        asm volatile("" : "+v"(k_at), "+v"(v_at));
        if (page < my_last && now.id >= 0) {
            kv_f32x16 s[2];
            s[0] = s[1] = kv_f32x16{};
#pragma unroll
            for (int c = 0; c < DIM / 16; ++c)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const kv_half8 k = *reinterpret_cast<const kv_half8*>((const char*)k_tile + (k_at ^ (c * 32)) + t * 32 * KR * 16);
#pragma unroll
                    for (int e = 0; e < T; ++e) s[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[c][e], s[t], 0, 0, 0);
                }
            const int32_t key0 = (int32_t)(page * kPage);
            const float shrink_all = unit.next(now.vs);
            if (shrink_all != 1.0f)
#pragma unroll
                for (int d = 0; d < DIM / 32; ++d) o[d] *= shrink_all;
            float factor = now.ks * undo;
            if (key0 + kPage > all_see) {
                // register k of tile t is key 32 t + 16 (k / 8) + 8 g + k % 8
                const int32_t sees = limit - key0 - (int32_t)g * 8;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        s[t][k] = 32 * t + 16 * (k / 8) + k % 8 < sees ? s[t][k] * factor : -INFINITY;
                factor = 1.0f;
            }
            float m = max3(s[0][15], s[1][15], s[0][14]);
            float m1 = max3(s[1][14], s[0][13], s[1][13]);
#pragma unroll
            for (int k = 0; k < 12; k += 2) {
                m = max3(m, s[0][k], s[0][k + 1]);
                m1 = max3(m1, s[1][k], s[1][k + 1]);
            }
            m = max3(m, s[0][12], s[1][12]);
            m = fmaxf(max_over_32(fmaxf(m, m1)) * factor, top);
            // outputs and sums are taken to the new maximum when it has grown by
            // 2^1.5, which the numerators' type has room for
            if (__any(m > top + 1.5f)) {
                const float shrink = __builtin_amdgcn_exp2f(top - m);
                total *= shrink;
#pragma unroll
                for (int d = 0; d < DIM / 32; ++d) o[d] *= shrink;
                top = m;
            }
            const float off = unit.lift - top;
            kv_half8 p[4][T];
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u / 2][u % 2 * 8 + k], factor, off));
                sum += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
                half_terms<T>(x, p[u]);
            }
            total = __builtin_fmaf(sum, unit.drop, total);
            // neighbouring products add to different tiles: none waits for the one before it
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int d = 0; d < DIM / 32; ++d) {
                    const kv_half8 v = *reinterpret_cast<const kv_half8*>((const char*)v_tile + (v_at ^ (u * 32)) + d * 32 * 128);
#pragma unroll
                    for (int e = 0; e < T; ++e) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[u][e], o[d], 0, 0, 0);
                }
        }
        now = next, next = after;
    }
    loads_done();                                    // nothing may write to LDS that is no longer this workgroup's

    total = sum_over_32(total);
    if (row >= a.rows) return;
    const bool seen = there && total != 0.0f;
    const float f = a.splits > 1 ? unit.unit : seen ? unit.unit / total : 0.0f;
    const size_t at = a.splits > 1 ? (((size_t)bh * a.splits + split) * a.rows + row) * DIM : query_row(a, b, h, row) * DIM;
    // register k of tile d is channel 32 d + 8 (k / 4) + 4 g + k % 4
#pragma unroll
    for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const kv_f32x4 y = {o[d][k] * f, o[d][k + 1] * f, o[d][k + 2] * f, o[d][k + 3] * f};
            const size_t to = at + d * 32 + k * 2 + g * 4;
            if (a.splits > 1)
                *reinterpret_cast<kv_f32x4*>(a.part + to) = y;
            else
                merge4<IN>(a.out, to, seen ? y : kv_f32x4{});
        }
    if (g) return;
    if (a.splits > 1)
        a.stats[at / DIM * 2] = top, a.stats[at / DIM * 2 + 1] = total;
    else if (a.lse)
        a.lse[(size_t)bh * a.rows + row] = seen ? top - kLift + __builtin_amdgcn_logf(total) : INFINITY;
}

// --- the weights that the keys received: with every row's log2 sum known, a
// wave forms a page's scores again (reading its keys only), and adds up their
// exponentials over the rows.  Each weight belongs to one wave, which adds in
// one order: no atomics.  16 rows at most: their queries stay in registers
// over the wave's pages.

// Of 2 N values a lane keeps the upper N if it is `upper`, else the lower, and
// adds what its partner has of them.
template <int CTRL, int N>
__device__ __forceinline__ void halve(float (&v)[16], bool upper) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float keep = upper ? v[i + N] : v[i], give = upper ? v[i] : v[i + N];
        v[i] = keep + dpp_move<CTRL>(give);
    }
}

template <int DIM, int IN>
__global__ __launch_bounds__(kThreads) void kv8_weights_kernel(AttendArgs a) {
    constexpr int T = IN == kInBF16 ? 1 : 2;
    constexpr int KC = DIM / 64;
    const uint32_t lane = threadIdx.x % 64, r = lane % 16, g = lane / 16;
    const uint32_t waves = a.splits * (kThreads / 64);
    const uint32_t bh = blockIdx.x / a.splits, h = bh % a.c.heads, b = bh / a.c.heads;
    const uint32_t wave = blockIdx.x % a.splits * (kThreads / 64) + threadIdx.x / 64;
    const Sequence seq(a, b);
    const uint32_t pages = (uint32_t)(seq.n + kPage - 1) / kPage;
    // a wave has a run of pages, at most 64, whose numbers and scales its lanes hold
    const uint32_t run = (pages + waves - 1) / waves, first = wave * run, last = min(first + run, pages);
    if (first >= last || seq.m == 0) return;
    const int32_t my_id = valid_page(a.c.table[(size_t)b * a.c.width + min(first + lane, last - 1)], a.c.pages);
    const float my_ks = my_id < 0 ? 0.0f : a.c.k_scales[(size_t)my_id * a.c.heads + h];

    Query<IN, DIM, 16, 64> raw;
    kv_half8 q[DIM / 32][T];
    float undo = 0.0f, lse = INFINITY;
    int32_t limit = 0;
    if (seq.counts(r)) {
        raw.load(a.q, query_row(a, b, h, r), g * 16, true);
        lse = a.lse[(size_t)bh * a.rows + r];
        limit = seq.limit(r);
    } else {
        raw.load(a.q, 0, 0, false);
    }
    const uint32_t k_at = (r / 4 * 16 + r % 4) * DIM + g * 16;
    float* weights = a.weights + (size_t)bh * a.c.width * kPage;
    uint4 kr[4][KC];
    float next_old = 0.0f;
    auto load_page = [&](uint32_t page, int32_t page_id) {
        const int8_t* k = a.c.k + ((size_t)max(page_id, 0) * a.c.heads + h) * (kPage * DIM) + k_at;
        next_old = weights[page * kPage + lane];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int c = 0; c < KC; ++c) kr[t][c] = *reinterpret_cast<const uint4*>(k + t * 4 * DIM + c * 64);
    };
    int32_t id = __builtin_amdgcn_readlane(my_id, 0);
    load_page(first, id);
    undo = raw.template convert<16, T>(a.negative, q) * a.scale;
    for (uint32_t page = first; page < last; ++page) {
        const uint32_t i = page - first;
        const float ks = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_ks), i));
        const float old = next_old;
        const int32_t next_id = __builtin_amdgcn_readlane(my_id, min(i + 1, last - first - 1));
        kv_f32x4 sum[4] = {};
        const int32_t key0 = (int32_t)(page * kPage + g * 16);
        kv_f32x4 s[4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const kv_half8 k = u ? half_codes(kr[t][c].z, kr[t][c].w) : half_codes(kr[t][c].x, kr[t][c].y);
#pragma unroll
                    for (int e = 0; e < T; ++e)
                        s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[2 * c + u][e], s[t], 0, 0, 0);
                }
        if (page + 1 < last) load_page(page + 1, next_id);
        const float factor = ks * undo;
        const int32_t sees = id < 0 ? 0 : limit - key0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sum[t][k] = 4 * t + k < sees ? __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][k], factor, -lse)) : 0.0f;
        // over the 16 lanes of a row: each exchange halves the keys that a lane
        // still sums, and lane r is left with key 16 g + r
        float v[16];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * t + k] = sum[t][k];
        halve<kDppRowRotate8, 8>(v, r & 8);
        halve<kDppRowHalfMirror, 4>(v, r & 4);
        halve<kDppSwapPairs, 2>(v, r & 2);
        halve<kDppSwapAdjacent, 1>(v, r & 1);
        const float mine = v[0];
        const int32_t key = key0 + (int32_t)r;
        if (key < seq.n && id >= 0) weights[key] = old + mine;
        id = next_id;
    }
}

// The same for more rows.  Their queries are converted once, into fragments
// that a wave of the second kernel reads whole lines of; a wave there has 32
// keys in registers and runs over a share of the row tiles, whose sums are
// added in order by the third kernel where there are several shares.

constexpr int kShareThreads = 256, kShareKeys = kShareThreads / 64 * 32;

struct Row {
    float factor, lse;     // log2 sum: infinite for rows without a query
    int32_t limit;
};

struct ShareArgs {
    AttendArgs a;
    kv_half8* fragments;   // [sequence and head][tile of 32 rows][dim / 16][term][lane]
    Row* rows;             // [sequence and head][tiles * 32]
    float* sums;           // [share][sequence and head][width * kPage], where shares > 1
    uint32_t row_tiles, shares, key_groups;
};

template <int DIM, int IN>
__global__ __launch_bounds__(kShareThreads) void kv8_fragments_kernel(ShareArgs s) {
    constexpr int T = IN == kInBF16 ? 1 : 2;
    const AttendArgs& a = s.a;
    const uint32_t lane = threadIdx.x % 64, r = lane % 32, g = lane / 32;
    const size_t unit = (size_t)blockIdx.x * (kShareThreads / 64) + threadIdx.x / 64;
    if (unit >= (size_t)a.c.batch * a.c.heads * s.row_tiles) return;
    const uint32_t tile = unit % s.row_tiles, bh = unit / s.row_tiles, h = bh % a.c.heads, b = bh / a.c.heads;
    const Sequence seq(a, b);
    const uint32_t row = tile * 32 + r;
    const bool there = seq.counts(row);
    Query<IN, DIM, 8, 16> raw;
    raw.load(a.q, there ? query_row(a, b, h, row) : 0, g * 8, there);
    kv_half8 q[DIM / 16][T];
    const float undo = raw.template convert<32, T>(a.negative, q) * a.scale;
#pragma unroll
    for (int c = 0; c < DIM / 16; ++c)
#pragma unroll
        for (int e = 0; e < T; ++e) s.fragments[((unit * (DIM / 16) + c) * T + e) * 64 + lane] = q[c][e];
    if (g == 0)
        s.rows[unit * 32 + r] = Row{undo, there ? a.lse[(size_t)bh * a.rows + row] : INFINITY, there ? seq.limit(row) : 0};
}

template <int DIM, int IN>
__global__ __launch_bounds__(kShareThreads) void kv8_shares_kernel(ShareArgs s) {
    constexpr int T = IN == kInBF16 ? 1 : 2, N = DIM / 16;
    const AttendArgs& a = s.a;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, r = lane % 32, g = lane / 32;
    const uint32_t share = blockIdx.x % s.shares, rest = blockIdx.x / s.shares;
    const uint32_t bh = rest / s.key_groups, h = bh % a.c.heads, b = bh / a.c.heads;
    const uint32_t key0 = rest % s.key_groups * kShareKeys + wave * 32, page = key0 / kPage;
    if (page >= a.c.width) return;
    const Sequence seq(a, b);
    const int32_t id = valid_page(a.c.table[(size_t)b * a.c.width + page], a.c.pages);
    const size_t tokens = (size_t)a.c.width * kPage;
    float* out = (s.shares > 1 ? s.sums + ((size_t)share * a.c.batch * a.c.heads + bh) * tokens : a.weights + bh * tokens) + key0;

    float mine = 0.0f;
    if ((int32_t)key0 < seq.n && seq.m > 0 && id >= 0) {
        // row m of the products is the key with bits 2 and 3 exchanged, as above
        const size_t at = (size_t)id * a.c.heads + h;
        const float ks = a.c.k_scales[at];
        const int8_t* codes = a.c.k + at * (kPage * DIM) + (key0 % kPage + exchange_bits_2_3(r)) * DIM + g * 8;
        kv_half8 k[N];
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const uint2 w = *reinterpret_cast<const uint2*>(codes + c * 16);
            k[c] = half_codes(w.x, w.y);
        }
        // the first tile with a row that sees key0, and this share of the tiles from there on
        const int32_t before = (int32_t)key0 - (seq.n - seq.m);
        const uint32_t first_tile = before > 0 ? (uint32_t)((size_t)before * seq.group / 32) : 0;
        const uint32_t end_tile = min(s.row_tiles, (uint32_t)(((size_t)seq.m * seq.group + 31) / 32));
        const uint32_t count = end_tile > first_tile ? end_tile - first_tile : 0, per = (count + s.shares - 1) / s.shares;
        const uint32_t from = first_tile + min(share * per, count), to = first_tile + min((share + 1) * per, count);
        kv_f32x16 sum = {};
        kv_half8 q[N][T];
        Row row;
        auto load = [&](uint32_t tile) {
            const size_t unit = (size_t)bh * s.row_tiles + tile;
#pragma unroll
            for (int c = 0; c < N; ++c)
#pragma unroll
                for (int e = 0; e < T; ++e) q[c][e] = s.fragments[((unit * N + c) * T + e) * 64 + lane];
            row = s.rows[unit * 32 + r];
        };
        if (from < to) load(from);
        for (uint32_t tile = from; tile < to; ++tile) {
            // two sums, so that neighbouring products do not wait for each other
            kv_f32x16 even = {}, odd = {};
#pragma unroll
            for (int c = 0; c < N; ++c)
#pragma unroll
                for (int e = 0; e < T; ++e) {
                    if ((c * T + e) % 2)
                        odd = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[c], q[c][e], odd, 0, 0, 0);
                    else
                        even = __builtin_amdgcn_mfma_f32_32x32x16_f16(k[c], q[c][e], even, 0, 0, 0);
                }
            const Row now = row;
            if (tile + 1 < to) load(tile + 1);
            const float factor = ks * now.factor;
            const auto share_of = [&](int i) {
                return __builtin_amdgcn_exp2f(__builtin_fmaf(even[i] + odd[i], factor, -now.lse));
            };
            // the tile's first row sees the fewest keys; rows without a query give 0 by their sum
            if (__builtin_amdgcn_readfirstlane(now.limit) >= (int32_t)key0 + 32) {
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] += share_of(i);
            } else {
                const int32_t sees = now.limit - (int32_t)key0 - (int32_t)g * 8;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[i] += 16 * (i / 8) + i % 8 < sees ? share_of(i) : 0.0f;
            }
        }
        // over the 32 lanes of a half; lane r < 16 of it keeps register r's key
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = sum[i];
            v += dpp_move<kDppSwapAdjacent>(v);
            v += dpp_move<kDppSwapPairs>(v);
            v += dpp_move<kDppRowHalfMirror>(v);
            v += dpp_move<kDppRowMirror>(v);
            const Pair p = with_lane_16(v);
            v = p.a + p.b;
            if (r == (uint32_t)i) mine = v;
        }
    }
    if (r >= 16) return;
    const uint32_t key = 16 * (r / 8) + 8 * g + r % 8;
    if (s.shares > 1)
        out[key] = mine;
    else if ((int32_t)(key0 + key) < seq.n)
        out[key] += mine;
}

__global__ __launch_bounds__(kShareThreads) void kv8_add_shares_kernel(ShareArgs s) {
    const AttendArgs& a = s.a;
    const size_t tokens = (size_t)a.c.width * kPage, all = (size_t)a.c.batch * a.c.heads * tokens;
    const size_t i = (size_t)blockIdx.x * kShareThreads + threadIdx.x;
    if (i >= all || (int32_t)(i % tokens) >= clamp_length(a.c.lengths[i / tokens / a.c.heads], a.c.width * kPage)) return;
    float y = 0.0f;
    for (uint32_t share = 0; share < s.shares; ++share) y += s.sums[share * all + i];
    a.weights[i] += y;
}

// ---------------------------------------------------------------------------
// evict.  First the choice: one workgroup for each sequence and head finds the
// weight of the last token that stays by three histograms (11, 11 and 10 bits
// of the weights' order-preserving bit patterns), then writes the kept
// indexes in order: each thread counts what it keeps of its own tokens, and
// then places it.  The lower index stays where weights are equal.

constexpr int kBins = 2048;

struct EvictArgs {
    Kv8 c, into;
    const float* weights;
    uint32_t recent, keep;
    int32_t* kept;
    float* moved;
};

// Ascending unsigned integers for ascending weights; -0 counts as 0, NaN above everything.
__device__ __forceinline__ uint32_t order_of(float w) {
    if (w != w) return ~0u;
    const uint32_t bits = __builtin_bit_cast(uint32_t, w + 0.0f);
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

// The weight with that order (0 for -0, one NaN for all).
__device__ __forceinline__ float weight_of(uint32_t order) {
    return __builtin_bit_cast(float, order & 0x80000000u ? order ^ 0x80000000u : ~order);
}

// A thread has `own` consecutive tokens (a multiple of four).  The order of
// the first HELD stays in registers; tokens behind them are read again where
// needed.  0 stands for no token: no weight's order is that low.
template <int THREADS, int HELD>
struct Tokens {
    const float* w;
    uint32_t first, end;
    uint32_t held[HELD];
    __device__ __forceinline__ Tokens(const float* weights, uint32_t all, uint32_t own) : w(weights) {
        first = min((uint32_t)threadIdx.x * own, all);
        end = min(first + own, all);
#pragma unroll
        for (int j = 0; j < HELD; j += 4) {
            mine4(first + j, held + j);
        }
    }
    __device__ __forceinline__ void mine4(uint32_t i, uint32_t* o) const {
        kv_f32x4 x = {};
        if (i + 4 <= end)
            x = *reinterpret_cast<const kv_f32x4*>(w + i);
        else
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < end) x[k] = w[i + k];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = i + k < end ? order_of(x[k]) : 0;
    }
    template <class F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll
        for (int j = 0; j < HELD; ++j) f(first + j, held[j]);
        for (uint32_t i = first + HELD; i < end; ++i) f(i, order_of(w[i]));
    }
};

template <int THREADS, int HELD>
__global__ __launch_bounds__(THREADS) void kv8_select_kernel(EvictArgs a) {
    constexpr int WAVES = THREADS / 64, OWN = kBins / THREADS;
    __shared__ uint32_t bins[kBins], wave_sum[WAVES], wave_more[WAVES], wave_equal[WAVES];
    __shared__ uint32_t found_bin, found_above;
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const uint32_t bh = blockIdx.x, h = bh % a.c.heads, b = bh / a.c.heads;
    const uint32_t n = (uint32_t)clamp_length(a.c.lengths[b], a.c.width * kPage);
    const uint32_t recent = min(a.recent, a.keep);
    const float* w = a.weights + (size_t)bh * a.c.width * kPage;
    int32_t* kept = a.kept + (size_t)bh * a.keep;
    float* moved = a.moved + (size_t)bh * a.keep;
    if (h == 0 && tid == 0) a.into.lengths[b] = (int32_t)min(n, a.keep);
    if (n <= a.keep) {
        for (uint32_t i = tid; i < a.keep; i += THREADS) {
            kept[i] = i < n ? (int32_t)i : -1;
            moved[i] = i < n ? w[i] : 0.0f;
        }
        return;
    }
    const uint32_t free = n - recent, need = a.keep - recent;      // `need` of the first `free` tokens stay
    const Tokens<THREADS, HELD> tokens(w, free, (free + 4 * THREADS - 1) / (4 * THREADS) * 4);
    for (uint32_t i = tid; i < recent; i += THREADS) {
        kept[need + i] = (int32_t)(free + i);
        moved[need + i] = w[free + i];
    }
    if (need == 0) return;

    uint32_t prefix = 0, mask = 0, left = need;        // the threshold's bits so far, and which they are
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t top = pass == 2 ? 1023 : 2047;
        for (uint32_t i = tid; i < kBins; i += THREADS) bins[i] = 0;
        __syncthreads();
        tokens.each([&](uint32_t, uint32_t o) {
            if (o != 0 && (o & mask) == prefix) atomicAdd(&bins[(o >> shift) & top], 1u);
        });
        __syncthreads();
        // tokens in this thread's bins and in all above them
        uint32_t bin[OWN], suffix = 0;
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            bin[i] = bins[OWN * tid + i];
            suffix += bin[i];
        }
        uint32_t above = suffix;
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t other = __shfl_down(suffix, d);
            if (lane + d < 64) suffix += other;
        }
        if (lane == 0) wave_sum[wave] = suffix;
        __syncthreads();
        above = suffix - above;
#pragma unroll
        for (uint32_t v = 1; v < WAVES; ++v) above += v > wave ? wave_sum[v] : 0;
#pragma unroll
        for (int i = OWN - 1; i >= 0; --i) {
            if (above < left && above + bin[i] >= left) {
                found_bin = OWN * tid + i;
                found_above = above;
            }
            above += bin[i];
        }
        __syncthreads();
        prefix |= found_bin << shift;
        mask |= top << shift;
        left -= found_above;
    }

    // all above the threshold stay, and the first `left` equal to it
    uint32_t more = 0, equal = 0;
    tokens.each([&](uint32_t, uint32_t o) {
        more += o > prefix;
        equal += o == prefix;
    });
    // what the threads before this one have
    uint32_t more_before = more, equal_before = equal;
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t m = __shfl_up(more_before, d), e = __shfl_up(equal_before, d);
        if (lane >= (uint32_t)d) more_before += m, equal_before += e;
    }
    if (lane == 63) wave_more[wave] = more_before, wave_equal[wave] = equal_before;
    __syncthreads();
    more_before -= more;
    equal_before -= equal;
#pragma unroll
    for (uint32_t v = 0; v + 1 < WAVES; ++v) {
        more_before += v < wave ? wave_more[v] : 0;
        equal_before += v < wave ? wave_equal[v] : 0;
    }
    tokens.each([&](uint32_t i, uint32_t o) {
        const bool is_more = o > prefix, is_equal = o == prefix;
        if (is_more || (is_equal && equal_before < left)) {
            const uint32_t at = more_before + min(equal_before, left);
            kept[at] = (int32_t)i;
            // reading w[i] again cost 2 of 22 us for 128 heads of 16,384 tokens
            moved[at] = weight_of(o);
        }
        more_before += is_more;
        equal_before += is_equal;
    });
}

// Then the move: a workgroup gathers one page of one head, keys and values,
// keeps their codes in registers between the maxima and the new codes, and
// writes the page.  Values are gathered byte by byte, a lane for each token:
// neighbouring kept tokens mostly share the lines of a source page.  Keys and
// values go together because a workgroup's time is the chain of loads before
// them (length, position, page, scale): apart they took 113 us for 128 heads
// of 4,096 kept tokens.
template <int DIM>
__global__ __launch_bounds__(kThreads) void kv8_move_kernel(EvictArgs a, uint32_t out_pages) {
    constexpr int Q = DIM / 4, U = kPage * Q / kThreads;
    __shared__ float shared[2][kThreads / 64];
    __shared__ uint32_t tile[kPage][Q + 1];
    __shared__ int64_t source[kPage];                  // each token's page and head, -1: none
    __shared__ int32_t token[kPage];
    __shared__ float source_k_scale[kPage], source_v_scale[kPage];
    // a source page feeds neighbouring pages: these run on one XCD, whose L2 then has it
    const uint32_t unit = xcd_tile(blockIdx.x, gridDim.x), page = unit % out_pages, bh = unit / out_pages;
    const uint32_t h = bh % a.c.heads, b = bh / a.c.heads, tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
    const uint32_t n = (uint32_t)min(clamp_length(a.c.lengths[b], a.c.width * kPage), (int32_t)a.keep);
    if (page * kPage >= n) return;
    const int32_t id = valid_page(a.into.table[(size_t)b * a.into.width + page], a.into.pages);
    if (id < 0) return;
    if (tid < kPage) {
        const uint32_t j = page * kPage + tid;
        int64_t at = -1;
        int32_t t = 0;
        if (j < n) {
            t = a.kept[(size_t)bh * a.keep + j];
            const int32_t from = valid_page(a.c.table[(size_t)b * a.c.width + t / kPage], a.c.pages);
            if (from >= 0) at = (int64_t)from * a.c.heads + h;
        }
        source[tid] = at;
        token[tid] = t % kPage;
        source_k_scale[tid] = at < 0 ? 0.0f : a.c.k_scales[at];
        source_v_scale[tid] = at < 0 ? 0.0f : a.c.v_scales[at];
    }
    __syncthreads();
    const size_t to = (size_t)id * a.into.heads + h;
    uint32_t kw[U], vw[U];
    // values: a lane has a token; four channels make a word
    const int64_t v_at = source[lane];
    const int8_t* v = a.c.v + (v_at < 0 ? 0 : v_at) * (kPage * DIM) + token[lane];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int q = u * (kThreads / 64) + wave;
        uint32_t x = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) x |= (uint32_t)(uint8_t)v[(q * 4 + k) * kPage] << (8 * k);
        vw[u] = v_at < 0 ? 0 : x;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = u * kThreads + tid, t = i / Q, q = i % Q;
        const int64_t at = source[t];
        const uint32_t x = *reinterpret_cast<const uint32_t*>(a.c.k + ((at < 0 ? 0 : at) * kPage + token[t]) * DIM + q * 4);
        kw[u] = at < 0 ? 0 : x;
    }
    float mk = 0.0f, mv = 0.0f;
    const float v_scale = source_v_scale[lane];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        mk = absmax4(values4(kw[u], source_k_scale[(u * kThreads + tid) / Q]), mk);
        mv = absmax4(values4(vw[u], v_scale), mv);
    }
    const float k_new = group_max(mk, shared[0]) / 127.0f, v_new = group_max(mv, shared[1]) / 127.0f;
    if (tid == 0) a.into.k_scales[to] = k_new, a.into.v_scales[to] = v_new;
    with_codes(v_new, [&](auto codes4) {
#pragma unroll
        for (int u = 0; u < U; ++u) tile[lane][u * (kThreads / 64) + wave] = codes4(values4(vw[u], v_scale));
    });
    uint32_t* k_codes = reinterpret_cast<uint32_t*>(a.into.k + to * (kPage * DIM));
    with_codes(k_new, [&](auto codes4) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = u * kThreads + tid;
            k_codes[i] = codes4(values4(kw[u], source_k_scale[i / Q]));
        }
    });
    __syncthreads();
    uint32_t* v_codes = reinterpret_cast<uint32_t*>(a.into.v + to * (kPage * DIM));
#pragma unroll
    for (int u = 0; u < U / 4; ++u) {
        const int i = u * kThreads + tid, q = i / (kPage / 4), t = i % (kPage / 4);
        uint32_t x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = tile[t * 4 + k][q];
        transpose4(x);
#pragma unroll
        for (int k = 0; k < 4; ++k) v_codes[(q * 4 + k) * (kPage / 4) + t] = x[k];
    }
}

// ---------------------------------------------------------------------------
// launches

template <int D>
using Dim = std::integral_constant<int, D>;

template <class F>
hipError_t with_dim(int dim, F f) {
    return dim == 64 ? f(Dim<64>{}) : dim == 128 ? f(Dim<128>{}) : f(Dim<256>{});
}

template <class F>
hipError_t with_kind(int kind, F f) {
    return kind == kInBF16 ? f(std::integral_constant<int, kInBF16>{}) : f(std::integral_constant<int, kInF32>{});
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// How an attention call is cut.  The cache's lengths are on the device, so cuts
// follow the page table's width; workgroups behind a sequence's end leave at
// once.  Few rows: a workgroup's four waves take a page each in turn; about
// two workgroups to a CU, unless that leaves a wave fewer than four pages
// (2,048 workgroups against 512: 64 sequences of 8,000 tokens with weights
// 109.6 against 104.3 us, 64 x 12 heads of 2,000 tokens 32.1 against 27.9, 4 x
// 16 heads of 20,000 tokens 50.1 against 50.9), and at least one to a CU while
// a wave has one page.  Many rows: cut only where the tiles leave CUs idle, to
// about one workgroup a CU with 256 channels, of which no two fit one (two:
// 1,000 queries x 16 heads 82 against 52 us), else two; a cut has eight pages or
// more where half the CUs have a tile without (four: 654 queries x 32 heads x 128
// channels 31.9 against 29.6).
// Two tiles of 16 rows at 256 channels would not fit a wave's registers.
constexpr uint32_t few_rows_of(int dim) { return dim == 256 ? 16 : 32; }

struct Plan {
    bool few;
    uint32_t tiles, splits, pages_per_split;
};

Plan plan_for(uint32_t batch, uint32_t kv_heads, uint32_t rows, int dim, uint32_t width) {
    Plan p = {};
    p.few = rows <= few_rows_of(dim);
    p.tiles = p.few ? 1 : (rows + kTileRows - 1) / kTileRows;
    const size_t units = (size_t)batch * kv_heads * p.tiles;
    auto cut = [&](size_t target, uint32_t least) {
        const size_t want = (target + units - 1) / units, most = (width + least - 1) / least;
        return (uint32_t)(want < most ? want : most);
    };
    uint32_t splits;
    if (p.few) {
        splits = cut(512, 16);
        if (units * splits < 256) splits = cut(256, 4);
    } else {
        splits = units >= 256 ? 1 : cut(dim == 256 ? 256 : 512, units >= 128 ? 8 : 4);
    }
    if (splits < 1) splits = 1;
    p.pages_per_split = (width + splits - 1) / splits;
    if (p.pages_per_split < 1) p.pages_per_split = 1;
    p.splits = (width + p.pages_per_split - 1) / p.pages_per_split;
    if (p.splits < 1) p.splits = 1;
    return p;
}

} // namespace

hipError_t launch_kv8_append(const Kv8& c, const int32_t* starts, const void* k_new, const void* v_new, int kind,
                             uint32_t tokens, hipStream_t st) {
    AppendArgs a = {c, starts, k_new, v_new, tokens, (tokens + kPage - 2) / kPage + 1};
    const uint32_t groups = c.batch * a.touched * c.heads * 2;
    return with_dim(c.dim, [&](auto D) {
        return with_kind(kind, [&](auto K) { return launch_threads(kv8_append_kernel<D(), K()>, groups, kThreads, st, a); });
    });
}

hipError_t launch_kv8_read(const Kv8& c, const int32_t* starts, uint32_t tokens, void* k_out, void* v_out, int kind,
                           hipStream_t st) {
    ReadArgs a = {c, starts, k_out, v_out, tokens, (tokens + kPage - 2) / kPage + 1};
    const uint32_t groups = c.batch * a.touched * c.heads * 2;
    return with_dim(c.dim, [&](auto D) {
        return with_kind(kind, [&](auto K) { return launch_threads(kv8_read_kernel<D(), K()>, groups, kThreads, st, a); });
    });
}

namespace {

// Where a call's scratch lies in its workspace.
struct Layout {
    size_t lse, stats, part, fragments, rows, sums, end;
    uint32_t row_tiles, shares, key_groups;
};

// Rows whose queries one tile of the few-row weights kernel holds.
constexpr uint32_t kOneTile = 16;

Layout layout_for(const Plan& p, uint32_t batch, uint32_t kv_heads, uint32_t rows, int dim, uint32_t width, int terms,
                  bool weights) {
    Layout l = {};
    const size_t heads = (size_t)batch * kv_heads, items = heads * rows;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    if (weights) l.lse = take(items * 4);
    if (p.splits > 1) {
        l.stats = take(items * p.splits * 8);
        l.part = take(items * p.splits * dim * 4);
    }
    if (weights && rows > kOneTile) {
        l.row_tiles = (rows + 31) / 32;
        l.key_groups = (width * kPage + kShareKeys - 1) / kShareKeys;
        // enough workgroups for the chip, at least four row tiles to each
        const size_t units = heads * l.key_groups, want = (1536 + units - 1) / units, most = (l.row_tiles + 3) / 4;
        l.shares = (uint32_t)(want < most ? want : most);
        l.fragments = take(heads * l.row_tiles * 32 * dim * 2 * terms);
        l.rows = take(heads * l.row_tiles * 32 * sizeof(Row));
        if (l.shares > 1) l.sums = take(l.shares * heads * width * kPage * 4);
    }
    l.end = at;
    return l;
}

} // namespace

size_t kv8_attention_workspace(uint32_t batch, uint32_t kv_heads, uint32_t rows, int dim, uint32_t width, int kind,
                               bool weights) {
    const Plan p = plan_for(batch, kv_heads, rows, dim, width);
    return layout_for(p, batch, kv_heads, rows, dim, width, kind == kInBF16 ? 1 : 2, weights).end;
}

hipError_t launch_kv8_attention(const Kv8& c, const void* q, int kind, uint32_t queries, uint32_t heads,
                                const int32_t* q_lens, float scale, float* weights, void* out, void* workspace,
                                hipStream_t st) {
    AttendArgs a = {};
    a.c = c, a.q = q, a.q_lens = q_lens, a.out = out, a.weights = weights;
    a.queries = queries, a.heads = heads, a.group = heads / c.heads, a.rows = queries * a.group;
    a.scale = (scale < 0 ? -scale : scale) * 1.44269504088896340736f;
    a.negative = scale < 0;
    const Plan p = plan_for(c.batch, c.heads, a.rows, c.dim, c.width);
    const Layout l = layout_for(p, c.batch, c.heads, a.rows, c.dim, c.width, kind == kInBF16 ? 1 : 2, weights != nullptr);
    a.tiles = p.tiles, a.splits = p.splits, a.pages_per_split = p.pages_per_split;
    const size_t items = (size_t)c.batch * c.heads * a.rows;
    uint8_t* scratch = (uint8_t*)workspace;
    if (weights) a.lse = (float*)(scratch + l.lse);
    if (a.splits > 1) {
        a.stats = (float*)(scratch + l.stats);
        a.part = (float*)(scratch + l.part);
    }
    return with_dim(c.dim, [&](auto D) {
        return with_kind(kind, [&](auto K) {
            const uint32_t groups = c.batch * c.heads * a.tiles * a.splits;
            hipError_t e;
            if (!p.few)
                e = launch_threads(kv8_attend_many_kernel<D(), K()>, groups, kThreads, st, a);
            else if (few_rows_of(D()) == 16 || a.rows <= 16)
                e = launch_threads(kv8_attend_few_kernel<D(), 1, K(), 4>, groups, kThreads, st, a);
            else
                e = launch_threads(kv8_attend_few_kernel<D(), few_rows_of(D()) / 16, K(), 4>, groups, kThreads, st, a);
            if (e == hipSuccess && a.splits > 1)
                e = a.splits > 4
                        ? launch_threads(kv8_join_kernel<D(), K(), kJoinRows>, (uint32_t)items, kJoinRows * D() / 4, st, a)
                        : launch_threads(kv8_join_kernel<D(), K(), 1>, (uint32_t)((items + kJoinRows - 1) / kJoinRows),
                                         kJoinRows * D() / 4, st, a);
            if (e != hipSuccess || !weights) return e;
            if (a.rows <= kOneTile) {
                // about eight pages to a wave
                a.splits = (c.width + 31) / 32;
                return launch_threads(kv8_weights_kernel<D(), K()>, c.batch * c.heads * a.splits, kThreads, st, a);
            }
            ShareArgs s = {a, (kv_half8*)(scratch + l.fragments), (Row*)(scratch + l.rows), (float*)(scratch + l.sums),
                           l.row_tiles, l.shares, l.key_groups};
            const size_t heads_all = (size_t)c.batch * c.heads;
            constexpr int waves = kShareThreads / 64;
            e = launch_threads(kv8_fragments_kernel<D(), K()>, (uint32_t)((heads_all * l.row_tiles + waves - 1) / waves),
                               kShareThreads, st, s);
            if (e == hipSuccess)
                e = launch_threads(kv8_shares_kernel<D(), K()>, (uint32_t)(heads_all * l.key_groups * l.shares),
                                   kShareThreads, st, s);
            if (e == hipSuccess && l.shares > 1)
                e = launch_threads(kv8_add_shares_kernel,
                                   (uint32_t)((heads_all * c.width * kPage + kShareThreads - 1) / kShareThreads),
                                   kShareThreads, st, s);
            return e;
        });
    });
}

hipError_t launch_kv8_evict(const Kv8& c, const Kv8& into, const float* weights, uint32_t recent, uint32_t keep,
                            int32_t* kept, float* moved, hipStream_t st) {
    EvictArgs a = {c, into, weights, recent, keep, kept, moved};
    // The table's width bounds the tokens: their order stays in registers up to
    // 24,576.  Four waves meet at a barrier sooner than sixteen: eviction of 4 x 8
    // heads of 1,100 tokens, with the read, 20.6 against 22.9 us; at 3,900 tokens,
    // where they would read half of the tokens again in every pass, 43.5 against 38.
    const uint32_t tokens = c.width * kPage, groups = c.batch * c.heads;
    const hipError_t e = tokens <= 256 * 8    ? launch_threads(kv8_select_kernel<256, 8>, groups, 256, st, a)
                         : tokens <= 1024 * 8 ? launch_threads(kv8_select_kernel<1024, 8>, groups, 1024, st, a)
                                              : launch_threads(kv8_select_kernel<1024, 24>, groups, 1024, st, a);
    if (e != hipSuccess) return e;
    const uint32_t out_pages = (keep + kPage - 1) / kPage;
    return with_dim(c.dim, [&](auto D) {
        return launch_threads(kv8_move_kernel<D()>, c.batch * c.heads * out_pages, kThreads, st, a, out_pages);
    });
}

} // namespace qar
