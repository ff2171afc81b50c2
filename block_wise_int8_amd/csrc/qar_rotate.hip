// qar_rotate.hip -- queries, keys and values out of a joint projection on
// gfx950: every head of the queries and keys is normed by its root mean square
// and its channels are rotated by their position, the values are set apart, in
// one pass over the tensor.
//
//   y = x / sqrt(mean(x^2) + eps) * gain
//   (a, b) = (a cos t - b sin t, b cos t + a sin t),   t = position * frequency
//
// for every pair (a, b) of the rotated channels.  Bound by memory: each
// element is read once and written once, and the arithmetic between, some
// twenty instructions for a pair, fits under that.  What is not obvious is
// where the pairs lie.  A lane owns two runs of eight channels (16 bytes of
// bf16) of a head, chosen so that a pair is never split between lanes: with
// pairs that lie half the rotated channels apart, run l and the run of its
// partners; with neighbouring pairs, runs 2 l and 2 l + 1.  A head is then 4, 8
// or 16 lanes, whose sum of squares is a few DPP moves, and a lane's sines and
// cosines are the same for every head of a token: a workgroup computes a
// token's once, and its lanes keep theirs in registers over the heads.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qar_device.h"
#include "qar_launch.h"
#include "qar_serve.h"

namespace qar {
namespace {

enum : int { kHalves = 0, kNeighbours = 1, kSplitHalves = 2 };

// Eight elements as binary32.
template <int IN>
__device__ __forceinline__ void load_run(const void* x, size_t e, float (&y)[8]) {
    if constexpr (IN == kInBF16) {
        const uint4 q = load_b128((const uint16_t*)x + e);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) y[2 * i] = bf16_lo(w[i]), y[2 * i + 1] = bf16_hi(w[i]);
    } else {
        const uint4 a = load_b128((const float*)x + e), b = load_b128((const float*)x + e + 4);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __builtin_bit_cast(float, w[i]);
    }
}

template <int OUT>
__device__ __forceinline__ void store_run(void* x, size_t e, const float (&y)[8]) {
    if constexpr (OUT == kInBF16) {
        store_b128((uint16_t*)x + e, make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                                pack_bf16x2(y[6], y[7])));
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            store_b128((float*)x + e + i,
                       make_uint4(__builtin_bit_cast(uint32_t, y[i]), __builtin_bit_cast(uint32_t, y[i + 1]),
                                  __builtin_bit_cast(uint32_t, y[i + 2]), __builtin_bit_cast(uint32_t, y[i + 3])));
    }
}

// The sum over a head's lanes.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    v += dpp_move<kDppSwapAdjacent>(v);
    v += dpp_move<kDppSwapPairs>(v);
    if constexpr (L >= 8) v += dpp_move<kDppRowHalfMirror>(v);
    if constexpr (L >= 16) v += dpp_move<kDppRowMirror>(v);
    return v;
}

// Sine and cosine of position * frequency.  The angle is reduced in 64 bits to
// an eighth of a turn on either side of a quarter: in 32 bits position 10^6
// would be off by 2^-4 of a radian.  What is left enters binary32 with an error
// of 2^-25 of a radian.
__device__ __forceinline__ float2 cos_sin(int32_t position, float frequency) {
    const double turns = (double)position * ((double)frequency * 0.15915494309189533577);
    const double part = turns - __builtin_rint(turns);              // -1/2 .. 1/2
    const double quarter = __builtin_rint(part * 4.0);
    float s, c;
    sincospif((float)((part - quarter * 0.25) * 2.0), &s, &c);
    const int k = (int)quarter & 3;
    const float a = k & 1 ? s : c, b = k & 1 ? c : s;               // cos, sin up to their signs
    return make_float2(k == 1 || k == 2 ? -a : a, k >= 2 ? -b : b);
}

// PAIRS: kSplitHalves is kHalves where the pairs are no multiple of eight and
// partners meet in LDS.
template <int DIM, int IN, int PAIRS>
__global__ __launch_bounds__(kThreads) void norm_rotate_kernel(RotateCall a) {
    constexpr int L = DIM / 16, H = kThreads / L;                   // lanes of a head, heads at a time
    __shared__ float2 table[DIM / 2];
    __shared__ float rows[PAIRS == kSplitHalves ? H : 1][PAIRS == kSplitHalves ? DIM + 4 : 1];
    const uint32_t tid = threadIdx.x, l = tid % L, mine = tid / L;
    const size_t token = blockIdx.x / a.parts;
    const uint32_t part = blockIdx.x % a.parts, all = a.heads + 2 * a.kv_heads, rotated = a.heads + a.kv_heads;
    const uint32_t per = (all + a.parts - 1) / a.parts, first = part * per, last = min(first + per, all);

    // the lane's runs of eight channels
    uint32_t run[2];
    if (PAIRS == kHalves && l < a.pairs / 8)
        run[0] = l, run[1] = l + a.pairs / 8;
    else
        run[0] = 2 * l, run[1] = 2 * l + 1;

    float x[2][8] = {};
    uint32_t h = first + mine;
    auto load = [&](uint32_t head) {
#pragma unroll
        for (int i = 0; i < 2; ++i) load_run<IN>(a.x, (token * all + head) * DIM + run[i] * 8, x[i]);
    };
    if (h < last) load(h);

    if (first < rotated && tid < a.pairs) {
        const size_t b = token / a.tokens;
        const int32_t position = a.each_token ? a.positions[token] : (int32_t)((uint32_t)a.positions[b] + (uint32_t)(token - b * a.tokens));
        table[tid] = cos_sin(position, a.frequencies[tid]);
    }
    __syncthreads();
    // of the lane's pairs: eight with halves, four of each run with neighbours
    float2 turn[8];
    if constexpr (PAIRS != kSplitHalves) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t pair = l * 8 + i;
            turn[i] = pair < a.pairs ? table[pair] : make_float2(1.0f, 0.0f);
        }
    }

    for (uint32_t base = first; base < last; base += H) {
        float y[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) y[i][k] = x[i][k];
        const uint32_t head = base + mine;
        if (head + H < last) load(head + H);
        const bool turned = head < rotated, there = head < last;
        if (a.norm) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) sum = __builtin_fmaf(y[i][k], y[i][k], sum);
            sum = lanes_sum<L>(sum);
            if (turned) {
                const float r = 1.0f / sqrtf(sum * (1.0f / DIM) + a.eps);
                const void* gain = head < a.heads ? a.q_gain : a.k_gain;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float g[8];
                    if (gain) load_run<IN>(gain, run[i] * 8, g);
#pragma unroll
                    for (int k = 0; k < 8; ++k) y[i][k] = gain ? y[i][k] * r * g[k] : y[i][k] * r;
                }
            }
        }
        if constexpr (PAIRS == kHalves) {
            if (turned && l < a.pairs / 8) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float u = y[0][k], v = y[1][k];
                    y[0][k] = u * turn[k].x - v * turn[k].y;
                    y[1][k] = v * turn[k].x + u * turn[k].y;
                }
            }
        } else if constexpr (PAIRS == kNeighbours) {
            if (turned) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        const float2 t = turn[i * 4 + k / 2];
                        const float u = y[i][k], v = y[i][k + 1];
                        y[i][k] = u * t.x - v * t.y;
                        y[i][k + 1] = v * t.x + u * t.y;
                    }
            }
        } else {
            // a head's lanes are of one wave, which writes and reads in order
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) rows[mine][run[i] * 8 + k] = y[i][k];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t c = run[i] * 8 + k;
                    if (turned && c < 2 * a.pairs) {
                        const bool upper = c >= a.pairs;
                        const float2 t = table[upper ? c - a.pairs : c];
                        const float partner = rows[mine][upper ? c - a.pairs : c + a.pairs];
                        y[i][k] = y[i][k] * t.x + (upper ? partner : -partner) * t.y;
                    }
                }
            __builtin_amdgcn_wave_barrier();
        }
        if (!there) continue;
        void* out = head < a.heads ? a.q : turned ? a.k : a.v;
        const uint32_t of = head < a.heads ? a.heads : a.kv_heads, index = head < a.heads ? head : (head - a.heads) % a.kv_heads;
#pragma unroll
        for (int i = 0; i < 2; ++i) store_run<IN>(out, (token * of + index) * DIM + run[i] * 8, y[i]);
    }
}

template <int DIM, int IN>
hipError_t launch(const RotateCall& a, uint32_t groups, hipStream_t st) {
    if (a.interleaved) return launch_threads(norm_rotate_kernel<DIM, IN, kNeighbours>, groups, kThreads, st, a);
    if (a.pairs % 8 == 0) return launch_threads(norm_rotate_kernel<DIM, IN, kHalves>, groups, kThreads, st, a);
    return launch_threads(norm_rotate_kernel<DIM, IN, kSplitHalves>, groups, kThreads, st, a);
}

} // namespace

hipError_t launch_norm_rotate(RotateCall a, int kind, int dim, hipStream_t st) {
    // few tokens: a token's heads spread over workgroups, each at least one pass
    const uint32_t at_once = kThreads / (dim / 16), all = a.heads + 2 * a.kv_heads, most = (all + at_once - 1) / at_once;
    a.parts = a.rows >= 1024 ? 1 : (uint32_t)std::min<size_t>(most, (1024 + a.rows - 1) / a.rows);
    const uint32_t groups = (uint32_t)a.rows * a.parts;
    const auto go = [&](auto IN) {
        constexpr int K = decltype(IN)::value;
        return dim == 64 ? launch<64, K>(a, groups, st) : dim == 128 ? launch<128, K>(a, groups, st) : launch<256, K>(a, groups, st);
    };
    return kind == kInBF16 ? go(std::integral_constant<int, kInBF16>{}) : go(std::integral_constant<int, kInF32>{});
}

} // namespace qar
