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
// where the pairs lie.  A lane owns pieces of 16 bytes of a head, two or (for
// binary32) four, chosen so that a pair is never split between lanes and that
// neighbouring lanes read neighbouring pieces: with pairs that lie half the
// rotated channels apart, pieces and the pieces of their partners.  A head is
// then 4, 8 or 16 lanes, whose sum of squares is a few DPP moves, and a lane's
// sines and cosines are the same for every head of a token: a workgroup
// computes a token's once, and its lanes keep theirs in registers over the heads.
// Measured: 8,191 tokens of 32 and 16 heads x 128 in bf16 53 us, 2,331 of 16 and
// 8 x 256 in binary32 with 64 channels rotated 32 us (5.1 and 4.7 TB/s of the
// 5.1 that a copy reaches), 32 tokens 3.9 us, which is the chain position ->
// sine -> store; 16-byte pieces in place of 4-byte ones took the second from 64.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qar_device.h"
#include "qar_launch.h"
#include "qar_serve.h"

namespace qar {
namespace {

enum : int { kHalves = 0, kNeighbours = 1, kSplitHalves = 2 };

// The elements of 16 bytes.
template <int IN>
constexpr int kPiece = IN == kInBF16 ? 8 : 4;

template <int IN>
__device__ __forceinline__ void load_piece(const void* x, size_t e, float (&y)[kPiece<IN>]) {
    const uint4 q = load_b128((const char*)x + e * (16 / kPiece<IN>));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (IN == kInBF16)
            y[2 * i] = bf16_lo(w[i]), y[2 * i + 1] = bf16_hi(w[i]);
        else
            y[i] = __builtin_bit_cast(float, w[i]);
    }
}

template <int OUT>
__device__ __forceinline__ void store_piece(void* x, size_t e, const float (&y)[kPiece<OUT>]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (OUT == kInBF16)
            w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
        else
            w[i] = __builtin_bit_cast(uint32_t, y[i]);
    }
    store_b128((char*)x + e * (16 / kPiece<OUT>), make_uint4(w[0], w[1], w[2], w[3]));
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

// PAIRS: kSplitHalves is kHalves where the pairs are no multiple of a piece, and
// partners meet in LDS.
template <int DIM, int IN, int PAIRS>
__global__ __launch_bounds__(kThreads) void norm_rotate_kernel(RotateCall a) {
    constexpr int L = DIM / 16, H = kThreads / L;                   // lanes of a head, heads at a time
    constexpr int E = kPiece<IN>, U = 8 / E, HALF = DIM / 2 / E;    // a lane's units of two pieces; half a head's pieces
    __shared__ float2 table[DIM / 2];
    __shared__ float rows[PAIRS == kSplitHalves ? H : 1][PAIRS == kSplitHalves ? DIM + 4 : 1];
    const uint32_t tid = threadIdx.x, l = tid % L, mine = tid / L;
    const size_t token = a.first + blockIdx.x / a.parts;
    const uint32_t part = blockIdx.x % a.parts, all = a.heads + 2 * a.kv_heads, rotated = a.heads + a.kv_heads;
    const uint32_t per = (all + a.parts - 1) / a.parts, first = part * per, last = min(first + per, all);

    // Unit u of a head is a piece of first partners and that of their second
    // ones, u and u + pairs / E; behind these, two pieces that are not rotated
    // (with neighbours all units are of that kind, and turn within themselves).
    const uint32_t paired = PAIRS == kHalves ? a.pairs / E : 0;
    uint32_t unit[U], at[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        unit[i] = i * L + l;
        at[i][0] = (unit[i] < paired ? unit[i] : unit[i] + paired) * E;
        at[i][1] = (unit[i] < paired ? unit[i] + paired : unit[i] + HALF) * E;
    }

    float x[U][2][E] = {};
    auto load = [&](uint32_t head) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) load_piece<IN>(a.x, (token * all + head) * DIM + at[i][j], x[i][j]);
    };
    if (first + mine < last) load(first + mine);

    if (first < rotated && tid < a.pairs) {
        const size_t b = token / a.tokens;
        const int32_t position = a.each_token ? a.positions[token] : (int32_t)((uint32_t)a.positions[b] + (uint32_t)(token - b * a.tokens));
        table[tid] = cos_sin(position, a.frequencies[tid]);
    }
    __syncthreads();
    // the lane's pairs: E of a unit with halves, E / 2 of each piece with neighbours
    float2 turn[U][E];
    if constexpr (PAIRS != kSplitHalves) {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const uint32_t pair = PAIRS == kHalves ? unit[i] * E + k : (at[i][k / (E / 2)] + k % (E / 2) * 2) / 2;
                turn[i][k] = table[std::min(pair, (uint32_t)DIM / 2 - 1)];    // behind the pairs unused
            }
    }

    for (uint32_t base = first; base < last; base += H) {
        float y[U][2][E];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int k = 0; k < E; ++k) y[i][j][k] = x[i][j][k];
        const uint32_t head = base + mine;
        if (head + H < last) load(head + H);
        const bool turned = head < rotated, there = head < last;
        if (a.norm) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < E; ++k) sum = __builtin_fmaf(y[i][j][k], y[i][j][k], sum);
            sum = lanes_sum<L>(sum);
            if (turned) {
                const float r = 1.0f / sqrtf(sum * (1.0f / DIM) + a.eps);
                const void* gain = head < a.heads ? a.q_gain : a.k_gain;
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float g[E];
                        if (gain) load_piece<IN>(gain, at[i][j], g);
#pragma unroll
                        for (int k = 0; k < E; ++k) y[i][j][k] = gain ? y[i][j][k] * r * g[k] : y[i][j][k] * r;
                    }
            }
        }
        if constexpr (PAIRS == kHalves) {
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (turned && unit[i] < paired) {
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const float u = y[i][0][k], v = y[i][1][k];
                        y[i][0][k] = u * turn[i][k].x - v * turn[i][k].y;
                        y[i][1][k] = v * turn[i][k].x + u * turn[i][k].y;
                    }
                }
        } else if constexpr (PAIRS == kNeighbours) {
            if (turned) {
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const float2 t = turn[i][k];
                        float* z = y[i][k / (E / 2)] + k % (E / 2) * 2;
                        const float u = z[0], v = z[1];
                        // behind the pairs neither is touched, were the other infinite
                        const bool pair = (at[i][k / (E / 2)] + k % (E / 2) * 2) / 2 < a.pairs;
                        z[0] = pair ? u * t.x - v * t.y : u;
                        z[1] = pair ? v * t.x + u * t.y : v;
                    }
            }
        } else {
            // a head's lanes are of one wave, which writes and reads in order
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < E; ++k) rows[mine][at[i][j] + k] = y[i][j][k];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const uint32_t c = at[i][j] + k;
                        if (turned && c < 2 * a.pairs) {
                            const bool upper = c >= a.pairs;
                            const float2 t = table[upper ? c - a.pairs : c];
                            const float partner = rows[mine][upper ? c - a.pairs : c + a.pairs];
                            y[i][j][k] = y[i][j][k] * t.x + (upper ? partner : -partner) * t.y;
                        }
                    }
            __builtin_amdgcn_wave_barrier();
        }
        if (!there) continue;
        void* out = head < a.heads ? a.q : turned ? a.k : a.v;
        const uint32_t of = head < a.heads ? a.heads : a.kv_heads, index = head < a.heads ? head : (head - a.heads) % a.kv_heads;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) store_piece<IN>(out, (token * of + index) * DIM + at[i][j], y[i][j]);
    }
}

template <int DIM, int IN>
hipError_t launch(const RotateCall& a, uint32_t groups, hipStream_t st) {
    if (a.interleaved) return launch_threads(norm_rotate_kernel<DIM, IN, kNeighbours>, groups, kThreads, st, a);
    if (a.pairs % kPiece<IN> == 0) return launch_threads(norm_rotate_kernel<DIM, IN, kHalves>, groups, kThreads, st, a);
    return launch_threads(norm_rotate_kernel<DIM, IN, kSplitHalves>, groups, kThreads, st, a);
}

} // namespace

hipError_t launch_norm_rotate(RotateCall a, int kind, int dim, hipStream_t st) {
    // few tokens: a token's heads spread over workgroups, each at least one pass
    const uint32_t at_once = kThreads / (dim / 16), all = a.heads + 2 * a.kv_heads, most = (all + at_once - 1) / at_once;
    a.parts = a.rows >= 1024 ? 1 : (uint32_t)std::min<size_t>(most, (1024 + a.rows - 1) / a.rows);
    const auto go = [&](auto IN, uint32_t groups) {
        constexpr int K = decltype(IN)::value;
        return dim == 64 ? launch<64, K>(a, groups, st) : dim == 128 ? launch<128, K>(a, groups, st) : launch<256, K>(a, groups, st);
    };
    // a launch has less than 2^32 threads
    constexpr size_t most_rows = ((size_t)1 << 32) / kThreads - 1;
    hipError_t e = hipSuccess;
    for (a.first = 0; e == hipSuccess && a.first < a.rows; a.first += most_rows) {
        const uint32_t groups = (uint32_t)std::min(a.rows - a.first, most_rows) * a.parts;
        e = kind == kInBF16 ? go(std::integral_constant<int, kInBF16>{}, groups) : go(std::integral_constant<int, kInF32>{}, groups);
    }
    return e;
}

} // namespace qar
