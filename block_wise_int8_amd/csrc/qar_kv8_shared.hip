// qar_kv8_shared.hip -- attention over the 8-bit cache for sequences whose
// first tokens are the same pages, on gfx950.
//
// A softmax over a prefix and over a sequence's own tokens is joined from the
// two parts' maxima, sums and outputs.  So the prefix is attended to once for
// all: the queries of a group's sequences (with the heads that share a key
// head) are the rows of one product, and a page of the prefix is read, and its
// codes converted, once for all rows of a tile instead of once for each
// sequence.  The own tokens are attended to sequence by sequence.  Either is
// cut into slots of pages, whose lengths are found on the device from the
// prefix and the sequence's length, and the slots of a row are joined last.
#include <float.h>
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qar_kv8_device.h"

namespace qar {
namespace {

struct SharedArgs {
    Kv8 c;
    const void* q;
    const int32_t *starts, *prefix;     // [groups + 1], [groups]
    const int32_t* q_lens;              // may be null: every sequence has `queries`
    void* out;
    float *part, *stats;                // [row][slot][dim], [row][slot]: maximum and sum
    uint32_t queries, heads, group, rows, groups;
    uint32_t prefix_tiles, own_tiles;   // of rows: of all groups, of a sequence
    uint32_t prefix_slots, own_slots;
    float scale;                        // of the scores, times log2(e), without its sign
    bool negative;                      // its sign, which the queries take
};

// ---------------------------------------------------------------------------
// which rows and pages

// A group's sequences, and the pages that they have in common.
struct Group {
    uint32_t start, end, pages;
};

// The last group with first(start, g) <= top, where first ascends; {0, 0, 0}
// if there is none.  A wave looks at 64 groups at once, and at all that it
// may want of them, so that one load follows no other.
template <class F>
__device__ __forceinline__ Group last_group(const SharedArgs& a, uint32_t top, uint32_t& index, F first) {
    const uint32_t lane = threadIdx.x % 64;
    Group found = {0, 0, 0};
    for (uint32_t base = 0; base < a.groups; base += 64) {
        const uint32_t g = min(base + lane, a.groups - 1);
        const uint32_t start = (uint32_t)clamp_length(a.starts[g], a.c.batch), end = (uint32_t)clamp_length(a.starts[g + 1], a.c.batch);
        const uint32_t pages = (uint32_t)clamp_length(a.prefix[g], a.c.width * kPage) / kPage;
        const uint64_t mask = __ballot(base + lane < a.groups && first(start, g) <= top);
        if (!mask) break;
        const int i = 63 - __builtin_clzll(mask);
        found = Group{(uint32_t)__builtin_amdgcn_readlane((int)start, i), (uint32_t)__builtin_amdgcn_readlane((int)end, i),
                      (uint32_t)__builtin_amdgcn_readlane((int)pages, i)};
        index = base + i;
        if (~mask) break;
    }
    return found;
}

// Pages before sequence b's own.
__device__ __forceinline__ uint32_t pages_before(const SharedArgs& a, uint32_t b) {
    uint32_t index;
    const Group g = last_group(a, b, index, [](uint32_t start, uint32_t) { return start; });
    return b < g.end ? g.pages : 0;
}

// `pages` cut into at most `slots` slots.
struct Cut {
    uint32_t per, used;
    __device__ __forceinline__ Cut(uint32_t pages, uint32_t slots) {
        per = max((pages + slots - 1) / slots, 4u);          // a page for each of a workgroup's waves
        used = (pages + per - 1) / per;
    }
};

// A sequence's numbers.
struct Seq {
    int32_t n, m;
    __device__ __forceinline__ Seq(const SharedArgs& a, uint32_t b)
        : n(clamp_length(a.c.lengths[b], a.c.width * kPage)),
          m(a.q_lens ? clamp_length(a.q_lens[b], a.queries) : (int32_t)a.queries) {}
};

// The group that has tile number `tile` of all groups' tiles of rows, and its
// first tile's number; {0, 0, 0} behind the last tile.  So the workgroups
// without work are the last: spare ones between others leave CUs idle beside
// CUs with two.
__device__ __forceinline__ Group group_of_tile(const SharedArgs& a, uint32_t tile, uint32_t tile_rows, uint32_t& first_tile) {
    const uint32_t lane = threadIdx.x % 64;
    uint32_t before = 0;
    for (uint32_t base = 0; base < a.groups; base += 64) {
        const uint32_t g = min(base + lane, a.groups - 1);
        const uint32_t start = (uint32_t)clamp_length(a.starts[g], a.c.batch), end = (uint32_t)clamp_length(a.starts[g + 1], a.c.batch);
        const uint32_t pages = (uint32_t)clamp_length(a.prefix[g], a.c.width * kPage) / kPage;
        const uint32_t count = base + lane < a.groups && end > start ? ((end - start) * a.rows + tile_rows - 1) / tile_rows : 0;
        uint32_t sum = count;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const uint32_t other = __shfl_up(sum, d);
            if (lane >= (uint32_t)d) sum += other;
        }
        const uint64_t mask = __ballot(before + sum > tile);
        if (mask) {
            const int i = __builtin_ctzll(mask);
            first_tile = before + (uint32_t)__builtin_amdgcn_readlane((int)(sum - count), i);
            return Group{(uint32_t)__builtin_amdgcn_readlane((int)start, i), (uint32_t)__builtin_amdgcn_readlane((int)end, i),
                         (uint32_t)__builtin_amdgcn_readlane((int)pages, i)};
        }
        before += (uint32_t)__builtin_amdgcn_readlane((int)sum, 63);
    }
    first_tile = tile;
    return Group{0, 0, 0};
}

// What a workgroup does: a tile of rows of one key head, a slot of pages.  Row
// r is row r % a.rows of sequence first_seq + r / a.rows; that is its query
// r / a.group with head r % a.group of the key head's group.
struct Work {
    uint32_t head, slot, first_seq, first_row, row_count;
    uint32_t first, last;                // pages
    bool any;
    __device__ __forceinline__ void of_prefix(const SharedArgs& a, uint32_t unit, uint32_t tile_rows) {
        slot = unit % a.prefix_slots;
        head = unit / a.prefix_slots % a.c.heads;
        const uint32_t tile = unit / a.prefix_slots / a.c.heads;
        uint32_t first_tile;
        const Group g = group_of_tile(a, tile, tile_rows, first_tile);
        first_seq = g.start;
        row_count = (g.end - g.start) * a.rows;
        first_row = (tile - first_tile) * tile_rows;
        const Cut cut(g.pages, a.prefix_slots);
        first = slot * cut.per;
        last = min(first + cut.per, g.pages);
        any = first_row < row_count && first < last;
    }
    __device__ __forceinline__ void of_own(const SharedArgs& a, uint32_t unit, uint32_t tile_rows) {
        const uint32_t of_slot = unit % a.own_slots, rest = unit / a.own_slots;
        slot = a.prefix_slots + of_slot;
        head = rest % a.c.heads;
        first_seq = rest / a.c.heads % a.c.batch;
        first_row = (a.own_tiles - 1 - rest / a.c.heads / a.c.batch) * tile_rows;   // the longest first
        row_count = a.rows;
        const int32_t n = clamp_length(a.c.lengths[first_seq], a.c.width * kPage);
        const uint32_t before = pages_before(a, first_seq), pages = (uint32_t)(n + kPage - 1) / kPage;
        const Cut cut(pages > before ? pages - before : 0, a.own_slots);
        first = before + of_slot * cut.per;
        last = min(first + cut.per, pages);
        any = first < last;
    }
};

// The sequence whose table names the pages that `work` has of a prefix: the
// first of the group, or, where that holds fewer tokens (it ended or was cut back,
// and its entries are gone), the group's longest, which holds all that any row
// sees.  And where they end: pages behind the longest sequence hold nothing yet,
// their scales neither.  The lengths are asked for while the first one's entries
// are on their way.
struct Holder {
    uint32_t seq, last;
    __device__ __forceinline__ Holder(const SharedArgs& a, const Work& work) : seq(work.first_seq), last(work.last) {
        const int32_t top = a.c.width * kPage;
        if ((uint32_t)clamp_length(a.c.lengths[seq], top) >= last * kPage) return;
        const uint32_t count = work.row_count / a.rows;
        int32_t most = -1;
        uint32_t which = 0;
        for (uint32_t i = threadIdx.x % 64; i < count; i += 64) {
            const int32_t n = clamp_length(a.c.lengths[work.first_seq + i], top);
            if (n > most) most = n, which = i;
        }
        int32_t longest = most;
#pragma unroll
        for (int d = 32; d; d /= 2) longest = max(longest, __shfl_xor(longest, d));
        longest = __builtin_amdgcn_readfirstlane(longest);
        seq += (uint32_t)__builtin_amdgcn_readlane((int)which, __builtin_ctzll(__ballot(most == longest)));
        last = min(last, (uint32_t)(longest + kPage - 1) / kPage);
    }
};

// A row of the queries, and of the parts.
struct Row {
    bool there;
    int32_t limit;                       // it sees the keys below
    size_t query, item;
    __device__ __forceinline__ Row(const SharedArgs& a, const Work& w, uint32_t r) {
        there = r < w.row_count;
        const uint32_t safe = there ? r : 0, b = w.first_seq + safe / a.rows, mine = safe % a.rows;
        const Seq seq(a, b);
        const int32_t i = (int32_t)(mine / a.group);
        there = there && i < seq.m;
        limit = seq.n - seq.m + i + 1;
        query = ((size_t)b * a.queries + i) * a.heads + w.head * a.group + mine % a.group;
        item = ((size_t)b * a.c.heads + w.head) * a.rows + mine;
    }
};

// The smallest and the largest over each 16 lanes.
__device__ __forceinline__ int32_t lanes16_min(int32_t v) {
#pragma unroll
    for (int d = 8; d; d /= 2) v = min(v, __shfl_xor(v, d));
    return v;
}

// ---------------------------------------------------------------------------
// few rows: a wave takes a page at a time, from memory to registers (the
// layout of kv8_attend_few_kernel, qar_kv8.hip).

constexpr int kFewWaves = 4, kFewRows = 16;

template <int DIM>
constexpr int kFewLds = kFewWaves * 16 * (DIM + 4) * 4 + 2 * kFewWaves * 16 * 4 + 16 * 8;

template <int DIM, int IN>
__device__ __forceinline__ void attend_few(const SharedArgs& a, const Work& work, bool own, char* lds) {
    constexpr int NW = kFewWaves;
    constexpr int T = IN == kInBF16 ? 1 : 2;
    constexpr int KC = DIM / 64, VC = DIM / 16;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64, r = lane % 16, g = lane / 16;
    const uint32_t h = work.head, first = work.first;
    uint32_t seq = work.first_seq, last = work.last;
    int32_t my_id;
    float my_ks, my_vs;
    auto look_up_id = [&](uint32_t page) {
        my_id = page < last ? valid_page(a.c.table[(size_t)seq * a.c.width + page], a.c.pages) : -1;
    };
    auto look_up_scales = [&] {
        my_ks = my_vs = 0.0f;
        if (my_id >= 0) {
            my_ks = a.c.k_scales[(size_t)my_id * a.c.heads + h];
            my_vs = a.c.v_scales[(size_t)my_id * a.c.heads + h];
        }
    };
    look_up_id(first + wave + lane * NW);
    if (!own) {
        const Holder holder(a, work);
        last = holder.last;
        if (holder.seq != seq || last != work.last) {
            seq = holder.seq;
            look_up_id(first + wave + lane * NW);
        }
    }
    look_up_scales();

    const Row row(a, work, work.first_row + r);
    Query<IN, DIM, 16, 64> raw;
    raw.load(a.q, row.there ? row.query : 0, g * 16, row.there);
    const int32_t limit = row.there ? row.limit : INT32_MAX; // rows that are not there are not stored
    const int32_t all_see = __builtin_amdgcn_readfirstlane(lanes16_min(limit));   // every row sees the keys below
    kv_half8 q[DIM / 32][T];
    float undo;

    kv_f32x4 o[VC] = {};
    Unit unit;
    float top = -FLT_MAX, total = 0.0f;

    const size_t head_bytes = (size_t)kPage * DIM;
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
        for (int c = 0; c < VC; ++c) vr[c] = *reinterpret_cast<const uint4*>(p + c * 16 * kPage);
    };

    for (uint32_t base = first + wave; base < last; base += 64 * NW) {
        if (base != first + wave) {
            look_up_id(base + lane * NW);
            look_up_scales();
        }
        const uint32_t count = min(64u, (last - base + NW - 1) / NW);
        int32_t id = __builtin_amdgcn_readlane(my_id, 0);
        load_k(id);
        load_v(id);
        if (base == first + wave) undo = raw.template convert<16, T>(a.negative, q) * a.scale;
        for (uint32_t i = 0; i < count; ++i) {
            const int32_t next = __builtin_amdgcn_readlane(my_id, min(i + 1, count - 1));
            const float ks = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_ks), i));
            const float vs = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_vs), i));
            const int32_t key0 = (int32_t)((base + i * NW) * kPage);

            kv_f32x4 s[4] = {};
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    kv_half8 k[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        k[t] = u ? half_codes(kr[t][c].z, kr[t][c].w) : half_codes(kr[t][c].x, kr[t][c].y);
#pragma unroll
                    for (int e = 0; e < T; ++e)
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k[t], q[2 * c + u][e], s[t], 0, 0, 0);
                }
            if (i + 1 < count) load_k(next);

            const float shrink_all = unit.next(vs);
            if (shrink_all != 1.0f)
#pragma unroll
                for (int c = 0; c < VC; ++c) o[c] *= shrink_all;
            kv_half8 p[2][T];
            float factor = ks * undo;
            if (key0 + kPage > all_see || id < 0) {
                const int32_t sees = (id < 0 ? 0 : limit) - key0 - (int32_t)g * 16;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[t][k] = 4 * t + k < sees ? s[t][k] * factor : -INFINITY;
                factor = 1.0f;
            }
            float m = max3(s[0][0], s[0][1], s[0][2]);
#pragma unroll
            for (int k = 3; k < 15; k += 2) m = max3(m, s[k / 4][k % 4], s[(k + 1) / 4][(k + 1) % 4]);
            m = fmaxf(max_over_16(fmaxf(m, s[3][3])) * factor, top);
            if (__any(m > top)) {
                const float shrink = __builtin_amdgcn_exp2f(top - m);
                total *= shrink;
#pragma unroll
                for (int c = 0; c < VC; ++c) o[c] *= shrink;
                top = m;
            }
            const float off = unit.lift - m;
            float sum = 0.0f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * u + k / 4][k % 4], factor, off));
                sum += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
                half_terms<T>(x, p[u]);
            }
            total = __builtin_fmaf(sum, unit.drop, total);
#pragma unroll
            for (int c = 0; c < VC; c += 2) {
                const kv_half8 v[2][2] = {{half_codes(vr[c].x, vr[c].y), half_codes(vr[c + 1].x, vr[c + 1].y)},
                                          {half_codes(vr[c].z, vr[c].w), half_codes(vr[c + 1].z, vr[c + 1].w)}};
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < T; ++e)
#pragma unroll
                        for (int d = 0; d < 2; ++d)
                            o[c + d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v[u][d], p[u][e], o[c + d], 0, 0, 0);
            }
            if (i + 1 < count) load_v(next);
            id = next;
        }
    }

    // the waves' results meet in LDS
    size_t* items = reinterpret_cast<size_t*>(lds);
    auto tops = reinterpret_cast<float (*)[16]>(lds + 16 * 8), totals = tops + NW;
    auto os = reinterpret_cast<float (*)[16][DIM + 4]>(totals + NW);
    total = sum_over_16(total);
    if (g == 0) tops[wave][r] = top, totals[wave][r] = total;
    if (threadIdx.x < 16) items[r] = row.item;
#pragma unroll
    for (int c = 0; c < VC; ++c) *reinterpret_cast<kv_f32x4*>(&os[wave][r][c * 16 + g * 4]) = o[c] * unit.unit;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < 16 * DIM; i += NW * 64) {
        const uint32_t row16 = i / DIM, d = i % DIM;
        if (work.first_row + row16 >= work.row_count) break;
        float m = tops[0][row16], l = 0.0f, y = 0.0f;
#pragma unroll
        for (int w = 1; w < NW; ++w) m = fmaxf(m, tops[w][row16]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = __builtin_amdgcn_exp2f(tops[w][row16] - m);
            l = __builtin_fmaf(totals[w][row16], f, l);
            y = __builtin_fmaf(os[w][row16][d], f, y);
        }
        const size_t at = items[row16] * (a.prefix_slots + a.own_slots) + work.slot;
        a.part[at * DIM + d] = y;
        if (d == 0) a.stats[at * 2] = m, a.stats[at * 2 + 1] = l;
    }
}

// ---------------------------------------------------------------------------
// many rows: four waves of 32 rows share a page in LDS (the layout of
// kv8_attend_many_kernel, qar_kv8.hip).

constexpr int kTileRows = 128;
constexpr int kAhead = 6;

// The order of a chain of N products of T terms and the LDS reads before them,
// which the compiler would otherwise put right before their use.
template <int N, int T>
__device__ __forceinline__ void lay_out_products() {
    constexpr int kMatrix = 0x8, kLdsRead = 0x100;
    __builtin_amdgcn_sched_group_barrier(kLdsRead, kAhead, 0);
#pragma unroll
    for (int f = 0; f < N; ++f) {
        __builtin_amdgcn_sched_group_barrier(kMatrix, T, 0);
        if (f + kAhead < N) __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// Where a tile's own pages end: as far as its last row sees.
__device__ __forceinline__ uint32_t own_pages_end(const SharedArgs& a, const Work& work) {
    const Seq seq(a, work.first_seq);
    const int32_t i = min((int32_t)(min(work.first_row + kTileRows, a.rows) - 1) / (int32_t)a.group, seq.m - 1);
    const int32_t keys = seq.n - seq.m + i + 1;
    return min(work.last, seq.m > 0 && keys > 0 ? (uint32_t)(keys + kPage - 1) / kPage : 0u);
}

template <int DIM, int IN>
constexpr bool kScoresAhead = DIM == 128 && IN == kInBF16;
template <int DIM, int IN>         // a page in binary16 and the next one's codes, or two in binary16
constexpr int kManyLds = kPage * DIM * 2 * (kScoresAhead<DIM, IN> ? 4 : 3);

template <int DIM, int IN>
__device__ __forceinline__ void attend_many(const SharedArgs& a, const Work& work, bool own, char* lds) {
    constexpr int T = IN == kInBF16 ? 1 : 2;
    constexpr int U = DIM / 64;                        // 16-byte loads of a thread, keys and values each
    constexpr int KR = DIM / 8;                        // slots of a row of keys
    const auto k_swizzle = [](uint32_t row) { return DIM == 64 ? row / 2 % 8 : row % 16; };
    auto k_tile = reinterpret_cast<kv_half8*>(lds), v_tile = k_tile + kPage * KR;
    auto k_codes = reinterpret_cast<uint4*>(v_tile + DIM * 8), v_codes = k_codes + U * kThreads;
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), r = lane % 32,
                   g = lane / 32;
    const uint32_t h = work.head, first = work.first;
    const uint32_t first_row = work.first_row + wave * 32;

    uint32_t seq = work.first_seq, last = work.last;
    struct Page {
        int32_t id;
        float ks, vs;          // 0 for a page that is not there: what page 0 holds must not matter
    };
    uint32_t base = first;
    int32_t my_id;
    float my_ks, my_vs;
    auto look_up_id = [&] {
        my_id = valid_page(a.c.table[(size_t)seq * a.c.width + min(base + lane, work.last - 1)], a.c.pages);
    };
    auto look_up_scales = [&] {
        const size_t at = (size_t)max(my_id, 0) * a.c.heads + h;
        my_ks = my_id < 0 ? 0.0f : a.c.k_scales[at];
        my_vs = my_id < 0 ? 0.0f : a.c.v_scales[at];
    };
    auto page_at = [&](uint32_t page) {
        if (page - base >= 64) {
            base = page;
            look_up_id();
            look_up_scales();
        }
        const uint32_t i = page - base;
        return Page{__builtin_amdgcn_readlane(my_id, i),
                    __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_ks), i)),
                    __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_vs), i))};
    };
    auto fetch = [&](int32_t id) {
        const size_t at = ((size_t)max(id, 0) * a.c.heads + h) * (kPage * DIM) + tid * 16;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            to_lds(a.c.k + at + u * kThreads * 16, k_codes + u * kThreads + wave * 64);
            to_lds(a.c.v + at + u * kThreads * 16, v_codes + u * kThreads + wave * 64);
        }
    };
    look_up_id();
    if (own) {
        last = own_pages_end(a, work);
    } else {
        const Holder holder(a, work);
        last = holder.last;
        if (holder.seq != seq) {
            seq = holder.seq;
            look_up_id();
        }
    }
    look_up_scales();
    Page now = page_at(first), next = page_at(first + 1);
    fetch(now.id);

    const Row row(a, work, first_row + r);
    Query<IN, DIM, 8, 16> raw;
    raw.load(a.q, row.there ? row.query : 0, g * 8, row.there);
    // what the wave's rows see: all of them the keys below all_see, none a page from my_last on
    int32_t all_see = row.there ? row.limit : INT32_MAX, most = row.there ? row.limit : 0;
#pragma unroll
    for (int d = 16; d; d /= 2) {
        all_see = min(all_see, __shfl_xor(all_see, d));
        most = max(most, __shfl_xor(most, d));
    }
    all_see = __builtin_amdgcn_readfirstlane(all_see);
    most = __builtin_amdgcn_readfirstlane(most);
    const uint32_t my_last = min(last, most > 0 ? (uint32_t)(most + kPage - 1) / kPage : 0u);
    const int32_t limit = row.there ? row.limit : INT32_MAX;

    kv_half8 q[DIM / 16][T];
    const float undo = raw.template convert<32, T>(a.negative, q) * a.scale;

    kv_f32x16 o[DIM / 32] = {};
    Unit unit;
    float top = -FLT_MAX, total = 0.0f;
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
            // fragments of both products are read kAhead products before they are used
            constexpr int FK = DIM / 8;
            kv_half8 kf[FK];
            const auto read_k = [&](int f) {
                kf[f] = *reinterpret_cast<const kv_half8*>((const char*)k_tile + (k_at ^ (f / 2 * 32)) + f % 2 * 32 * KR * 16);
            };
#pragma unroll
            for (int f = 0; f < kAhead; ++f) read_k(f);
#pragma unroll
            for (int f = 0; f < FK; ++f) {
                if (f + kAhead < FK) read_k(f + kAhead);
#pragma unroll
                for (int e = 0; e < T; ++e)
                    s[f % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[f], q[f / 2][e], s[f % 2], 0, 0, 0);
            }
            lay_out_products<FK, T>();
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
            constexpr int D = DIM / 32, FV = 4 * D;
            kv_half8 vf[FV];
            const auto read_v = [&](int f) {
                vf[f] = *reinterpret_cast<const kv_half8*>((const char*)v_tile + (v_at ^ (f / D * 32)) + f % D * 32 * 128);
            };
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int f = 0; f < kAhead; ++f) read_v(f);
#pragma unroll
            for (int f = 0; f < FV; ++f) {
                if (f + kAhead < FV) read_v(f + kAhead);
#pragma unroll
                for (int e = 0; e < T; ++e)
                    o[f % D] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[f], p[f / D][e], o[f % D], 0, 0, 0);
            }
            lay_out_products<FV, T>();
        }
        now = next, next = after;
    }
    loads_done();                                    // nothing may write to LDS that is no longer this workgroup's

    total = sum_over_32(total);
    if (first_row + r >= work.row_count) return;
    const size_t at = Row(a, work, first_row + r).item * (a.prefix_slots + a.own_slots) + work.slot;
    // register k of tile d is channel 32 d + 8 (k / 4) + 4 g + k % 4
#pragma unroll
    for (int d = 0; d < DIM / 32; ++d)
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<kv_f32x4*>(a.part + at * DIM + d * 32 + k * 2 + g * 4) =
                kv_f32x4{o[d][k], o[d][k + 1], o[d][k + 2], o[d][k + 3]} * unit.unit;
    if (g == 0) a.stats[at * 2] = top, a.stats[at * 2 + 1] = total;
}

// The same a page ahead: the scores of the next page are formed between the
// exponentials of this one, the next codes go into the other half of LDS between
// the products with the values, and one barrier a page is enough.  A wave has
// its matrix and its vector instructions side by side that way, which a second
// workgroup on the CU gives the other bodies.  For bf16 and 128 channels only:
// 64 leave too few products to hide the exponentials behind (8 prompts x 8
// sequences, in tiles of 128 rows, 28.7 -> 33.5 us), 256 and fp32 have no
// registers for a second page.
// 64 sequences behind 32,768 tokens 78.4 -> 72.1 us, 65,536 tokens 130 -> 115
// us in this kernel, 800 query rows a head 172 -> 166 us, from four pages a
// workgroup on no worse.

template <int DIM, int IN>
__device__ __forceinline__ void attend_many_ahead(const SharedArgs& a, const Work& work, bool own, char* lds) {
    constexpr int U = DIM / 64;                        // 16-byte loads of a thread, keys and values each
    constexpr int KR = DIM / 8;                        // slots of a row of keys
    constexpr int FK = DIM / 8, FV = DIM / 8, D = DIM / 32;   // fragments of keys, of values; tiles of outputs
    constexpr int AHEAD = 4;
    enum : int { kVector = 0x2, kMatrix = 0x8, kLdsRead = 0x100, kLdsWrite = 0x200, kExp = 0x400 };
    static_assert(kScoresAhead<DIM, IN>);
    const auto k_swizzle = [](uint32_t row) { return row % 16; };
    constexpr int BYTES = kPage * DIM * 2;             // of a page's keys, or values
    const uint32_t tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64), r = lane % 32,
                   g = lane / 32;
    const uint32_t h = work.head, first = work.first;
    const uint32_t first_row = work.first_row + wave * 32;
    uint32_t seq = work.first_seq, last = work.last;
    struct Page {
        int32_t id;
        float ks, vs;          // 0 for a page that is not there
    };
    uint32_t base = first;
    int32_t my_id;
    float my_ks, my_vs;
    auto look_up_id = [&] {
        my_id = valid_page(a.c.table[(size_t)seq * a.c.width + min(base + lane, work.last - 1)], a.c.pages);
    };
    auto look_up_scales = [&] {
        const size_t at = (size_t)max(my_id, 0) * a.c.heads + h;
        my_ks = a.c.k_scales[at], my_vs = a.c.v_scales[at];
        __builtin_amdgcn_s_waitcnt(0x0f70);            // the loads: here, not before every use
        if (my_id < 0) my_ks = my_vs = 0.0f;
    };
    auto page_at = [&](uint32_t page) {
        if (page - base >= 64) {
            base = page;
            look_up_id();
            look_up_scales();
        }
        const uint32_t i = page - base;
        return Page{__builtin_amdgcn_readlane(my_id, i),
                    __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_ks), i)),
                    __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, my_vs), i))};
    };
    uint4 kr[U], vr[U];
    auto fetch = [&](const int8_t* codes, int32_t id, uint4 (&to)[U]) {
        const int8_t* from = codes + ((size_t)max(id, 0) * a.c.heads + h) * (kPage * DIM) + tid * 16;
#pragma unroll
        for (int u = 0; u < U; ++u) to[u] = *reinterpret_cast<const uint4*>(from + u * kThreads * 16);
    };
    auto write_k = [&](int buffer) {
        auto k_tile = reinterpret_cast<kv_half8*>(lds + buffer * BYTES);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = u * kThreads + tid;
            const uint32_t key = i / (DIM / 16), lr = exchange_bits_2_3(key), c = i % (DIM / 16) * 2;
            k_tile[lr * KR + (c ^ k_swizzle(lr))] = half_codes(kr[u].x, kr[u].y);
            k_tile[lr * KR + ((c + 1) ^ k_swizzle(lr))] = half_codes(kr[u].z, kr[u].w);
        }
    };
    auto write_v = [&](int buffer) {
        auto v_tile = reinterpret_cast<kv_half8*>(lds + (2 + buffer) * BYTES);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = u * kThreads + tid, d = i / 4, e = i % 4 * 2;
            v_tile[d * 8 + (e ^ d / 2 % 8)] = half_codes(vr[u].x, vr[u].y);
            v_tile[d * 8 + ((e + 1) ^ d / 2 % 8)] = half_codes(vr[u].z, vr[u].w);
        }
    };
    look_up_id();
    if (own) {
        last = own_pages_end(a, work);
    } else {
        const Holder holder(a, work);
        last = holder.last;
        if (holder.seq != seq) {
            seq = holder.seq;
            look_up_id();
        }
    }
    look_up_scales();
    Page now = page_at(first), next = page_at(first + 1), after = page_at(first + 2);
    fetch(a.c.k, now.id, kr);
    fetch(a.c.v, now.id, vr);

    kv_half8 q[DIM / 16][1];
    float undo;
    int32_t limit, all_see;
    {
        const Row row(a, work, first_row + r);
        Query<IN, DIM, 8, 16> raw;
        raw.load(a.q, row.there ? row.query : 0, g * 8, row.there);
        limit = row.there ? row.limit : INT32_MAX;
        all_see = limit;
#pragma unroll
        for (int d = 16; d; d /= 2) all_see = min(all_see, __shfl_xor(all_see, d));
        all_see = __builtin_amdgcn_readfirstlane(all_see);
        undo = raw.template convert<32, 1>(a.negative, q) * a.scale;
    }
    const uint32_t k_first = r * (KR * 16) + (g ^ k_swizzle(r)) * 16, v_first = r * 128 + (g ^ r / 2 % 8) * 16;
    uint32_t k_at = k_first, v_at = v_first;
    auto k_fragment = [&](int buffer, int f) {
        return *reinterpret_cast<const kv_half8*>(lds + buffer * BYTES + (k_at ^ (f / 2 * 32)) + f % 2 * 32 * KR * 16);
    };
    auto v_fragment = [&](int buffer, int f) {
        return *reinterpret_cast<const kv_half8*>(lds + (2 + buffer) * BYTES + (v_at ^ (f / D * 32)) + f % D * 32 * 128);
    };

    kv_f32x16 o[D] = {};
    Unit unit;
    float top = -FLT_MAX, total = 0.0f;
    kv_f32x16 s0[2] = {}, s1[2];                       // scores of even and odd pages, counted from the first
    write_k(0);
    fetch(a.c.k, next.id, kr);
    write_v(0);
    fetch(a.c.v, next.id, vr);
    lds_barrier();
#pragma unroll
    for (int f = 0; f < FK; ++f) s0[f % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k_fragment(0, f), q[f / 2][0], s0[f % 2], 0, 0, 0);
    write_k(1);
    fetch(a.c.k, after.id, kr);
    lds_barrier();

    // Enters with page's scores in s, its values and the next page's keys in LDS
    // and the codes of the next values and the keys after them in registers.
    uint32_t page = first;
    auto step = [&](auto PARITY, kv_f32x16 (&s)[2], kv_f32x16 (&s_next)[2]) {
        constexpr int even = decltype(PARITY)::value, odd = 1 - even;
        const int32_t key0 = (int32_t)(page * kPage);
        float factor = now.ks * undo;
        if (key0 + kPage > all_see || now.id < 0) {
            const int32_t sees = (now.id < 0 ? 0 : limit) - key0 - (int32_t)g * 8;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    s[t][k] = 32 * t + 16 * (k / 8) + k % 8 < sees ? s[t][k] * factor : -INFINITY;
            factor = 1.0f;
        }
        // new to the compiler at each page: it would keep an address for every fragment
        k_at = k_first, v_at = v_first;
        asm volatile("" : "+v"(k_at), "+v"(v_at));
        constexpr int N1 = FK / 4;
        kv_half8 kf[FK];
        s_next[0] = s_next[1] = kv_f32x16{};
#pragma unroll
        for (int f = 0; f < AHEAD; ++f) kf[f] = k_fragment(odd, f);
#pragma unroll
        for (int f = 0; f < N1; ++f) {
            if (f + AHEAD < FK) kf[f + AHEAD] = k_fragment(odd, f + AHEAD);
            s_next[f % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[f], q[f / 2][0], s_next[f % 2], 0, 0, 0);
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
        const float shrink_all = unit.next(now.vs);
        if (__any(m > top + 1.5f) || shrink_all != 1.0f) {
            const float grown = m > top + 1.5f ? m : top, shrink = __builtin_amdgcn_exp2f(top - grown);
            total *= shrink;
#pragma unroll
            for (int d = 0; d < D; ++d) o[d] *= shrink * shrink_all;
            top = grown;
        }
        __builtin_amdgcn_sched_barrier(0);
        const float off = unit.lift - top;
        kv_half8 p[4][1];
        float sum = 0.0f;
#pragma unroll
        for (int f = N1; f < FK; ++f) {
            if (f + AHEAD < FK) kf[f + AHEAD] = k_fragment(odd, f + AHEAD);
            s_next[f % 2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[f], q[f / 2][0], s_next[f % 2], 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u / 2][u % 2 * 8 + k], factor, off));
            sum += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
            half_terms<1>(x, p[u]);
        }
        total = __builtin_fmaf(sum, unit.drop, total);
        constexpr int N2 = FK - N1;
#pragma unroll
        for (int f = N1; f < FK; ++f) {
            __builtin_amdgcn_sched_group_barrier(kMatrix, 1, 0);
            if (f + AHEAD < FK) __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
            __builtin_amdgcn_sched_group_barrier(kVector, (32 + N2 - 1) / N2, 0);
            __builtin_amdgcn_sched_group_barrier(kExp, (32 + N2 - 1) / N2, 0);
            __builtin_amdgcn_sched_group_barrier(kVector, 52 / N2, 0);
        }
        // the numerators are wanted here, not where they are used
        asm volatile("" : "+v"(p[0][0]), "+v"(p[1][0]), "+v"(p[2][0]), "+v"(p[3][0]), "+v"(total));
        __builtin_amdgcn_sched_barrier(0);
        const Page last_but = page_at(page + 3);
        __builtin_amdgcn_sched_barrier(0);
        kv_half8 vf[FV];
#pragma unroll
        for (int f = 0; f < AHEAD; ++f) vf[f] = v_fragment(even, f);
#pragma unroll
        for (int f = 0; f < FV; ++f) {
            if (f + AHEAD < FV) vf[f + AHEAD] = v_fragment(even, f + AHEAD);
            o[f % D] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[f], p[f / D][0], o[f % D], 0, 0, 0);
        }
        write_k(even);
        write_v(odd);
        __builtin_amdgcn_sched_group_barrier(kLdsRead, AHEAD, 0);
#pragma unroll
        for (int f = 0; f < FV; ++f) {
            __builtin_amdgcn_sched_group_barrier(kMatrix, 1, 0);
            if (f + AHEAD < FV) __builtin_amdgcn_sched_group_barrier(kLdsRead, 1, 0);
            __builtin_amdgcn_sched_group_barrier(kVector, 40 * U / FV, 0);
            if (f % 2) __builtin_amdgcn_sched_group_barrier(kLdsWrite, 4 * U * 2 / FV, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        fetch(a.c.v, after.id, vr);
        fetch(a.c.k, last_but.id, kr);
        lds_barrier();                               // the next pages are there, these have been read
        now = next, next = after, after = last_but;
        ++page;
    };
    while (page + 1 < last) {
        step(std::integral_constant<int, 0>{}, s0, s1);
        step(std::integral_constant<int, 1>{}, s1, s0);
    }
    if (page < last) step(std::integral_constant<int, 0>{}, s0, s1);

    total = sum_over_32(total);
    if (first_row + r >= work.row_count) return;
    const size_t at = Row(a, work, first_row + r).item * (a.prefix_slots + a.own_slots) + work.slot;
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<kv_f32x4*>(a.part + at * DIM + d * 32 + k * 2 + g * 4) =
                kv_f32x4{o[d][k], o[d][k + 1], o[d][k + 2], o[d][k + 3]} * unit.unit;
    if (g == 0) a.stats[at * 2] = top, a.stats[at * 2 + 1] = total;
}

// ---------------------------------------------------------------------------
// the kernels: one form for both kinds of tiles, or many rows for the prefix
// and few for the own pages.  The prefix comes first and leaves a CU half empty
// (see `plan_for`); there the own pages, which wait for memory, run beside it:
// 64 sequences of 32 heads x 128 behind 32,768 tokens 77 us, in two launches
// 87, in turn eight by eight 93, all before the scores were formed a page ahead.

enum : int { kFew = 0, kMany = 1, kManyFew = 2 };

template <int DIM, int IN, int FORM>
__global__ __launch_bounds__(kThreads, DIM == 256 ? 1 : 2)
    void kv8_shared_kernel(SharedArgs a, uint32_t prefix_units) {
    constexpr int FEW = FORM == kMany ? 0 : kFewLds<DIM>, MANY = FORM == kFew ? 0 : kManyLds<DIM, IN>;
    constexpr int BYTES = std::max(FEW, MANY);
    __shared__ alignas(16) char lds[BYTES];
    const bool own = blockIdx.x >= prefix_units;
    const uint32_t unit = own ? blockIdx.x - prefix_units : blockIdx.x;
    Work work;
    if (own)
        work.of_own(a, unit, FORM == kMany ? kTileRows : kFewRows);
    else
        work.of_prefix(a, unit, FORM == kFew ? kFewRows : kTileRows);
    if (!work.any) return;
    if (FORM == kFew || (FORM == kManyFew && own)) {
        if constexpr (FORM != kMany) attend_few<DIM, IN>(a, work, own, lds);
    } else if constexpr (FORM != kFew) {
        if constexpr (kScoresAhead<DIM, IN>)
            attend_many_ahead<DIM, IN>(a, work, own, lds);
        else
            attend_many<DIM, IN>(a, work, own, lds);
    }
}

// ---------------------------------------------------------------------------
// a row's slots joined: DIM / 4 lanes with four channels each take a row, or
// GROUPS times as many, each time some of its slots.

constexpr int kJoinRows = 8;                // rows times groups of a workgroup

template <int DIM, int OUT, int GROUPS>
__global__ __launch_bounds__(kJoinRows * DIM / 4) void kv8_shared_join_kernel(SharedArgs a) {
    constexpr int Q = DIM / 4, ROWS = kJoinRows / GROUPS;
    __shared__ kv_f32x4 ys[ROWS][GROUPS][Q];
    __shared__ float tops[ROWS][GROUPS], totals[ROWS][GROUPS];
    const uint32_t q = threadIdx.x % Q, group = threadIdx.x / Q % GROUPS, of_group = threadIdx.x / Q / GROUPS;
    const size_t item = (size_t)blockIdx.x * ROWS + of_group, all = (size_t)a.c.batch * a.c.heads * a.rows;
    const size_t safe = min(item, all - 1);
    const uint32_t mine = safe % a.rows, bh = safe / a.rows, h = bh % a.c.heads, b = bh / a.c.heads;
    // a wave's rows may be of several sequences: each is looked up by all of the wave
    uint32_t before = 0;
    if constexpr (GROUPS * Q >= 64) {
        before = pages_before(a, __builtin_amdgcn_readfirstlane(b));
    } else {
        for (uint32_t lane = 0; lane < 64; lane += Q) {
            const uint32_t other = pages_before(a, __builtin_amdgcn_readlane(b, lane));
            if (threadIdx.x % 64 / Q == lane / Q) before = other;
        }
    }
    const Seq seq(a, b);
    const int32_t i = (int32_t)(mine / a.group);
    const uint32_t pages = (uint32_t)(seq.n + kPage - 1) / kPage;
    const Cut prefix(before, a.prefix_slots), own(pages > before ? pages - before : 0, a.own_slots);
    float m = -FLT_MAX, l = 0.0f;
    kv_f32x4 y = {};
    if (i < seq.m) {
        const uint32_t slots = a.prefix_slots + a.own_slots, count = prefix.used + own.used;
#pragma unroll 4
        for (uint32_t s = group; s < count; s += GROUPS) {
            const size_t at = safe * slots + (s < prefix.used ? s : a.prefix_slots + s - prefix.used);
            const float2 stat = *reinterpret_cast<const float2*>(a.stats + at * 2);
            const kv_f32x4 x = *reinterpret_cast<const kv_f32x4*>(a.part + at * DIM + q * 4);
            const float top = fmaxf(m, stat.x), f = __builtin_amdgcn_exp2f(m - top), e = __builtin_amdgcn_exp2f(stat.x - top);
            m = top;
            l = __builtin_fmaf(stat.y, e, l * f);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __builtin_fmaf(x[k], e, y[k] * f);
        }
    }
    if constexpr (GROUPS > 1) {
        ys[of_group][group][q] = y;
        if (q == 0) tops[of_group][group] = m, totals[of_group][group] = l;
        __syncthreads();
        if (group) return;
        m = tops[of_group][0];
#pragma unroll
        for (int s = 1; s < GROUPS; ++s) m = fmaxf(m, tops[of_group][s]);
        l = 0.0f;
        y = kv_f32x4{};
#pragma unroll
        for (int s = 0; s < GROUPS; ++s) {
            const float f = __builtin_amdgcn_exp2f(tops[of_group][s] - m);
            l = __builtin_fmaf(totals[of_group][s], f, l);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = __builtin_fmaf(ys[of_group][s][q][k], f, y[k]);
        }
    }
    if (item >= all) return;
    const bool seen = l != 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) y[k] = seen ? y[k] / l : 0.0f;
    store4<OUT>(a.out, (((size_t)b * a.queries + i) * a.heads + h * a.group + mine % a.group) * DIM + q * 4, y);
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

// Rows that go to tiles of 16, which read the same pages at the same time, and
// not to one of 128.  16, 32 and 64 rows a tile's worth at a time, against 128:
// 32 rows x 256 channels behind 32,768 tokens 53 against 77 us, 64 rows 78
// against 86; 48 rows x 64 20.6 against 26.4, 64 rows of 8 prompts 25.2 against
// 27.4; 32 rows x 128 24.7 against 33.6, but 48 rows of 8 prompts 43.5 against
// 38.4.  (A tile of two times 16 rows reads a page once, but holds so many
// registers that a SIMD has one wave: 32 rows x 128 33, x 64 23.8 against 17.3.)
bool is_few(int dim, size_t rows) { return rows <= (dim == 128 ? 32 : 64); }

// How a call is cut.  Group sizes, prefixes and lengths are on the device; the
// host goes by their averages and bounds.  A slot more for a row is a row of
// outputs more to write and to read again, so there are no more than fill the
// CUs: of many rows one workgroup a CU with 128 or 256 channels (64 sequences
// behind 32,768 tokens, 32 heads x 128: one 66 us, one and a half 69, two 73,
// three 81; 16 heads x 256, 32 sequences: 89, 99, 118), three with 64, whose
// pages are shorter (64 heads: 89, 76, 70); of few rows one with 128 or 256 (eight
// sequences behind 32,768 tokens 25 us, with two 29; behind 131,072 tokens 63 and
// 84), two with 64 (8 prompts x 8 sequences of 4,000 tokens: one 25.3, two 23.1,
// three 24.2; 8,000 tokens: 39, 32, 32); of own pages one.  Where a slot of many
// rows would be more than 56 pages long, two workgroups share a CU's units better
// than one uses them (64 sequences behind 65,536 tokens 105 against 112 us, behind
// 131,072 190 against 212; fp32 156 against 175 and 285 against 330; at 48 pages
// bf16 90 against 86), but not more than two: 800 rows behind 8,000 tokens, in two
// slots as it is, 135 us and in four 168.
struct Plan {
    bool prefix_few, own_few;
    uint32_t prefix_rows, own_rows;      // of a tile
    uint32_t prefix_tiles, own_tiles, prefix_slots, own_slots;
};

// As many slots as give `target` workgroups, or up to twice as many where that
// leaves a tenth or more of the CUs' time empty (20 groups x 8 heads: 320
// workgroups are two rounds, 480 as well: 66 -> 56 us).
uint32_t slots_for(size_t units, uint32_t width, size_t target) {
    const size_t want = (target + units - 1) / units, most = (width + 3) / 4;
    if (want >= most) return (uint32_t)most;
    // a CU's longest share, in pages of the axis: rounds of workgroups by slots
    const auto rounds = [&](size_t slots) { return (units * slots + 255) / 256; };
    size_t best = want;
    if (units * want * 10 < rounds(want) * 256 * 9)
        for (size_t s = want + 1; s <= 2 * want && s <= most; ++s)
            if (rounds(s) * best * 10 < rounds(best) * s * 9) best = s;
    return (uint32_t)best;
}

Plan plan_for(uint32_t batch, uint32_t kv_heads, uint32_t rows, int dim, uint32_t width, uint32_t groups) {
    Plan p = {};
    const size_t all = (size_t)batch * rows, mean = (all + groups - 1) / groups;
    p.prefix_few = is_few(dim, mean);
    p.prefix_rows = p.prefix_few ? kFewRows : kTileRows;
    p.prefix_tiles = (uint32_t)(all / p.prefix_rows) + groups;
    const size_t likely = groups * ((mean + p.prefix_rows - 1) / p.prefix_rows);   // groups of one size
    p.prefix_slots = slots_for(likely * kv_heads, width, dim != 64 ? 256 : p.prefix_few ? 512 : 768);
    if (!p.prefix_few && dim == 128 && width / p.prefix_slots > 56)
        p.prefix_slots = std::max(p.prefix_slots, (uint32_t)(512 / (likely * kv_heads)));
    p.own_few = is_few(dim, rows);
    p.own_rows = p.own_few ? kFewRows : kTileRows;
    p.own_tiles = (rows + p.own_rows - 1) / p.own_rows;
    p.own_slots = slots_for((size_t)batch * kv_heads * p.own_tiles, width, 256);
    return p;
}

bool joined_by_eight(const Plan& p) { return p.prefix_slots + p.own_slots > 4; }

} // namespace

bool kv8_shared_fits(uint32_t batch, uint32_t kv_heads, uint32_t rows, int dim, uint32_t width, uint32_t groups) {
    const Plan p = plan_for(batch, kv_heads, rows, dim, width, groups);
    const size_t units = (size_t)p.prefix_tiles * kv_heads * p.prefix_slots + (size_t)batch * kv_heads * p.own_tiles * p.own_slots;
    const size_t join = (size_t)batch * kv_heads * rows * (dim / 4) * (joined_by_eight(p) ? kJoinRows : 1);
    return units * kThreads <= UINT32_MAX && join + kJoinRows * dim / 4 <= UINT32_MAX;
}

size_t kv8_shared_workspace(uint32_t batch, uint32_t kv_heads, uint32_t rows, int dim, uint32_t width, uint32_t groups) {
    const Plan p = plan_for(batch, kv_heads, rows, dim, width, groups);
    const size_t parts = (size_t)batch * kv_heads * rows * (p.prefix_slots + p.own_slots);
    return align256(parts * 8) + align256(parts * dim * 4);
}

hipError_t launch_kv8_shared(const Kv8& c, const void* q, int kind, uint32_t queries, uint32_t heads, const int32_t* starts,
                             const int32_t* prefix, uint32_t groups, const int32_t* q_lens, float scale, void* out,
                             void* workspace, hipStream_t st) {
    SharedArgs a = {};
    a.c = c, a.q = q, a.starts = starts, a.prefix = prefix, a.groups = groups, a.q_lens = q_lens, a.out = out;
    a.queries = queries, a.heads = heads, a.group = heads / c.heads, a.rows = queries * a.group;
    a.scale = (scale < 0 ? -scale : scale) * 1.44269504088896340736f;
    a.negative = scale < 0;
    const Plan p = plan_for(c.batch, c.heads, a.rows, c.dim, c.width, groups);
    a.prefix_tiles = p.prefix_tiles, a.own_tiles = p.own_tiles, a.prefix_slots = p.prefix_slots, a.own_slots = p.own_slots;
    const size_t items = (size_t)c.batch * c.heads * a.rows, parts = items * (p.prefix_slots + p.own_slots);
    a.stats = (float*)workspace;
    a.part = (float*)((uint8_t*)workspace + align256(parts * 8));
    return with_dim(c.dim, [&](auto D) {
        return with_kind(kind, [&](auto K) {
            const uint32_t prefix_units = p.prefix_tiles * c.heads * p.prefix_slots;
            const uint32_t own_units = c.batch * c.heads * p.own_tiles * p.own_slots;
            const auto attend = [&](auto kernel) { return launch_threads(kernel, prefix_units + own_units, kThreads, st, a, prefix_units); };
            // a group's rows are a sequence's at least: few of all are few of each
            const hipError_t e = p.prefix_few  ? attend(kv8_shared_kernel<D(), K(), kFew>)
                                 : p.own_few ? attend(kv8_shared_kernel<D(), K(), kManyFew>)
                                             : attend(kv8_shared_kernel<D(), K(), kMany>);
            if (e != hipSuccess) return e;
            return joined_by_eight(p)
                       ? launch_threads(kv8_shared_join_kernel<D(), K(), kJoinRows>, (uint32_t)items, kJoinRows * D() / 4, st, a)
                       : launch_threads(kv8_shared_join_kernel<D(), K(), 1>, (uint32_t)((items + kJoinRows - 1) / kJoinRows),
                                        kJoinRows * D() / 4, st, a);
        });
    });
}

} // namespace qar
