// qar_kv8_pages.hip -- who owns the 8-bit cache's pages, on gfx950: sequences
// fork and share pages, are cut back, take pages for new tokens, and live
// pages move to the pool's front.
//
// refs[p] counts the page-table entries that name page p; a page without any
// is free.  All of it happens on the device, so that a step that forks, takes
// pages and appends can be captured, and every result is that of serving the
// sequences one after another, the lowest free page first: equal calls give
// equal tables.  The calls on tables and counts move a few kilobytes and are
// bound by their chain of dependent loads; only what has to be private or to
// move is copied, which is bound by memory.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "qar_device.h"
#include "qar_launch.h"
#include "qar_serve.h"

namespace qar {
namespace {

constexpr int kPage = 64;

__device__ __forceinline__ bool is_page(int32_t id, uint32_t pages) { return (uint32_t)id < pages; }

__device__ __forceinline__ uint32_t clamp_length(int32_t n, uint32_t top) {
    return n < 0 ? 0 : (uint32_t)n > top ? top : (uint32_t)n;
}

__device__ __forceinline__ uint32_t pages_of(uint32_t tokens) { return (tokens + kPage - 1) / kPage; }

// ---------------------------------------------------------------------------
// fork: a workgroup writes one new sequence's table from its parent's (64 from
// one of 125 pages 4.4 us, most of it parent -> length -> table -> count).

struct ForkArgs {
    const int32_t *table, *lengths, *parents;
    int32_t *into, *into_lengths, *refs;
    uint32_t batch, width, into_width, pages;
};

__global__ __launch_bounds__(kThreads) void kv8_fork_kernel(ForkArgs a) {
    const uint32_t b = blockIdx.x;
    const int32_t parent = a.parents[b];
    const bool has = (uint32_t)parent < a.batch;
    const uint32_t n = has ? clamp_length(a.lengths[parent], a.width * kPage) : 0, used = pages_of(n);
    for (uint32_t w = threadIdx.x; w < a.into_width; w += kThreads) {
        const int32_t id = w < used ? a.table[(size_t)parent * a.width + w] : -1;
        const bool there = is_page(id, a.pages);
        if (there) atomicAdd(a.refs + id, 1);
        a.into[(size_t)b * a.into_width + w] = there ? id : -1;
    }
    if (threadIdx.x == 0) a.into_lengths[b] = (int32_t)n;
}

// ---------------------------------------------------------------------------
// free: a workgroup gives back what one sequence has behind its kept tokens (64
// of up to 33 pages 2.6 us).

struct FreeArgs {
    int32_t *table, *lengths, *refs;
    const int32_t* keep;                 // may be null: nothing is kept
    uint32_t width, pages;
};

__global__ __launch_bounds__(kThreads) void kv8_free_kernel(FreeArgs a) {
    const uint32_t b = blockIdx.x;
    const uint32_t n = min(clamp_length(a.lengths[b], a.width * kPage),
                           a.keep ? clamp_length(a.keep[b], a.width * kPage) : 0u);
    for (uint32_t w = pages_of(n) + threadIdx.x; w < a.width; w += kThreads) {
        int32_t* entry = a.table + (size_t)b * a.width + w;
        const int32_t id = *entry;
        if (is_page(id, a.pages)) atomicSub(a.refs + id, 1);
        *entry = -1;
    }
    __syncthreads();                     // all have read the length
    if (threadIdx.x == 0) a.lengths[b] = (int32_t)n;
}

// ---------------------------------------------------------------------------
// One workgroup decides who gets which page: what a sequence gets depends on
// what all before it took.  Its scans are shuffles within a wave and the waves'
// counts in LDS.

// This thread's offset among the threads' counts, in thread order, and their
// sum.  `sums` is used again by the next call, after a barrier of its own.
template <int WAVES>
__device__ __forceinline__ uint32_t scan(uint32_t count, uint32_t& total, uint32_t (&sums)[WAVES]) {
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    uint32_t sum = count;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t other = __shfl_up(sum, d);
        if (lane >= (uint32_t)d) sum += other;
    }
    __syncthreads();                     // the call before has been read
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    uint32_t before = sum - count;
    total = 0;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) {
        before += (uint32_t)v < wave ? sums[v] : 0;
        total += sums[v];
    }
    return before;
}

// --- reserve.  A sequence goes on at its length n.  It wants a page for every
// page behind n that has none, and one in place of the page that holds n if
// that is partly filled and others own it at the sequence's turn: `rank`
// sequences before it went on in the same page and took copies, so refs - rank
// owners are left.  Wanted pages are numbered in the order of sequences and
// positions; number i takes the i-th free page.

struct ReserveArgs {
    int32_t *table, *refs;
    const int32_t *lengths, *tokens;
    int32_t *room, *source, *target;
    uint32_t batch, width, pages;
};

constexpr int kSequences = 4096;         // what the arrays below hold
constexpr uint32_t kHasAll = ~0u, kLastOwner = ~1u;

// Four waves meet at a barrier sooner than sixteen, and meet a dozen times (64
// beams: 7.8 against 8.6 us); more than 256 sequences take sixteen.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void kv8_reserve_kernel(ReserveArgs a) {
    constexpr int RUN = 4096 / THREADS;           // neighbouring pages that a thread looks at
    __shared__ alignas(16) int32_t shared_page[kSequences];   // the page that a sequence goes on in, -1: at a page's start; -2: nowhere
    __shared__ uint32_t begin[kSequences + 1];    // of the sequence's looked-at entries, among all sequences'
    __shared__ uint32_t short_of[kSequences];     // the first page that it did not get, or one of the two above
    __shared__ int32_t found[RUN * THREADS];      // free pages that nobody has taken yet
    __shared__ uint32_t sums[THREADS / 64];
    const uint32_t tid = threadIdx.x;
    // which of its pages from `first` on are free; the first are asked for at once
    const auto look = [&](uint32_t first) {
        uint32_t mask = 0;
#pragma unroll
        for (int k = 0; k < RUN; ++k) mask |= (uint32_t)(a.refs[min(first + RUN * tid + k, a.pages - 1)] <= 0 && first + RUN * tid + k < a.pages) << k;
        return mask;
    };
    uint32_t free_mask = look(0);
    const auto length_of = [&](uint32_t b) { return clamp_length(a.lengths[b], a.width * kPage); };
    const auto end_of = [&](uint32_t b, uint32_t n) {
        return (uint32_t)min((uint64_t)n + (uint32_t)max(a.tokens[b], 0), (uint64_t)a.width * kPage);
    };

    for (uint32_t b = tid; b < a.batch; b += THREADS) {
        const uint32_t n = length_of(b), end = end_of(b, n);
        int32_t id = -1;
        if (end == n) {
            id = -2;
        } else if (n % kPage) {
            id = a.table[(size_t)b * a.width + n / kPage];
            if (!is_page(id, a.pages)) id = -2;
        }
        shared_page[b] = id;
        short_of[b] = kHasAll;
        a.source[b] = a.target[b] = -1;
    }
    __syncthreads();

    // copies, and the entries that each sequence looks at
    uint32_t entries = 0;
    for (uint32_t base = 0; base < a.batch; base += THREADS) {
        const uint32_t b = base + tid;
        uint32_t count = 0;
        if (b < a.batch && shared_page[b] != -2) {
            const uint32_t n = length_of(b);
            count = pages_of(end_of(b, n)) - pages_of(n);
            const int32_t id = shared_page[b];
            if (id >= 0) {
                const int32_t owners = a.refs[id];
                if (owners > 1) {
                    // sixteen at a time: one by one, each would wait for LDS
                    uint32_t rank = 0;
#pragma unroll 4
                    for (uint32_t j = 0; j < b; j += 4) {
                        const int4 four = *reinterpret_cast<const int4*>(shared_page + j);
                        rank += (four.x == id) + (four.y == id && j + 1 < b) + (four.z == id && j + 2 < b) +
                                (four.w == id && j + 3 < b);
                    }
                    count += owners - (int32_t)rank > 1;
                    // the last owner keeps the page, if those before it got theirs
                    if (owners - (int32_t)rank <= 1) short_of[b] = kLastOwner;
                }
            }
        }
        uint32_t total;
        const uint32_t before = scan(count, total, sums);
        if (b < a.batch) begin[b] = entries + before;
        entries += total;
    }
    if (tid == 0) begin[a.batch] = entries;
    __syncthreads();

    // the entries in order, a thread each; free pages are looked for from the
    // front as far as they are needed
    bool ran_out = false;
    uint32_t next_page = 0, have = 0, taken = 0;  // pages looked at; found and not taken: found[taken .. taken + have)
    for (uint32_t base = 0; base < entries; base += THREADS) {
        const uint32_t e = base + tid;
        uint32_t b = 0, w = 0;
        bool copies = false, wants = false;
        if (e < entries) {
            uint32_t lo = 0, hi = a.batch;        // the last sequence that begins at e or before, and has entries
            while (hi - lo > 1) {
                const uint32_t mid = (lo + hi) / 2;
                if (begin[mid] <= e) lo = mid;
                else hi = mid;
            }
            b = lo;
            const uint32_t n = length_of(b), i = e - begin[b], all = begin[b + 1] - begin[b];
            const uint32_t fresh = pages_of(end_of(b, n)) - pages_of(n);
            copies = all > fresh && i == 0;
            w = copies ? n / kPage : pages_of(n) + i - (all - fresh);
            wants = copies || !is_page(a.table[(size_t)b * a.width + w], a.pages);
        }
        uint32_t total;
        const uint32_t number = scan(wants, total, sums);
        uint32_t served = 0;
        while (served < total) {
            if (have == 0) {
                if (next_page >= a.pages) break;
                if (next_page) free_mask = look(next_page);
                uint32_t sum;
                uint32_t at = scan(__popc(free_mask), sum, sums);
#pragma unroll
                for (int k = 0; k < RUN; ++k)
                    if (free_mask >> k & 1) found[at++] = (int32_t)(next_page + RUN * tid + k);
                next_page += RUN * THREADS;
                have = sum, taken = 0;
                __syncthreads();
                continue;
            }
            const uint32_t now = min(have, total - served);
            if (wants && number >= served && number < served + now) {
                const int32_t page = found[taken + number - served];
                int32_t* entry = a.table + (size_t)b * a.width + w;
                if (copies) {
                    a.source[b] = *entry;
                    a.target[b] = page;
                    atomicSub(a.refs + *entry, 1);
                }
                *entry = page;
                a.refs[page] = 1;
            }
            served += now, taken += now, have -= now;
            __syncthreads();
        }
        // the pool is empty
        if (wants && number >= served) atomicMin(&short_of[b], w);
        ran_out |= served < total;
        __syncthreads();
    }

    for (uint32_t b = tid; b < a.batch; b += THREADS) {
        const uint32_t n = length_of(b), end = end_of(b, n);
        const uint32_t lacks = short_of[b];
        uint32_t room = shared_page[b] == -2 ? 0 : end - n;
        if (ran_out && lacks != kHasAll) {
            bool fails = n % kPage && lacks == n / kPage;
            // the last owner of a page: one of those before it may have stayed without a copy
            if (shared_page[b] >= 0)
                for (uint32_t j = 0; j < b && !fails; ++j)
                    fails = shared_page[j] == shared_page[b] && short_of[j] == length_of(j) / kPage;
            room = fails ? 0 : lacks == kLastOwner ? room : min(room, lacks * kPage - n);
        }
        a.room[b] = (int32_t)room;
    }
}

// --- compact.  With L live pages, the live ones from L on move, in ascending
// order, to the free places below L.  Lists in one workgroup, which walks the
// counts twice (2,186 pages 6.2 us), then the table and the counts in parallel.

struct CompactArgs {
    int32_t *table, *refs, *source, *target;
    uint32_t pages;
    size_t entries;                      // of the table
};

constexpr int kScan = 1024, kRun = 8;    // threads, neighbouring pages to each

__global__ __launch_bounds__(kScan) void kv8_compact_kernel(CompactArgs a) {
    __shared__ uint32_t sums[kScan / 64];
    const uint32_t tid = threadIdx.x, half = a.pages / 2;
    uint32_t count = 0;
    for (uint32_t p = tid; p < a.pages; p += kScan) count += a.refs[p] > 0;
    uint32_t live;
    scan(count, live, sums);
    uint32_t from = 0, to = 0;
    for (uint32_t base = 0; base < a.pages; base += kScan * kRun) {
        const uint32_t p0 = base + tid * kRun;
        uint32_t leaves = 0, takes = 0;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const uint32_t p = p0 + k;
            if (p < a.pages) {
                const int32_t owners = a.refs[p];
                if (owners > 0 && p >= live) leaves |= 1u << k;
                if (owners <= 0 && p < live) takes |= 1u << k;
                if (owners < 0) a.refs[p] = 0;    // below, negative counts stand for places
            }
        }
        uint32_t all_leave, all_take;
        uint32_t i = from + scan(__popc(leaves), all_leave, sums), j = to + scan(__popc(takes), all_take, sums);
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            if (leaves >> k & 1) a.source[i++] = (int32_t)(p0 + k);
            if (takes >> k & 1) a.target[j++] = (int32_t)(p0 + k);
        }
        from += all_leave, to += all_take;
    }
    __syncthreads();                     // the lists are written
    for (uint32_t i = tid; i < half; i += kScan) {
        if (i < from) {
            const int32_t s = a.source[i], t = a.target[i];
            a.refs[t] = a.refs[s];
            a.refs[s] = -1 - t;          // where the page went, for the table
        } else {
            a.source[i] = a.target[i] = -1;
        }
    }
}

__global__ __launch_bounds__(kThreads) void kv8_remap_kernel(CompactArgs a) {
    const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.entries) return;
    const int32_t id = a.table[i];
    if (!is_page(id, a.pages)) return;
    const int32_t place = a.refs[id];
    if (place < 0) a.table[i] = -1 - place;
}

__global__ __launch_bounds__(kThreads) void kv8_settle_kernel(CompactArgs a) {
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    if (i < a.pages / 2 && a.source[i] >= 0) a.refs[a.source[i]] = 0;
}

// ---------------------------------------------------------------------------
// copy.  A workgroup takes pieces of 16 KB of the listed pages, sixteen
// loads' worth of a wave each, all under way before the first is stored.
// Lists are mostly empty towards their end (a compaction's is as long as half
// the pool): a wave looks up 64 pieces at once.  A compaction's 504 pages of 8
// heads x 128 take 25 us, 5.2 TB/s as any copy; some twenty pages that beams must not share 4.7.

struct CopyArgs {
    const int8_t *k, *v;
    const float *k_scales, *v_scales;
    int8_t *to_k, *to_v;
    float *to_k_scales, *to_v_scales;
    const int32_t *source, *target;
    uint32_t count, pages, to_pages, heads;
    uint32_t bytes, pieces;              // of a page, keys or values; of both
};

constexpr int kPieceLoads = 4;
constexpr uint32_t kPiece = kThreads * 16 * kPieceLoads;

__global__ __launch_bounds__(kThreads) void kv8_copy_kernel(CopyArgs a) {
    const uint32_t lane = threadIdx.x % 64;
    const size_t units = (size_t)a.count * a.pieces, step = gridDim.x;
    for (size_t base = blockIdx.x; base < units; base += 64 * step) {
        const size_t mine = base + lane * step;
        int32_t from = -1, to = -1;
        if (mine < units) {
            from = a.source[mine / a.pieces];
            to = a.target[mine / a.pieces];
        }
        uint64_t there = __ballot(is_page(from, a.pages) && is_page(to, a.to_pages));
        while (there) {
            const int i = __builtin_ctzll(there);
            there &= there - 1;
            const int32_t s = __builtin_amdgcn_readlane(from, i), t = __builtin_amdgcn_readlane(to, i);
            const uint32_t piece = (uint32_t)((base + i * step) % a.pieces), half = a.pieces / 2, which = piece >= half;
            const uint32_t at = piece % half * kPiece + threadIdx.x * 16;
            const int8_t* in = (which ? a.v : a.k) + (size_t)s * a.bytes;
            int8_t* out = (which ? a.to_v : a.to_k) + (size_t)t * a.bytes;
            uint4 q[kPieceLoads];
#pragma unroll
            for (int u = 0; u < kPieceLoads; ++u)
                if (at + u * kThreads * 16 < a.bytes) q[u] = load_b128(in + at + u * kThreads * 16);
#pragma unroll
            for (int u = 0; u < kPieceLoads; ++u)
                if (at + u * kThreads * 16 < a.bytes) store_b128(out + at + u * kThreads * 16, q[u]);
            if (piece % half == 0) {
                const float* scales = which ? a.v_scales : a.k_scales;
                float* to_scales = which ? a.to_v_scales : a.to_k_scales;
                for (uint32_t h = threadIdx.x; h < a.heads; h += kThreads)
                    to_scales[(size_t)t * a.heads + h] = scales[(size_t)s * a.heads + h];
            }
        }
    }
}

} // namespace

hipError_t launch_kv8_fork(const Kv8& c, int32_t* refs, const int32_t* parents, const Kv8& into, hipStream_t st) {
    const ForkArgs a = {c.table, c.lengths, parents, const_cast<int32_t*>(into.table), into.lengths, refs,
                        c.batch, c.width, into.width, c.pages};
    return launch_threads(kv8_fork_kernel, into.batch, kThreads, st, a);
}

hipError_t launch_kv8_free(const Kv8& c, int32_t* refs, const int32_t* keep, hipStream_t st) {
    const FreeArgs a = {const_cast<int32_t*>(c.table), c.lengths, refs, keep, c.width, c.pages};
    return launch_threads(kv8_free_kernel, c.batch, kThreads, st, a);
}

hipError_t launch_kv8_reserve(const Kv8& c, int32_t* refs, const int32_t* tokens, int32_t* room, int32_t* source,
                              int32_t* target, hipStream_t st) {
    static_assert(kSequences == kKv8MaxSequences, "arrays");
    const ReserveArgs a = {const_cast<int32_t*>(c.table), refs, c.lengths, tokens, room, source, target, c.batch, c.width, c.pages};
    return c.batch <= 256 ? launch_threads(kv8_reserve_kernel<256>, 1, 256, st, a)
                          : launch_threads(kv8_reserve_kernel<1024>, 1, 1024, st, a);
}

hipError_t launch_kv8_compact(const Kv8& c, int32_t* refs, int32_t* source, int32_t* target, hipStream_t st) {
    const CompactArgs a = {const_cast<int32_t*>(c.table), refs, source, target, c.pages, (size_t)c.batch * c.width};
    hipError_t e = launch_threads(kv8_compact_kernel, 1, kScan, st, a);
    if (e == hipSuccess) e = launch_threads(kv8_remap_kernel, (uint32_t)((a.entries + kThreads - 1) / kThreads), kThreads, st, a);
    if (e == hipSuccess) e = launch_threads(kv8_settle_kernel, (a.pages / 2 + kThreads - 1) / kThreads, kThreads, st, a);
    return e;
}

hipError_t launch_kv8_copy(const Kv8& c, const Kv8& into, const int32_t* source, const int32_t* target, uint32_t count,
                           hipStream_t st) {
    CopyArgs a = {c.k, c.v, c.k_scales, c.v_scales, into.k, into.v, into.k_scales, into.v_scales, source, target,
                  count, c.pages, into.pages, c.heads, 0, 0};
    a.bytes = c.heads * kPage * (uint32_t)c.dim;
    a.pieces = 2 * ((a.bytes + kPiece - 1) / kPiece);
    const size_t units = (size_t)count * a.pieces;
    return launch_threads(kv8_copy_kernel, (uint32_t)std::min<size_t>(units, 4096), kThreads, st, a);
}

} // namespace qar
