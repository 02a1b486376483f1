// Pages shared between sequences: forking a sequence, copying the pages that
// a fork or a compaction names, releasing sequences that share pages, and
// closing up a fragmented pool.  Beside block_alloc.cu, whose pool state
// (block tables, lengths, free stack) these calls work on.
//
// extra_refs counts a block's owners beyond the first.  A block in use by one
// sequence, and a free one, has 0, so the allocator need not know of it.
// A fork shares full pages alone: it gives each child its own copy of the parent's
// unfinished page.  A shared page becomes unfinished only where a truncation ends in
// it; before the next append the sequence is forked once more, and its slot released.
//
// Every result is the same on every run: entries are ranked by scans over
// the caller's order or over the block ids, never by the order in which
// atomics arrive.
//
// The integer work is a few kilobytes to a few megabytes and bound by latency:
// one launch each, whose phases are separated by barriers of one thread-block
// cluster (a single CTA for a small pool).  Releasing and compacting rank the
// block ids: each CTA of the cluster has a contiguous part of them, each warp
// of it a contiguous part of that, which it counts, then (after the counts
// have met in shared memory, across the cluster) writes in order.  Both so take
// time in proportion to the pool: releasing 64 sequences of 1K tokens 5 us in a pool
// of 4K blocks, 6 us of 32K, 18 us of 262,144; a compaction's plan 14, 18 and 48 us.
#include <climits>

#include <cooperative_groups.h>

#include "xs_common.cuh"

namespace xs {
namespace {

namespace cg = cooperative_groups;

constexpr int kShareThreads = 1024;
constexpr int kShareWarps = kShareThreads / 32;
constexpr int kShareCluster = 8;
constexpr int64_t kShareSmall = 4096;   // block ids, and table entries, of a single CTA
constexpr int32_t kGivenBack = -1;      // in a sequence's row: its page was given back before

// One warp's part [lo, hi) of [0, n), cut over the cluster's CTAs and warps.
struct Part {
    int64_t lo, hi;
};
__device__ __forceinline__ Part warp_part(int64_t n, int rank, int ranks) {
    const int warps = blockDim.x >> 5;
    const int64_t w = static_cast<int64_t>(rank) * warps + (threadIdx.x >> 5);
    const int64_t all = static_cast<int64_t>(ranks) * warps;
    const int64_t per = ((n + all - 1) / all + 31) / 32 * 32;
    return Part{min(w * per, n), min(w * per + per, n)};
}

// How many of the warp's part satisfy pred; every lane gets the count.
template <typename F> __device__ __forceinline__ int count_part(const Part &part, F &&pred) {
    const int lane = threadIdx.x & 31;
    int count = 0;
#pragma unroll 4
    for (int64_t i = part.lo; i < part.hi; i += 32)
        count += __popc(__ballot_sync(0xffffffffu, i + lane < part.hi && pred(i + lane)));
    return count;
}
// put(k, i) for the k-th (from `at` on) element i of the part that satisfies pred.
template <typename F, typename P>
__device__ __forceinline__ void write_part(const Part &part, int64_t at, F &&pred, P &&put) {
    const int lane = threadIdx.x & 31;
#pragma unroll 4
    for (int64_t i = part.lo; i < part.hi; i += 32) {
        const bool yes = i + lane < part.hi && pred(i + lane);
        const uint32_t all = __ballot_sync(0xffffffffu, yes);
        if (yes) put(at + __popc(all & ((1u << lane) - 1)), i + lane);
        at += __popc(all);
    }
}

// Counts of every warp of the cluster, in order.
struct ShareCounts {
    int of[kShareCluster * kShareWarps];
};
// The sum before this warp, and of all; `mine` alike in the warp's lanes.
// Synchronises the cluster.
__device__ __forceinline__ int64_t cluster_scan(cg::cluster_group &cluster, ShareCounts &counts,
                                                int mine, int64_t *total) {
    const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    const int me = rank * warps + (threadIdx.x >> 5);
    if (ranks == 1) {
        if (lane == 0) counts.of[me] = mine;
        __syncthreads();
    } else {
        if (lane < ranks) cluster.map_shared_rank(&counts, lane)->of[me] = mine;
        cluster.sync();
    }
    // Block ids, so also their counts, fit 31 bits.
    int before = 0, all = 0;
    for (int i = lane; i < ranks * warps; i += 32) {
        const int v = counts.of[i];
        all += v;
        if (i < me) before += v;
    }
    *total = __reduce_add_sync(0xffffffffu, all);
    return __reduce_add_sync(0xffffffffu, before);
}
// All threads of the launch, and what they wrote.
__device__ __forceinline__ void launch_sync(cg::cluster_group &cluster) {
    if (cluster.num_blocks() == 1)
        __syncthreads();
    else
        cluster.sync();
}

// Exclusive sum of v over the block's threads; `total` gets the sum.
__device__ __forceinline__ int block_scan(int v, int *total, int *sm /* 33 ints */) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
    }
    __syncthreads();
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const int own = lane < static_cast<int>(blockDim.x >> 5) ? sm[lane] : 0;
        int w = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += y;
        }
        sm[lane] = w - own;
        if (lane == 31) sm[32] = w;
    }
    __syncthreads();
    *total = sm[32];
    return sm[warp] + inc - v;
}

__device__ __forceinline__ int pages_of(int n, int bs, int max_blocks) {
    return n > 0 ? static_cast<int>(min((static_cast<int64_t>(n) + bs - 1) / bs,
                                        static_cast<int64_t>(max_blocks)))
                 : 0;
}

// One CTA.  A child slot named twice goes to the first entry that may have it.
// Up to kForkDirect entries are compared with one another in shared memory; of
// more, a slot's length holds the lowest index of its claimants (INT_MIN + i)
// between two passes, at the cost of two more trips to memory.
constexpr int kForkDirect = 256;
__global__ void __launch_bounds__(kShareThreads)
    block_fork_kernel(const int32_t *__restrict__ parents, const int32_t *__restrict__ children,
                      int n, int32_t *tables, int max_blocks, int32_t *lens, int B, int bs,
                      const int32_t *__restrict__ free_stack, int32_t *free_top,
                      int32_t *extra_refs, int64_t num_blocks, int64_t *copies, int *err_flag) {
    after_previous();
    __shared__ int sm[33];
    __shared__ int32_t row_from[kShareThreads], row_to[kShareThreads], row_len[kShareThreads],
        row_new[kShareThreads];
    auto length = [&](int b) { return *static_cast<volatile int32_t *>(lens + b); };
    auto usable = [&](int i, int &p, int &c, int &len) {
        if (!XS_BOUNDS(i >= 0 && i < n, err_flag)) return false;
        p = parents[i], c = children[i];
        if (p < 0 || p >= B || c < 0 || c >= B) return false;
        len = length(p);
        return len >= 0 && length(c) < 0;
    };
    const bool direct = n <= kForkDirect && n <= static_cast<int>(blockDim.x);
    if (!direct) {
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            int p, c, len;
            if (usable(i, p, c, len)) atomicMin(lens + c, INT_MIN + i);
        }
        __syncthreads();
    }
    const int top = *free_top;
    int popped = 0;
    for (int base = 0; base < n; base += blockDim.x) {
        const int i = base + threadIdx.x;
        int p = -1, c = -1, len = 0;
        bool ok = false;
        if (i < n) {
            if (direct) {
                ok = usable(i, p, c, len);
            } else {
                p = parents[i], c = children[i];
                ok = p >= 0 && p < B && c >= 0 && c < B;
                if (ok) {
                    len = length(p);
                    ok = len >= 0 && length(c) == INT_MIN + i;
                }
            }
        }
        if (direct) {
            row_to[threadIdx.x] = ok ? c : -1;
            __syncthreads();
            for (int k = 0; ok && k < i; ++k) ok = row_to[k] != c;
        }
        if (i < n && !ok) raise_flag(err_flag, XS_FLAG_BAD_SLOT);
        bool fits = ok;
        if (ok && (static_cast<int64_t>(len) + bs - 1) / bs > max_blocks) {
            raise_flag(err_flag, XS_FLAG_BAD_LEN);
            fits = false;
        }
        const bool tail = fits && len % bs != 0;
        int count;
        const int rank = popped + block_scan(tail, &count, sm);
        popped += count;
        if (tail && rank >= top) {
            raise_flag(err_flag, XS_FLAG_POOL_EMPTY);
            fits = false;
        }
        int32_t blk = -1;
        int64_t src = -1;
        if (tail && fits) {
            const int at = top - 1 - rank;      // a stack holds a block at most once
            if (XS_BOUNDS(at >= 0 && at < num_blocks, err_flag)) blk = free_stack[at];
            if (XS_BOUNDS(p >= 0 && p < B && len / bs < max_blocks, err_flag))
                src = tables[static_cast<int64_t>(p) * max_blocks + len / bs];
            if (src < 0 || src >= num_blocks || blk < 0 || blk >= num_blocks) {
                raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
                src = -1;
            }
        }
        if (i < n && XS_BOUNDS(i >= 0, err_flag)) {
            copies[2 * static_cast<int64_t>(i)] = src;
            copies[2 * static_cast<int64_t>(i) + 1] = src < 0 ? -1 : blk;
        }
        row_from[threadIdx.x] = p;
        row_to[threadIdx.x] = fits ? c : -1;
        row_len[threadIdx.x] = len;
        row_new[threadIdx.x] = blk;
        __syncthreads();
        const int rows = min(n - base, static_cast<int>(blockDim.x));
        const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        for (int k = warp; k < rows; k += warps) {
            if (row_to[k] < 0) continue;
            const int32_t *from = tables + static_cast<int64_t>(row_from[k]) * max_blocks;
            int32_t *to = tables + static_cast<int64_t>(row_to[k]) * max_blocks;
            const int full = row_len[k] / bs;
            if (!XS_BOUNDS(row_from[k] >= 0 && row_from[k] < B && row_to[k] < B && full <= max_blocks,
                           err_flag))
                continue;
#pragma unroll 4
            for (int col = lane; col < max_blocks; col += 32) {
                int32_t id = -1;
                if (col < full) {
                    id = from[col];
                    if (id >= 0 && id < num_blocks)
                        atomicAdd(extra_refs + id, 1);
                    else if (id != kGivenBack)
                        raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
                } else if (col == full) {
                    id = row_new[k];
                }
                to[col] = id;
            }
        }
        __syncthreads();
        if (ok && XS_BOUNDS(c >= 0 && c < B, err_flag)) lens[c] = fits ? len : -1;
        __syncthreads();
    }
    if (threadIdx.x == 0) *free_top = top - min(popped, top);
}

// The blocks whose count fell below zero go on the free stack, the highest id
// first, so that the lowest is the next one taken; their counts become 0.
__device__ __forceinline__ void push_freed(cg::cluster_group &cluster, ShareCounts &counts,
                                           int32_t *free_stack, int64_t top, int32_t *free_top,
                                           int64_t capacity, int32_t *extra_refs, int64_t num_blocks,
                                           int *err_flag) {
    const int rank = cluster.block_rank(), ranks = cluster.num_blocks(), lane = threadIdx.x & 31;
    const Part part = warp_part(num_blocks, rank, ranks);
    // 1,024 ids at a time: lane i has the bits of 32 of them from its 32 i on, so that most
    // pools are read once (twice: 200,000 blocks 5 us more).
    constexpr int kLook = 1024, kAtOnce = 8;
    uint32_t bits;
    auto look = [&](int64_t base) {
        bits = 0;
        for (int c = 0; c < kLook / 32 && base + 32 * c < part.hi; c += kAtOnce) {
            bool freed[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int64_t i = base + 32 * (c + u) + lane;
                freed[u] = i < part.hi && __ldcg(extra_refs + (num_blocks - 1 - i)) < 0;
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const uint32_t all = __ballot_sync(0xffffffffu, freed[u]);
                if (lane == c + u) bits = all;
            }
        }
    };
    int mine = 0;
    for (int64_t base = part.lo; base < part.hi; base += kLook) {
        look(base);
        mine += __popc(bits);
    }
    int64_t total;
    int64_t at = top + cluster_scan(cluster, counts, __reduce_add_sync(0xffffffffu, mine), &total);
    for (int64_t base = part.lo; base < part.hi; base += kLook) {
        if (part.hi - part.lo > kLook) look(base);      // (else they are still there)
        for (uint32_t some = __ballot_sync(0xffffffffu, bits != 0); some; some &= some - 1) {
            const int from = __ffs(some) - 1;
            const uint32_t all = __shfl_sync(0xffffffffu, bits, from);
            const int64_t id = num_blocks - 1 - (base + 32 * from + lane);
            const int64_t k = at + __popc(all & ((1u << lane) - 1));
            at += __popc(all);
            if (!(all >> lane & 1) || !XS_BOUNDS(k >= 0 && id >= 0 && id < num_blocks, err_flag)) continue;
            if (k < capacity)
                free_stack[k] = static_cast<int32_t>(id);
            else
                raise_flag(err_flag, XS_FLAG_POOL_EMPTY);
            extra_refs[id] = 0;
        }
    }
    if (rank == 0 && threadIdx.x == 0) *free_top = static_cast<int32_t>(min(top + total, capacity));
}

// A block whose count falls below zero is marked by that until the scan over
// the block ids has pushed it.
__global__ void __launch_bounds__(kShareThreads)
    block_release_kernel(const int32_t *__restrict__ seq_ids, int n, int32_t *tables,
                         int max_blocks, int32_t *lens, int B, int bs, int32_t *free_stack,
                         int32_t *free_top, int64_t capacity, int32_t *extra_refs,
                         int64_t num_blocks, int *err_flag) {
    after_previous();
    __shared__ ShareCounts counts;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t top = *free_top;
    for (int k = rank + warp * ranks; k < n; k += ranks * static_cast<int>(blockDim.x >> 5)) {
        const int b = seq_ids[k];
        if (b < 0 || b >= B) {
            if (lane == 0) raise_flag(err_flag, XS_FLAG_BAD_SLOT);
            continue;
        }
        int32_t *row = tables + static_cast<int64_t>(b) * max_blocks;
        int len = 0;
        if (lane == 0) len = atomicExch(lens + b, -1);  // a slot listed twice is released once
        int32_t early[4];       // the row's first entries, while the length comes
#pragma unroll
        for (int u = 0; u < 4; ++u) early[u] = 32 * u + lane < max_blocks ? row[32 * u + lane] : -1;
        len = __shfl_sync(0xffffffffu, len, 0);
        if (len < 0) continue;
        const int pages = pages_of(len, bs, max_blocks);
        auto drop = [&](int col, int32_t id) {
            if (col < pages) {
                if (id >= 0 && id < num_blocks)
                    atomicSub(extra_refs + id, 1);
                else if (id != kGivenBack)
                    raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
            }
            if (XS_BOUNDS(col >= 0 && col < max_blocks, err_flag)) row[col] = -1;
        };
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (32 * u + lane < max_blocks) drop(32 * u + lane, early[u]);
#pragma unroll 4
        for (int col = 128 + lane; col < max_blocks; col += 32) drop(col, row[col]);
    }
    launch_sync(cluster);
    push_freed(cluster, counts, free_stack, top, free_top, capacity, extra_refs, num_blocks, err_flag);
}

// Gives back the pages behind a new length: like a release of these alone.
__global__ void __launch_bounds__(kShareThreads)
    block_truncate_kernel(const int32_t *__restrict__ seq_ids, const int32_t *__restrict__ new_lens,
                          int n, int32_t *tables, int max_blocks, int32_t *lens, int B, int bs,
                          int32_t *free_stack, int32_t *free_top, int64_t capacity,
                          int32_t *extra_refs, int64_t num_blocks, int *err_flag) {
    after_previous();
    __shared__ ShareCounts counts;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t top = *free_top;
    for (int k = rank + warp * ranks; k < n; k += ranks * static_cast<int>(blockDim.x >> 5)) {
        const int b = seq_ids[k], to = new_lens[k];
        // An entry of a slot that an earlier one has is not done.
        bool again = false;
        for (int i = lane; i < k; i += 32) again |= seq_ids[i] == b;
        if (__any_sync(0xffffffffu, again) || b < 0 || b >= B) {
            if (lane == 0) raise_flag(err_flag, XS_FLAG_BAD_SLOT);
            continue;
        }
        const int len = lens[b];
        if (to < 0 || to >= len) continue;
        int32_t *row = tables + static_cast<int64_t>(b) * max_blocks;
        const int pages = pages_of(len, bs, max_blocks);
        // (Read before any is written: one after another, 320 entries took 3 us more.)
        constexpr int kAtOnce = 8;
        for (int col0 = pages_of(to, bs, max_blocks) + lane; col0 - lane < pages; col0 += 32 * kAtOnce) {
            int32_t id[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) id[u] = col0 + 32 * u < pages ? row[col0 + 32 * u] : -1;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int col = col0 + 32 * u;
                if (col >= pages) continue;
                if (id[u] >= 0 && id[u] < num_blocks)
                    atomicSub(extra_refs + id[u], 1);
                else if (id[u] != kGivenBack)
                    raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
                if (XS_BOUNDS(col >= 0 && col < max_blocks, err_flag)) row[col] = -1;
            }
        }
        __syncwarp();
        if (lane == 0 && XS_BOUNDS(b >= 0 && b < B, err_flag)) lens[b] = to;
    }
    launch_sync(cluster);
    push_freed(cluster, counts, free_stack, top, free_top, capacity, extra_refs, num_blocks, err_flag);
}

// remap first marks the live blocks (0), then holds the new ids.
__global__ void __launch_bounds__(kShareThreads)
    block_compact_kernel(const int32_t *tables, int32_t *tables_out, int max_blocks,
                         const int32_t *__restrict__ lens, int B, int bs, const int32_t *extra,
                         int32_t *extra_out, int32_t *free_stack, int32_t *free_top,
                         int64_t num_blocks, int32_t *remap, int64_t *moves, int32_t *n_moves,
                         int *err_flag) {
    after_previous();
    __shared__ ShareCounts counts[3];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
    const int64_t thread = static_cast<int64_t>(rank) * blockDim.x + threadIdx.x;
    const int64_t threads = static_cast<int64_t>(ranks) * blockDim.x;
    const int64_t warp = thread >> 5, warps = threads >> 5;
    const int lane = threadIdx.x & 31;
    for (int64_t id = thread; id < num_blocks; id += threads) remap[id] = -1;
    launch_sync(cluster);
    // A warp takes 128 columns of a row at a time.
    const int pieces = (max_blocks + 127) / 128;
    for (int64_t piece = warp; piece < static_cast<int64_t>(B) * pieces; piece += warps) {
        const int b = static_cast<int>(piece / pieces), col0 = static_cast<int>(piece % pieces) * 128;
        const int n = lens[b];
        if (col0 == 0 && n > 0 && (static_cast<int64_t>(n) + bs - 1) / bs > max_blocks && lane == 0)
            raise_flag(err_flag, XS_FLAG_BAD_LEN);
        const int pages = pages_of(n, bs, max_blocks);
        int32_t id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = col0 + 32 * u + lane;
            id[u] = col < pages ? tables[static_cast<int64_t>(b) * max_blocks + col] : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (col0 + 32 * u + lane >= pages) continue;
            if (!XS_BOUNDS(b < B && col0 + 32 * u + lane < max_blocks, err_flag)) continue;
            if (id[u] >= 0 && id[u] < num_blocks)
                remap[id[u]] = 0;
            else if (id[u] != kGivenBack)
                raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
        }
    }
    launch_sync(cluster);
    const Part part = warp_part(num_blocks, rank, ranks);
    auto used = [&](int64_t id) { return __ldcg(remap + id) == 0; };
    int64_t live, movers, holes;
    cluster_scan(cluster, counts[0], count_part(part, used), &live);
    auto mover = [&](int64_t id) { return id >= live && used(id); };
    auto hole = [&](int64_t id) { return id < live && !used(id); };
    const int64_t m0 = cluster_scan(cluster, counts[1], count_part(part, mover), &movers);
    const int64_t h0 = cluster_scan(cluster, counts[2], count_part(part, hole), &holes);
    auto in_moves = [&](int64_t k) { return XS_BOUNDS(k >= 0 && k < num_blocks / 2, err_flag); };
    write_part(part, m0, mover, [&](int64_t k, int64_t id) {
        if (in_moves(k)) moves[2 * k] = id;
    });
    write_part(part, h0, hole, [&](int64_t k, int64_t id) {
        if (in_moves(k)) moves[2 * k + 1] = id;
    });
    launch_sync(cluster);
    for (int64_t id = thread; id < live; id += threads)
        if (__ldcg(remap + id) == 0) remap[id] = static_cast<int32_t>(id);
    for (int64_t k = thread; k < num_blocks / 2; k += threads) {
        if (k < movers) {
            const int64_t src = __ldcg(moves + 2 * k), dst = __ldcg(moves + 2 * k + 1);
            if (!XS_BOUNDS(src >= live && src < num_blocks && dst >= 0 && dst < live, err_flag)) continue;
            remap[src] = static_cast<int32_t>(dst);
            extra_out[dst] = extra[src];
        } else {
            moves[2 * k] = moves[2 * k + 1] = -1;
        }
    }
    launch_sync(cluster);
    for (int64_t id = thread; id < num_blocks; id += threads) {
        if (id >= live)
            extra_out[id] = 0;
        else if (__ldcg(remap + id) == id)      // (a hole's came with its mover)
            extra_out[id] = extra[id];
        if (id < num_blocks - live && XS_BOUNDS(live >= 0, err_flag))
            free_stack[id] = static_cast<int32_t>(num_blocks - 1 - id);
    }
    for (int64_t piece = warp; piece < static_cast<int64_t>(B) * pieces; piece += warps) {
        const int b = static_cast<int>(piece / pieces), col0 = static_cast<int>(piece % pieces) * 128;
        const int pages = pages_of(lens[b], bs, max_blocks);
        int32_t id[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = col0 + 32 * u + lane;
            id[u] = col < max_blocks ? tables[static_cast<int64_t>(b) * max_blocks + col] : 0;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = col0 + 32 * u + lane;
            if (col < pages && id[u] >= 0 && id[u] < num_blocks) id[u] = __ldcg(remap + id[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = col0 + 32 * u + lane;
            if (col < max_blocks && XS_BOUNDS(b >= 0 && b < B, err_flag))
                tables_out[static_cast<int64_t>(b) * max_blocks + col] = id[u];
        }
    }
    if (thread == 0) {
        *free_top = static_cast<int32_t>(num_blocks - live);
        *n_moves = static_cast<int32_t>(movers);
    }
}

// Launches `kernel` as one cluster, or as a single CTA if the work is small
// (a cluster's barriers cost more than it saves: releasing 4 sequences of a
// pool of 100 blocks takes 3.5 us as a CTA of 8 warps, 6 us as a cluster; at
// 8K blocks and 33K table entries compacting takes 31 us as one CTA, 16 us as
// a cluster).
template <typename K, typename... A>
int launch_share(K kernel, int64_t work, cudaStream_t stream, A... args) {
    const int ctas = work <= kShareSmall ? 1 : kShareCluster;
    return launch_after(kernel, dim3(ctas), work <= kShareSmall / 4 ? kShareThreads / 4 : kShareThreads,
                        0, stream, ctas, args...);
}

constexpr int kCopyThreads = 256, kCopyUnroll = 8;

// Items of kCopyThreads * kCopyUnroll 16-byte pieces of one (pair, layer, K or V).
__global__ void __launch_bounds__(kCopyThreads)
    block_copy_kernel(uint4 *k_pools, uint4 *v_pools, int layers, int64_t layer_chunks,
                      const int64_t *__restrict__ pairs, int64_t n,
                      const int32_t *__restrict__ count, int64_t block_chunks, int64_t num_blocks,
                      int *err_flag) {
    after_previous();
    constexpr int64_t kPiece = kCopyThreads * kCopyUnroll;
    if (count) n = min(n, max(static_cast<int64_t>(*count), int64_t(0)));
    const int64_t pieces = (block_chunks + kPiece - 1) / kPiece;
    const int64_t per_pair = pieces * layers * 2;
    for (int64_t item = blockIdx.x; item < n * per_pair; item += gridDim.x) {
        const int64_t pair = item / per_pair, rest = item - pair * per_pair;
        const int64_t lv = rest / pieces, piece = rest - lv * pieces;
        const int64_t s = pairs[2 * pair], d = pairs[2 * pair + 1];
        if (s < 0 || d < 0) continue;
        if (s >= num_blocks || d >= num_blocks) {
            if (rest == 0 && threadIdx.x == 0) raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
            continue;
        }
        if (!XS_BOUNDS(pair < n && (lv >> 1) < layers && piece < pieces &&
                           (layers == 1 || num_blocks * block_chunks <= layer_chunks), err_flag))
            continue;
        uint4 *pool = ((lv & 1) ? v_pools : k_pools) + (lv >> 1) * layer_chunks;
        const uint4 *from = pool + s * block_chunks;
        uint4 *to = pool + d * block_chunks;
        uint4 x[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            const int64_t c = piece * kPiece + u * kCopyThreads + threadIdx.x;
            if (c < block_chunks) x[u] = from[c];
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            const int64_t c = piece * kPiece + u * kCopyThreads + threadIdx.x;
            if (c < block_chunks) to[c] = x[u];
        }
    }
}

}  // namespace
XS_DEFINE_BOUNDS_COUNTER(bounds_failures_share)

}  // namespace xs

extern "C" int xs_block_fork(const int32_t *parents, const int32_t *children, int n,
                             int32_t *block_tables, int max_blocks_per_seq, int32_t *context_lens,
                             int B, int block_size, const int32_t *free_stack, int32_t *free_top,
                             int32_t *extra_refs, int64_t num_blocks, int64_t *copies,
                             int *err_flag, cudaStream_t stream) {
    if (!parents || !children || !block_tables || !context_lens || !free_stack || !free_top ||
        !extra_refs || !copies)
        return XS_ENULL;
    if (n < 0 || B < 0 || max_blocks_per_seq < 0 || block_size <= 0 || num_blocks < 0 ||
        num_blocks > INT_MAX)
        return XS_ESHAPE;
    if (n == 0) return XS_OK;
    const int threads = n <= 8 ? xs::kShareThreads / 4 : xs::kShareThreads;
    return xs::launch_after(xs::block_fork_kernel, dim3(1), threads, 0, stream, 1, parents, children,
                            n, block_tables, max_blocks_per_seq, context_lens, B, block_size,
                            free_stack, free_top, extra_refs, num_blocks, copies, err_flag);
}

extern "C" int xs_block_release(const int32_t *seq_ids, int n, int32_t *block_tables,
                                int max_blocks_per_seq, int32_t *context_lens, int B,
                                int block_size, int32_t *free_stack, int32_t *free_top,
                                int64_t stack_capacity, int32_t *extra_refs, int64_t num_blocks,
                                int *err_flag, cudaStream_t stream) {
    if (!seq_ids || !block_tables || !context_lens || !free_stack || !free_top || !extra_refs)
        return XS_ENULL;
    if (n < 0 || B < 0 || max_blocks_per_seq < 0 || block_size <= 0 || stack_capacity < 0 ||
        num_blocks < 0 || num_blocks > INT_MAX)
        return XS_ESHAPE;
    if (n == 0) return XS_OK;
    const int64_t entries = static_cast<int64_t>(n) * max_blocks_per_seq;
    return xs::launch_share(xs::block_release_kernel, num_blocks > entries ? num_blocks : entries,
                            stream, seq_ids, n, block_tables, max_blocks_per_seq, context_lens, B,
                            block_size, free_stack, free_top, stack_capacity, extra_refs,
                            num_blocks, err_flag);
}

extern "C" int xs_block_truncate(const int32_t *seq_ids, const int32_t *new_lens, int n,
                                 int32_t *block_tables, int max_blocks_per_seq,
                                 int32_t *context_lens, int B, int block_size, int32_t *free_stack,
                                 int32_t *free_top, int64_t stack_capacity, int32_t *extra_refs,
                                 int64_t num_blocks, int *err_flag, cudaStream_t stream) {
    if (!seq_ids || !new_lens || !block_tables || !context_lens || !free_stack || !free_top ||
        !extra_refs)
        return XS_ENULL;
    if (n < 0 || B < 0 || max_blocks_per_seq < 0 || block_size <= 0 || stack_capacity < 0 ||
        num_blocks < 0 || num_blocks > INT_MAX)
        return XS_ESHAPE;
    if (n == 0) return XS_OK;
    const int64_t entries = static_cast<int64_t>(n) * max_blocks_per_seq;
    return xs::launch_share(xs::block_truncate_kernel, num_blocks > entries ? num_blocks : entries,
                            stream, seq_ids, new_lens, n, block_tables, max_blocks_per_seq,
                            context_lens, B, block_size, free_stack, free_top, stack_capacity,
                            extra_refs, num_blocks, err_flag);
}

extern "C" int xs_block_compact(const int32_t *block_tables, int32_t *block_tables_out,
                                int max_blocks_per_seq, const int32_t *context_lens, int B,
                                int block_size, const int32_t *extra_refs, int32_t *extra_refs_out,
                                int32_t *free_stack, int32_t *free_top, int64_t num_blocks,
                                int32_t *remap, int64_t *moves, int32_t *n_moves, int *err_flag,
                                cudaStream_t stream) {
    if (!block_tables || !block_tables_out || !context_lens || !extra_refs || !extra_refs_out ||
        !free_stack || !free_top || !remap || (!moves && num_blocks > 1) || !n_moves)
        return XS_ENULL;
    if (B < 0 || max_blocks_per_seq < 0 || block_size <= 0 || num_blocks < 0 ||
        num_blocks > INT_MAX)
        return XS_ESHAPE;
    const int64_t entries = static_cast<int64_t>(B) * max_blocks_per_seq;
    return xs::launch_share(xs::block_compact_kernel, num_blocks > entries ? num_blocks : entries,
                            stream, block_tables, block_tables_out, max_blocks_per_seq,
                            context_lens, B, block_size, extra_refs, extra_refs_out, free_stack,
                            free_top, num_blocks, remap, moves, n_moves, err_flag);
}

extern "C" int xs_block_copy(void *k_pools, void *v_pools, int layers, int64_t layer_stride_bytes,
                             const int64_t *pairs, int64_t n, const int32_t *count,
                             int64_t block_bytes, int64_t num_blocks, int *err_flag,
                             cudaStream_t stream) {
    if (!k_pools || !v_pools || !pairs) return XS_ENULL;
    if (layers < 0 || n < 0 || block_bytes <= 0 || num_blocks < 0 ||
        num_blocks > INT64_MAX / block_bytes ||
        (layers > 1 && layer_stride_bytes < num_blocks * block_bytes))
        return XS_ESHAPE;
    if (block_bytes % 16 != 0 || layer_stride_bytes % 16 != 0) return XS_EUNSUPPORTED;
    if (!xs::aligned16(k_pools) || !xs::aligned16(v_pools)) return XS_EALIGN;
    if (n == 0 || layers == 0) return XS_OK;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return XS_EDEVICE;
    const int64_t chunks = block_bytes / 16;
    const int64_t piece = static_cast<int64_t>(xs::kCopyThreads) * xs::kCopyUnroll;
    const int64_t per_pair = (chunks + piece - 1) / piece * layers * 2;
    const int64_t most = static_cast<int64_t>(sms) * 8;
    int64_t grid = most;
    if (n <= most / per_pair && n * per_pair < most) grid = n * per_pair;
    return xs::launch_after(xs::block_copy_kernel, dim3(static_cast<int>(grid)), xs::kCopyThreads, 0,
                            stream, 1, static_cast<uint4 *>(k_pools), static_cast<uint4 *>(v_pools),
                            layers, layer_stride_bytes / 16, pairs, n, count, chunks, num_blocks,
                            err_flag);
}
