// Pages shared between sequences: forking a sequence, copying the pages that
// a fork or a compaction names, releasing sequences that share pages, and
// closing up a fragmented pool.  Beside block_alloc.cu, whose pool state
// (block tables, lengths, free stack) these calls work on.
//
// extra_refs counts a block's owners beyond the first.  A block in use by one
// sequence, and a free one, has 0, so the allocator need not know of it.
// Only full pages are ever shared: a fork gives each child its own copy of
// the parent's unfinished page, so no append meets a shared page.
//
// Every result is the same on every run: entries are ranked by scans over
// the caller's order or over the block ids, never by the order in which
// atomics arrive.
#include <climits>

#include "xs_common.cuh"

namespace xs {
namespace {

constexpr int kShareThreads = 1024;

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

// One CTA.  A child slot named twice goes to the first entry that names it:
// the slot's length holds the lowest index of its claimants (INT_MIN + i)
// between the two passes.
__global__ void __launch_bounds__(kShareThreads)
    block_fork_kernel(const int32_t *__restrict__ parents, const int32_t *__restrict__ children,
                      int n, int32_t *tables, int max_blocks, int32_t *lens, int B, int bs,
                      const int32_t *__restrict__ free_stack, int32_t *free_top,
                      int32_t *extra_refs, int64_t num_blocks, int64_t *copies, int *err_flag) {
    __shared__ int sm[33];
    __shared__ int32_t row_from[kShareThreads], row_to[kShareThreads], row_len[kShareThreads],
        row_new[kShareThreads];
    auto usable = [&](int i, int &p, int &c, int &len) {
        p = parents[i], c = children[i];
        if (p < 0 || p >= B || c < 0 || c >= B) return false;
        len = *static_cast<volatile int32_t *>(lens + p);
        return len >= 0 && *static_cast<volatile int32_t *>(lens + c) < 0;
    };
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        int p, c, len;
        if (usable(i, p, c, len)) atomicMin(lens + c, INT_MIN + i);
    }
    __syncthreads();
    const int top = *free_top;
    int popped = 0;
    for (int base = 0; base < n; base += blockDim.x) {
        const int i = base + threadIdx.x;
        int p = -1, c = -1, len = 0;
        bool ok = false;
        if (i < n) {
            p = parents[i], c = children[i];
            ok = p >= 0 && p < B && c >= 0 && c < B;
            if (ok) {
                len = *static_cast<volatile int32_t *>(lens + p);
                ok = len >= 0 && *static_cast<volatile int32_t *>(lens + c) == INT_MIN + i;
            }
            if (!ok) raise_flag(err_flag, XS_FLAG_BAD_SLOT);
        }
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
            blk = free_stack[top - 1 - rank];
            src = tables[static_cast<int64_t>(p) * max_blocks + len / bs];
            if (src < 0 || src >= num_blocks || blk < 0 || blk >= num_blocks) {
                raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
                src = -1;
            }
        }
        if (i < n) {
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
            for (int col = lane; col < max_blocks; col += 32) {
                int32_t id = -1;
                if (col < full) {
                    id = from[col];
                    if (id >= 0 && id < num_blocks)
                        atomicAdd(extra_refs + id, 1);
                    else
                        raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
                } else if (col == full) {
                    id = row_new[k];
                }
                to[col] = id;
            }
        }
        __syncthreads();
        if (ok) lens[c] = fits ? len : -1;
        __syncthreads();
    }
    if (threadIdx.x == 0) *free_top = top - min(popped, top);
}

// One CTA.  A block whose count falls below zero is marked by that (-1) until
// the scan over the block ids has pushed it.
__global__ void __launch_bounds__(kShareThreads)
    block_release_kernel(const int32_t *__restrict__ seq_ids, int n, int32_t *tables,
                         int max_blocks, int32_t *lens, int B, int bs, int32_t *free_stack,
                         int32_t *free_top, int64_t capacity, int32_t *extra_refs,
                         int64_t num_blocks, int *err_flag) {
    __shared__ int sm[33];
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    for (int k = warp; k < n; k += warps) {
        const int b = seq_ids[k];
        if (b < 0 || b >= B) {
            if (lane == 0) raise_flag(err_flag, XS_FLAG_BAD_SLOT);
            continue;
        }
        int len = 0;
        if (lane == 0) len = atomicExch(lens + b, -1);  // a slot listed twice is released once
        len = __shfl_sync(0xffffffffu, len, 0);
        if (len < 0) continue;
        int32_t *row = tables + static_cast<int64_t>(b) * max_blocks;
        const int pages = pages_of(len, bs, max_blocks);
        for (int col = lane; col < max_blocks; col += 32) {
            if (col < pages) {
                const int32_t id = row[col];
                if (id >= 0 && id < num_blocks)
                    atomicSub(extra_refs + id, 1);
                else
                    raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
            }
            row[col] = -1;
        }
    }
    __syncthreads();
    // Highest id first, so that the lowest is the next one taken.
    int64_t at = *free_top;
    for (int64_t base = num_blocks; base > 0; base -= blockDim.x) {
        const int64_t id = base - 1 - threadIdx.x;
        const bool freed = id >= 0 && *static_cast<volatile int32_t *>(extra_refs + id) < 0;
        int count;
        const int64_t idx = at + block_scan(freed, &count, sm);
        if (freed) {
            extra_refs[id] = 0;
            if (idx < capacity)
                free_stack[idx] = static_cast<int32_t>(id);
            else
                raise_flag(err_flag, XS_FLAG_POOL_EMPTY);
        }
        at += count;
    }
    if (threadIdx.x == 0) *free_top = static_cast<int32_t>(min(at, capacity));
}

// One CTA.  remap first marks the live blocks (0), then holds the new ids.
__global__ void __launch_bounds__(kShareThreads)
    block_compact_kernel(const int32_t *tables, int32_t *tables_out, int max_blocks,
                         const int32_t *__restrict__ lens, int B, int bs, const int32_t *extra,
                         int32_t *extra_out, int32_t *free_stack, int32_t *free_top,
                         int64_t num_blocks, int32_t *remap, int64_t *moves, int32_t *n_moves,
                         int *err_flag) {
    __shared__ int sm[33];
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    for (int64_t id = threadIdx.x; id < num_blocks; id += blockDim.x) remap[id] = -1;
    __syncthreads();
    for (int b = warp; b < B; b += warps) {
        const int n = lens[b];
        if (n > 0 && (static_cast<int64_t>(n) + bs - 1) / bs > max_blocks && lane == 0)
            raise_flag(err_flag, XS_FLAG_BAD_LEN);
        const int pages = pages_of(n, bs, max_blocks);
        for (int col = lane; col < pages; col += 32) {
            const int32_t id = tables[static_cast<int64_t>(b) * max_blocks + col];
            if (id >= 0 && id < num_blocks)
                remap[id] = 0;
            else
                raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
        }
    }
    __syncthreads();
    int64_t live = 0;
    int count;
    for (int64_t base = 0; base < num_blocks; base += blockDim.x) {
        const int64_t id = base + threadIdx.x;
        block_scan(id < num_blocks && remap[id] == 0, &count, sm);
        live += count;
    }
    int64_t movers = 0, holes = 0;
    for (int64_t base = 0; base < num_blocks; base += blockDim.x) {
        const int64_t id = base + threadIdx.x;
        const bool in = id < num_blocks, used = in && remap[id] == 0;
        const bool mover = used && id >= live, hole = in && !used && id < live;
        int64_t k = movers + block_scan(mover, &count, sm);
        movers += count;
        if (mover) moves[2 * k] = id;
        k = holes + block_scan(hole, &count, sm);
        holes += count;
        if (hole) moves[2 * k + 1] = id;
    }
    __syncthreads();
    for (int64_t id = threadIdx.x; id < live; id += blockDim.x)
        if (remap[id] == 0) remap[id] = static_cast<int32_t>(id);
    for (int64_t k = threadIdx.x; k < num_blocks / 2; k += blockDim.x) {
        if (k < movers) {
            const int64_t src = moves[2 * k], dst = moves[2 * k + 1];
            remap[src] = static_cast<int32_t>(dst);
            extra_out[dst] = extra[src];
        } else {
            moves[2 * k] = moves[2 * k + 1] = -1;
        }
    }
    __syncthreads();
    for (int64_t id = threadIdx.x; id < num_blocks; id += blockDim.x) {
        if (id >= live)
            extra_out[id] = 0;
        else if (remap[id] >= 0)
            extra_out[id] = extra[id];
        if (id < num_blocks - live) free_stack[id] = static_cast<int32_t>(num_blocks - 1 - id);
    }
    for (int b = warp; b < B; b += warps) {
        const int pages = pages_of(lens[b], bs, max_blocks);
        for (int col = lane; col < max_blocks; col += 32) {
            const int64_t e = static_cast<int64_t>(b) * max_blocks + col;
            int32_t id = tables[e];
            if (col < pages && id >= 0 && id < num_blocks) id = remap[id];
            tables_out[e] = id;
        }
    }
    if (threadIdx.x == 0) {
        *free_top = static_cast<int32_t>(num_blocks - live);
        *n_moves = static_cast<int32_t>(movers);
    }
}

constexpr int kCopyThreads = 256, kCopyUnroll = 8;

// Items of kCopyThreads * kCopyUnroll 16-byte pieces of one (pair, layer, K or V).
__global__ void __launch_bounds__(kCopyThreads)
    block_copy_kernel(uint4 *k_pools, uint4 *v_pools, int layers, int64_t layer_chunks,
                      const int64_t *__restrict__ pairs, int64_t n,
                      const int32_t *__restrict__ count, int64_t block_chunks, int64_t num_blocks,
                      int *err_flag) {
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
    xs::block_fork_kernel<<<1, xs::kShareThreads, 0, stream>>>(
        parents, children, n, block_tables, max_blocks_per_seq, context_lens, B, block_size,
        free_stack, free_top, extra_refs, num_blocks, copies, err_flag);
    return xs::launch_status();
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
    xs::block_release_kernel<<<1, xs::kShareThreads, 0, stream>>>(
        seq_ids, n, block_tables, max_blocks_per_seq, context_lens, B, block_size, free_stack,
        free_top, stack_capacity, extra_refs, num_blocks, err_flag);
    return xs::launch_status();
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
    xs::block_compact_kernel<<<1, xs::kShareThreads, 0, stream>>>(
        block_tables, block_tables_out, max_blocks_per_seq, context_lens, B, block_size,
        extra_refs, extra_refs_out, free_stack, free_top, num_blocks, remap, moves, n_moves,
        err_flag);
    return xs::launch_status();
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
    const int grid = static_cast<int>(n < most / per_pair + 1 ? n * per_pair < most ? n * per_pair : most : most);
    xs::block_copy_kernel<<<grid, xs::kCopyThreads, 0, stream>>>(
        static_cast<uint4 *>(k_pools), static_cast<uint4 *>(v_pools), layers,
        layer_stride_bytes / 16, pairs, n, count, chunks, num_blocks, err_flag);
    return xs::launch_status();
}
