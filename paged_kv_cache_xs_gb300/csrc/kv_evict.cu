// Eviction from a paged cache by accumulated attention weight: sequences longer
// than a limit are cut to a budget of tokens, in every layer and for every KV
// head by itself: the first ones, the last ones and, of those between, the ones
// of largest score (of equal ones the earlier).  What is kept moves together to
// the sequence's first pages, in order.
//
// Two launches.  The first ranks: a CTA for each (layer, sequence, KV head), or a
// cluster of kRankCtas where tables are long, finds the score that is the last to
// be kept by radix selection on the scores' bits, 11, 11 and 10 of them at a time,
// counted in shared memory (11 bits: sign, exponent and two more, so that scores
// of one magnitude spread over bins), and writes the kept positions.  Each CTA of
// a cluster counts a contiguous part of the positions and adds the bins that it
// has met to those of all the others.  The scores stay in shared memory for the
// passes.  Each warp counts, then writes, a contiguous part, so there are no
// barriers within a pass and the order of atomics decides nothing.  What is kept
// is found once, as bits, a lane for 32 positions, and written from these (looked
// for again at the writing: 2 to 9 us more).
//
// The second moves rows, in place.  Position j takes the row of position
// kept[j] >= j, so a CTA that goes through j upwards and reads a tile before it
// writes one overwrites nothing that is still to be read, and may have the tile
// after it under way.  CTAs share a (layer, sequence, KV head) by K, V and slices
// of the rows' bytes, never by tokens.  Rows that stay where they are (the first
// tokens) are neither read nor written.
//
// What bounds it: the move its bytes (48 sequences cut to 2K tokens in 4 layers, 3.2 GB
// read and written: 497 us of the call's 532, 6.5 TB/s; rows of 256 bytes at
// random places), the ranking the instructions and latencies of its passes (a
// call that moves nothing takes 29 us there, and 15 for one sequence of 32K, whose
// whole call takes 38).
#include <atomic>
#include <climits>

#include "xs_common.cuh"

namespace xs {
namespace {

constexpr int kPage = 16;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;      // 16-byte pieces of a thread in a tile
constexpr int kLongTokens = 4096;   // of a table: beyond, a cluster ranks
// (Eviction of one sequence of 32K tokens in 4 layers, us: clusters of 4 CTAs of 512
// threads 47, of 4 of 1024 48, of 8 of 256 54, of 8 of 1024 58, one CTA of 1024 67.)
constexpr int kRankCtas = 4, kRankThreads = 512;
constexpr int kScoresHeld = 40960;  // of a CTA, in shared memory; of more, they are read again for each pass

struct EvictParams {
    const int32_t *seq_ids;
    int n;
    char *k_pools, *v_pools;
    int64_t layer_bytes;        // between two layers' pools
    float *scores;              // [layers, B, Hkv, max_blocks * 16]
    const int32_t *tables, *lens, *extra;
    int max_blocks, B, Hkv, layers, row_bytes;
    int64_t num_blocks;
    int first, recent, budget, limit;
    int held;                   // scores that a CTA's shared memory has room for
    int32_t *kept, *new_lens;
    int *err_flag;
};

// Larger for a larger score; NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
    if ((bits & 0x7fffffffu) > 0x7f800000u) bits = 0xff800000u;
    if (bits == 0x80000000u) bits = 0;
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
}

// Sum of v over the block's threads before this one; `total`: over all.
template <int kThreads> __device__ __forceinline__ int scan_threads(int v, int *sm, int *total) {
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
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before = all;
        all += sm[w];
    }
    *total = all;
    return before + inc - v;
}

// The threads of the launch's cluster (kCtas 1: of the CTA), and what they wrote.
template <int kCtas> __device__ __forceinline__ void all_sync() {
    if (kCtas == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void *own, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(own)), "r"(rank));
    return a;
}

template <int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
    after_previous();
    extern __shared__ uint32_t held[];      // the keys of this CTA's part of the scores, where they fit
    // The CTA's counts, and of all the candidates for each pass.
    __shared__ int hist[kBins], all_hist[kCtas > 1 ? 3 : 1][kCtas > 1 ? kBins : 1];
    __shared__ int sm[kThreads / 32], bin, left, counts[2];
    __shared__ int2 tally[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x % kCtas;
    const int head = blockIdx.x / kCtas;
    const int hk = head % p.Hkv, entry = head / p.Hkv % p.n, layer = head / p.Hkv / p.n;
    const bool tells = layer == 0 && hk == 0 && rank == 0;      // of this entry, what is not a head's own
    int32_t *kept = p.kept + static_cast<int64_t>(head) * p.budget;

    if (kCtas > 1) {        // (waited for before the first counts are added)
        for (int i = tid; i < 3 * kBins; i += kThreads) (&all_hist[0][0])[i] = 0;
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    }
    // Whether the sequence is cut: the same for all its heads and layers.
    const int b = XS_BOUNDS(entry < p.n && layer < p.layers, p.err_flag) ? p.seq_ids[entry] : -1;
    int flag = b < 0 || b >= p.B ? XS_FLAG_BAD_SLOT : 0, len = -1;
    if (!flag) {
        len = p.lens[b];
        for (int i = tid; i < entry; i += kThreads)
            if (p.seq_ids[i] == b) flag = XS_FLAG_BAD_SLOT;
    }
    const int n = min(len, p.max_blocks * kPage);
    // (The scores are on their way while the pages are looked at.)
    const uint32_t *score = reinterpret_cast<const uint32_t *>(
        p.scores + ((static_cast<int64_t>(layer) * p.B + (n > p.limit ? b : 0)) * p.Hkv + hk) * p.max_blocks * kPage);
    // This CTA's positions [mine, end), of which [lo, hi) are chosen from.
    const int part = ((n + kCtas - 1) / kCtas + 31) / 32 * 32;
    const int mine = min(rank * part, n), end = min(mine + part, n);
    const int lo = max(p.first, mine), hi = min(n - p.recent, end);
    const bool fits = end - mine <= p.held;
    if (n > p.limit && fits) {
#pragma unroll 4
        for (int t = lo + tid; t < hi; t += kThreads) held[t - mine] = key_of(score[t]);
    }
    if (n > p.limit) {
        const int32_t *row = p.tables + static_cast<int64_t>(b) * p.max_blocks;
        for (int c = p.first / kPage + tid; c < (n + kPage - 1) / kPage; c += kThreads) {
            const int32_t id = row[c];
            if (id < 0 || id >= p.num_blocks)
                flag |= XS_FLAG_BAD_BLOCK;
            else if (p.extra && p.budget > p.first && c <= (p.budget - 1) / kPage && p.extra[id] > 0)
                flag |= XS_FLAG_SHARED;
        }
    }
    const bool stop = __syncthreads_or(flag);
    if (tells && flag) raise_flag(p.err_flag, flag);
    if (tells && tid == 0 && len > n) raise_flag(p.err_flag, XS_FLAG_BAD_LEN);
    const bool cut = !stop && n > p.limit;
    if (tells && tid == 0) p.new_lens[entry] = cut ? p.budget : -1;
    if (!cut) {
        if (kCtas > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
        for (int j = rank * kThreads + tid; j < p.budget; j += kCtas * kThreads) kept[j] = -1;
        return;         // the whole cluster
    }

    auto key_at = [&](int t) { return fits ? held[t - mine] : key_of(__ldg(score + t)); };

    // The threshold: keys above it are kept, and `need` of those equal to it.
    uint32_t threshold = 0xffffffffu;       // above every key
    int need = p.budget - p.first - p.recent;
    if (need > 0) {
        uint32_t prefix = 0;
        int shift = 32;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int bits = pass < 2 ? 11 : 10, above = shift;
            shift -= bits;
            for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int t = lo + tid; t < hi; t += kThreads) {
                const uint32_t key = key_at(t);
                if (pass == 0 || key >> above == prefix) atomicAdd(&hist[key >> shift & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            const int *bins = hist;
            if (kCtas > 1) {
                bins = all_hist[pass];
                if (pass == 0) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
                for (int i = tid; i < kBins; i += kThreads) {
                    const int c = hist[i];
                    if (!c) continue;
#pragma unroll
                    for (int r = 0; r < kCtas; ++r)
                        asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(
                                         peer_addr(&all_hist[pass][i], r)),
                                     "r"(c)
                                     : "memory");
                }
                all_sync<kCtas>();
            }
            // A thread's bins, from the highest of all on.
            constexpr int kPer = kBins / kThreads;
            int sum = 0, total;
#pragma unroll
            for (int i = 0; i < kPer; ++i) sum += bins[kBins - 1 - (tid * kPer + i)];
            int before = scan_threads<kThreads>(sum, sm, &total);
            if (before < need && before + sum >= need) {
                for (int i = 0; i < kPer; ++i) {
                    const int at = kBins - 1 - (tid * kPer + i), c = bins[at];
                    if (before < need && before + c >= need) bin = at, left = need - before;
                    before += c;
                }
            }
            __syncthreads();
            prefix = pass == 0 ? static_cast<uint32_t>(bin) : prefix << bits | static_cast<uint32_t>(bin);
            need = left;
        }
        threshold = prefix;
    } else {
        if (kCtas > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
        __syncthreads();
    }

    // Each warp's part of the positions, in order, 1,024 at a time: lane i has the bits
    // of 32 of them from its 32 i on that are kept, and of those equal to the threshold.
    constexpr int kWarps = kThreads / 32, kLook = 1024, kSparse = 4;
    const int per = ((end - mine + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int from = min(mine + warp * per, end), to = min(from + per, end);
    uint32_t over, even;
    auto look = [&](int base) {
        over = even = 0;
#pragma unroll 4
        for (int i = 0; i < min((to - base + 31) / 32, 32); ++i) {
            const int t = base + 32 * i + lane;
            bool o = false, e = false;
            if (t < to) {
                o = t < p.first || t >= n - p.recent;
                if (!o) {
                    const uint32_t key = key_at(t);
                    o = key > threshold, e = key == threshold;
                }
            }
            const uint32_t os = __ballot_sync(0xffffffffu, o), es = __ballot_sync(0xffffffffu, e);
            if (lane == i) over = os, even = es;
        }
    };
    int overs = 0, evens = 0;
    for (int base = from; base < to; base += kLook) {
        look(base);
        overs += __popc(over), evens += __popc(even);
    }
    overs = __reduce_add_sync(0xffffffffu, overs), evens = __reduce_add_sync(0xffffffffu, evens);
    if (lane == 0) tally[warp] = make_int2(overs, evens);
    __syncthreads();
    int overs0 = 0, evens0 = 0, all_overs = 0, all_evens = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) overs0 = all_overs, evens0 = all_evens;
        all_overs += tally[w].x, all_evens += tally[w].y;
    }
    if (kCtas > 1) {        // and what the CTAs before this one have
        if (tid == 0) counts[0] = all_overs, counts[1] = all_evens;
        all_sync<kCtas>();
        int o = 0, e = 0;
        if (lane < rank) {
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(o) : "r"(peer_addr(&counts[0], lane)) : "memory");
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(e) : "r"(peer_addr(&counts[1], lane)) : "memory");
        }
        overs0 += __reduce_add_sync(0xffffffffu, o), evens0 += __reduce_add_sync(0xffffffffu, e);
        // No CTA leaves before all have read its counts.
        asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    }
    for (int base = from; base < to; base += kLook) {
        if (to - from > kLook) look(base);      // (else they are still there)
        // What this lane's positions have before them, and all lanes' together.
        const int mine_too = __popc(over) | __popc(even) << 16;
        int upto = mine_too;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += y;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31), before = upto - mine_too;
        const int evens1 = evens0 + (before >> 16);
        // Of those equal to the threshold the first `need` of all are kept.
        uint32_t rest = even;
        for (int i = min(max(need - evens1, 0), __popc(even)); i > 0; --i) rest &= rest - 1;
        int j = overs0 + (before & 0xffff) + min(evens1, need);
        uint32_t bits = over | (even ^ rest);
        auto put = [&](int k, int t) {
            if (XS_BOUNDS(k >= 0 && k < p.budget, p.err_flag)) kept[k] = t;
        };
        // A lane with many of them (the last tokens) has them written by the warp.
        for (uint32_t dense = __ballot_sync(0xffffffffu, __popc(bits) > kSparse); dense; dense &= dense - 1) {
            const int l = __ffs(dense) - 1, j0 = __shfl_sync(0xffffffffu, j, l);
            const uint32_t set = __shfl_sync(0xffffffffu, bits, l);
            if (set >> lane & 1) put(j0 + __popc(set & ((1u << lane) - 1)), base + 32 * l + lane);
        }
        if (__popc(bits) <= kSparse)
            for (; bits; bits &= bits - 1, ++j) put(j, base + 32 * lane + __ffs(bits) - 1);
        overs0 += all & 0xffff, evens0 += all >> 16;
    }
    if (kCtas > 1) asm volatile("barrier.cluster.wait;" ::: "memory");
}

constexpr int kMoveChunk = 1024;    // positions whose places are looked up at a time

// Goes through positions [first, budget) in tiles: where position j takes
// another's piece, put(j, get(j)) - once the whole tile has been got.  A tile is
// kMoveUnroll positions of each thread, `step` apart from `own` on.  look(j)
// finds j's places for a chunk of positions; moves(j): whether it takes another's.
template <typename V, typename L, typename M, typename G, typename P>
__device__ __forceinline__ void move_tiles(int first, int budget, int own, int step, L &&look, M &&moves, G &&get,
                                           P &&put) {
    for (int chunk = first; chunk < budget; chunk += kMoveChunk) {
        const int end = min(chunk + kMoveChunk, budget);
        __syncthreads();
        look(chunk, end);
        __syncthreads();
        for (int base = chunk; base < end; base += kMoveUnroll * step) {
            V v[kMoveUnroll];
            bool yes[kMoveUnroll];
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u) {
                const int j = base + u * step + own;
                yes[u] = j < end && moves(j);
                if (yes[u]) v[u] = get(j);
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u)
                if (yes[u]) put(base + u * step + own, v[u]);
        }
    }
}

// CTAs (layer, entry, KV head) x (K's slices, V's slices, the scores).
__global__ void __launch_bounds__(kMoveThreads, 4)
    evict_move_kernel(const __grid_constant__ EvictParams p, const int slices) {
    after_previous();
    __shared__ int32_t from[kMoveChunk], from_id[kMoveChunk], to_id[kMoveChunk / kPage + 1];
    const int32_t *kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.budget;
    if (__ldcg(kept) < 0) return;       // not cut
    const int hk = blockIdx.x % p.Hkv, entry = blockIdx.x / p.Hkv % p.n;
    const int layer = blockIdx.x / p.Hkv / p.n;
    const int b = XS_BOUNDS(entry < p.n && layer < p.layers, p.err_flag) ? p.seq_ids[entry] : 0;
    const int plane = blockIdx.y / slices, slice = blockIdx.y % slices, tid = threadIdx.x;
    const int tokens = p.max_blocks * kPage;
    int at = p.first;                   // of `from` and the others: the chunk's start
    auto moves = [&](int j) { return from[j - at] != j; };
    auto checked = [&](int t) { return XS_BOUNDS(t >= 0 && t < tokens, p.err_flag) ? t : 0; };
    if (plane == 2) {
        float *score = p.scores + ((static_cast<int64_t>(layer) * p.B + b) * p.Hkv + hk) * tokens;
        move_tiles<float>(
            p.first, p.budget, tid, kMoveThreads,
            [&](int chunk, int end) {
                at = chunk;
                for (int j = chunk + tid; j < end; j += kMoveThreads) from[j - chunk] = checked(__ldcg(kept + j));
            },
            moves, [&](int j) { return score[from[j - at]]; }, [&](int j, float v) { score[checked(j)] = v; });
        return;
    }
    char *pool = (plane ? p.v_pools : p.k_pools) + layer * p.layer_bytes;
    const int32_t *row = p.tables + static_cast<int64_t>(b) * p.max_blocks;
    // A slice of a row: `wide` pieces of 16 bytes, one each for neighbouring threads.
    const int wide = p.row_bytes / 16 / slices, piece = tid % wide;
    const int64_t in_row = static_cast<int64_t>(slice * wide + piece) * 16 + hk * kPage * static_cast<int64_t>(p.row_bytes);
    const int64_t block_bytes = static_cast<int64_t>(p.Hkv) * kPage * p.row_bytes;
    auto place = [&](int id, int t) {
        return reinterpret_cast<uint4 *>(pool + id * block_bytes + (t % kPage) * p.row_bytes + in_row);
    };
    auto block_of = [&](int t) {
        const int32_t id = __ldg(row + checked(t) / kPage);
        return XS_BOUNDS(id >= 0 && id < p.num_blocks, p.err_flag) ? id : 0;
    };
    move_tiles<uint4>(
        p.first, p.budget, tid / wide, kMoveThreads / wide,
        [&](int chunk, int end) {
            at = chunk;
#pragma unroll 4
            for (int j = chunk + tid; j < end; j += kMoveThreads) {
                const int t = __ldcg(kept + j);
                from[j - chunk] = t;
                from_id[j - chunk] = block_of(t);
            }
            for (int c = chunk / kPage + tid; c <= (end - 1) / kPage; c += kMoveThreads)
                to_id[c - chunk / kPage] = block_of(c * kPage);
        },
        moves, [&](int j) { return *place(from_id[j - at], from[j - at]); },
        [&](int j, const uint4 &v) { *place(to_id[j / kPage - at / kPage], j) = v; });
}

}  // namespace
XS_DEFINE_BOUNDS_COUNTER(bounds_failures_evict)

}  // namespace xs

extern "C" int xs_kv_evict(const int32_t *seq_ids, int n, void *k_pools, void *v_pools, int layers,
                           int64_t layer_stride_bytes, float *scores, const int32_t *block_tables,
                           int max_blocks_per_seq, const int32_t *context_lens, int B,
                           const int32_t *extra_refs, int first, int recent, int budget, int limit, int Hkv,
                           int D, int block_size, int64_t num_blocks, int dtype, int32_t *kept,
                           int32_t *new_lens, int *err_flag, cudaStream_t stream) {
    if (!seq_ids || !k_pools || !v_pools || !scores || !block_tables || !context_lens || !kept || !new_lens)
        return XS_ENULL;
    const int size = xs::elem_bytes(dtype);
    if (!size) return XS_EDTYPE;
    if (n < 0 || layers <= 0 || B < 0 || Hkv <= 0 || D <= 0 || block_size <= 0 || max_blocks_per_seq < 0 ||
        num_blocks < 0 || first < 0 || recent < 0 || budget <= 0 || limit < budget ||
        static_cast<int64_t>(first) + recent > budget)
        return XS_ESHAPE;
    if ((D != 64 && D != 128) || block_size != xs::kPage || max_blocks_per_seq > (1 << 26) ||
        layer_stride_bytes % 16 != 0)
        return XS_EUNSUPPORTED;
    const int row_bytes = D * size;
    const int64_t block_bytes = static_cast<int64_t>(Hkv) * xs::kPage * row_bytes;
    if (num_blocks > INT64_MAX / block_bytes || (layers > 1 && layer_stride_bytes < num_blocks * block_bytes))
        return XS_ESHAPE;
    if (!xs::aligned16(k_pools) || !xs::aligned16(v_pools)) return XS_EALIGN;
    const int64_t heads = static_cast<int64_t>(layers) * n;
    if (heads > INT_MAX / Hkv) return XS_EUNSUPPORTED;
    if (heads == 0) return XS_OK;
    xs::EvictParams p = {};
    p.seq_ids = seq_ids, p.n = n;
    p.k_pools = static_cast<char *>(k_pools), p.v_pools = static_cast<char *>(v_pools);
    p.layer_bytes = layer_stride_bytes, p.scores = scores;
    p.tables = block_tables, p.lens = context_lens, p.extra = extra_refs;
    p.max_blocks = max_blocks_per_seq, p.B = B, p.Hkv = Hkv, p.layers = layers, p.row_bytes = row_bytes;
    p.num_blocks = num_blocks;
    p.first = first, p.recent = recent, p.budget = budget, p.limit = limit;
    p.kept = kept, p.new_lens = new_lens, p.err_flag = err_flag;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return XS_EDEVICE;
    const int ctas = static_cast<int>(heads) * Hkv;
    const int64_t tokens = static_cast<int64_t>(max_blocks_per_seq) * xs::kPage;
    int rc;
    if (tokens <= xs::kLongTokens) {
        p.held = static_cast<int>(tokens);
        rc = xs::launch_after(xs::evict_select_kernel<256, 1>, dim3(ctas), 256, tokens * sizeof(uint32_t), stream, 1, p);
    } else {
        if (ctas > INT_MAX / xs::kRankCtas) return XS_EUNSUPPORTED;
        const auto select = xs::evict_select_kernel<xs::kRankThreads, xs::kRankCtas>;
        static std::atomic<bool> may[64];      // each device has been told of its shared memory
        if (dev >= 64 || !may[dev].load(std::memory_order_acquire)) {
            if (cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     xs::kScoresHeld * sizeof(uint32_t)) != cudaSuccess) {
                cudaGetLastError();
                return XS_EDEVICE;
            }
            if (dev < 64) may[dev].store(true, std::memory_order_release);
        }
        const int64_t part = (tokens + xs::kRankCtas - 1) / xs::kRankCtas + 32;
        p.held = static_cast<int>(part < xs::kScoresHeld ? part : 0);
        rc = xs::launch_after(select, dim3(ctas * xs::kRankCtas), xs::kRankThreads, p.held * sizeof(uint32_t), stream,
                              xs::kRankCtas, p);
    }
    if (rc != XS_OK) return rc;
    // Slices of no less than 64 bytes (of 128: 10% slower, of 32 the same), while they
    // leave SMs without work.
    int slices = 1;
    while (row_bytes / slices > 64 && static_cast<int64_t>(ctas) * 2 * slices < 4 * sms) slices *= 2;
    return xs::launch_after(xs::evict_move_kernel, dim3(ctas, 2 * slices + 1), xs::kMoveThreads, 0, stream, 1, p,
                            slices);
}
