// Per-head RMSNorm of q and k, the rotary position rotation, and the append
// of the new K/V rows into their pages (in the rows' own type or in 4 bits),
// in one pass over a projection's output; and the 4-bit append by itself,
// which is the same pass without q, norm and rotation.
//
// With x a row of D values (one head of one token), w the weights and
// p the token's position:
//     y = x / sqrt(mean(x^2) + eps) * w
//     (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
// over the pairs (a, b) of the first rotary_dim dims, with cos and sin of
// p theta_i from the caller's table (fp32, so that far positions keep their
// angles).  All of it is fp32, rounded once to the row's type; a 4-bit page
// quantises that rounded row, so the fused append stores what an append of
// the rotated rows would.
//
// A row is D / 8 lanes.  Each lane holds two chunks of 4 dims that the
// rotation pairs with one another (dims 4 j.. and rotary_dim / 2 + 4 j.. of
// split halves, 8 j.. of neighbouring pairs), so the rotation needs no
// exchange.  A prompt's pass is short of issue slots and of rows on their way
// before it is short of bytes: fp32 goes two to an operation, the weights lie
// in shared memory as fp32, addresses advance by a step, and a lane holds so
// little that many warps are resident.  (8K tokens of 32q/8kv x 128 in bf16:
// 58 us with one value to an operation, 47 us with one row ahead, 35 us so; a copy of
// as many bytes takes 32 us.)
//
// A warp takes kRows consecutive tokens, one for each of its lane groups, and
// a run of heads: position, page, cosines and sines are fetched once for the
// run, and the next head's row while the current one is worked on.  A prompt
// is bound by the bytes of its rows; a decode batch by the latency of length
// -> table -> page, so its runs are single heads.  Consecutive tokens also lie
// in one page, where two rows of 4-bit V share their words: a pair of groups
// writes whole words.
#include <climits>

#include "kv4.cuh"

namespace xs {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeCtas = 7;        // on an SM: 72 registers, a few of them spilled (6 and
                                    // none spilled: 8K tokens 39 us, 7: 36, before runs
                                    // were chosen by their waves, which made it 35)
constexpr int kRopeAheadBytes = 8;  // rows of a lane on their way, times the size of a value
constexpr int kRopeRun = 48;        // heads of a run at most
constexpr int kRopeStart = 4;       // rows that a warp's start costs as much as

struct RopeParams {
    const void *q, *k, *v;      // rows of head h of token t at t * stride + h * D
    int64_t q_stride, k_stride, v_stride;
    void *q_out, *k_out;        // contiguous [T, H, D]; k_out only without pages
    const void *q_weight, *k_weight;
    float eps;
    const float *cos_sin;       // [max_pos][rot]: rot / 2 cosines, rot / 2 sines
    int max_pos, rot;
    const int32_t *positions;   // [T], or nullptr (paged form; no rotation)
    const int64_t *slots;       // [T], or nullptr
    const int32_t *tables;      // paged form: [T, max_blocks] and lens [T]
    const int32_t *lens;
    int max_blocks;
    void *k_cache, *v_cache;    // nullptr: no append
    int64_t num_blocks;
    int T, Hq, Hkv;
    int rows_per_token;         // Hq + Hkv, and Hkv more for V with an append
    int run;                    // heads that a warp takes one after the other
    bool interleaved, kv4;
    int *err_flag;
};

// N values at p as they come from memory (8 to 32 bytes, as aligned), and as fp32.
template <typename T, int N> struct Chunk {
    static constexpr int kWords = N * sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kWords == 2) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4 *>(p)[i] =
                    make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
    }
    __device__ __forceinline__ void to_f32(float *f) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) {
                f[i] = __uint_as_float(w[i]);
            } else {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void from_f32(const float *f) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = __float_as_uint(f[i]);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
};

// Mean of the squares of a row, of which each of its lanes holds 8 values.
template <int kLanes> __device__ __forceinline__ float mean_square(const F2 *x) {
    F2 sum = mul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sum = fma2(x[i], x[i], sum);
    float s = sum.x + sum.y;
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    return s * (1.0f / (8 * kLanes));
}

// The slot that row t's token is appended to, or -1 (none, or flagged).
__device__ __forceinline__ int64_t append_slot(const RopeParams &p, int64_t t, int64_t pos,
                                               int *err_flag) {
    if (p.slots) {
        const int64_t s = p.slots[t];
        if (s >= p.num_blocks * 16) {
            raise_flag(err_flag, XS_FLAG_BAD_SLOT);
            return -1;
        }
        return s;
    }
    const int64_t page = pos >> 4;
    if (page >= p.max_blocks) {
        raise_flag(err_flag, XS_FLAG_BAD_LEN);
        return -1;
    }
    if (!XS_BOUNDS(t >= 0 && t < p.T && page >= 0, p.err_flag)) return -1;
    const int32_t blk = p.tables[t * p.max_blocks + page];
    if (blk < 0 || blk >= p.num_blocks) {
        raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
        return -1;
    }
    return static_cast<int64_t>(blk) * 16 + (pos & 15);
}

template <typename T, int D, bool kKv4>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kLanes = D / 8;               // lanes of a row
    constexpr int kRows = 32 / kLanes;          // rows of a warp
    __shared__ __align__(16) uint32_t keys[kKv4 ? kRopeThreads / 32 : 1][kRows][D / 4];
    __shared__ __align__(16) float weights[2][D];
    after_previous();
    constexpr int kMine = 2 * D / kRopeThreads;     // weights of a thread
    float weight[kMine];    // on their way to shared memory while the first rows are found
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int e = threadIdx.x + i * kRopeThreads;
        const T *w = static_cast<const T *>(e < D ? p.q_weight : p.k_weight);
        weight[i] = w ? Elem<T>::to_f32(w[e % D]) : 1.0f;
    }
    const int lane = threadIdx.x & 31, j = lane % kLanes, warp = threadIdx.x >> 5;
    const int runs = (p.rows_per_token + p.run - 1) / p.run;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + warp;
    const int64_t block = item < (int64_t(1) << 32)
                              ? static_cast<uint32_t>(item) / static_cast<uint32_t>(runs)
                              : item / runs;
    const int run_begin = static_cast<int>(item - block * runs) * p.run;
    const int run_end = min(run_begin + p.run, p.rows_per_token);
    const int64_t t = block * kRows + lane / kLanes;    // past T for an item past the last
    // A lane's chunks of a rotated row.
    const bool rotates = j < p.rot / 8;
    const bool halves = rotates && !p.interleaved;
    const int r0 = halves ? j : 2 * j, r1 = halves ? p.rot / 8 + j : 2 * j + 1;
    // The rows of the next kAhead heads are on their way (a row that is not
    // there counts as zeros): q's, k's or v's, the run's first ones before
    // anything else is known of the token.
    constexpr int kAhead = kKv4 ? 2 : kRopeAheadBytes / sizeof(T);
    Chunk<T, 4> ahead[kAhead][2];
    // Whether chunks c0 and c1 of head h of the token's q, k or v are its own.
    auto inside = [&](int kind, int h, int c0, int c1) {
        return XS_BOUNDS(t >= 0 && t < p.T && h >= 0 && h < (kind == 0 ? p.Hq : p.Hkv) && c0 >= 0 &&
                             4 * c0 + 4 <= D && c1 >= 0 && 4 * c1 + 4 <= D, p.err_flag);
    };
    auto fetch = [&](int kind, int h, int count) {
        const int c0 = kind < 2 ? r0 : 2 * j, c1 = kind < 2 ? r1 : 2 * j + 1;
        const T *src = kind == 0   ? static_cast<const T *>(p.q) + t * p.q_stride
                       : kind == 1 ? static_cast<const T *>(p.k) + t * p.k_stride
                                   : static_cast<const T *>(p.v) + t * p.v_stride;
        src += h * D;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
#pragma unroll
            for (int w = 0; w < Chunk<T, 4>::kWords; ++w) ahead[i][0].w[w] = ahead[i][1].w[w] = 0;
            if (t < p.T && i < count && inside(kind, h + i, c0, c1)) {
                ahead[i][0].load(src + i * D + 4 * c0);
                ahead[i][1].load(src + i * D + 4 * c1);
            }
        }
        return src + kAhead * D;
    };
    auto first_of = [&](int kind) { return kind == 0 ? 0 : kind == 1 ? p.Hq : p.Hq + p.Hkv; };
    auto count_of = [&](int kind) {     // heads of the kind in the run
        const int first = first_of(kind), last = kind == 0 ? p.Hq : min(first + p.Hkv, p.rows_per_token);
        return min(run_end, last) - max(run_begin, first);
    };
    const int kind0 = run_begin < p.Hq ? 0 : run_begin < p.Hq + p.Hkv ? 1 : 2;
    const T *src = fetch(kind0, run_begin - first_of(kind0), count_of(kind0));

    bool live = t < p.T;
    int64_t pos = 0;
    if (live) {
        if (p.lens)
            pos = static_cast<int64_t>(p.lens[t]) - 1;
        else if (p.positions)
            pos = p.positions[t];
        live = pos >= 0;
    }
    if (live && p.rot > 0 && pos >= p.max_pos) {
        if (j == 0 && run_begin == 0) raise_flag(p.err_flag, XS_FLAG_BAD_LEN);
        live = false;
        // A step's attention goes on with q_out: NaN, not an earlier step's query.
        if (p.lens)
            for (int h = run_begin; h < min(run_end, p.Hq); ++h) {
                Chunk<T, 8> none;
#pragma unroll
                for (int w = 0; w < Chunk<T, 8>::kWords; ++w) none.w[w] = 0x7fffffffu;
                if (inside(0, h, 2 * j, 2 * j + 1))
                    none.store(static_cast<T *>(p.q_out) + (t * p.Hq + h) * D + 8 * j);
            }
    }
    int64_t slot = -1;
    if (live && p.k_cache && run_end > p.Hq)
        slot = append_slot(p, t, pos, j == 0 && run_begin <= p.Hq ? p.err_flag : nullptr);
    if (slot >= 0 && !XS_BOUNDS((slot >> 4) < p.num_blocks && run_end <= p.rows_per_token, p.err_flag))
        slot = -1;
    const int64_t page0 = slot < 0 ? 0 : (slot >> 4) * p.Hkv;
    const int o = static_cast<int>(slot & 15);

    // The lane's cosines and sines.
    F2 c[2], s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = F2{1.0f, 1.0f}, s[i] = F2{0.0f, 0.0f};
    if (live && rotates && run_begin < p.Hq + p.Hkv &&
        XS_BOUNDS(pos < p.max_pos && 4 * j + 4 <= p.rot / 2, p.err_flag)) {
        const float *row = p.cos_sin + pos * p.rot + 4 * j;
        Chunk<float, 4> v;
        v.load(row);
        v.to_f32(&c[0].x);
        v.load(row + p.rot / 2);
        v.to_f32(&s[0].x);
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) (&weights[0][0])[threadIdx.x + i * kRopeThreads] = weight[i];
    __syncthreads();

    // q, then k, then v heads of the run.
#pragma unroll 1
    for (int kind = kind0; kind < 3; ++kind) {
        const int count = count_of(kind);
        if (count <= 0) break;
        const int h = max(run_begin - first_of(kind), 0);
        const int c0 = kind < 2 ? r0 : 2 * j, c1 = kind < 2 ? r1 : 2 * j + 1;
        if (kind != kind0) src = fetch(kind, h, count);
        const bool paged = kind > 0 && p.k_cache;
        const bool norm = kind == 0 ? p.q_weight != nullptr : kind == 1 && p.k_weight != nullptr;
        const bool turn = kind < 2 && rotates;
        const bool writes = paged ? slot >= 0 : live;
        // Where the row goes, and how far on the next head's does.
        T *dst;
        uint8_t *page = nullptr;
        int step = D;
        if (!paged) {
            dst = kind == 0 ? static_cast<T *>(p.q_out) + (t * p.Hq + h) * D
                            : static_cast<T *>(p.k_out) + (t * p.Hkv + h) * D;
        } else {
            void *cache = kind == 1 ? p.k_cache : p.v_cache;
            dst = static_cast<T *>(cache) + ((page0 + h) * 16 + o) * D;
            page = static_cast<uint8_t *>(cache) + (page0 + h) * kv4_page_bytes(D);
            step = 16 * D;
        }
        // Whether the next group's row (an even one's), or the one before (an
        // odd one's), is the other row of this one's V pair.
        const bool paired =
            kKv4 && __shfl_xor_sync(0xffffffffu, slot, kLanes) == (slot ^ 1) && slot >= 0;
        const float *g = weights[kind == 0 ? 0 : 1];

#pragma unroll 1
        for (int k0 = 0; k0 < count; k0 += kAhead)
#pragma unroll
        for (int i0 = 0; i0 < kAhead; ++i0) {
            if (k0 + i0 >= count) break;
            F2 x[4];
            ahead[i0][0].to_f32(&x[0].x);
            ahead[i0][1].to_f32(&x[2].x);
            if (t < p.T && k0 + i0 + kAhead < count && inside(kind, h + k0 + i0 + kAhead, c0, c1)) {
                ahead[i0][0].load(src + 4 * c0);
                ahead[i0][1].load(src + 4 * c1);
            }
            src += D;
            if (norm) {
                float mean = mean_square<kLanes>(x) + p.eps;
                // Squares that leave fp32 (|x| beyond 2^60, or below 2^-50 under an
                // eps that does not cover it) are taken of x 2^-96 or x 2^96 instead.
                const float lift = mean > 0x1p125f ? 0x1p-96f : mean < 0x1p-100f ? 0x1p96f : 1.0f;
                if (__any_sync(0xffffffffu, lift != 1.0f)) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], F2{lift, lift});
                    mean = mean_square<kLanes>(x) + p.eps * lift * lift;
                }
                const float rms = rsqrtf(mean);
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(g + 4 * (i ? c1 : c0));
                    x[i] = mul2(mul2(x[i], F2{rms, rms}), F2{v.x, v.y});
                    x[i + 1] = mul2(mul2(x[i + 1], F2{rms, rms}), F2{v.z, v.w});
                }
            }
            if (turn) {
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float cc = i & 1 ? c[i / 2].y : c[i / 2].x;
                        const float ss = i & 1 ? s[i / 2].y : s[i / 2].x;
                        x[i] = F2{x[i].x * cc - x[i].y * ss, x[i].y * cc + x[i].x * ss};
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const F2 a = x[i], b = x[2 + i];
                        x[i] = sub2(mul2(a, c[i]), mul2(b, s[i]));
                        x[2 + i] = fma2(b, c[i], mul2(a, s[i]));
                    }
                }
            }
            Chunk<T, 4> y0, y1;
            y0.from_f32(&x[0].x);
            y1.from_f32(&x[2].x);
            if (!kKv4 || !paged) {
                if (writes && inside(kind, h + k0 + i0, c0, c1)) {
                    y0.store(dst + 4 * c0);
                    y1.store(dst + 4 * c1);
                }
                dst += step;
                continue;
            }
            if constexpr (kKv4) {
                y0.to_f32(&x[0].x);
                y1.to_f32(&x[2].x);
                uint32_t key[2] = {max_u16x2(kv4_keys(y0.w[0]), kv4_keys(y0.w[1])),
                                   max_u16x2(kv4_keys(y1.w[0]), kv4_keys(y1.w[1]))};
                // Where the lane's chunks are neighbours, four lanes hold a group; where
                // they are of the halves of a whole row, eight lanes hold two; else they
                // meet in shared memory.
                uint32_t both;          // the keys of the two chunks' groups
                if (kind == 2 || p.interleaved || p.rot == 0) {
                    uint32_t k = max_u16x2(key[0], key[1]);
                    k = max_u16x2(k, __shfl_xor_sync(0xffffffffu, k, 1));
                    k = max_u16x2(k, __shfl_xor_sync(0xffffffffu, k, 2));
                    both = kv4_fold(k);
                } else if (p.rot == D) {
                    uint32_t k = max_u16x2(__byte_perm(key[0], key[1], 0x5410),
                                           __byte_perm(key[0], key[1], 0x7632));
                    k = max_u16x2(k, __shfl_xor_sync(0xffffffffu, k, 1));
                    k = max_u16x2(k, __shfl_xor_sync(0xffffffffu, k, 2));
                    k = max_u16x2(k, __shfl_xor_sync(0xffffffffu, k, 4));
                    both = k;
                } else {
                    uint32_t *row_keys = keys[warp][lane / kLanes];
                    __syncwarp();
                    row_keys[c0] = key[0];
                    row_keys[c1] = key[1];
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 *k4 = reinterpret_cast<const uint4 *>(row_keys + ((u ? c1 : c0) & ~7));
                        const uint4 a = k4[0], b = k4[1];
                        key[u] = kv4_fold(max_u16x2(max_u16x2(max_u16x2(a.x, a.y), max_u16x2(a.z, a.w)),
                                                    max_u16x2(max_u16x2(b.x, b.y), max_u16x2(b.z, b.w))));
                    }
                    both = __byte_perm(key[0], key[1], 0x5410);
                }
                uint32_t scales = kv4_scales(both);
                uint32_t half[2];       // four codes each
                kv4_pack(half, &x[0].x, scales);
                // The word (8 dims) this lane stores: its own two chunks, or, of
                // split halves, the first chunk's with the next lane's, or the
                // second's with the lane before's.
                uint32_t word = half[0] | half[1] << 16;
                const uint32_t other = __shfl_xor_sync(0xffffffffu, j & 1 ? half[0] : half[1], 1);
                int ch = j;
                if (kind == 1 && halves) {
                    word = j & 1 ? other | half[1] << 16 : half[0] | other << 16;
                    ch = (j & 1 ? c1 : c0) >> 1;
                }
                const uint16_t word_scale =
                    static_cast<uint16_t>(kind == 1 && halves && (j & 1) ? scales >> 16 : scales);
                const uint32_t theirs = __shfl_xor_sync(0xffffffffu, word, kLanes);
                if (writes && inside(kind, h + k0 + i0, 2 * ch, 2 * ch + 1)) {
                    if (kind == 2 && paired)
                        kv4_store_pair<D>(page, o, ch, word, theirs, word_scale);
                    else
                        kv4_store_chunk<D>(page, kind == 2, o, ch, word, word_scale);
                }
                page += kv4_page_bytes(D);
            }
        }
    }
}

bool strided_ok(const void *ptr, int64_t stride, int eb) {
    return aligned16(ptr) && (stride * eb) % 16 == 0;
}

int launch(RopeParams &p, int D, int dtype, cudaStream_t stream) {
    p.rows_per_token = p.Hq + p.Hkv + (p.k_cache ? p.Hkv : 0);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return XS_EDEVICE;
    // Single heads while the warps all fit; else the run whose waves of warps take the
    // fewest rows (4K tokens into a 4-bit cache, two runs of 24 heads in one
    // wave: 23.6 us; three of 16 in two: 28.4 us).
    const int rows = 256 / D;   // tokens of a warp
    const int64_t blocks = (static_cast<int64_t>(p.T) + rows - 1) / rows;
    const int64_t held = static_cast<int64_t>(sms) * (kRopeCtas * kRopeThreads / 32);
    p.run = 1;
    if (blocks * p.rows_per_token > held) {
        int64_t least = INT64_MAX;
        for (int run = 1; run <= kRopeRun && run <= p.rows_per_token; ++run) {
            const int64_t runs = (p.rows_per_token + run - 1) / run, waves = (blocks * runs + held - 1) / held;
            if (waves * (run + kRopeStart) < least) least = waves * (run + kRopeStart), p.run = run;
        }
    }
    const int64_t items = blocks * ((p.rows_per_token + p.run - 1) / p.run);
    const int64_t want = (items + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    if (want > INT_MAX) return XS_EUNSUPPORTED;
    const int grid = static_cast<int>(want);
    auto go = [&](auto kernel) {
        return launch_after(kernel, dim3(grid), kRopeThreads, 0, stream, 1, p);
    };
    if (dtype == XS_F32)
        return D == 128 ? go(qk_norm_rope_kernel<float, 128, false>)
                        : go(qk_norm_rope_kernel<float, 64, false>);
    if (p.kv4)
        return D == 128 ? go(qk_norm_rope_kernel<__nv_bfloat16, 128, true>)
                        : go(qk_norm_rope_kernel<__nv_bfloat16, 64, true>);
    return D == 128 ? go(qk_norm_rope_kernel<__nv_bfloat16, 128, false>)
                    : go(qk_norm_rope_kernel<__nv_bfloat16, 64, false>);
}

// Checks that every form shares; fills the fields they share.  `append`: the
// call has pages (then v and the pools are required, k_out is not).
int prepare(RopeParams &p, bool append, bool paged, bool kv4, int D, int block_size, int dtype) {
    const int eb = elem_bytes(dtype);
    if (p.Hq > 0 && (!p.q || !p.q_out)) return XS_ENULL;
    if (!p.k || (append ? (!p.v || !p.k_cache || !p.v_cache) : !p.k_out)) return XS_ENULL;
    if (append && (paged ? (!p.tables || !p.lens) : !p.slots)) return XS_ENULL;
    if (p.rot != 0 && (!p.cos_sin || (!paged && !p.positions))) return XS_ENULL;
    if (!eb) return XS_EDTYPE;
    if (p.T < 0 || p.Hq < 0 || p.Hkv <= 0 || D <= 0 || p.rot < 0 || p.rot > D || p.max_pos < 0 ||
        (append && (block_size <= 0 || p.num_blocks < 0)) || (paged && p.max_blocks < 0))
        return XS_ESHAPE;
    // A row must not run into the next one's.
    if ((p.Hq > 0 && p.q_stride < static_cast<int64_t>(p.Hq) * D) ||
        p.k_stride < static_cast<int64_t>(p.Hkv) * D ||
        (append && p.v_stride < static_cast<int64_t>(p.Hkv) * D))
        return XS_ESHAPE;
    if ((D != 64 && D != 128) || p.rot % 16 != 0 || (append && block_size != 16))
        return XS_EUNSUPPORTED;
    if (kv4 && dtype != XS_BF16) return XS_EUNSUPPORTED;
    if (p.Hq > (1 << 20) || p.Hkv > (1 << 20)) return XS_EUNSUPPORTED;
    if ((p.Hq > 0 && (!strided_ok(p.q, p.q_stride, eb) || !aligned16(p.q_out))) ||
        !strided_ok(p.k, p.k_stride, eb) || (!append && !aligned16(p.k_out)) ||
        (append && (!strided_ok(p.v, p.v_stride, eb) || !aligned16(p.k_cache) ||
                    !aligned16(p.v_cache))) ||
        !aligned16(p.q_weight) || !aligned16(p.k_weight) || (p.rot != 0 && !aligned16(p.cos_sin)))
        return XS_EALIGN;
    p.kv4 = kv4;
    return XS_OK;
}

}  // namespace
XS_DEFINE_BOUNDS_COUNTER(bounds_failures_rope)

}  // namespace xs

extern "C" int xs_qk_norm_rope(void *q_out, void *k_out, const void *q, int64_t q_stride,
                               const void *k, int64_t k_stride, const void *q_weight,
                               const void *k_weight, float eps, const float *cos_sin, int max_pos,
                               int rotary_dim, const int32_t *positions, int T, int Hq, int Hkv,
                               int D, int flags, int dtype, int *err_flag, cudaStream_t stream) {
    if (flags & ~XS_ROPE_INTERLEAVED) return XS_EUNSUPPORTED;
    if (!q || !q_out) return XS_ENULL;
    if (Hq <= 0) return XS_ESHAPE;
    xs::RopeParams p = {};
    p.q = q, p.k = k, p.q_stride = q_stride, p.k_stride = k_stride;
    p.q_out = q_out, p.k_out = k_out, p.q_weight = q_weight, p.k_weight = k_weight;
    p.eps = eps, p.cos_sin = cos_sin, p.max_pos = max_pos, p.rot = rotary_dim;
    p.positions = positions, p.T = T, p.Hq = Hq, p.Hkv = Hkv;
    p.interleaved = flags & XS_ROPE_INTERLEAVED, p.err_flag = err_flag;
    const int rc = xs::prepare(p, false, false, false, D, 16, dtype);
    if (rc != XS_OK || T == 0) return rc;
    return xs::launch(p, D, dtype, stream);
}

extern "C" int xs_qk_norm_rope_append(void *q_out, const void *q, int64_t q_stride, const void *k,
                                      int64_t k_stride, const void *v, int64_t v_stride,
                                      const void *q_weight, const void *k_weight, float eps,
                                      const float *cos_sin, int max_pos, int rotary_dim,
                                      const int32_t *positions, void *k_cache, void *v_cache,
                                      const int64_t *slot_mapping, int T, int Hq, int Hkv, int D,
                                      int block_size, int64_t num_blocks, int flags, int dtype,
                                      int *err_flag, cudaStream_t stream) {
    if (flags & ~(XS_ROPE_INTERLEAVED | XS_CACHE_KV4)) return XS_EUNSUPPORTED;
    if (!q || !q_out) return XS_ENULL;
    if (Hq <= 0) return XS_ESHAPE;
    xs::RopeParams p = {};
    p.q = q, p.k = k, p.v = v, p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
    p.q_out = q_out, p.q_weight = q_weight, p.k_weight = k_weight;
    p.eps = eps, p.cos_sin = cos_sin, p.max_pos = max_pos, p.rot = rotary_dim;
    p.positions = positions, p.slots = slot_mapping, p.k_cache = k_cache, p.v_cache = v_cache;
    p.num_blocks = num_blocks, p.T = T, p.Hq = Hq, p.Hkv = Hkv;
    p.interleaved = flags & XS_ROPE_INTERLEAVED, p.err_flag = err_flag;
    const int rc =
        xs::prepare(p, true, false, (flags & XS_CACHE_KV4) != 0, D, block_size, dtype);
    if (rc != XS_OK || T == 0) return rc;
    return xs::launch(p, D, dtype, stream);
}

extern "C" int xs_qk_norm_rope_append_paged(
    void *q_out, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
    int64_t v_stride, const void *q_weight, const void *k_weight, float eps, const float *cos_sin,
    int max_pos, int rotary_dim, void *k_cache, void *v_cache, const int32_t *block_tables,
    int max_blocks_per_seq, const int32_t *context_lens, int B, int Hq, int Hkv, int D,
    int block_size, int64_t num_blocks, int flags, int dtype, int *err_flag, cudaStream_t stream) {
    if (flags & ~(XS_ROPE_INTERLEAVED | XS_CACHE_KV4)) return XS_EUNSUPPORTED;
    if (!q || !q_out) return XS_ENULL;
    if (Hq <= 0) return XS_ESHAPE;
    xs::RopeParams p = {};
    p.q = q, p.k = k, p.v = v, p.q_stride = q_stride, p.k_stride = k_stride, p.v_stride = v_stride;
    p.q_out = q_out, p.q_weight = q_weight, p.k_weight = k_weight;
    p.eps = eps, p.cos_sin = cos_sin, p.max_pos = max_pos, p.rot = rotary_dim;
    p.tables = block_tables, p.max_blocks = max_blocks_per_seq, p.lens = context_lens;
    p.k_cache = k_cache, p.v_cache = v_cache;
    p.num_blocks = num_blocks, p.T = B, p.Hq = Hq, p.Hkv = Hkv;
    p.interleaved = flags & XS_ROPE_INTERLEAVED, p.err_flag = err_flag;
    const int rc = xs::prepare(p, true, true, (flags & XS_CACHE_KV4) != 0, D, block_size, dtype);
    if (rc != XS_OK || B == 0) return rc;
    return xs::launch(p, D, dtype, stream);
}

extern "C" int xs_kv4_append(const void *k_new, int64_t k_stride, const void *v_new,
                             int64_t v_stride, void *k_cache, void *v_cache,
                             const int64_t *slot_mapping, int T, int Hkv, int D, int block_size,
                             int64_t num_blocks, int dtype, int *err_flag, cudaStream_t stream) {
    xs::RopeParams p = {};
    p.k = k_new, p.v = v_new, p.k_stride = k_stride, p.v_stride = v_stride;
    p.slots = slot_mapping, p.k_cache = k_cache, p.v_cache = v_cache;
    p.num_blocks = num_blocks, p.T = T, p.Hkv = Hkv, p.err_flag = err_flag;
    const int rc = xs::prepare(p, true, false, true, D, block_size, dtype);
    if (rc != XS_OK || T == 0) return rc;
    return xs::launch(p, D, dtype, stream);
}

extern "C" int xs_kv4_append_paged(const void *k_new, int64_t k_stride, const void *v_new,
                                   int64_t v_stride, void *k_cache, void *v_cache,
                                   const int32_t *block_tables, int max_blocks_per_seq,
                                   const int32_t *context_lens, int B, int Hkv, int D,
                                   int block_size, int64_t num_blocks, int dtype, int *err_flag,
                                   cudaStream_t stream) {
    xs::RopeParams p = {};
    p.k = k_new, p.v = v_new, p.k_stride = k_stride, p.v_stride = v_stride;
    p.tables = block_tables, p.max_blocks = max_blocks_per_seq, p.lens = context_lens;
    p.k_cache = k_cache, p.v_cache = v_cache;
    p.num_blocks = num_blocks, p.T = B, p.Hkv = Hkv, p.err_flag = err_flag;
    const int rc = xs::prepare(p, true, true, true, D, block_size, dtype);
    if (rc != XS_OK || B == 0) return rc;
    return xs::launch(p, D, dtype, stream);
}
