// Decode attention over a bounded part of a paged cache, and with the weights
// that each cached token got.  Each sequence's one query token attends to
//
//     out[b, h] = sum_t p_ht V_t,  p_h = softmax_t(scale q[b, h] . K_t)
//
// over the tokens t < first and t >= n - window (every token: window 0), and,
// in the form with weights,
//
//     scores[b, hk, t] = old + sum over the heads h of KV head hk of p_ht
//
// (old: 0 for tokens that were not scored before).
//
// A page of one KV head serves the G = Hq / Hkv query heads of its group.  bf16
// pages are worked on with m16n8k16 matrix instructions, keys (and dims of the
// output) on the rows, heads on the columns; fp32 pages with fp32 products and
// sums of the ordinary pipes.  The softmax is online, in fp32: its reference leads
// the largest logit by kLead powers of two and is set again only when a logit
// exceeds it, so most pages take no exchange between lanes.  A weight enters
// the second product of the bf16 form as the sum of two bf16 values (the
// weight cut to 8 bits, and the rest rounded to 8: 2^-16 of it is lost); with
// the first alone the output's error grows by a third.
//
// Pages reach a warp's own ring of places in shared memory by bulk copies (one
// tensor copy each for a bf16 K and V page, whose 128-byte swizzle keeps the
// fragments' loads free of bank conflicts) that its lanes start ahead; a page
// is waited for, read and given back with no barrier but the warp's own.
//
// Split, over segments (sequence, KV head):
//  - few: a thread-block cluster of 2, 4 or 8 CTAs for each, whose warps' states
//    meet in shared memory;
//  - more: a CTA for each, of 8 warps where the device holds all at once and tables
//    are short, else of 4 warps, two on an SM, whose starts and ends hide behind
//    one another's pages;
//  - many of unlike lengths: the pages of all sequences form one line, each
//    sequence with kSegmentCost more for its end, and the line is cut into equal
//    shares, one for each group of Hkv warps of the grid, a warp for each KV head
//    (so that a block's pages are read at about one time).  Copies run on across
//    the ends of sequences.  A segment that one warp does is written at once; one
//    that is cut leaves fp32 partials in the workspace, at most two for each warp,
//    and the warp that finishes it last joins them in order: the result does not
//    depend on which that is.
// The lengths, on the device, decide between the last two, and where a warp works,
// so the host needs to know none of them and a captured call follows them.
//
// Weights.  p_ht needs the final maximum and sum of its row, which no warp
// knows while it has the logit.  So logits are kept, 4 bytes for a token and
// head beside 4 D bytes of bf16 K and V for a token and KV head.  A CTA or cluster
// with a whole segment keeps them in shared memory (or, beyond its room, in the
// workspace) and turns them into weights itself; the line leaves them in the
// workspace, most of it in L2, for a second kernel.  (The warp that ends a segment
// doing that took 4 us more for 64 sequences of 17 to 8193 tokens than the kernel.)
//
// What bounds it: DRAM where there is enough of it (bf16, 32q/8kv x 128: 128 sequences
// that see 4112 tokens each 301 us, 7.2 TB/s where a copy has 6.8; 128 of 2049 to 4097
// with weights 265 us, of which the logits beyond shared memory take 8 and the scores
// 10), and the chain length - ids - page - join where there is not (one
// sequence: 5.0 us up to 1K tokens, 7.1 at 4K, 8.1 with weights).
#include <atomic>
#include <type_traits>

#include <cuda.h>

#include "tensor_map.h"
#include "xs_common.cuh"

namespace xs {
namespace bounded {
namespace {     // (the release and the debug library may be loaded side by side)

constexpr int kBlock = 16;
constexpr int kLineWarps = 4;       // warps of a CTA of the line, two CTAs on an SM
constexpr int kClusterWarps = 8;    // of a cluster's CTA, one on an SM
constexpr int kMaxWarps = 1280;     // the workspace holds partials for so many
constexpr int kSegmentCost = 6;     // pages (4: many short segments 8% faster, few long ones 4% slower; 8: the reverse)
constexpr int kMinShare = 4;        // pages
constexpr int kShortTable = 128;    // pages
constexpr int kScannedB = 256;      // sequences whose lengths a CTA for each segment may look at
// Segments of up to so many pages are not cut (61 x 12 of 7 pages: 9.1 us so, 10.1 cut;
// 61 x 12 of up to 64: 11.7 us, 12.8 with 16).
constexpr int kWholePages = 8;
constexpr int kMaxCluster = 8;
// For the choice between the two forms of many segments, in units of a page at the
// device's full rate (1.1 ns for 8 KB of K and V): what a page takes a CTA of
// kLineWarps that has the device for itself, and a CTA's start and end.
template <typename T, int D> constexpr int64_t kAlone = kBlock * D * sizeof(T) < 4096 ? 200 : 100;
template <typename T, int D> constexpr int64_t kEnds = 2600 * 4096 / (kBlock * D * static_cast<int>(sizeof(T)));
// Logits that a CTA keeps in shared memory (with weights).
template <typename T, int D, int W> __host__ __device__ constexpr int logit_floats() {
    return W == kClusterWarps ? 6144 : sizeof(T) == 2 ? 10240 : D == 128 ? 4096 : 2048;
}
constexpr float kLead = 8.0f;       // of a reference before the largest logit
constexpr float kLowest = -3.402823466e38f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kWaitLimitNs = 4000000000ull;
// In the debug library the limit can be set, and a page of CTA 0's first warp
// left out, so that its wait runs out (xs_debug_bounded_wait_injection).
#ifdef XS_DEBUG_BOUNDS
__device__ unsigned long long g_wait_limit_ns = kWaitLimitNs;
__device__ int g_skip_page = -1;    // the warp's page, counted since the launch
__device__ __forceinline__ uint64_t wait_limit() { return g_wait_limit_ns; }
__device__ __forceinline__ bool skip_page(uint32_t page) {
    return blockIdx.x == 0 && threadIdx.x == 0 && static_cast<int>(page) == g_skip_page;
}
#else
__device__ __forceinline__ constexpr uint64_t wait_limit() { return kWaitLimitNs; }
__device__ __forceinline__ constexpr bool skip_page(uint32_t) { return false; }
#endif

// Places (a K and a V page) of a warp's ring: 96 KB for a CTA of four warps, so that
// two share an SM, or 64 KB beside the logits of bf16 pages (128 sequences of 2K to 4K
// tokens 244 us so, 258 with 96 and fewer logits; without logits 64 of 1K take 41.6 us with
// 96, 45.9 with 64), and 192 KB for a cluster's (fp32 pages of 128: 192 and 128 KB).
template <typename T, int D, bool kWeights> __host__ __device__ constexpr int line_stages() {
    return sizeof(T) == 4 && D == 128
               ? 3
               : ((kWeights && sizeof(T) == 2 ? 64 : 96) << 10) / (kLineWarps * 2 * kBlock * D * static_cast<int>(sizeof(T)));
}
template <typename T, int D> __host__ __device__ constexpr int cluster_stages() {
    return (192 << 10) / (kClusterWarps * 2 * kBlock * D * static_cast<int>(sizeof(T)));
}

struct Params {
    void *out;
    const void *q;
    int64_t q_stride;       // elements between two sequences' queries
    const void *k_cache, *v_cache;
    const int32_t *tables, *lens;
    const void *sinks;
    int max_blocks, first, window, B, Hq, Hkv, G;
    int64_t num_blocks;
    float scale_log2;
    int *err_flag;
    int *counters;      // [kMaxWarps]: arrivals at the segment that warp i begins and does not end
    float *partials;    // [kMaxWarps][2] of partial_floats(D)
    // With weights:
    float *scores;      // [B, Hkv, max_blocks * 16]
    const int32_t *scored;  // [B] or null: n - 1
    float *logits;      // [B, Hkv, max_blocks * 16, G], in powers of two
    float2 *ends;       // [B, Hq]: a row's reference and the reciprocal of its sum
};

// f(integral_constant<int, G>) for G in {1, 2, 4, 8}.
template <typename F> __device__ __forceinline__ void by_heads(int G, F &&f) {
    if (G == 1)
        f(std::integral_constant<int, 1>());
    else if (G == 2)
        f(std::integral_constant<int, 2>());
    else if (G == 4)
        f(std::integral_constant<int, 4>());
    else
        f(std::integral_constant<int, 8>());
}

// A lane's registers of 8 heads x D values, then 8 references and 8 sums.
__host__ __device__ constexpr int partial_floats(int D) { return 8 * D + 16; }

// What sequence b's query sees: tokens [0, f) and [low, n), on `pages` pages,
// the first `fp` of which are pages 0 .. fp - 1 and the others page0 and on.
struct Span {
    int n, low, f, fp, page0, pages;
    __device__ __forceinline__ int page(int i) const { return i < fp ? i : i - fp + page0; }
    __device__ __forceinline__ bool sees(int t) const { return t < n && (t >= low || t < f); }
    __device__ __forceinline__ bool sees_page(int tok0) const {
        return tok0 + kBlock <= n && (tok0 >= low || tok0 + kBlock <= f);
    }
};
__device__ __forceinline__ Span span_of(const Params &p, int b) {
    Span s;
    s.n = XS_BOUNDS(b >= 0 && b < p.B, p.err_flag) ? p.lens[b] : 0;
    if (s.n > p.max_blocks * kBlock) {
        if (blockIdx.x == 0) raise_flag(p.err_flag, XS_FLAG_BAD_LEN);
        s.n = p.max_blocks * kBlock;
    }
    s.n = max(s.n, 0);
    s.low = p.window > 0 && s.n > p.window ? s.n - p.window : 0;
    s.f = min(p.first, s.low);
    s.page0 = s.low / kBlock;
    s.fp = min((s.f + kBlock - 1) / kBlock, s.page0);
    s.pages = s.fp + (s.n + kBlock - 1) / kBlock - s.page0;
    return s;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void ldsm(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, turned over between the lanes.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float4 lds128(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// ------------------------------------------------------------------ a warp's work on pages
// State<T, D>: references m, sums l and values acc of the 8 heads of a group (those
// from G on are never read).  A lane has kHeads heads' m and l (head(k)), its
// own share of l until sum_up(), and D / 4 of the values: acc[4 k + c] is dim
// dim(k, c) of head head_of(k, c).
template <typename T, int D> struct State;

template <int D> struct State<__nv_bfloat16, D> {
    static constexpr int kHeads = 2;
    uint32_t q[D / 16][2];
    float m[2], l[2], acc[D / 4];

    static __device__ __forceinline__ int head(int lane, int k) { return 2 * (lane & 3) + k; }
    static __device__ __forceinline__ int head_of(int lane, int, int c) { return 2 * (lane & 3) + (c & 1); }
    static __device__ __forceinline__ int dim(int lane, int k, int c) {
        return 16 * k + (lane >> 2) + 8 * (c >> 1);
    }
    // The second operand of the logits: lane (g, t) has dims 16 i + 2 t, + 1, and 8 more, of head g.
    __device__ __forceinline__ void load_q(const Params &p, const void *q0, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(q0) +
                                                                 static_cast<int64_t>(g) * D) + t;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) q[i][u] = g < p.G ? src[8 * i + 4 * u] : 0u;
    }
    __device__ __forceinline__ void scale(const float (&f)[2]) {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) acc[i] *= f[i & 1];
    }
    __device__ __forceinline__ void sum_up(const Params &) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], d);
    }
    // A page (its swizzled K rows at shared address kp, V rows at vp) whose first
    // token is tok0.  logits: where token tok0's go, or null.
    template <bool kWeights>
    __device__ __forceinline__ void page(const Params &p, uint32_t kp, uint32_t vp, const Span &sp,
                                         int tok0, float *logits, float *, int lane) {
        const int g = lane >> 2, t = lane & 3;
        // Row and 16-byte chunk of this lane's part of a 16 x 16 tile (both products).
        const int row = (lane >> 4) * 8 + (lane & 7), half = (lane >> 3) & 1;
        auto at = [&](uint32_t base, int i) {
            return base + (i >> 2) * (kBlock * 128) + row * 128 + (((2 * (i & 3) + half) ^ (row & 7)) << 4);
        };
        float s[2][4] = {};
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];
            ldsm(at(kp, i), a);
            mma(s[i & 1], a[0], a[2], a[1], a[3], q[i][0], q[i][1]);
        }
        float x[4];     // key g, heads 2 t and 2 t + 1; key g + 8, the same
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = (s[0][c] + s[1][c]) * p.scale_log2;
        const bool whole = sp.sees_page(tok0);
        if (!whole) {   // hidden rows hold whatever they hold
            const bool in0 = sp.sees(tok0 + g), in1 = sp.sees(tok0 + g + 8);
            x[0] = in0 ? x[0] : -INFINITY, x[1] = in0 ? x[1] : -INFINITY;
            x[2] = in1 ? x[2] : -INFINITY, x[3] = in1 ? x[3] : -INFINITY;
        }
        if (kWeights) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float *to = logits + (g + 8 * u) * p.G + 2 * t;
                if (2 * t + 1 < p.G)
                    *reinterpret_cast<float2 *>(to) = make_float2(x[2 * u], x[2 * u + 1]);
                else if (2 * t < p.G)
                    *to = x[2 * u];
            }
        }
        float hi[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
        if (__any_sync(0xffffffffu, hi[0] > m[0] || hi[1] > m[1])) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) hi[k] = fmaxf(hi[k], __shfl_xor_sync(0xffffffffu, hi[k], d));
                // A head without a logit above -infinity (or with NaN alone) stays at
                // kLowest, below every logit to come.
                const float to = hi[k] > m[k] ? hi[k] + kLead : m[k];
                f[k] = fast_exp2(m[k] - to);
                m[k] = to;
                l[k] *= f[k];
            }
            scale(f);
        }
        uint32_t w[2], rest[2];     // the weights of keys g and of keys g + 8, turned over
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float e[2], cut[2], more[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                e[k] = fast_exp2(x[2 * u + k] - m[k]);
                l[k] += e[k];
                cut[k] = __uint_as_float(__float_as_uint(e[k]) & 0xffff0000u);
                // Never negative, and not 0: an infinite V stays one.
                more[k] = fmaxf(e[k] - cut[k], e[k] * 0x1p-20f);
            }
            w[u] = turned(__byte_perm(__float_as_uint(cut[0]), __float_as_uint(cut[1]), 0x7632));
            rest[u] = turned(pack_bf16(more[0], more[1]));
        }
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};      // keys 2 t, 2 t + 1, and 8 more
        if (!whole) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                keep[u] = (sp.sees(tok0 + 2 * t + 8 * u) ? 0x0000ffffu : 0u) |
                          (sp.sees(tok0 + 2 * t + 8 * u + 1) ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];
            ldsm_trans(at(vp, i), a);
            a[0] &= keep[0], a[1] &= keep[0], a[2] &= keep[1], a[3] &= keep[1];
            mma(&acc[4 * i], a[0], a[1], a[2], a[3], w[0], w[1]);
            mma(&acc[4 * i], a[0], a[1], a[2], a[3], rest[0], rest[1]);
        }
    }
    // The output, acc times f (as scale()).
    __device__ __forceinline__ void write(const Params &p, void *out0, const float (&f)[2], int lane) {
        const int g = lane >> 2, t = lane & 3;
        uint32_t *to = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(out0) +
                                                    static_cast<int64_t>(g) * D) + t;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t v = turned(pack_bf16(acc[4 * i + 2 * u] * f[0], acc[4 * i + 2 * u + 1] * f[1]));
                if (g < p.G) to[8 * i + 4 * u] = v;
            }
    }
};

// fp32: 8 lanes share a key's dims in the logits; then lane (j, r) has the logits
// of head r and keys j, j + 4, j + 8, j + 12.  In the values a lane has D / 32 dims
// of every head, and the weights come through shared memory.  With one head in a
// group (G = 1) a lane has the logit of one key, and its weight is passed by a
// shuffle: 2.2 times fewer instructions.
template <int D> struct State<float, D> {
    static constexpr int kHeads = 1;
    static constexpr int kDims = D / 32;
    const float *q;
    float4 q1[D / 32];      // G = 1: dims 32 i + 4 r .. of the head
    float m[1], l[1], acc[D / 4];

    static __device__ __forceinline__ int head(int lane, int) { return lane & 7; }
    static __device__ __forceinline__ int head_of(int, int k, int c) { return (4 * k + c) / kDims; }
    static __device__ __forceinline__ int dim(int lane, int k, int c) { return lane * kDims + (4 * k + c) % kDims; }
    __device__ __forceinline__ void load_q(const Params &p, const void *q0, int lane) {
        q = static_cast<const float *>(q0);
        if (p.G == 1) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) q1[i] = __ldg(reinterpret_cast<const float4 *>(q) + 8 * i + (lane & 7));
        }
    }
    __device__ __forceinline__ void scale(const float (&f)[1]) {
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const float fh = __shfl_sync(0xffffffffu, f[0], h);
#pragma unroll
            for (int i = 0; i < kDims; ++i) acc[h * kDims + i] *= fh;
        }
    }
    __device__ __forceinline__ void sum_up(const Params &p) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], 8);
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], 16);
        if (p.G == 1) {     // keys r & 3, on lanes r and r + 4 alike
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], 1);
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], 2);
        }
    }
    template <bool kWeights>
    __device__ __forceinline__ void page1(const Params &p, uint32_t kp, uint32_t vp, const Span &sp, int tok0,
                                          float *logits, int lane) {
        const int j = lane >> 3, r = lane & 7;
        float s[4] = {};
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 k = lds128(kp + ((4 * u + j) * D + 32 * i + 4 * r) * 4);
                s[u] = fmaf(k.w, q1[i].w, fmaf(k.z, q1[i].z, fmaf(k.y, q1[i].y, fmaf(k.x, q1[i].x, s[u]))));
            }
#pragma unroll
        for (int d = 1; d < 8; d <<= 1)
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], d);
        const int key = 4 * (r & 3) + j;
        const float mine = r & 2 ? (r & 1 ? s[3] : s[2]) : (r & 1 ? s[1] : s[0]);
        const float x = sp.sees(tok0 + key) ? mine * p.scale_log2 : -INFINITY;
        if (kWeights && r < 4) logits[key] = x;
        if (__any_sync(0xffffffffu, x > m[0])) {
            float hi = x;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
            const float to = hi > m[0] ? hi + kLead : m[0];
            const float f = fast_exp2(m[0] - to);
            m[0] = to;
            l[0] *= f;
#pragma unroll
            for (int i = 0; i < kDims; ++i) acc[i] *= f;
        }
        const float e = fast_exp2(x - m[0]);
        l[0] += e;
#pragma unroll
        for (int t = 0; t < kBlock; ++t) {
            const float w = __shfl_sync(0xffffffffu, e, (t & 3) * 8 + (t >> 2));
            float v[kDims];
            load_v(v, vp, t, lane);
            const bool in = sp.sees(tok0 + t);      // a hidden row holds whatever it holds
#pragma unroll
            for (int i = 0; i < kDims; ++i) acc[i] = fmaf(w, in ? v[i] : 0.0f, acc[i]);
        }
    }
    static __device__ __forceinline__ void load_v(float (&v)[kDims], uint32_t vp, int t, int lane) {
        if constexpr (kDims == 4) {
            const float4 y = lds128(vp + (t * D + 4 * lane) * 4);
            v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
        } else {
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                         : "=f"(v[0]), "=f"(v[1])
                         : "r"(vp + (t * D + 2 * lane) * 4)
                         : "memory");
        }
    }
    template <bool kWeights>
    __device__ __forceinline__ void page(const Params &p, uint32_t kp, uint32_t vp, const Span &sp,
                                         int tok0, float *logits, float *weights, int lane) {
        if (p.G == 1) return page1<kWeights>(p, kp, vp, sp, tok0, logits, lane);
        const int j = lane >> 3, r = lane & 7;
        float s[4][8] = {};
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            float4 k[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) k[u] = lds128(kp + ((4 * u + j) * D + 32 * i + 4 * r) * 4);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                if (h >= p.G) break;
                const float4 v = __ldg(reinterpret_cast<const float4 *>(q + h * D + 32 * i + 4 * r));
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    s[u][h] = fmaf(k[u].w, v.w, fmaf(k[u].z, v.z, fmaf(k[u].y, v.y, fmaf(k[u].x, v.x, s[u][h]))));
            }
        }
        // Sums over the 8 lanes of a key; lane r keeps head r.
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float a[4], b[2];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                a[h] = (r & 4 ? s[u][h + 4] : s[u][h]) +
                       __shfl_xor_sync(0xffffffffu, r & 4 ? s[u][h] : s[u][h + 4], 4);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                b[h] = (r & 2 ? a[h + 2] : a[h]) + __shfl_xor_sync(0xffffffffu, r & 2 ? a[h] : a[h + 2], 2);
            x[u] = (r & 1 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, r & 1 ? b[0] : b[1], 1);
            x[u] = sp.sees(tok0 + 4 * u + j) ? x[u] * p.scale_log2 : -INFINITY;
            if (kWeights && r < p.G) logits[(4 * u + j) * p.G + r] = x[u];
        }
        float hi = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        if (__any_sync(0xffffffffu, hi > m[0])) {
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 8));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 16));
            const float to = hi > m[0] ? hi + kLead : m[0];
            const float f[1] = {fast_exp2(m[0] - to)};
            m[0] = to;
            l[0] *= f[0];
            scale(f);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float e = fast_exp2(x[u] - m[0]);
            l[0] += e;
            weights[(4 * u + j) * 8 + r] = e;
        }
        __syncwarp();
        const uint32_t w0 = smem_addr(weights);
#pragma unroll 4
        for (int t = 0; t < kBlock; ++t) {
            if (!sp.sees(tok0 + t)) continue;
            const float4 a = lds128(w0 + t * 32), b = lds128(w0 + t * 32 + 16);
            const float w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            float v[kDims];
            load_v(v, vp, t, lane);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                if (h >= p.G) break;
#pragma unroll
                for (int i = 0; i < kDims; ++i) acc[h * kDims + i] = fmaf(w[h], v[i], acc[h * kDims + i]);
            }
        }
    }
    __device__ __forceinline__ void write(const Params &p, void *out0, const float (&f)[1], int lane) {
        float *to = static_cast<float *>(out0) + lane * kDims;
#pragma unroll
        for (int h = 0; h < 8; ++h) {
            const float fh = __shfl_sync(0xffffffffu, f[0], h);
            if (h >= p.G) continue;
#pragma unroll
            for (int i = 0; i < kDims; i += 2)
                *reinterpret_cast<float2 *>(to + h * D + i) =
                    make_float2(acc[h * kDims + i] * fh, acc[h * kDims + i + 1] * fh);
        }
    }
};

template <typename T, int D> __device__ __forceinline__ void clear(State<T, D> &s) {
#pragma unroll
    for (int k = 0; k < State<T, D>::kHeads; ++k) s.m[k] = kLowest, s.l[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 4; ++i) s.acc[i] = 0.0f;
}

__device__ __forceinline__ float sink_of(const Params &p, int h, bool f32) {
    const float s = f32 ? static_cast<const float *>(p.sinks)[h]
                        : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.sinks)[h]);
    return s * kLog2e;
}

// ------------------------------------------------------------------ a warp's ring

// Starts the copies of a K and a V page to a place of the ring.
template <typename T, int D>
__device__ __forceinline__ void start_copy(const Params &p, const CUtensorMap *tmk, const CUtensorMap *tmv,
                                           uint32_t dst, int64_t page, uint32_t bar) {
    constexpr int kBytes = kBlock * D * static_cast<int>(sizeof(T));
    if constexpr (sizeof(T) == 2) {
        asm volatile(
            "{\n .reg .b64 pol;\n createpolicy.fractional.L2::evict_first.b64 pol, 1.0;\n"
            " mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%4], %5;\n"
            " cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%2, {%6, %6, %6, %7}], [%4], pol;\n"
            " cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%1], [%3, {%6, %6, %6, %7}], [%4], pol;\n}" ::"r"(dst),
            "r"(dst + kBytes), "l"(reinterpret_cast<uint64_t>(tmk)), "l"(reinterpret_cast<uint64_t>(tmv)),
            "r"(bar), "r"(2 * kBytes), "r"(0), "r"(static_cast<int>(page))
            : "memory");
    } else {
        const char *k = static_cast<const char *>(p.k_cache) + page * kBytes;
        const char *v = static_cast<const char *>(p.v_cache) + page * kBytes;
        asm volatile(
            "{\n .reg .b64 pol;\n createpolicy.fractional.L2::evict_first.b64 pol, 1.0;\n"
            " mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%4], %5;\n"
            " cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%0], [%2], %6, [%4], pol;\n"
            " cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint "
            "[%1], [%3], %6, [%4], pol;\n}" ::"r"(dst),
            "r"(dst + kBytes), "l"(k), "l"(v), "r"(bar), "r"(2 * kBytes), "r"(kBytes)
            : "memory");
    }
}

template <typename T, int D, int kStages> struct Ring {
    static constexpr int kBytes = 2 * kBlock * D * static_cast<int>(sizeof(T));
    uint32_t at, bars;      // shared addresses
    uint32_t issued = 0, taken = 0;
    bool dead = false;      // a wait ran out: nothing more is started, and all that follows is NaN

    __device__ __forceinline__ void init(const void *places, uint64_t *full) {
        at = smem_addr(places), bars = smem_addr(full);
        const int lane = threadIdx.x & 31;
        if (lane < kStages) mbar_init(full + lane, 1);
        mbar_fence_init();
        __syncwarp();
    }

    __device__ __forceinline__ void start(const Params &p, const CUtensorMap *tmk, const CUtensorMap *tmv,
                                          int32_t id, int hk, int lane) {
        const uint32_t st = issued % kStages;
        if (lane == 0 && !skip_page(issued) &&
            XS_BOUNDS(id >= 0 && id < p.num_blocks && hk >= 0 && hk < p.Hkv, p.err_flag))
            start_copy<T, D>(p, tmk, tmv, at + st * kBytes, static_cast<int64_t>(id) * p.Hkv + hk, bars + 8 * st);
        ++issued;
    }
    static __device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        return ok != 0;
    }
    static __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) {
        bool ok = arrived(bar, parity);
        if (!ok) {
            const uint64_t t0 = global_ns();
            do ok = arrived(bar, parity);
            while (!ok && global_ns() - t0 <= wait_limit());
        }
        return __all_sync(0xffffffffu, ok);
    }
    // Waits for the next page: its shared address; or it did not come (dead) and what
    // is on its way has landed, as far as it does.
    __device__ __forceinline__ uint32_t next(const Params &p, int lane) {
        const uint32_t st = taken % kStages;
        if (!wait(bars + 8 * st, (taken / kStages) & 1)) {
            dead = true;
            if (lane == 0) raise_flag(p.err_flag, XS_FLAG_TIMEOUT);
            for (; taken < issued; ++taken) wait(bars + 8 * (taken % kStages), (taken / kStages) & 1);
            return 0;
        }
        return at + st * kBytes;
    }
};

// The page ids of sequence b's visible pages from i on, one in each lane.
__device__ __forceinline__ int32_t load_ids(const Params &p, int b, const Span &sp, int i) {
    int32_t id = 0;
    if (i < sp.pages && XS_BOUNDS(b < p.B && i >= 0 && sp.page(i) < p.max_blocks, p.err_flag)) {
        id = __ldg(p.tables + static_cast<int64_t>(b) * p.max_blocks + sp.page(i));
        if (id < 0 || id >= p.num_blocks) {
            raise_flag(p.err_flag, XS_FLAG_BAD_BLOCK);
            id = 0;
        }
    }
    return id;
}

template <typename T, int D>
__device__ __forceinline__ const void *query_of(const Params &p, int b, int hk) {
    return static_cast<const T *>(p.q) + b * p.q_stride + static_cast<int64_t>(hk) * p.G * D;
}
template <typename T, int D> __device__ __forceinline__ void *out_of(const Params &p, int b, int hk) {
    return static_cast<T *>(p.out) + (static_cast<int64_t>(b) * p.Hq + hk * p.G) * D;
}
__device__ __forceinline__ int64_t logits_at(const Params &p, int b, int hk, int tok) {
    return ((static_cast<int64_t>(b) * p.Hkv + hk) * p.max_blocks * kBlock + tok) * p.G;
}

// ------------------------------------------------------------------ the line

// A warp's place on the line: sequence b, which starts at `start`, and the warp's
// pages [a, e) of it.
struct Cursor {
    int b, a, e, start;
    Span sp;
    __device__ __forceinline__ void settle(const Params &p, int lo, int hi) {
        sp = span_of(p, b);
        a = min(max(lo - start, 0), sp.pages);
        e = min(hi - start, sp.pages);
        if (sp.pages <= kWholePages) a = 0, e = start >= lo ? sp.pages : 0;
    }
    // To the next sequence; false at the end of the warp's share.
    __device__ __forceinline__ bool advance(const Params &p, int lo, int hi) {
        start += sp.pages + kSegmentCost;
        if (start >= hi) return false;
        ++b;
        settle(p, lo, hi);
        return true;
    }
};

__device__ __forceinline__ float *partial_of(const Params &p, int D, int64_t i, int slot) {
    if (!XS_BOUNDS(i >= 0 && i < kMaxWarps, p.err_flag)) i = 0;
    return p.partials + (2 * i + slot) * partial_floats(D);
}

// The row ends (weights: also kept for the second kernel): factors of the values.
template <typename T, int D, bool kWeights>
__device__ __forceinline__ void finish(const Params &p, State<T, D> &st, int b, int hk, int lane) {
    using S = State<T, D>;
    float f[S::kHeads];
#pragma unroll
    for (int k = 0; k < S::kHeads; ++k) {
        const int h = S::head(lane, k);
        float top = st.m[k], total = st.l[k];
        if (p.sinks && h < p.G) {
            const float sink = sink_of(p, hk * p.G + h, sizeof(T) == 4);
            const float to = fmaxf(top, sink);
            const float w = fast_exp2(top - to);
            total = fmaf(total, w, fast_exp2(sink - to));
            f[k] = w / total;
            top = to;
        } else {
            f[k] = 1.0f / total;
        }
        if (kWeights && h < p.G && lane < 8 && XS_BOUNDS(b < p.B && hk < p.Hkv, p.err_flag))
            p.ends[static_cast<int64_t>(b) * p.Hq + hk * p.G + h] = make_float2(top, 1.0f / total);
    }
    if (XS_BOUNDS(b < p.B && hk < p.Hkv, p.err_flag)) st.write(p, out_of<T, D>(p, b, hk), f, lane);
}

// Joins the partials that KV head hk's warps of groups f .. last left of a segment,
// in order: that of group f its second, the others their first.  kAtOnce are on
// their way at a time (an access to another SM's fresh results takes about 1 us;
// with 6 the line takes up to 4% longer).
template <typename T, int D>
__device__ __forceinline__ void join(const Params &p, State<T, D> &st, int hk, int f, int last, int lane) {
    using S = State<T, D>;
    constexpr int kAtOnce = 4;
    clear(st);
    for (int base = f; base <= last; base += kAtOnce) {
        float4 o[kAtOnce][D / 16];
        float m[kAtOnce][S::kHeads], l[kAtOnce][S::kHeads];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const bool in = base + u <= last;
            const int group = in ? base + u : last;
            const float *src = partial_of(p, D, static_cast<int64_t>(group) * p.Hkv + hk, group == f);
#pragma unroll
            for (int k = 0; k < S::kHeads; ++k) {
                m[u][k] = __ldcg(src + 8 * D + S::head(lane, k));
                l[u][k] = __ldcg(src + 8 * D + 8 + S::head(lane, k));
                if (!in) m[u][k] = kLowest, l[u][k] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                o[u][k] = __ldcg(reinterpret_cast<const float4 *>(src) + 32 * k + lane);
        }
        float to[S::kHeads], w[S::kHeads];
#pragma unroll
        for (int k = 0; k < S::kHeads; ++k) {
            to[k] = st.m[k];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) to[k] = fmaxf(to[k], m[u][k]);
            w[k] = fast_exp2(st.m[k] - to[k]);
            st.m[k] = to[k];
            st.l[k] *= w[k];
        }
        st.scale(w);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (base + u > last) break;
            float g[D / 4];
#pragma unroll
            for (int k = 0; k < S::kHeads; ++k) {
                w[k] = fast_exp2(m[u][k] - to[k]);
                st.l[k] = fmaf(w[k], l[u][k], st.l[k]);
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                g[4 * k] = o[u][k].x, g[4 * k + 1] = o[u][k].y, g[4 * k + 2] = o[u][k].z, g[4 * k + 3] = o[u][k].w;
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) st.acc[i] = fmaf(w[i & 1], g[i], st.acc[i]);
            } else {
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float wh = __shfl_sync(0xffffffffu, w[0], h);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        st.acc[h * (D / 32) + i] = fmaf(wh, g[h * (D / 32) + i], st.acc[h * (D / 32) + i]);
                }
            }
        }
    }
}

// CTAs of the line on an SM (fp32 pages of 128 fill it with one's ring).
template <typename T, int D> __host__ __device__ constexpr int line_ctas() {
    return sizeof(T) == 4 && D == 128 ? 1 : 2;
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, v, d);
        if (static_cast<int>(threadIdx.x & 31) >= d) v += y;
    }
    return v;
}

template <typename S> __device__ __forceinline__ S &shared_of() {
    extern __shared__ __align__(1024) unsigned char bounded_smem[];
    // (The start of the dynamic shared memory need not be a multiple of 1024.)
    return *reinterpret_cast<S *>(bounded_smem + (-smem_addr(bounded_smem) & 1023u));
}

// ------------------------------------------------------------------ weights from logits

// The weights of the tokens at(x), x < count, as far as they are below n, from
// their G logits each, at logits(x), added to their scores; ends: the G rows'
// references and factors.  A thread has kAtOnce tokens under way.
template <int G, typename F, typename L>
__device__ __forceinline__ void add_weights(const Params &p, int b, int hk, int count, F &&at, L &&logits, int n,
                                            int scored, const float2 *ends) {
    using V = typename std::conditional<G == 1, float, typename std::conditional<G == 2, float2, float4>::type>::type;
    constexpr int kPieces = G <= 4 ? 1 : 2, kAtOnce = 4;
    if (!XS_BOUNDS(b < p.B && hk < p.Hkv && n <= p.max_blocks * kBlock, p.err_flag)) return;
    float *scores = p.scores + (static_cast<int64_t>(b) * p.Hkv + hk) * p.max_blocks * kBlock;
    for (int x0 = threadIdx.x; x0 < count; x0 += kAtOnce * blockDim.x) {
        V x[kAtOnce][kPieces];
        float old[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int y = x0 + u * blockDim.x, t = y < count ? at(y) : n;
            if (t >= n) continue;
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                x[u][k] = reinterpret_cast<const V *>(logits(y))[k];
            old[u] = t < scored ? scores[t] : 0.0f;
        }
        float2 end[G];
#pragma unroll
        for (int h = 0; h < G; ++h) end[h] = ends[h];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int y = x0 + u * blockDim.x, t = y < count ? at(y) : n;
            if (t >= n) continue;
            const float *v = reinterpret_cast<const float *>(x[u]);
            float w = 0.0f;
#pragma unroll
            for (int h = 0; h < G; ++h) w = fmaf(fast_exp2(v[h] - end[h].x), end[h].y, w);
            scores[t] = old[u] + w;
        }
    }
}

// Whether the kernel for many segments gives each a CTA: so unless the longest would
// keep its CTA much longer than the others need, or the CTAs' starts and ends would.
// (us, a CTA for each and the line, bf16, 8 KV heads x 128, G = 4: 20 sequences of 300
// tokens 6.3 and 10.4, of 2000 25 and 31; 64 of 1024 41 and 46, of 4096 151 and 161; 128 of
// 3000 220 and 233; 25 of 17 to 8193 76 and 35, 64 of them 90 and 60; 100 of 16 9.2 and 6.0.)
__device__ __forceinline__ bool each_alone(const Params &p, int grid, int line_grid, uint32_t total, uint32_t longest,
                                           int64_t alone, int64_t ends) {
    const int segments = p.B * p.Hkv, waves = (segments + line_grid - 1) / line_grid;  // (32 bits: checked by the host)
    const int64_t all = static_cast<int64_t>(total) * p.Hkv;
    return segments <= grid && longest * alone <= (waves == 1 ? all + all / 4 : all / 2) + ends &&
           (waves - 1) * ends <= all;
}

constexpr int kWeightThreads = 256;
constexpr int kWeightTokens = 1024;     // of a CTA at a time

// How the first kernel was launched, and its constants.
struct FirstKernel {
    int grid, line_grid, alone, ends;
};

// Behind the line (nothing where each segment had a CTA, so few CTAs that take
// piece after piece of kWeightTokens: one for each piece cost 10 us there).  The
// lengths do not change behind the first kernel's own start, which this one's
// follows: they are looked at, and the first piece's old scores fetched, while that
// kernel works.
template <int G>
__global__ void __launch_bounds__(kWeightThreads)
    bounded_weights_kernel(const __grid_constant__ Params p, const int pieces, const FirstKernel first) {
    const int lane = threadIdx.x & 31;
    auto length = [&](int b) {
        return min(XS_BOUNDS(b >= 0 && b < p.B, p.err_flag) ? max(__ldcg(p.lens + b), 0) : 0, p.max_blocks * kBlock);
    };
    uint32_t total = 0, longest = 0;
    // (As the first kernel, which gives no segment a CTA if there are more than CTAs.)
    const int lengths = p.B * p.Hkv <= first.grid ? p.B : 0;
    for (int base = 0; base < lengths; base += 32) {
        const uint32_t pages = base + lane < p.B ? (length(base + lane) + kBlock - 1) / kBlock : 0;
        total += __reduce_add_sync(0xffffffffu, pages);
        longest = max(longest, pages);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    const bool idle = each_alone(p, first.grid, first.line_grid, total, longest, first.alone, first.ends);
    const int64_t items = static_cast<int64_t>(p.B) * p.Hkv * pieces;
    int b = 0, hk = 0, piece = 0, n = 0, scored = 0;
    auto take = [&](int64_t i) {
        const int segment = static_cast<int>(i / pieces);
        piece = static_cast<int>(i - static_cast<int64_t>(segment) * pieces);
        b = segment / p.Hkv, hk = segment - b * p.Hkv;
        n = length(b);
        scored = p.scored ? __ldcg(p.scored + b) : n - 1;
    };
    if (!idle && blockIdx.x < items) {
        take(blockIdx.x);
        const int t = piece * kWeightTokens + 32 * static_cast<int>(threadIdx.x);
        if (threadIdx.x < kWeightTokens / 32 && t < min(n, scored))
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                p.scores + (static_cast<int64_t>(b) * p.Hkv + hk) * p.max_blocks * kBlock + t));
    }
    after_previous();
    if (idle) return;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        if (i != blockIdx.x) take(i);
        for (int from = piece * kWeightTokens; from < n; from += pieces * kWeightTokens)
            add_weights<G>(
                p, b, hk, min(kWeightTokens, n - from), [&](int x) { return from + x; },
                [&](int x) { return p.logits + logits_at(p, b, hk, from + x); }, n, scored,
                p.ends + static_cast<int64_t>(b) * p.Hq + hk * G);
    }
}

// ------------------------------------------------------------------ a CTA's work on a segment

template <typename T, int D, int W, int S> struct alignas(1024) CtaSmem {
    // The pages on their way; when all have been read, the warps' values meet there.
    union {
        uint8_t ring[W][S][2 * kBlock * D * sizeof(T)];
        float4 o[W][8 * D / 4];
    };
    float weights[sizeof(T) == 4 ? W : 1][kBlock * 8];
    float4 part[8 * D / 4];             // what the CTA has
    float m[8], l[8];
    float warp_m[W][8], warp_l[W][8], warp_w[W][8];
    float rank_w[kMaxCluster][8];       // factors of the CTAs' values
    float2 ends[8];
    uint64_t full[W][S];
    alignas(16) float logits[logit_floats<T, D, W>()];      // (the form with weights has them)
};
template <typename T, int D> using ClusterSmem = CtaSmem<T, D, kClusterWarps, cluster_stages<T, D>()>;
template <typename T, int D, bool kWeights> using LineSmem = CtaSmem<T, D, kLineWarps, line_stages<T, D, kWeights>()>;
// (The start of the dynamic shared memory need not be a multiple of 1024.)
template <typename T, int D> constexpr int cluster_smem(bool weights) {
    return 1024 + static_cast<int>(sizeof(ClusterSmem<T, D>)) -
           (weights ? 0 : static_cast<int>(logit_floats<T, D, kClusterWarps>() * sizeof(float)));
}
template <typename T, int D, bool kWeights> constexpr int line_smem() {
    return 1024 + static_cast<int>(sizeof(LineSmem<T, D, kWeights>)) -
           (kWeights ? 0 : static_cast<int>(logit_floats<T, D, kLineWarps>() * sizeof(float)));
}

__device__ __forceinline__ uint32_t peer_addr(const void *own, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(own)), "r"(rank));
    return a;
}
__device__ __forceinline__ float peer_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_f32x4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// Segment (b, hk), or CTA `rank`'s part of it where `ctas` share it, by a CTA of W warps.
template <typename T, int D, bool kWeights, int W, int kStages> struct Segment {
    using S = State<T, D>;
    static constexpr int kGroup = W * kBlock;       // tokens
    static constexpr int kChunks = 8 * D / 4;
    const Params &p;
    CtaSmem<T, D, W, kStages> &sm;
    const int b, hk, rank, ctas;
    Span sp;
    int groups, held;       // groups of pages, and of how many the logits are in shared memory

    // The CTA's pages; what its warps have of them is left in shared memory.  False
    // if the segment is empty (then its output is written).
    __device__ __forceinline__ bool pages(Ring<T, D, kStages> &ring, const CUtensorMap *tmk, const CUtensorMap *tmv,
                                          bool tells) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        S st;
        clear(st);
        st.load_q(p, query_of<T, D>(p, b, hk), lane);
        // The CTA's pages: every ctas-th group of W without a window, which are
        // known before the length is, so that their ids come with it; or an equal run
        // of the window's.
        const bool all = p.window == 0;
        const int32_t *row = p.tables + static_cast<int64_t>(b) * p.max_blocks;
        const int stride = all ? ctas * W : W;
        int at0 = rank * W + warp;      // this warp's first page, the next `stride` behind
        int32_t ids = 0;
        if (all && at0 + lane * stride < p.max_blocks && XS_BOUNDS(b < p.B, p.err_flag))
            ids = __ldg(row + at0 + lane * stride);
        sp = span_of(p, b);
        // A length past its table is told of by the first CTA alone: it looks at all.
        if (tells)
            for (int i = tid; i < p.B; i += 32 * W) span_of(p, i);
        if (sp.pages == 0) {
            if (rank == 0) {
                T *out = static_cast<T *>(out_of<T, D>(p, b, hk));
                for (int x = tid; x < p.G * D; x += 32 * W) out[x] = Elem<T>::from_f32(0.0f);
            }
            return false;       // the whole cluster
        }
        int end = sp.pages;
        if (!all) {
            at0 = static_cast<int>(static_cast<int64_t>(sp.pages) * rank / ctas) + warp;
            end = static_cast<int>(static_cast<int64_t>(sp.pages) * (rank + 1) / ctas);
            ids = load_ids(p, b, sp, at0 + lane * stride);      // (those past `end` are not used)
        } else if (at0 + lane * stride < sp.pages) {
            if (ids < 0 || ids >= p.num_blocks) {
                raise_flag(p.err_flag, XS_FLAG_BAD_BLOCK);
                ids = 0;
            }
        }
        const int mine = (end - at0 + stride - 1) / stride;     // pages of this warp (or <= 0)
        int issued = 0;
        auto start = [&]() {
            if (issued >= mine || ring.dead) return;
            if (issued && (issued & 31) == 0) ids = load_ids(p, b, sp, at0 + (issued + lane) * stride);
            ring.start(p, tmk, tmv, __shfl_sync(0xffffffffu, ids, issued & 31), hk, lane);
            ++issued;
        };
#pragma unroll 1
        for (int k = 0; k < kStages; ++k) start();
        // The logits of the first groups of pages are kept together in shared memory, the
        // others by their tokens in the workspace.
        groups = kWeights ? max(0, (sp.pages - rank * W + stride - 1) / stride) : 0;
        held = kWeights ? min(groups, logit_floats<T, D, W>() / (kGroup * p.G)) : 0;
#pragma unroll 1
        for (int k = 0; k < mine && !ring.dead; ++k) {
            const uint32_t kp = ring.next(p, lane);
            if (ring.dead) break;
            const int tok0 = sp.page(at0 + k * stride) * kBlock;
            float *to = nullptr;
            if (kWeights && XS_BOUNDS(tok0 + kBlock <= p.max_blocks * kBlock, p.err_flag))
                to = k < held ? sm.logits + (k * W + warp) * kBlock * p.G : p.logits + logits_at(p, b, hk, tok0);
            st.template page<kWeights>(p, kp, kp + ring.kBytes / 2, sp, tok0, to,
                                       sm.weights[sizeof(T) == 4 ? warp : 0], lane);
            ++ring.taken;
            __syncwarp();
            start();
        }
        st.sum_up(p);
        if (ring.dead) {
#pragma unroll
            for (int k = 0; k < S::kHeads; ++k) st.l[k] = NAN;
        }
        __syncthreads();    // all pages have been read
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            sm.o[warp][32 * k + lane] = make_float4(st.acc[4 * k], st.acc[4 * k + 1], st.acc[4 * k + 2], st.acc[4 * k + 3]);
        if (lane < 8) {
#pragma unroll
            for (int k = 0; k < S::kHeads; ++k) {
                sm.warp_m[warp][S::head(lane, k)] = st.m[k];
                sm.warp_l[warp][S::head(lane, k)] = st.l[k];
            }
        }
        __syncthreads();
        if (tid < 8 * W) {
            const int w = tid >> 3, h = tid & 7;
            float top = sm.warp_m[0][h];
#pragma unroll
            for (int k = 1; k < W; ++k) top = fmaxf(top, sm.warp_m[k][h]);
            sm.warp_w[w][h] = fast_exp2(sm.warp_m[w][h] - top);
            if (w == 0) {
                float total = 0.0f;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    total = fmaf(fast_exp2(sm.warp_m[k][h] - top), sm.warp_l[k][h], total);
                sm.m[h] = top, sm.l[h] = total;
            }
        }
        __syncthreads();
        return true;
    }
    // Four values of the CTA's (in the layout of the lanes' registers).
    __device__ __forceinline__ float4 combined(int chunk) const {
        const int ln = chunk & 31, k = chunk >> 5;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float4 v = sm.o[w][chunk];
            o.x = fmaf(sm.warp_w[w][S::head_of(ln, k, 0)], v.x, o.x);
            o.y = fmaf(sm.warp_w[w][S::head_of(ln, k, 1)], v.y, o.y);
            o.z = fmaf(sm.warp_w[w][S::head_of(ln, k, 2)], v.z, o.z);
            o.w = fmaf(sm.warp_w[w][S::head_of(ln, k, 3)], v.w, o.w);
        }
        return o;
    }
    // Four values of the output, times the factors of CTA rank_of (-1: none).
    __device__ __forceinline__ void write(int chunk, int rank_of, const float (&v)[4]) const {
        T *out = static_cast<T *>(out_of<T, D>(p, b, hk));
        if (!XS_BOUNDS(b < p.B && hk < p.Hkv, p.err_flag)) return;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int h = S::head_of(chunk & 31, chunk >> 5, c);
            if (h < p.G)
                out[h * D + S::dim(chunk & 31, chunk >> 5, c)] =
                    Elem<T>::from_f32(rank_of < 0 ? v[c] : v[c] * sm.rank_w[rank_of][h]);
        }
    }
    __device__ __forceinline__ void weights() const {
        by_heads(p.G, [&](auto heads) {
            constexpr int G = decltype(heads)::value;
            auto token = [&](int x) { return (x / kGroup * ctas + rank) * kGroup + x % kGroup; };
            auto logits = [&](int x) {
                return x < held * kGroup ? sm.logits + x * G : p.logits + logits_at(p, b, hk, token(x));
            };
            add_weights<G>(p, b, hk, groups * kGroup, token, logits, sp.n, p.scored ? p.scored[b] : sp.n - 1, sm.ends);
        });
    }
    // All of it was this CTA's: the output, and the weights.
    __device__ __forceinline__ void whole() const {
        const int tid = threadIdx.x;
        if (tid < 8) {
            float top = sm.m[tid], total = sm.l[tid], w = 1.0f;
            if (p.sinks && tid < p.G) {
                const float sink = sink_of(p, hk * p.G + tid, sizeof(T) == 4);
                const float to = fmaxf(top, sink);
                w = fast_exp2(top - to);
                total = fmaf(total, w, fast_exp2(sink - to));
                top = to;
            }
            sm.rank_w[0][tid] = w / total;
            sm.ends[tid] = make_float2(top, 1.0f / total);
        }
        __syncthreads();
        for (int chunk = tid; chunk < kChunks; chunk += 32 * W) {
            const float4 o = combined(chunk);
            const float v[4] = {o.x, o.y, o.z, o.w};
            write(chunk, 0, v);
        }
        if (kWeights) weights();
    }
};

// ------------------------------------------------------------ many segments

// A CTA for each segment where the lengths allow it, else the line on the first
// line_grid CTAs.
template <typename T, int D, bool kWeights>
__global__ void __launch_bounds__(32 * kLineWarps, line_ctas<T, D>())
    bounded_many_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                        const __grid_constant__ Params p, const int line_grid) {
    constexpr int kStages = line_stages<T, D, kWeights>();
    LineSmem<T, D, kWeights> &sm = shared_of<LineSmem<T, D, kWeights>>();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int me = blockIdx.x * kLineWarps + warp, warps = line_grid * kLineWarps;
    Ring<T, D, kStages> ring;
    ring.init(sm.ring[warp][0], sm.full[warp]);
    griddep_wait();
    if (kWeights) griddep_launch_dependents();      // the second kernel waits beside this one

    // All pages, and the longest sequence's (every CTA looks at all lengths).
    auto pages_at = [&](int b) { return b < p.B ? static_cast<uint32_t>(span_of(p, b).pages) : 0u; };
    uint32_t pages0[4], longest = 0;
    uint32_t total = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) pages0[u] = pages_at(32 * u + lane);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        total += __reduce_add_sync(0xffffffffu, pages0[u]);
        longest = max(longest, pages0[u]);
    }
#pragma unroll 4
    for (int base = 128; base < p.B; base += 32) {
        const uint32_t pages = pages_at(base + lane);
        total += __reduce_add_sync(0xffffffffu, pages);
        longest = max(longest, pages);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (each_alone(p, static_cast<int>(gridDim.x), line_grid, total, longest, kAlone<T, D>, kEnds<T, D>)) {
        if (static_cast<int>(blockIdx.x) >= p.B * p.Hkv) return;
        const int b = blockIdx.x / p.Hkv, hk = blockIdx.x - b * p.Hkv;
        Segment<T, D, kWeights, kLineWarps, kStages> seg{p, sm, b, hk, 0, 1};
        if (seg.pages(ring, &tmk, &tmv, false)) seg.whole();
        return;
    }
    if (static_cast<int>(blockIdx.x) >= line_grid) return;
    // The line; then the sequence in which this warp's share begins.
    const int line = static_cast<int>(total) + p.B * kSegmentCost;      // (32 bits hold it: checked by the host)
    // Shares no smaller than is best for the longest segment, whose n / share parts
    // are joined one after the other while a part takes its share's time.
    const int least = max(kMinShare, static_cast<int>(sqrtf(0.5f * longest)));
    const int groups = min(warps / p.Hkv, max(line / least, 1));
    const int group = me / p.Hkv, hk = me - group * p.Hkv;
    if (group >= groups) return;
    // The first `longer` shares are one page longer than the others.
    const int share = line / groups, longer = line - share * groups;
    const int lo = share * group + min(group, longer), hi = lo + share + (group < longer);
    auto group_at = [&](int x) {
        const int y = x - longer * (share + 1);
        return y < 0 ? x / (share + 1) : longer + y / share;
    };
    Cursor at;
    {
        int before = 0;
        bool found = false;
        auto look = [&](int base, uint32_t pages) {     // among sequences base .. base + 31
            const int units = base + lane < p.B ? static_cast<int>(pages) + kSegmentCost : 0;
            const int sum = static_cast<int>(warp_scan(units)), end = before + sum, s = end - units;
            before = __shfl_sync(0xffffffffu, end, 31);
            const uint32_t who = __ballot_sync(0xffffffffu, lo >= s && lo < end);
            if (!who) return;
            found = true;
            const int src = __ffs(who) - 1;
            at.b = base + src;
            at.start = __shfl_sync(0xffffffffu, s, src);
        };
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (!found && 32 * u < p.B) look(32 * u, pages0[u]);
        for (int base = 128; !found && base < p.B; base += 32) look(base, pages_at(base + lane));
        if (!found) return;
    }
    at.settle(p, lo, hi);

    // Copies run ahead of the work, across the ends of segments.
    Cursor ahead = at;
    int next = ahead.a, chunk = next;
    bool more = true;
    int32_t ids = load_ids(p, ahead.b, ahead.sp, chunk + lane);
    auto start = [&]() {
        while (more && next >= ahead.e) {
            more = ahead.advance(p, lo, hi);
            if (!more) return;
            next = chunk = ahead.a;
            if (next < ahead.e) ids = load_ids(p, ahead.b, ahead.sp, chunk + lane);
        }
        if (!more) return;
        if (next - chunk == 32) {
            chunk = next;
            ids = load_ids(p, ahead.b, ahead.sp, chunk + lane);
        }
        ring.start(p, &tmk, &tmv, __shfl_sync(0xffffffffu, ids, next - chunk), hk, lane);
        ++next;
    };
#pragma unroll 1
    for (int k = 0; k < kStages; ++k) start();

    State<T, D> st;
    do {
        const Span &sp = at.sp;
        if (sp.pages == 0) {
            if (at.start >= lo && XS_BOUNDS(at.b < p.B && hk < p.Hkv, p.err_flag)) {
                T *out = static_cast<T *>(out_of<T, D>(p, at.b, hk));
                for (int x = lane; x < p.G * D; x += 32) out[x] = Elem<T>::from_f32(0.0f);
            }
            continue;
        }
        if (at.a >= at.e) continue;
        clear(st);
        st.load_q(p, query_of<T, D>(p, at.b, hk), lane);
#pragma unroll 1
        for (int k = at.a; k < at.e && !ring.dead; ++k) {
            const uint32_t kp = ring.next(p, lane);
            if (ring.dead) break;
            const int tok0 = sp.page(k) * kBlock;
            float *logits = nullptr;
            if (kWeights && XS_BOUNDS(tok0 + kBlock <= p.max_blocks * kBlock, p.err_flag))
                logits = p.logits + logits_at(p, at.b, hk, tok0);
            st.template page<kWeights>(p, kp, kp + ring.kBytes / 2, sp, tok0, logits,
                                       sm.weights[sizeof(T) == 4 ? warp : 0], lane);
            ++ring.taken;
            __syncwarp();
            start();
        }
        st.sum_up(p);
        if (ring.dead) {
#pragma unroll
            for (int k = 0; k < State<T, D>::kHeads; ++k) st.l[k] = NAN;
        }
        if (at.a > 0 || at.e < sp.pages) {
            // A part: the last of the segment's warps joins them all.
            float *part = partial_of(p, D, me, at.a == 0);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                __stcg(reinterpret_cast<float4 *>(part) + 32 * k + lane,
                       make_float4(st.acc[4 * k], st.acc[4 * k + 1], st.acc[4 * k + 2], st.acc[4 * k + 3]));
            if (lane < 8) {
#pragma unroll
                for (int k = 0; k < State<T, D>::kHeads; ++k) {
                    __stcg(part + 8 * D + State<T, D>::head(lane, k), st.m[k]);
                    __stcg(part + 8 * D + 8 + State<T, D>::head(lane, k), st.l[k]);
                }
            }
            const int f = group_at(at.start);
            const int last = group_at(at.start + sp.pages - 1);
            __syncwarp();
            int joins = 0;
            if (lane == 0 && XS_BOUNDS(f >= 0 && f <= last && last < groups, p.err_flag)) {
                int *count = p.counters + f * p.Hkv + hk;
                joins = atomic_add_acq_rel_gpu(count, 1) == last - f;
                if (joins) *count = 0;
            }
            joins = __shfl_sync(0xffffffffu, joins, 0);
            __syncwarp();
            if (!joins) continue;
            join<T, D>(p, st, hk, f, last, lane);
        }
        finish<T, D, kWeights>(p, st, at.b, hk, lane);
    } while (at.advance(p, lo, hi));
}

// ------------------------------------------------------------------ clusters

// A cluster of `ctas` (a power of two) for each segment.
template <typename T, int D, bool kWeights>
__global__ void __launch_bounds__(32 * kClusterWarps, 1)
    bounded_cluster_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                           const __grid_constant__ Params p, const int ctas) {
    using Seg = Segment<T, D, kWeights, kClusterWarps, cluster_stages<T, D>()>;
    using S = State<T, D>;
    constexpr int kChunks = Seg::kChunks;
    ClusterSmem<T, D> &sm = shared_of<ClusterSmem<T, D>>();
    const int tid = threadIdx.x;
    Ring<T, D, cluster_stages<T, D>()> ring;
    ring.init(sm.ring[tid >> 5][0], sm.full[tid >> 5]);
    griddep_wait();
    const int rank = blockIdx.x % ctas, segment = blockIdx.x / ctas;
    const int b = segment / p.Hkv, hk = segment - b * p.Hkv;
    Seg seg{p, sm, b, hk, rank, ctas};
    if (!seg.pages(ring, &tmk, &tmv, blockIdx.x == 0)) return;
    if (ctas == 1) return seg.whole();
    if (tid < kChunks) sm.part[tid] = seg.combined(tid);
    // The CTAs' parts meet.
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    const int per = (kChunks + ctas - 1) / ctas;        // chunks of this CTA
    const int from = tid % ctas, mine_at = tid / ctas, chunk = rank * per + mine_at;
    const bool valid = mine_at < per && chunk < kChunks;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (valid) o = peer_f32x4(peer_addr(&sm.part[chunk], from));
    if (tid < 8 * ctas) {
        const int h = tid / ctas;
        const float mr = peer_f32(peer_addr(&sm.m[h], from)), lr = peer_f32(peer_addr(&sm.l[h], from));
        const uint32_t who = ctas == 2 ? 0xffffu : 0xffffffffu;     // (8 ctas threads)
        float top = mr;
        for (int d = ctas / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(who, top, d));
        float sink = 0.0f;
        const bool sinks = p.sinks && h < p.G;
        if (sinks) {
            sink = sink_of(p, hk * p.G + h, sizeof(T) == 4);
            top = fmaxf(top, sink);
        }
        const float w = fast_exp2(mr - top);
        float total = w * lr;
        for (int d = ctas / 2; d > 0; d >>= 1) total += __shfl_xor_sync(who, total, d);
        if (sinks) total += fast_exp2(sink - top);
        sm.rank_w[from][h] = w / total;
        if (from == 0) sm.ends[h] = make_float2(top, 1.0f / total);
    }
    __syncthreads();
    {
        const int ln = chunk & 31, k = chunk >> 5;
        float v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (valid) v[c] *= sm.rank_w[from][S::head_of(ln, k, c)];
            for (int d = ctas / 2; d > 0; d >>= 1) v[c] += __shfl_xor_sync(0xffffffffu, v[c], d);
        }
        if (valid && from == 0) seg.write(chunk, -1, v);
    }
    // No CTA leaves before all have read its shared memory (what they read has
    // been used above).
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    if (kWeights) seg.weights();
    asm volatile("barrier.cluster.wait;" ::: "memory");
}

// ------------------------------------------------------------------ host side

template <typename T, int D, bool kWeights> int clusters_held(int ctas) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * kClusterWarps);
    cfg.dynamicSmemBytes = cluster_smem<T, D>(kWeights);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, bounded_cluster_kernel<T, D, kWeights>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return n;
}

// What a device holds of the cluster kernel at once, in clusters of 2, 4 and 8.
// Asked for once for each device (by two threads at once: twice, with one answer).
struct Held {
    int of[3];
};
template <typename T, int D, bool kWeights> int configure(int dev, Held *held) {
    static std::atomic<uint64_t> known[64];     // 20 bits each, and 1 in the top one; 0: not yet
    uint64_t v = dev < 64 ? known[dev].load(std::memory_order_acquire) : 0;
    if (!v) {
        if (cudaFuncSetAttribute(bounded_many_kernel<T, D, kWeights>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 line_smem<T, D, kWeights>()) != cudaSuccess ||
            cudaFuncSetAttribute(bounded_cluster_kernel<T, D, kWeights>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 cluster_smem<T, D>(kWeights)) != cudaSuccess) {
            cudaGetLastError();
            return XS_EDEVICE;
        }
        v = 1ull << 63;
        for (int i = 0; i < 3; ++i) {
            const int n = clusters_held<T, D, kWeights>(2 << i);
            if (n < 0) return XS_EDEVICE;
            v |= static_cast<uint64_t>(n) << (20 * i);
        }
        if (dev < 64) known[dev].store(v, std::memory_order_release);
    }
    for (int i = 0; i < 3; ++i) held->of[i] = static_cast<int>(v >> (20 * i) & 0xfffff);
    return XS_OK;
}

template <typename T, int D, bool kWeights> int launch(const Params &p, int dev, int sms, cudaStream_t stream) {
    Held held;
    int rc = configure<T, D, kWeights>(dev, &held);
    if (rc != XS_OK) return rc;
    CUtensorMap tmk = {}, tmv = {};
    if (sizeof(T) == 2) {
        // The pool as (64, 16, D / 64, pages): a page's copy is D / 64 swizzled halves of 16 rows.
        const cuuint64_t dims[4] = {64, kBlock, D / 64, static_cast<cuuint64_t>(p.num_blocks) * p.Hkv};
        const cuuint64_t strides[3] = {D * 2, 128, kBlock * D * 2};
        const cuuint32_t box[4] = {64, kBlock, D / 64, 1};
        rc = encode_bf16_map<4>(&tmk, p.k_cache, dims, strides, box);
        if (rc == XS_OK) rc = encode_bf16_map<4>(&tmv, p.v_cache, dims, strides, box);
        if (rc != XS_OK) return rc;
    }
    const int64_t segments = static_cast<int64_t>(p.B) * p.Hkv;
    const int64_t most = p.window > 0 ? min(p.max_blocks, p.first / kBlock + p.window / kBlock + 3) : p.max_blocks;
    // The largest clusters that the device holds at once (15 of 8 CTAs, 36 of 4 and 76
    // of 2: their CTAs are of one group of SMs).  us, clusters of 8, 4, 2, and the line:
    // one sequence of 8 KV heads and 4K tokens 7.1, 9.5, 14.6, 22.7; 16 KV heads, one
    // too many for 8, 13.4, 9.6, 14.7; 36 (1K tokens) -, 5.9, 6.8, 12.3; 37 -, 10.2, 6.8.
    int ctas = 0;
    for (int i = 0; i < 3; ++i)
        if (segments <= held.of[i]) ctas = 2 << i;
    // Or a CTA of 8 warps for each, all at once; under a wide table one long sequence
    // could keep the others waiting.  (us, so and by the kernel for many: 100 segments of
    // 300 tokens 4.9 and 5.4, of 1024 8.5 and 11.9; one of 4000 and 99 of 100 24 and 17.)
    if (!ctas && segments <= sms && most <= kShortTable) ctas = 1;
    if (ctas)
        return launch_after(bounded_cluster_kernel<T, D, kWeights>, dim3(static_cast<int>(segments) * ctas),
                            32 * kClusterWarps, cluster_smem<T, D>(kWeights), stream, ctas, tmk, tmv, p, ctas);
    const int fill = min(sms * line_ctas<T, D>(), kMaxWarps / kLineWarps);
    if (p.Hkv > fill * kLineWarps) return XS_EUNSUPPORTED;
    // The line is at most so long, and no group takes less than kMinShare of it.
    const int64_t want_groups = (static_cast<int64_t>(p.B) * (most + kSegmentCost) + kMinShare - 1) / kMinShare;
    const int64_t want = (want_groups * p.Hkv + kLineWarps - 1) / kLineWarps;
    const int line_grid = static_cast<int>(want < fill ? want : fill);
    const int grid = static_cast<int>(p.B <= kScannedB && segments > line_grid ? segments : line_grid);
    rc = launch_after(bounded_many_kernel<T, D, kWeights>, dim3(grid), 32 * kLineWarps, line_smem<T, D, kWeights>(),
                      stream, 1, tmk, tmv, p, line_grid);
    if (!kWeights || rc != XS_OK) return rc;
    const int pieces = max(1, min((p.max_blocks * kBlock + kWeightTokens - 1) / kWeightTokens, 8));
    const auto second = p.G == 1   ? bounded_weights_kernel<1>
                        : p.G == 2 ? bounded_weights_kernel<2>
                        : p.G == 4 ? bounded_weights_kernel<4>
                                   : bounded_weights_kernel<8>;
    const int64_t items = segments * pieces, at_once = static_cast<int64_t>(sms) * 5;
    return launch_after(second, dim3(static_cast<int>(items < at_once ? items : at_once)), kWeightThreads, 0, stream, 1,
                        p, pieces,
                        FirstKernel{grid, line_grid, static_cast<int>(kAlone<T, D>), static_cast<int>(kEnds<T, D>)});
}

constexpr size_t kCounterBytes = kMaxWarps * sizeof(int);
size_t partial_bytes(int D) { return static_cast<size_t>(kMaxWarps) * 2 * partial_floats(D) * sizeof(float); }

int check_and_launch(Params &p, bool weights, int D, int block_size, float scale, int dtype, void *workspace,
                     size_t workspace_bytes, cudaStream_t stream) {
    if (!p.out || !p.q || !p.k_cache || !p.v_cache || !p.tables || !p.lens || (weights && !p.scores))
        return XS_ENULL;
    const int size = elem_bytes(dtype);
    if (!size) return XS_EDTYPE;
    if (p.B < 0 || p.Hq <= 0 || p.Hkv <= 0 || p.Hq % p.Hkv != 0 || D <= 0 || block_size <= 0 || p.max_blocks < 0 ||
        p.num_blocks < 0 || p.first < 0 || p.window < 0 || p.q_stride < static_cast<int64_t>(p.Hq) * D)
        return XS_ESHAPE;
    p.G = p.Hq / p.Hkv;
    if ((D != 64 && D != 128) || block_size != kBlock || (p.G != 1 && p.G != 2 && p.G != 4 && p.G != 8) ||
        p.Hkv > 512 || p.max_blocks > (1 << 26) || p.q_stride * size % 16 != 0 ||
        p.num_blocks > 0x7fffffff / p.Hkv ||                                  // a tensor copy's coordinate
        static_cast<int64_t>(p.B) * p.Hkv > 0x7fffffff / kMaxCluster ||
        static_cast<int64_t>(p.B) * (p.max_blocks + kSegmentCost) > 0x7fffffff)    // the line, in pages
        return XS_EUNSUPPORTED;
    if (!aligned16(p.out) || !aligned16(p.q) || !aligned16(p.k_cache) || !aligned16(p.v_cache) || !aligned16(workspace))
        return XS_EALIGN;
    if (p.B == 0) return XS_OK;
    if (p.num_blocks == 0) return XS_ESHAPE;
    const size_t need = weights ? xs_paged_decode_weights_workspace_bytes(p.B, p.Hq, p.Hkv, D, p.max_blocks)
                                : xs_paged_decode_first_workspace_bytes(p.B, p.Hq, p.Hkv, D);
    if (!workspace || workspace_bytes < need) return XS_EWORKSPACE;
    p.scale_log2 = scale * kLog2e;
    char *at = static_cast<char *>(workspace);
    p.counters = reinterpret_cast<int *>(at), at += kCounterBytes;
    p.partials = reinterpret_cast<float *>(at), at += partial_bytes(D);
    if (weights) {
        p.ends = reinterpret_cast<float2 *>(at);
        at += (static_cast<size_t>(p.B) * p.Hq * sizeof(float2) + 15) / 16 * 16;
        p.logits = reinterpret_cast<float *>(at);
    }
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return XS_EDEVICE;
    if (dtype == XS_F32)
        return D == 128 ? (weights ? launch<float, 128, true>(p, dev, sms, stream) : launch<float, 128, false>(p, dev, sms, stream))
                        : (weights ? launch<float, 64, true>(p, dev, sms, stream) : launch<float, 64, false>(p, dev, sms, stream));
    using H = __nv_bfloat16;
    return D == 128 ? (weights ? launch<H, 128, true>(p, dev, sms, stream) : launch<H, 128, false>(p, dev, sms, stream))
                    : (weights ? launch<H, 64, true>(p, dev, sms, stream) : launch<H, 64, false>(p, dev, sms, stream));
}

}  // namespace
}  // namespace bounded
XS_DEFINE_BOUNDS_COUNTER(bounds_failures_bounded)

}  // namespace xs

extern "C" int xs_debug_bounded_wait_injection(int64_t wait_limit_ns, int skip_page) {
#ifdef XS_DEBUG_BOUNDS
    if (wait_limit_ns <= 0 || skip_page < -1) return XS_ESHAPE;
    const unsigned long long limit = static_cast<unsigned long long>(wait_limit_ns);
    if (cudaMemcpyToSymbol(xs::bounded::g_wait_limit_ns, &limit, sizeof(limit)) != cudaSuccess ||
        cudaMemcpyToSymbol(xs::bounded::g_skip_page, &skip_page, sizeof(skip_page)) != cudaSuccess) {
        cudaGetLastError();
        return XS_EDEVICE;
    }
    return XS_OK;
#else
    (void)wait_limit_ns;
    (void)skip_page;
    return XS_EUNSUPPORTED;
#endif
}

extern "C" size_t xs_paged_decode_first_workspace_bytes(int B, int Hq, int Hkv, int D) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return 0;
    return xs::bounded::kCounterBytes + xs::bounded::partial_bytes(D);
}

extern "C" size_t xs_paged_decode_weights_workspace_bytes(int B, int Hq, int Hkv, int D, int max_blocks_per_seq) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_blocks_per_seq < 0) return 0;
    return xs_paged_decode_first_workspace_bytes(B, Hq, Hkv, D) +
           (static_cast<size_t>(B) * Hq * sizeof(float2) + 15) / 16 * 16 +
           static_cast<size_t>(B) * Hq * max_blocks_per_seq * xs::bounded::kBlock * sizeof(float);
}

extern "C" int xs_paged_decode_first(void *out, const void *q, int64_t q_stride, const void *k_cache,
                                     const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                                     const int32_t *context_lens, const void *sinks, int first, int window, int B,
                                     int Hq, int Hkv, int D, int block_size, int64_t num_blocks, float scale,
                                     void *workspace, size_t workspace_bytes, int dtype, int *err_flag,
                                     cudaStream_t stream) {
    xs::bounded::Params p = {};
    p.out = out, p.q = q, p.q_stride = q_stride, p.k_cache = k_cache, p.v_cache = v_cache;
    p.tables = block_tables, p.lens = context_lens, p.sinks = sinks;
    p.max_blocks = max_blocks_per_seq, p.first = first, p.window = window;
    p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.num_blocks = num_blocks, p.err_flag = err_flag;
    return xs::bounded::check_and_launch(p, false, D, block_size, scale, dtype, workspace, workspace_bytes, stream);
}

extern "C" int xs_paged_decode_weights(void *out, float *scores, const int32_t *scored_lens, const void *q,
                                       int64_t q_stride, const void *k_cache, const void *v_cache,
                                       const int32_t *block_tables, int max_blocks_per_seq,
                                       const int32_t *context_lens, const void *sinks, int B, int Hq, int Hkv, int D,
                                       int block_size, int64_t num_blocks, float scale, void *workspace,
                                       size_t workspace_bytes, int dtype, int *err_flag, cudaStream_t stream) {
    xs::bounded::Params p = {};
    p.out = out, p.q = q, p.q_stride = q_stride, p.k_cache = k_cache, p.v_cache = v_cache;
    p.tables = block_tables, p.lens = context_lens, p.sinks = sinks;
    p.max_blocks = max_blocks_per_seq;
    p.scores = scores, p.scored = scored_lens;
    p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.num_blocks = num_blocks, p.err_flag = err_flag;
    return xs::bounded::check_and_launch(p, true, D, block_size, scale, dtype, workspace, workspace_bytes, stream);
}
