// Decode attention over a cache held in 4 bits (pages as in kv4.cuh): each
// sequence's one query token attends over all of its pages.
//
//     out[b, h] = sum_t softmax_t(scale q[b, h] . K_t) V_t
//     K_t = s_tc (n_td - 8) for d in group c, V_t the same
//
// A page of one KV head serves the G = Hq / Hkv query heads of its group, on
// m16n8k16 matrix instructions:
//
//   logits   S[h, t] = sum_c s_tc (sum_{d in c} n_td q_hd - 8 sum_{d in c} q_hd),
//            keys on the 16 rows, heads on the 8 columns, fp16.  A
//            pair of codes masked out of its word is the fp16 pair n 2^-24
//            (or n 2^-20 one nibble higher), exactly: no conversion.  q is
//            scaled by a power of two to below 2^16, by 1 / 16 more where it
//            meets the higher nibbles; its bf16 significand fits fp16.  The
//            group's scale is applied to the fp32 sum, so a logit is an fp32
//            sum of exact products.  - 8 sum q is what the sum starts at.  The
//            16 x 8 logits are then turned over between the lanes (8 shuffles),
//            since the second product wants p with its keys along a lane.
//            (Heads on the rows need no turning, but half of the rows and twice
//            the matrix instructions: 158 us where this took 154 us, both with
//            weights of a single rounding.)
//   values   O[d, h] = sum_t (n_td - 8) (p_th s_tc), dims on the rows, heads on
//            the columns, bf16, whose range p s needs.  p s is one product in
//            fp32, which enters as the sum of two bf16 values, what it rounds to
//            and what that leaves (2^-16 of it is lost): with the first alone
//            (2^-8) the output was off by 0.0023 of its size where fp32 weights
//            leave 0.0017, its own rounding, and the long batch took 154 us in
//            place of 171.  n - 8 is exact.  The scale meets p, not the codes:
//            4 products for a token and head in place of D.
//
// What bounds it (32 sequences of 4K to 32K tokens, 32q/8kv x 128, 680 MB): 171 us,
// 4.0 TB/s, by the instructions of a page and their latencies.  An earlier form
// took 113 us with both products left out (copies, waits and softmax alone).  A
// page takes 397 instructions of a warp; the integer pipe, which takes one every
// other cycle, is busy 55% of the time, issue slots 59%, the matrix pipe 29%, DRAM
// 50%.  With weights of a single rounding, more or fewer warps, two pages at a
// time, the next page's logits beside this one's values, multiplications for
// shifts, and 8-bit matrix instructions all measured the same or slower.
//
// The softmax is online, in fp32.  Its reference is set 8 above the running
// maximum (of logits in powers of two), and again only when a logit exceeds it, so
// most pages take no exchange between lanes, and no weight is above 1: a weight
// times the scale of a V group near the end of bf16 stays finite.
//
// Each warp works on pages of its own, which reach its ring of kStages places
// in shared memory by bulk copies (one for K, one for V) that lane 0 starts
// kStages pages ahead.  A lane's share of a page is a few 16-byte pieces that
// need no further exchange, so a page is waited for, read and given back with
// no barrier but the warp's own.
//
// Split: the pages of all sequences and KV heads form one line, each sequence
// and head ("segment") with kSegmentCost more for its start and end.  The line
// is cut into equal shares, one for each CTA, whatever the lengths are: CTA i
// finds its place from the lengths themselves, so the host needs to know none
// of them and a captured call follows them.  A segment that one CTA does is
// written at once.  One that is cut leaves fp32 partials in the workspace, at
// most two for each CTA whatever the batch, and the CTA that finishes it last
// joins them in order: the result does not depend on which that is.  Where
// segments are few, or short and not too many, thread-block clusters take them
// (kv4_decode_few_kernel, kv4_decode_short_kernel).
#include <atomic>

#include <cuda_fp16.h>

#include "kv4.cuh"

namespace xs {
namespace {

// Warps of a CTA, and CTAs on an SM (16 warps of 128 registers): small CTAs
// where segments are many and often end, larger ones where a segment has many
// CTAs and what they leave is joined (a 64-sequence step 48 us with 8 warps, 41 us with 4).
__host__ __device__ constexpr int dec_warps(bool few) { return few ? 8 : 4; }
__host__ __device__ constexpr int ctas_per_sm(bool few) { return 16 / dec_warps(few); }
constexpr int kMaxCtas = 1024;     // the workspace holds partials for so many
constexpr int kSegmentCost = 16;   // pages
constexpr int kMinShare = 16;      // pages
// Segments up to so many pages are not cut: a join costs more (64 segments of
// 100, 300, 500 tokens 5.9, 8.0, 9.5 us so, 8.7, 10.3, 10.7 us cut; of 1000 15.4 us so, 11.9 us).
constexpr int kWholePages = 32;
constexpr int kCluster = 8;        // CTAs of a cluster (of 16: 1.5 us more for a start)
constexpr int kClusterPages = 256; // of a segment: up to so many a cluster always does it
constexpr int kLineCluster = 4;    // CTAs of 4 warps of a cluster, for tables of up to
constexpr int kShortTable = 128;   // so many pages
// Of a cluster's segment: up to so many pages (2 of a warp) one CTA does alone (18
// sequences of 200 tokens, 13 pages: 8.3 us so, 6.3 us by a cluster).
__host__ __device__ constexpr int alone_pages(int warps) { return 2 * warps; }
constexpr int kStages = 4;         // pages of a warp's ring
constexpr float kLead = 8.0f;      // of a reference before the largest logit
constexpr float kLowest = -3.402823466e38f;     // a reference before any logit above it
constexpr uint64_t kWaitLimitNs = 4000000000ull;
// In the debug library the limit can be set, and a page of CTA 0's first warp
// left out, so that its wait runs out (xs_debug_kv4_wait_injection).
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

// d = A B + d
__device__ __forceinline__ void mma_f16(float *d, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float *c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes j and j + 4 of a word, as fp16: n 2^-24 for even j, n 2^-20 for odd.
__device__ __forceinline__ uint32_t codes_f16(uint32_t w, int j) {
    return (j & 2 ? w >> 8 : w) & (j & 1 ? 0x00f000f0u : 0x000f000fu);
}
// The same codes as bf16 n - 8: 0x4300 | n is 128 + n, and the difference is exact.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, int j) {
    uint32_t x;
    const uint32_t off = 0x43084308u;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w >> (4 * j)), "r"(0x000f000fu), "r"(0x43004300u));
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&off));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t pack_bf16(F2 v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N 32-bit words (8 or 16 bytes) at shared address a.
template <int N> __device__ __forceinline__ void load_words(uint32_t *r, uint32_t a) {
    if constexpr (N == 1)
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(a) : "memory");
    else if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(a)
                     : "memory");
    else
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}

struct Kv4DecodeParams {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const uint8_t *k_cache, *v_cache;
    const int32_t *tables, *lens;
    const __nv_bfloat16 *sinks;
    int max_blocks, window, B, Hq, Hkv, G;
    int64_t num_blocks;
    float scale_log2;
    int *counters;      // [gridDim.x]: arrivals at the segment that CTA i begins and does not end
    float *partials;    // [gridDim.x][2] of partial_floats(G, D)
    int *err_flag;
};

// The pages that sequence b's window covers: the first, and how many.
struct Span {
    int n, first, page0, pages;  // tokens [first, n)
};
__device__ __forceinline__ Span span_of(const Kv4DecodeParams &p, int b) {
    Span s;
    s.n = XS_BOUNDS(b >= 0 && b < p.B, p.err_flag) ? p.lens[b] : 0;
    if (s.n > p.max_blocks * 16) {
        if (blockIdx.x == 0) raise_flag(p.err_flag, XS_FLAG_BAD_LEN);
        s.n = p.max_blocks * 16;
    }
    s.n = max(s.n, 0);
    s.first = p.window > 0 && s.n > p.window ? s.n - p.window : 0;
    s.page0 = s.first >> 4;
    s.pages = ((s.n + 15) >> 4) - s.page0;
    return s;
}

// Floats of one CTA's partial: o [G][D], then m [G] and l [G]; whole 16 bytes.
__host__ __device__ constexpr int64_t partial_floats(int G, int D) {
    return (static_cast<int64_t>(G) * (D + 2) + 3) / 4 * 4;
}

// Partial `slot` of CTA i.
__device__ __forceinline__ float *partial_of(const Kv4DecodeParams &p, int D, int64_t i, int slot) {
    if (!XS_BOUNDS(i >= 0 && i < gridDim.x && gridDim.x <= kMaxCtas, p.err_flag)) i = 0;
    return p.partials + (2 * i + slot) * partial_floats(p.G, D);
}

template <int D, bool kFew> struct alignas(16) DecodeSmem {
    static constexpr int kDecWarps = dec_warps(kFew);
    // The pages on their way (K page, V page).  Between segments, when none are,
    // the warps' values meet there (rows padded, for the banks).
    union {
        uint8_t ring[kDecWarps][kStages][2][kv4_page_bytes(D)];
        float o[kDecWarps][8][D + 4];
    };
    uint64_t full[kDecWarps][kStages];
    // The logits' second operand for each group, two steps of 16 dims, as a lane's
    // four registers, and what the sums of heads 2 t, 2 t + 1 start at, twice.
    uint4 q[D / 32][32];
    float4 start_at[D / 32][4];
    float m[kDecWarps][8], l[kDecWarps][8];
    float weight[kDecWarps * 8];
    alignas(16) float part[8 * (D + 2)];    // what the CTA leaves for its cluster
    // The CTA's place: segment (b, hk), pages [a, e) of it, shared by the CTAs
    // f .. last.  Here so that it holds no registers while a segment runs.
    int b, hk, a, e, f, last, joins;
    int64_t start, share, line;         // on a line: where the segment starts, ...
};

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, v, d);
        if (static_cast<int>(threadIdx.x & 31) >= d) v += y;
    }
    return v;
}

// Copies of a K and a V page to shared address dst and behind it, counted on
// the barrier at shared address bar.  Each byte is read once: evict first.
__device__ __forceinline__ void start_copy(uint32_t dst, const uint8_t *k, int bytes,
                                           const uint8_t *v, uint32_t bar) {
    asm volatile(
        "{\n .reg .b64 pol;\n createpolicy.fractional.L2::evict_first.b64 pol, 1.0;\n"
        " mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%4], %5;\n"
        " cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1], %2, [%4], pol;\n"
        " cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%6], [%3], %2, [%4], pol;\n}" ::"r"(dst),
        "l"(k), "r"(bytes), "l"(v), "r"(bar), "r"(2 * bytes), "r"(dst + bytes)
        : "memory");
}

// Waits for a ring place with a limit, all lanes alike: false if it ran out.
__device__ __forceinline__ bool warp_waits(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, wait_limit()));
}

// A warp's ring since the launch: the pages taken from it, and whether a wait
// ran out (then nothing more is started, and all that the CTA does is NaN).
struct RingState {
    uint32_t taken = 0;
    bool dead = false;
};

// Pages [a, e) of one segment: what the CTA's warps leave in shared memory is
// joined and either written out (whole) or left at `part`.
template <int D, bool kFew>
__device__ __forceinline__ void run_segment(const Kv4DecodeParams &p, DecodeSmem<D, kFew> &sm,
                                            RingState &ring, int b, int hk, const Span &sp, int a,
                                            int e, bool whole, float *part) {
    constexpr int NG = D / 32, kDecWarps = dec_warps(kFew), kDecThreads = 32 * kDecWarps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int h0 = hk * p.G;
    const int32_t *row = p.tables + static_cast<int64_t>(b) * p.max_blocks + sp.page0;

    const int mine = (e - a - warp + kDecWarps - 1) / kDecWarps;   // pages of this warp (or <= 0)
    // Lane j holds the id of the warp's page k + j, for the k last loaded at.
    auto load_ids = [&](int k) {
        const int i = a + warp + (k + lane) * kDecWarps;
        int32_t id = 0;
        if (i < e && XS_BOUNDS(i >= 0 && sp.page0 + i < p.max_blocks, p.err_flag)) {
            id = __ldg(row + i);
            if (id < 0 || id >= p.num_blocks) {
                raise_flag(p.err_flag, XS_FLAG_BAD_BLOCK);
                id = 0;
            }
        }
        return id;
    };
    int32_t ids = load_ids(0);
    // Lane (g, t): 8 dims of every group of head g's query (on its way while the ids are).
    uint4 qx[NG];
    {
        const __nv_bfloat16 *q = p.q + (static_cast<int64_t>(b) * p.Hq + h0 + (g < p.G ? g : 0)) * D;
#pragma unroll
        for (int c = 0; c < NG; ++c)
            qx[c] = XS_BOUNDS(b < p.B && hk < p.Hkv && h0 + p.G <= p.Hq, p.err_flag)
                        ? *reinterpret_cast<const uint4 *>(q + 32 * c + 8 * t)
                        : make_uint4(0, 0, 0, 0);
    }
    // Starts the copies of the warp's page k into the ring's next place.
    const uint32_t ring0 = smem_addr(sm.ring[warp]), bar0 = smem_addr(sm.full[warp]);
    const uint32_t base = ring.taken;
    auto start = [&](int k) {
        if (k >= mine) return;
        if (k && (k & 31) == 0) ids = load_ids(k);
        const int32_t id = __shfl_sync(0xffffffffu, ids, k & 31);
        if (lane == 0 && !skip_page(base + k) &&
            XS_BOUNDS(id >= 0 && id < p.num_blocks && hk >= 0 && hk < p.Hkv, p.err_flag)) {
            const uint32_t st = (base + k) % kStages;
            const uint32_t dst = ring0 + st * (2 * kv4_page_bytes(D)), bar = bar0 + 8 * st;
            const int64_t at = (static_cast<int64_t>(id) * p.Hkv + hk) * kv4_page_bytes(D);
            start_copy(dst, p.k_cache + at, kv4_page_bytes(D), p.v_cache + at, bar);
        }
    };
    if (!ring.dead) {
#pragma unroll 1
        for (int k = 0; k < kStages; ++k) start(k);
    }

    // q as the second operand: column g is head g (heads past G are zero); words
    // j = 0..3 of group c hold dims 32 c + 8 t + j and + j + 4.
    float to_log2;
    bool far;
    {
        const bool head = g < p.G;
        float f[NG][8], top = 0.0f;
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            const uint4 x = head ? qx[c] : make_uint4(0, 0, 0, 0);
            unpack16(x, f[c], static_cast<__nv_bfloat16 *>(nullptr));
#pragma unroll
            for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(f[c][k]));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^15 <= top 2^up < 2^16; a subnormal or zero head counts as 2^-126.
        const int ex = max(static_cast<int>(__float_as_uint(top) >> 23), 1) - 127;
        const int up = 15 - ex;
        const float u0 = __uint_as_float(static_cast<uint32_t>(up / 2 + 127) << 23);
        const float u1 = __uint_as_float(static_cast<uint32_t>(up - up / 2 + 127) << 23);
        // For q near the end of bf16 (beyond 2^100) in two factors, since one overflows.
        far = up < -85;
        to_log2 = ldexpf(p.scale_log2, (far ? 24 - 64 : 24) - up);
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            float s = 0.0f;
            uint32_t qf[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float d = j & 1 ? 0.0625f : 1.0f;
                const __half2 h = __floats2half2_rn(f[c][j] * u0 * u1 * d, f[c][j + 4] * u0 * u1 * d);
                qf[j] = *reinterpret_cast<const uint32_t *>(&h);
                const float2 back = __half22float2(h);
                s += (back.x + back.y) * (j & 1 ? 16.0f : 1.0f);
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            if (warp == 0) {
                sm.q[c][lane] = make_uint4(qf[0], qf[1], qf[2], qf[3]);
                if (t == 0) {
                    float *to = &sm.start_at[c][g >> 1].x + (g & 1);
                    to[0] = to[2] = s * -0x1p-21f;
                }
            }
        }
    }
    __syncthreads();
    const uint32_t q0 = smem_addr(&sm.q[0][lane]), s0 = smem_addr(&sm.start_at[0][t]);

    float m = kLowest, l = 0.0f;    // head g: reference, and this lane's share of the sum
    float acc[NG][2][4];        // dims 32 c + 4 g + 2 jj (+ 1) of heads 2 t, 2 t + 1
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[c][jj][k] = 0.0f;

#pragma unroll 1
    for (int k = 0; k < mine && !ring.dead; ++k) {
        const int tok0 = (sp.page0 + a + warp + k * kDecWarps) * 16;
        const uint32_t st = (base + k) % kStages, parity = ((base + k) / kStages) & 1;
        if (!__all_sync(0xffffffffu, mbar_try_wait(&sm.full[warp][st], parity)) &&
            !warp_waits(&sm.full[warp][st], parity)) {
            ring.dead = true;
            if (lane == 0) raise_flag(p.err_flag, XS_FLAG_TIMEOUT);
            // Its copies and those behind it land before the ring serves another use.
            for (int i = 0; i < min(mine - k, kStages); ++i)
                warp_waits(&sm.full[warp][(base + k + i) % kStages], ((base + k + i) / kStages) & 1);
            break;
        }
        const uint32_t kp = ring0 + st * (2 * kv4_page_bytes(D)), vp = kp + kv4_page_bytes(D);
        uint32_t kw[2][NG], ks[2][NG / 2];  // rows g, g + 8, and their scales
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            load_words<NG>(kw[u], kp + (g + 8 * u) * (D / 2) + t * (4 * NG));
            load_words<NG / 2>(ks[u], kp + 8 * D + (g + 8 * u) * (2 * NG));
        }
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // (key g, heads 2 t, 2 t + 1), (key g + 8, the same)
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            uint32_t qf[4];
            float s[4];
            load_words<4>(qf, q0 + c * 512);
            load_words<4>(reinterpret_cast<uint32_t *>(s), s0 + c * 64);
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                mma_f16(s, codes_f16(kw[0][c], j), codes_f16(kw[1][c], j), codes_f16(kw[0][c], j + 1),
                        codes_f16(kw[1][c], j + 1), qf[j], qf[j + 1]);
            const float z0 = c & 1 ? bf_hi(ks[0][c / 2]) : bf_lo(ks[0][c / 2]);
            const float z1 = c & 1 ? bf_hi(ks[1][c / 2]) : bf_lo(ks[1][c / 2]);
            y[0] = fmaf(z0, s[0], y[0]), y[1] = fmaf(z0, s[1], y[1]);
            y[2] = fmaf(z1, s[2], y[2]), y[3] = fmaf(z1, s[3], y[3]);
        }
        // Turned over: keys 2 t, 2 t + 1, and 8 more, of head g.
        F2 x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int from = 8 * t + (g >> 1);
            const float a0 = __shfl_sync(0xffffffffu, y[2 * u], from);
            const float a1 = __shfl_sync(0xffffffffu, y[2 * u + 1], from);
            const float b0 = __shfl_sync(0xffffffffu, y[2 * u], from + 4);
            const float b1 = __shfl_sync(0xffffffffu, y[2 * u + 1], from + 4);
            x[u] = F2{g & 1 ? a1 : a0, g & 1 ? b1 : b0};
        }
        x[0].x *= to_log2, x[0].y *= to_log2;
        x[1].x *= to_log2, x[1].y *= to_log2;
        const bool ragged = tok0 < sp.first || tok0 + 16 > sp.n;
        if (ragged || far) {  // rows outside [first, n) hold whatever they hold
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int ta = tok0 + 2 * t + 8 * u;
                const bool in0 = ta >= sp.first && ta < sp.n;
                const bool in1 = ta + 1 >= sp.first && ta + 1 < sp.n;
                x[u].x = in0 ? x[u].x * (far ? 0x1p64f : 1.0f) : -INFINITY;
                x[u].y = in1 ? x[u].y * (far ? 0x1p64f : 1.0f) : -INFINITY;
            }
        }
        float hi = fmaxf(fmaxf(x[0].x, x[0].y), fmaxf(x[1].x, x[1].y));
        if (__any_sync(0xffffffffu, hi > m)) {
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 2));
            // A head without a logit above -infinity (or with NaN alone) stays at kLowest,
            // below every logit to come.
            const float to = hi > m ? hi + kLead : m;
            const float f = fast_exp2(m - to);
            m = to;
            l *= f;
            const float f0 = __shfl_sync(0xffffffffu, f, 8 * t);
            const float f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
            for (int c = 0; c < NG; ++c)
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    acc[c][jj][0] *= f0;
                    acc[c][jj][1] *= f1;
                    acc[c][jj][2] *= f0;
                    acc[c][jj][3] *= f1;
                }
        }
        F2 pr[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            pr[u] = F2{fast_exp2(x[u].x - m), fast_exp2(x[u].y - m)};
            l += pr[u].x + pr[u].y;
        }
        uint32_t vw[2][NG], vs[2][NG];  // row pairs t, t + 4: dims 32 c + 4 g .., scale pairs
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            load_words<NG>(vw[u], vp + (t + 4 * u) * D + g * (4 * NG));
            load_words<NG>(vs[u], vp + 8 * D + (t + 4 * u) * (4 * NG));
        }
        if (ragged) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int ta = tok0 + 2 * t + 8 * u;
                const uint32_t keep = (ta >= sp.first && ta < sp.n ? 0x0000ffffu : 0u) |
                                      (ta + 1 >= sp.first && ta + 1 < sp.n ? 0xffff0000u : 0u);
#pragma unroll
                for (int c = 0; c < NG; ++c) vs[u][c] &= keep;
            }
        }
        ring.taken = base + k + 1;
        __syncwarp();
        start(k + kStages);
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            uint32_t w[2], rest[2];     // the weights times the scales: w + rest
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const F2 ps = mul2(pr[u], F2{bf_lo(vs[u][c]), bf_hi(vs[u][c])});
                w[u] = pack_bf16(ps);
                rest[u] = pack_bf16(sub2(ps, F2{bf_lo(w[u]), bf_hi(w[u])}));
            }
            uint32_t n[2][4];
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                n[jj][0] = codes_bf16(vw[0][c], 2 * jj), n[jj][1] = codes_bf16(vw[0][c], 2 * jj + 1);
                n[jj][2] = codes_bf16(vw[1][c], 2 * jj), n[jj][3] = codes_bf16(vw[1][c], 2 * jj + 1);
                mma_bf16(acc[c][jj], n[jj][0], n[jj][1], n[jj][2], n[jj][3], w[0], w[1]);
            }
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
                mma_bf16(acc[c][jj], n[jj][0], n[jj][1], n[jj][2], n[jj][3], rest[0], rest[1]);
        }
    }

    // The warps' shares meet in shared memory.  A warp without pages counts
    // as l = 0 under kLowest.
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (ring.dead) l = NAN;     // this segment's output, and what the CTA does after it
    __syncthreads();    // all warps have read their last pages
    if (t == 0) {
        sm.m[warp][g] = m;
        sm.l[warp][g] = l;
    }
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float2 *>(&sm.o[warp][2 * t + k][32 * c + 4 * g + 2 * jj]) =
                    make_float2(acc[c][jj][k], acc[c][jj][k + 2]);
    __syncthreads();
    const bool sinks = whole && p.sinks;
    if (threadIdx.x < kDecWarps * 8) {      // (warp, head): its weight, over the sum if whole
        const int w = threadIdx.x >> 3, h = threadIdx.x & 7;
        float top = sm.m[0][h];
#pragma unroll
        for (int k = 1; k < kDecWarps; ++k) top = fmaxf(top, sm.m[k][h]);
        float sink = 0.0f;
        if (sinks && h < p.G) {
            sink = __bfloat162float(p.sinks[h0 + h]) * 1.4426950408889634f;
            top = fmaxf(top, sink);
        }
        float total = sinks ? fast_exp2(sink - top) : 0.0f;
#pragma unroll
        for (int k = 0; k < kDecWarps; ++k) total = fmaf(fast_exp2(sm.m[k][h] - top), sm.l[k][h], total);
        const float f = fast_exp2(sm.m[w][h] - top);
        sm.weight[threadIdx.x] = whole ? f / total : f;
        if (!whole && w == 0 && h < p.G) {
            if (XS_BOUNDS(p.G * (D + 1) + h < partial_floats(p.G, D), p.err_flag)) {
                part[p.G * D + h] = top;
                part[p.G * (D + 1) + h] = total;
            }
        }
    }
    __syncthreads();
    __nv_bfloat16 *out = p.out + (static_cast<int64_t>(b) * p.Hq + h0) * D;
    for (int x = 4 * threadIdx.x; x < p.G * D; x += 4 * kDecThreads) {
        if (!XS_BOUNDS(b < p.B && h0 + p.G <= p.Hq, p.err_flag)) continue;
        const int h = x / D, d = x % D;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            const float f = sm.weight[8 * w + h];
            const float4 v = *reinterpret_cast<const float4 *>(&sm.o[w][h][d]);
            o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
        }
        if (whole)
            *reinterpret_cast<uint2 *>(out + x) =
                make_uint2(pack_bf16(F2{o.x, o.y}), pack_bf16(F2{o.z, o.w}));
        else
            *reinterpret_cast<float4 *>(part + x) = o;
    }
    fence_proxy_async_shared();     // the rings go back to the bulk copies (after the next barrier)
}

// The partials of a segment that CTAs f .. last share, joined in order: CTA f
// left its second, the others their first.  As many as the rings hold come at
// once (an access to another CTA's fresh results takes about 1 us, so one
// after the other is what a join must not do); each thread then follows its
// own four values through them.
template <int D, bool kFew>
__device__ __noinline__ void join_partials(const Kv4DecodeParams &p, DecodeSmem<D, kFew> &sm, int b,
                                           int hk, int f, int last) {
    constexpr int kDecThreads = 32 * dec_warps(kFew);
    const int G = p.G, floats = static_cast<int>(partial_floats(G, D)), chunks = floats / 4;
    float *buf = reinterpret_cast<float *>(sm.ring);
    const int room = static_cast<int>(sizeof(sm.ring) / (4 * floats));
    constexpr int kPer = (8 * D / 4 + kDecThreads - 1) / kDecThreads;
    float4 o[kPer];
    float top[kPer], total[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        const int e = threadIdx.x + x * kDecThreads, h = 4 * e / D;
        o[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        top[x] = kLowest, total[x] = 0.0f;
        if (p.sinks && h < G) {
            top[x] = __bfloat162float(p.sinks[hk * G + h]) * 1.4426950408889634f;
            total[x] = 1.0f;
        }
    }
    for (int base = f; base <= last; base += room) {
        const int n = min(room, last - base + 1);
        for (int c = threadIdx.x; c < n * chunks; c += kDecThreads) {
            const int i = c / chunks, at = c - i * chunks;
            const float *src = partial_of(p, D, base + i, base + i == f);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(buf + 4 * c)),
                         "l"(src + 4 * at)
                         : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int e = threadIdx.x + x * kDecThreads, h = 4 * e / D;
            if (h >= G) continue;
            float to = top[x];
            for (int i = 0; i < n; ++i) to = fmaxf(to, buf[i * floats + G * D + h]);
            const float w0 = fast_exp2(top[x] - to);
            top[x] = to;
            total[x] *= w0;
            o[x].x *= w0, o[x].y *= w0, o[x].z *= w0, o[x].w *= w0;
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float w = fast_exp2(buf[i * floats + G * D + h] - to);
                const float4 v = *reinterpret_cast<const float4 *>(buf + i * floats + 4 * e);
                total[x] = fmaf(w, buf[i * floats + G * (D + 1) + h], total[x]);
                o[x].x = fmaf(w, v.x, o[x].x), o[x].y = fmaf(w, v.y, o[x].y);
                o[x].z = fmaf(w, v.z, o[x].z), o[x].w = fmaf(w, v.w, o[x].w);
            }
        }
        __syncthreads();
    }
    // The rings go back to the bulk copies.
    fence_proxy_async_shared();
    __syncthreads();
    __nv_bfloat16 *out = p.out + (static_cast<int64_t>(b) * p.Hq + hk * G) * D;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
        const int e = threadIdx.x + x * kDecThreads;
        if (4 * e / D < G && XS_BOUNDS(b < p.B && hk < p.Hkv, p.err_flag))
            reinterpret_cast<uint2 *>(out)[e] =
                make_uint2(pack_bf16(F2{o[x].x / total[x], o[x].y / total[x]}),
                           pack_bf16(F2{o[x].z / total[x], o[x].w / total[x]}));
    }
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
// Joins the parts that the CTAs of a cluster hold at `own`, and writes the output.
template <int kCtas, int kThreads>
__device__ __forceinline__ void join_cluster(const Kv4DecodeParams &p, const float *own,
                                             __nv_bfloat16 *out, int hk, int rank, int D) {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    // This CTA's part of the output, four values from each CTA of the cluster
    // by neighbouring lanes.
    const int G = p.G, chunks = G * D / 4, per = (chunks + kCtas - 1) / kCtas;
    const int from = threadIdx.x % kCtas;
    constexpr int kSlots = kThreads / kCtas, kTrips = 256 / kCtas / kSlots;    // G D / 4 <= 256
#pragma unroll
    for (int n = 0; n < kTrips; ++n) {
        if (n * kSlots >= per) break;
        const int i = n * kSlots + threadIdx.x / kCtas, chunk = rank * per + i, h = 4 * chunk / D;
        const bool valid = i < per && chunk < chunks && XS_BOUNDS(rank < kCtas && hk < p.Hkv, p.err_flag);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float top = kLowest, sum = 0.0f, sink = 0.0f;
        if (valid) {
            const uint32_t part = peer_addr(own, from);
            o = peer_f32x4(part + 16 * chunk);
            top = peer_f32(part + 4 * (G * D + h));
            sum = peer_f32(part + 4 * (G * (D + 1) + h));
        }
        float to = top;
#pragma unroll
        for (int d = kCtas / 2; d > 0; d >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, d));
        if (valid && p.sinks) {
            sink = __bfloat162float(p.sinks[hk * G + h]) * 1.4426950408889634f;
            to = fmaxf(to, sink);
        }
        const float f = fast_exp2(top - to);
        sum *= f;
        o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
        for (int d = kCtas / 2; d > 0; d >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
            o.x += __shfl_xor_sync(0xffffffffu, o.x, d), o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
            o.z += __shfl_xor_sync(0xffffffffu, o.z, d), o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
        }
        if (valid && from == 0) {
            if (p.sinks) sum += fast_exp2(sink - to);
            reinterpret_cast<uint2 *>(out)[chunk] = make_uint2(pack_bf16(F2{o.x / sum, o.y / sum}),
                                                               pack_bf16(F2{o.z / sum, o.w / sum}));
        }
    }
    // No CTA leaves before all have read its shared memory (what they read is in
    // registers; the barrier need not wait for the output).
    asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

// A part of a segment is done: the last of its CTAs joins them.
template <int D, bool kFew>
__device__ __forceinline__ void arrive_and_join(const Kv4DecodeParams &p, DecodeSmem<D, kFew> &sm) {
    // The barrier and the atomic's release carry all threads' partials, its
    // acquire and the next barrier the other CTAs'.
    __syncthreads();
    if (threadIdx.x == 0) {
        if (!XS_BOUNDS(sm.f >= 0 && sm.f <= sm.last && sm.last < gridDim.x, p.err_flag)) sm.f = sm.last = 0;
        sm.joins = atomic_add_acq_rel_gpu(p.counters + sm.f, 1) == sm.last - sm.f;
        if (sm.joins) p.counters[sm.f] = 0;
    }
    __syncthreads();
    if (sm.joins) join_partials<D, kFew>(p, sm, sm.b, sm.hk, sm.f, sm.last);
}

// A CTA's place is found by every warp for itself (a load of the lengths and a
// few shuffles; with barriers between the warps it took 0.2 us more).
template <int D>
__global__ void __launch_bounds__(32 * dec_warps(false), ctas_per_sm(false))
    kv4_decode_kernel(const __grid_constant__ Kv4DecodeParams p) {
    constexpr int kDecWarps = dec_warps(false), kDecThreads = 32 * kDecWarps;
    // Placed while the kernel before it ends.  It never lets the next one be
    // placed early: waiting CTAs of the next call on some SMs and not on others
    // upset the even spread of this call's (a 64-sequence step from 40 to 44 us
    // with weights of a single rounding).
    griddep_wait();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DecodeSmem<D, false> &sm = *reinterpret_cast<DecodeSmem<D, false> *>(smem_raw);
    if (threadIdx.x < kDecWarps * kStages) mbar_init(&sm.full[0][0] + threadIdx.x, 1);
    mbar_fence_init();
    RingState ring;
    // The line's length, then the segment in which this CTA's share begins.
    const int lane = threadIdx.x & 31;
    auto pages_at = [&](int b) { return b < p.B ? static_cast<uint32_t>(span_of(p, b).pages) : 0u; };
    uint32_t pages0[4];     // of the first 128 sequences; the sums of 32 fit 32 bits
    int64_t total = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) pages0[u] = pages_at(32 * u + lane);
#pragma unroll
    for (int u = 0; u < 4; ++u) total += __reduce_add_sync(0xffffffffu, pages0[u]);
#pragma unroll 4
    for (int base = 128; base < p.B; base += 32)
        total += __reduce_add_sync(0xffffffffu, pages_at(base + lane));
    const int64_t line = (total + static_cast<int64_t>(p.B) * kSegmentCost) * p.Hkv;
    const int64_t share = max((line + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(kMinShare));
    const int64_t target = share * blockIdx.x;
    int64_t before = 0;
    bool found = false;
    auto look = [&](int base, uint32_t pages) {     // among sequences base .. base + 31
        const uint32_t units = base + lane < p.B ? pages + kSegmentCost : 0;
        const uint32_t sum = warp_scan(units);
        const int64_t end = (before + sum) * p.Hkv, s = end - static_cast<int64_t>(units) * p.Hkv;
        before += __shfl_sync(0xffffffffu, sum, 31);
        const bool mine = target >= s && target < end;
        found = __any_sync(0xffffffffu, mine);
        if (mine && threadIdx.x < 32) {
            const int hk = static_cast<int>((target - s) / units);
            sm.b = base + lane;
            sm.hk = hk;
            sm.start = s + static_cast<int64_t>(hk) * units;
            sm.share = share;
            sm.line = line;
        }
    };
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (!found && 32 * u < p.B) look(32 * u, pages0[u]);
    for (int base = 128; !found && base < p.B; base += 32) look(base, pages_at(base + lane));
    if (!found) return;
    __syncthreads();
    while (true) {
        {
            const int b = sm.b, hk = sm.hk;
            const Span sp = span_of(p, b);
            if (threadIdx.x == 0) {
                const int64_t s = sm.start, share = sm.share, lo = share * blockIdx.x;
                const int64_t hi = min(lo + share, sm.line);
                sm.a = static_cast<int>(min(max(lo - s, int64_t(0)), static_cast<int64_t>(sp.pages)));
                sm.e = static_cast<int>(min(hi - s, static_cast<int64_t>(sp.pages)));
                sm.f = static_cast<int>(s / share);
                sm.last = static_cast<int>((s + sp.pages - 1) / share);
                if (sp.pages <= kWholePages)    // its first CTA does all of it
                    sm.last = sm.f, sm.a = 0, sm.e = s >= lo ? sp.pages : 0;
            }
            __syncthreads();
            const int a = sm.a, e = sm.e;
            if (sp.pages == 0) {
                if (sm.start >= sm.share * blockIdx.x) {
                    __nv_bfloat16 *out = p.out + (static_cast<int64_t>(b) * p.Hq + hk * p.G) * D;
                    for (int x = threadIdx.x; x < p.G * D; x += kDecThreads)
                        out[x] = __float2bfloat16_rn(0.0f);
                }
            } else if (a < e) {
                run_segment<D, false>(p, sm, ring, b, hk, sp, a, e, a == 0 && e == sp.pages,
                                      partial_of(p, D, blockIdx.x, a == 0));
            }
        }
        if (sm.a < sm.e && sm.f != sm.last) arrive_and_join(p, sm);
        const int b = sm.b, hk = sm.hk;
        const int64_t next = sm.start + span_of(p, b).pages + kSegmentCost;
        if (next >= min(sm.share * (blockIdx.x + 1), sm.line)) break;
        __syncthreads();   // all have read the old place
        if (threadIdx.x == 0) {
            sm.start = next;
            sm.hk = hk + 1 == p.Hkv ? 0 : hk + 1;
            sm.b = hk + 1 == p.Hkv ? b + 1 : b;
        }
        __syncthreads();
    }
}

// Few segments, in clusters of kCluster CTAs.  Either each segment has a cluster,
// whose CTAs cut it evenly and join their parts through shared memory (a
// short one its first CTA alone); or, where that leaves too much to one
// cluster, all segments are cut for all CTAs, as many as there are, and joined
// through the workspace.  Which, the lengths decide.  (32q/8kv x 128, us, clusters and
// pieces: one sequence of 300 tokens 5.2 and 8.2, of 2K 6.4 and 8.8, 4K 8.4 and
// 10.8, 8K 12.1 and 12.3, 12K 15.5 and 14.7; two of 4K 10.9 and 11.2, of 8K 15.8 and
// 13.9; four of 8K 16.3 and 17.5.)
template <int D>
__global__ void __launch_bounds__(32 * dec_warps(true), ctas_per_sm(true))
    kv4_decode_few_kernel(const __grid_constant__ Kv4DecodeParams p) {
    constexpr int kDecWarps = dec_warps(true), kDecThreads = 32 * kDecWarps;
    griddep_wait();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DecodeSmem<D, true> &sm = *reinterpret_cast<DecodeSmem<D, true> *>(smem_raw);
    if (threadIdx.x < kDecWarps * kStages) mbar_init(&sm.full[0][0] + threadIdx.x, 1);
    mbar_fence_init();
    RingState ring;
    const int lane = threadIdx.x & 31, rank = blockIdx.x % kCluster;
    uint32_t pages0[2], longest = 0;
    int64_t total = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
        pages0[u] = 32 * u + lane < p.B ? static_cast<uint32_t>(span_of(p, 32 * u + lane).pages) : 0u;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        total += __reduce_add_sync(0xffffffffu, pages0[u]);
        longest = max(longest, __reduce_max_sync(0xffffffffu, pages0[u]));
    }
    const int64_t segments = static_cast<int64_t>(p.B) * p.Hkv;
    total *= p.Hkv;
    // In units of a page of a warp, three times: a cluster's time is that of its longest
    // segment over 64 warps (less where CTAs have their SM for themselves);
    // with pieces all warps share the pages, and the join costs 4 pages more.
    const int weight = segments * kCluster * 4 > gridDim.x ? 3 : 2;
    const bool clusters =
        longest <= kClusterPages ||
        static_cast<int64_t>(longest) * weight <= 3 * (64 * 4 + total * kCluster / gridDim.x);
    int b = 0, hk = 0, a, e, whole;
    if (clusters) {
        const int segment = blockIdx.x / kCluster;
        b = segment / p.Hkv, hk = segment - b * p.Hkv;
        if (b >= p.B) return;           // the whole cluster
        const int pages = static_cast<int>(b < 32 ? __shfl_sync(0xffffffffu, pages0[0], b)
                                                  : __shfl_sync(0xffffffffu, pages0[1], b - 32));
        whole = pages <= alone_pages(kDecWarps);
        a = whole ? 0 : static_cast<int>(static_cast<int64_t>(pages) * rank / kCluster);
        e = whole ? pages : static_cast<int>(static_cast<int64_t>(pages) * (rank + 1) / kCluster);
        if (whole && rank) return;      // all but one
    } else {
        // Equal pieces of at least kMinShare pages, one for a CTA: as small as the
        // CTAs suffice for, or as they surely do (a sum of ceil(x) is at most
        // their number and the sum of x).
        auto pieces = [&](int u, uint32_t share) {
            return 32 * u + lane < p.B ? max((pages0[u] + share - 1) / share, 1u) : 0u;
        };
        auto share_for = [&](int64_t ctas) {
            return max(static_cast<uint32_t>((total + ctas - 1) / ctas), static_cast<uint32_t>(kMinShare));
        };
        uint32_t share = share_for(gridDim.x);
        const uint32_t all = __reduce_add_sync(0xffffffffu, pieces(0, share) + pieces(1, share));
        if (static_cast<int64_t>(all) * p.Hkv > gridDim.x) share = share_for(gridDim.x - segments);
        int before = 0;
        bool found = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (found) break;
            const uint32_t units = pieces(u, share), sum = warp_scan(units);
            const int end = (before + static_cast<int>(sum)) * p.Hkv, s = end - static_cast<int>(units) * p.Hkv;
            before += __shfl_sync(0xffffffffu, static_cast<int>(sum), 31);
            const int cta = blockIdx.x;
            const bool mine = cta >= s && cta < end;
            found = __any_sync(0xffffffffu, mine);
            if (mine && threadIdx.x < 32) {
                const int n = static_cast<int>(units), h = (cta - s) / n, j = cta - s - h * n;
                const int pages = static_cast<int>(pages0[u]), piece = (pages + n - 1) / n;
                sm.b = 32 * u + lane;
                sm.hk = h;
                sm.a = j * piece;
                sm.e = min((j + 1) * piece, pages);
                sm.f = cta - j;
                sm.last = sm.f + n - 1;
            }
        }
        if (!found) return;
    }
    __syncthreads();
    if (!clusters) b = sm.b, hk = sm.hk, a = sm.a, e = sm.e, whole = sm.f == sm.last;
    const int G = p.G;
    const Span sp = span_of(p, b);
    __nv_bfloat16 *out = p.out + (static_cast<int64_t>(b) * p.Hq + hk * G) * D;
    if (sp.pages == 0) {
        for (int x = threadIdx.x; x < G * D; x += kDecThreads) out[x] = __float2bfloat16_rn(0.0f);
        return;
    }
    run_segment<D, true>(p, sm, ring, b, hk, sp, a, e, whole,
                         clusters ? sm.part : partial_of(p, D, blockIdx.x, a == 0));
    if (whole) return;
    if (!clusters) {
        arrive_and_join(p, sm);
        return;
    }
    join_cluster<kCluster, kDecThreads>(p, sm.part, out, hk, rank, D);
}

// Short segments, not too many: a cluster of kLineCluster CTAs for each, in the line's
// form of a CTA (4 of them fill an SM).  A segment of up to alone_pages its
// first CTA does alone.  (12 sequences of 100, 300, 1K, 2K tokens, 32q/8kv x 128: 5.4, 6.2,
// 8.6, 13.1 us; on the line, which also takes them under a table or window of more
// pages, 6.0, 8.1, 13.5, 17.0.  The line's kernel itself cannot be launched in
// clusters for the sake of short calls: it then took 134 us where it took 98, for 18
// sequences of 20K tokens and weights of a single rounding.)
template <int D>
__global__ void __launch_bounds__(32 * dec_warps(false), ctas_per_sm(false))
    kv4_decode_short_kernel(const __grid_constant__ Kv4DecodeParams p) {
    constexpr int kDecWarps = dec_warps(false), kDecThreads = 32 * kDecWarps;
    griddep_wait();
    extern __shared__ __align__(16) uint8_t smem_raw[];
    DecodeSmem<D, false> &sm = *reinterpret_cast<DecodeSmem<D, false> *>(smem_raw);
    const int rank = blockIdx.x % kLineCluster, segment = blockIdx.x / kLineCluster;
    const int b = segment / p.Hkv, hk = segment - b * p.Hkv;
    // A length past its table is told of by the first CTA alone: it looks at all.
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.B; i += kDecThreads) span_of(p, i);
    const Span sp = span_of(p, b);
    const bool alone = sp.pages <= alone_pages(kDecWarps);
    if (alone && rank) return;          // all but one of the cluster
    __nv_bfloat16 *out = p.out + (static_cast<int64_t>(b) * p.Hq + hk * p.G) * D;
    if (sp.pages == 0) {
        for (int x = threadIdx.x; x < p.G * D; x += kDecThreads) out[x] = __float2bfloat16_rn(0.0f);
        return;
    }
    if (threadIdx.x < kDecWarps * kStages) mbar_init(&sm.full[0][0] + threadIdx.x, 1);
    mbar_fence_init();
    __syncthreads();
    RingState ring;
    const int a = alone ? 0 : sp.pages * rank / kLineCluster;
    const int e = alone ? sp.pages : sp.pages * (rank + 1) / kLineCluster;
    run_segment<D, false>(p, sm, ring, b, hk, sp, a, e, alone, sm.part);
    if (!alone) join_cluster<kLineCluster, kDecThreads>(p, sm.part, out, hk, rank, D);
}

// The clusters of a kernel that the device holds at once (as many as whole
// groups of SMs have room for), once it may have its shared memory; or -1.
template <typename K> int clusters_held(K kernel, int ctas, int threads, int smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return min(n, kMaxCtas / ctas);
}
struct Held {
    int few, brief;     // clusters of the few and of the short kernel
};
// Asked for once for each device (by two threads at once: twice, with one answer).
template <int D> int configure(int dev, Held *held) {
    static std::atomic<uint32_t> known[64];     // few and brief, and 1 more each; 0: not yet
    const uint32_t v = dev < 64 ? known[dev].load(std::memory_order_acquire) : 0;
    if (v) {
        *held = Held{static_cast<int>(v & 0xffff) - 1, static_cast<int>(v >> 16) - 1};
        return XS_OK;
    }
    if (cudaFuncSetAttribute(kv4_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             sizeof(DecodeSmem<D, false>)) != cudaSuccess) {
        cudaGetLastError();
        return XS_EDEVICE;
    }
    held->few = clusters_held(kv4_decode_few_kernel<D>, kCluster, 32 * dec_warps(true),
                              sizeof(DecodeSmem<D, true>));
    held->brief = clusters_held(kv4_decode_short_kernel<D>, kLineCluster, 32 * dec_warps(false),
                                sizeof(DecodeSmem<D, false>));
    if (held->few < 0 || held->brief < 0) return XS_EDEVICE;
    if (dev < 64)
        known[dev].store(static_cast<uint32_t>(held->few + 1) | static_cast<uint32_t>(held->brief + 1) << 16,
                         std::memory_order_release);
    return XS_OK;
}

template <int D> int launch(const Kv4DecodeParams &p, int dev, int sms, cudaStream_t stream) {
    Held held = {};
    const int rc = configure<D>(dev, &held);
    if (rc != XS_OK) return rc;
    const int64_t segments = static_cast<int64_t>(p.B) * p.Hkv;
    // The pages of a segment are at most those of the table, and of the window.
    const int most = p.window > 0 ? min(p.max_blocks, p.window / 16 + 2) : p.max_blocks;     // pages
    if (segments < held.few && p.B <= 64) {
        const int clusters = most <= kClusterPages ? static_cast<int>(segments) : held.few;
        return launch_after(kv4_decode_few_kernel<D>, dim3(clusters * kCluster), 32 * dec_warps(true),
                            sizeof(DecodeSmem<D, true>), stream, kCluster, p);
    }
    if (segments <= held.brief && most <= kShortTable)
        return launch_after(kv4_decode_short_kernel<D>, dim3(static_cast<int>(segments) * kLineCluster),
                            32 * dec_warps(false), sizeof(DecodeSmem<D, false>), stream, kLineCluster, p);
    // The line is at most so long, and no CTA takes less than kMinShare of it.
    const int64_t want =
        segments + (segments * (p.max_blocks + kSegmentCost) + kMinShare - 1) / kMinShare;
    const int fill = min(sms * ctas_per_sm(false), kMaxCtas);
    return launch_after(kv4_decode_kernel<D>, dim3(static_cast<int>(want < fill ? want : fill)),
                        32 * dec_warps(false), sizeof(DecodeSmem<D, false>), stream, 1, p);
}

}  // namespace
XS_DEFINE_BOUNDS_COUNTER(bounds_failures_kv4_decode)

}  // namespace xs

extern "C" int xs_debug_kv4_wait_injection(int64_t wait_limit_ns, int skip_page) {
#ifdef XS_DEBUG_BOUNDS
    if (wait_limit_ns <= 0 || skip_page < -1) return XS_ESHAPE;
    const unsigned long long limit = static_cast<unsigned long long>(wait_limit_ns);
    if (cudaMemcpyToSymbol(xs::g_wait_limit_ns, &limit, sizeof(limit)) != cudaSuccess ||
        cudaMemcpyToSymbol(xs::g_skip_page, &skip_page, sizeof(skip_page)) != cudaSuccess) {
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

extern "C" size_t xs_kv4_decode_workspace_bytes(int B, int Hq, int Hkv, int D) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return 0;
    const size_t counters = xs::kMaxCtas * sizeof(int);
    return counters + static_cast<size_t>(xs::kMaxCtas) * 2 * xs::partial_floats(Hq / Hkv, D) * sizeof(float);
}

extern "C" int xs_kv4_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
                             const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, const void *sinks, int window, int B,
                             int Hq, int Hkv, int D, int block_size, int64_t num_blocks,
                             float scale, void *workspace, size_t workspace_bytes, int dtype,
                             int *err_flag, cudaStream_t stream) {
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return XS_ENULL;
    if (!xs::elem_bytes(dtype)) return XS_EDTYPE;
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || block_size <= 0 ||
        max_blocks_per_seq < 0 || num_blocks < 0 || window < 0)
        return XS_ESHAPE;
    const int G = Hq / Hkv;
    if ((D != 64 && D != 128) || block_size != 16 || (G != 1 && G != 2 && G != 4 && G != 8) ||
        dtype != XS_BF16 || max_blocks_per_seq > (1 << 26))
        return XS_EUNSUPPORTED;
    if (!xs::aligned16(out) || !xs::aligned16(q) || !xs::aligned16(k_cache) ||
        !xs::aligned16(v_cache) || !xs::aligned16(workspace))
        return XS_EALIGN;
    if (B == 0) return XS_OK;
    if (num_blocks == 0) return XS_ESHAPE;
    if (!workspace || workspace_bytes < xs_kv4_decode_workspace_bytes(B, Hq, Hkv, D))
        return XS_EWORKSPACE;
    xs::Kv4DecodeParams p = {};
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.tables = block_tables, p.lens = context_lens;
    p.sinks = static_cast<const __nv_bfloat16 *>(sinks);
    p.max_blocks = max_blocks_per_seq, p.window = window;
    p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.G = G, p.num_blocks = num_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err_flag = err_flag;
    p.counters = static_cast<int *>(workspace);
    p.partials = reinterpret_cast<float *>(p.counters + xs::kMaxCtas);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return XS_EDEVICE;
    return D == 128 ? xs::launch<128>(p, dev, sms, stream) : xs::launch<64>(p, dev, sms, stream);
}
