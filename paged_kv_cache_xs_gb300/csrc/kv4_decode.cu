// Decode attention over a cache held in 4 bits (pages as in kv4.cuh): each
// sequence's one query token attends over all of its pages.
//
//     out[b, h] = sum_t softmax_t(scale q[b, h] . K_t) V_t
//     K_t = s_tc (n_td - 8) for d in group c, V_t the same
//
// A page of one KV head serves the G = Hq / Hkv query heads of its group.
// With keys (or dims) on the 16 rows of m16n8k16 and heads on its 8 columns:
//
//   logits   S[t, h] = sum_c s_tc (sum_{d in c} (128 + n_td) q_hd - 136 sum_{d in c} q_hd)
//            A code becomes the bf16 128 + n by one bitwise operation
//            (0x4300 | n); the -136 sum q is the accumulator's initial value,
//            and the group's scale is applied to the fp32 result.  128 + n
//            and q are exact, so the logits are fp32 sums of exact products.
//   values   O[d, h] = sum_t (n_td - 8) (p_th s_tc)
//            p is rounded to bf16 (2^-9) and its product with the scale once
//            more, as the operand of the matrix instruction has to be; n - 8
//            is exact.  p meets the scale, not the codes: 4 roundings for a
//            token and head in place of D.
//
// The softmax is online, in fp32, with a running maximum that is a multiple
// of nothing: it follows the true one only when a logit exceeds it by 2^8, so
// that most pages take no exchange between lanes (p up to 2^8 is harmless in
// fp32 and bf16).
//
// A lane's share of a page lies at one place of it (16 bytes of K codes for
// each of two rows, 16 of V codes for each of two row pairs), so pages go
// straight from global memory to registers, the next one while the current
// one is worked on.
#include "kv4.cuh"

namespace xs {
namespace {

constexpr int kDecWarps = 8;

__device__ __forceinline__ void mma_bf16(float *c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Codes j of both halves of a word as the bf16 pair 128 + n.
__device__ __forceinline__ uint32_t codes128(uint32_t w, int j) {
    return ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
    return *reinterpret_cast<const __nv_bfloat162 *>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) {
    return *reinterpret_cast<const uint32_t *>(&x);
}

// A lane's registers of one page.  NG = D / 32 words of each row / row pair.
template <int NG> struct PageRegs {
    uint32_t k[2][NG];   // rows g, g + 8
    uint32_t v[2][NG];   // row pairs t, t + 4
    uint32_t ks[2][(NG + 1) / 2];  // scales of rows g, g + 8: bf16 [NG]
    uint32_t vs[2][NG];  // scale pairs of row pairs t, t + 4
};

template <int N> __device__ __forceinline__ void load_words(uint32_t *r, const uint8_t *p) {
    if constexpr (N == 4) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p));
        r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w;
    } else if constexpr (N == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
        r[0] = x.x, r[1] = x.y;
    } else {
        r[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
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
    int *err_flag;
};

template <int D>
__global__ void __launch_bounds__(kDecWarps * 32) kv4_decode_kernel(const Kv4DecodeParams p) {
    constexpr int NG = D / 32;
    __shared__ float sm_m[kDecWarps][8], sm_l[kDecWarps][8];
    __shared__ float sm_o[kDecWarps][8][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int hk = blockIdx.x, b = blockIdx.y;
    int n = p.lens[b];
    if (n > p.max_blocks * 16) {
        if (threadIdx.x == 0 && hk == 0) raise_flag(p.err_flag, XS_FLAG_BAD_LEN);
        n = p.max_blocks * 16;
    }
    const int h0 = hk * p.G;
    __nv_bfloat16 *out = p.out + (static_cast<int64_t>(b) * p.Hq + h0) * D;
    if (n <= 0) {
        for (int i = threadIdx.x; i < p.G * D; i += blockDim.x) out[i] = __float2bfloat16_rn(0.0f);
        return;
    }
    const int first = p.window > 0 && n > p.window ? n - p.window : 0;
    const int page0 = first >> 4, pages = ((n + 15) >> 4) - page0;
    const int32_t *row = p.tables + static_cast<int64_t>(b) * p.max_blocks + page0;

    // q as the second operand: for group c and step ks, words j = 2 ks and
    // 2 ks + 1 hold dims 32 c + 8 t + j and + j + 4 of head g.
    uint32_t qf[NG][4];
    float cinit[NG][2];
    {
        const bool head = g < p.G;
        const __nv_bfloat16 *q = p.q + (static_cast<int64_t>(b) * p.Hq + h0 + (head ? g : 0)) * D;
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            uint4 x = *reinterpret_cast<const uint4 *>(q + 32 * c + 8 * t);
            if (!head) x = make_uint4(0, 0, 0, 0);
            // x holds dims 0..7 in pairs (0,1) (2,3) (4,5) (6,7)
            qf[c][0] = __byte_perm(x.x, x.z, 0x5410);
            qf[c][1] = __byte_perm(x.x, x.z, 0x7632);
            qf[c][2] = __byte_perm(x.y, x.w, 0x5410);
            qf[c][3] = __byte_perm(x.y, x.w, 0x7632);
            float f[8], s = 0.0f;
            unpack16(x, f, static_cast<__nv_bfloat16 *>(nullptr));
#pragma unroll
            for (int i = 0; i < 8; ++i) s += f[i];
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            cinit[c][0] = -136.0f * __shfl_sync(0xffffffffu, s, 8 * t);
            cinit[c][1] = -136.0f * __shfl_sync(0xffffffffu, s, 8 * t + 4);
        }
    }

    float m[2] = {0.0f, 0.0f}, l[2] = {0.0f, 0.0f};
    bool fresh = true;  // no finite maximum yet
    float acc[NG][2][4];
#pragma unroll
    for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int jj = 0; jj < 2; ++jj)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[c][jj][i] = 0.0f;

    auto page_id = [&](int i) {
        if (!XS_BOUNDS(i >= 0 && page0 + i < p.max_blocks, p.err_flag)) return 0;
        int32_t id = __ldg(row + i);
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) raise_flag(p.err_flag, XS_FLAG_BAD_BLOCK);
            id = 0;
        }
        return id;
    };
    PageRegs<NG> cur, nxt;
    auto load = [&](PageRegs<NG> &r, int32_t id) {
        const int64_t at = (static_cast<int64_t>(id) * p.Hkv + hk) * kv4_page_bytes(D);
        const uint8_t *kp = p.k_cache + at, *vp = p.v_cache + at;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            load_words<NG>(r.k[u], kp + (g + 8 * u) * (D / 2) + t * (4 * NG));
            load_words<NG>(r.v[u], vp + (t + 4 * u) * D + g * (4 * NG));
            load_words<NG / 2>(r.ks[u], kp + 8 * D + (g + 8 * u) * (2 * NG));
            load_words<NG>(r.vs[u], vp + 8 * D + (t + 4 * u) * (4 * NG));
        }
    };
    auto work = [&](PageRegs<NG> &r, int tok0) {
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            float s[4] = {cinit[c][0], cinit[c][1], cinit[c][0], cinit[c][1]};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                mma_bf16(s, codes128(r.k[0][c], 2 * ks), codes128(r.k[1][c], 2 * ks),
                         codes128(r.k[0][c], 2 * ks + 1), codes128(r.k[1][c], 2 * ks + 1),
                         qf[c][2 * ks], qf[c][2 * ks + 1]);
            const uint32_t w0 = r.ks[0][c / 2], w1 = r.ks[1][c / 2];
            const float s0 = __uint_as_float(c & 1 ? w0 & 0xffff0000u : w0 << 16);
            const float s1 = __uint_as_float(c & 1 ? w1 & 0xffff0000u : w1 << 16);
            x[0] = fmaf(s0, s[0], x[0]);
            x[1] = fmaf(s0, s[1], x[1]);
            x[2] = fmaf(s1, s[2], x[2]);
            x[3] = fmaf(s1, s[3], x[3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= p.scale_log2;
        if (tok0 < first || tok0 + 16 > n) {  // rows outside [first, n): whatever the page holds there
            const float none = -INFINITY;
            if (tok0 + g < first || tok0 + g >= n) x[0] = x[1] = none;
            if (tok0 + g + 8 < first || tok0 + g + 8 >= n) x[2] = x[3] = none;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int ta = tok0 + 2 * t + 8 * u;
                const uint32_t keep = (ta >= first && ta < n ? 0x0000ffffu : 0u) |
                                      (ta + 1 >= first && ta + 1 < n ? 0xffff0000u : 0u);
#pragma unroll
                for (int c = 0; c < NG; ++c) r.vs[u][c] &= keep;
            }
        }
        const float hi0 = fmaxf(x[0], x[2]), hi1 = fmaxf(x[1], x[3]);
        if (__any_sync(0xffffffffu, fresh || hi0 > m[0] + 8.0f || hi1 > m[1] + 8.0f)) {
            float h[2] = {hi0, hi1};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    h[i] = fmaxf(h[i], __shfl_xor_sync(0xffffffffu, h[i], d));
                // No usable maximum (nothing, or NaN): any finite reference does.
                const float to = h[i] > -INFINITY ? (fresh ? h[i] : fmaxf(m[i], h[i])) : m[i];
                const float f = fresh ? 1.0f : fast_exp2(m[i] - to);
                m[i] = to;
                l[i] *= f;
#pragma unroll
                for (int c = 0; c < NG; ++c)
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        acc[c][jj][i] *= f;
                        acc[c][jj][i + 2] *= f;
                    }
            }
            fresh = false;
        }
        const float p0 = fast_exp2(x[0] - m[0]), p1 = fast_exp2(x[1] - m[1]);
        const float p2 = fast_exp2(x[2] - m[0]), p3 = fast_exp2(x[3] - m[1]);
        l[0] += p0 + p2;
        l[1] += p1 + p3;
        const __nv_bfloat162 b0 = as_bf162(movmatrix_trans(pack_bf16(p0, p1)));
        const __nv_bfloat162 b1 = as_bf162(movmatrix_trans(pack_bf16(p2, p3)));
        const __nv_bfloat162 off = as_bf162(0x43084308u);  // 136
#pragma unroll
        for (int c = 0; c < NG; ++c) {
            const uint32_t w0 = as_u32(__hmul2(b0, as_bf162(r.vs[0][c])));
            const uint32_t w1 = as_u32(__hmul2(b1, as_bf162(r.vs[1][c])));
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
                mma_bf16(acc[c][jj], as_u32(__hsub2(as_bf162(codes128(r.v[0][c], 2 * jj)), off)),
                         as_u32(__hsub2(as_bf162(codes128(r.v[0][c], 2 * jj + 1)), off)),
                         as_u32(__hsub2(as_bf162(codes128(r.v[1][c], 2 * jj)), off)),
                         as_u32(__hsub2(as_bf162(codes128(r.v[1][c], 2 * jj + 1)), off)), w0, w1);
        }
    };

    int i = warp;
    if (i < pages) load(cur, page_id(i));
    for (; i < pages; i += kDecWarps) {
        const int next = i + kDecWarps;
        if (next < pages) load(nxt, page_id(next));
        work(cur, (page0 + i) * 16);
        cur = nxt;
    }

    // The warps' shares meet in shared memory.  A warp without pages counts
    // as l = 0 under the lowest reference.
#pragma unroll
    for (int i2 = 0; i2 < 2; ++i2) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i2] += __shfl_xor_sync(0xffffffffu, l[i2], d);
        if (g == 0) {
            sm_m[warp][2 * t + i2] = fresh ? -3.0e38f : m[i2];
            sm_l[warp][2 * t + i2] = l[i2];
        }
#pragma unroll
        for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                sm_o[warp][2 * t + i2][32 * c + 4 * g + 2 * jj] = acc[c][jj][i2];
                sm_o[warp][2 * t + i2][32 * c + 4 * g + 2 * jj + 1] = acc[c][jj][i2 + 2];
            }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.G * D; e += blockDim.x) {
        const int h = e / D, d = e % D;
        float top = -3.0e38f;
        for (int w = 0; w < kDecWarps; ++w) top = fmaxf(top, sm_m[w][h]);
        float sink = 0.0f;
        if (p.sinks) {
            sink = __bfloat162float(p.sinks[h0 + h]) * 1.4426950408889634f;
            top = fmaxf(top, sink);
        }
        float o = 0.0f, total = p.sinks ? fast_exp2(sink - top) : 0.0f;
        for (int w = 0; w < kDecWarps; ++w) {
            const float f = fast_exp2(sm_m[w][h] - top);
            o += f * sm_o[w][h][d];
            total += f * sm_l[w][h];
        }
        out[e] = __float2bfloat16_rn(o / total);
    }
}

}  // namespace
XS_DEFINE_BOUNDS_COUNTER(bounds_failures_kv4_decode)

}  // namespace xs

extern "C" size_t xs_kv4_decode_workspace_bytes(int B, int Hq, int Hkv, int D) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return 0;
    return 256;
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
    const dim3 grid(Hkv, B);
    if (D == 128)
        xs::kv4_decode_kernel<128><<<grid, xs::kDecWarps * 32, 0, stream>>>(p);
    else
        xs::kv4_decode_kernel<64><<<grid, xs::kDecWarps * 32, 0, stream>>>(p);
    return xs::launch_status();
}
