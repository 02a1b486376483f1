// The 4-bit page of the KV cache (layout and rounding), shared by the kernels
// that write it (qk_norm_rope.cu, kv4_cache.cu) and read it (kv4_cache.cu,
// kv4_decode.cu).
//
// A page of one (block, KV head) holds 16 rows of D values in 9 D bytes: 8 D
// bytes of 4-bit codes, then D bytes of bf16 scales, one for each group of 32
// dims of a row.  A code n in 0..15 under scale s stands for s (n - 8).
//
// Quantisation of a group: e = its element of largest magnitude (the positive
// one of a tie), s = bf16(-e / 8), n = clamp(rne(x / s), -8, 7) + 8; n = 8
// where s is 0.  The extreme is stored exactly (n = 0), and the sign in s lets
// the one code that has no partner (-8) serve whichever side is longer.  x and
// s have 8-bit significands, so x / s is a tie or at least 1/512 away from
// one: the fp32 quotient rounds as the true one does, and the codes are the
// same on any machine.
//
// The words lie in the order in which the decode attention's matrix
// instructions want them, so that a lane's fragment of a page is one 16-byte
// load (D = 128) and a 4-bit pair becomes a bf16 pair with a shift and one
// bitwise operation.  NG = D / 32 groups:
//   K: row o is D / 8 words; word t NG + c (t < 4, c < NG) has dims
//      32 c + 8 t + i (i < 8) in bits 4 i...  Scale of (o, c): o NG + c.
//   V: rows 2 i and 2 i + 1 share D / 4 words; word g NG + c (g < 8) has dims
//      32 c + 4 g + j (j < 4) of row 2 i in bits 4 j.. and of row 2 i + 1 in
//      bits 16 + 4 j...  Scale of (2 i + r, c): (i NG + c) 2 + r.
#pragma once

#include "xs_common.cuh"

namespace xs {

constexpr int kKv4Group = 32;
__host__ __device__ constexpr int kv4_page_bytes(int D) { return 9 * D; }

// Order of magnitude first, the positive of two equal ones above, NaN above all:
// the maximum of the keys is the key of a group's extreme.
__device__ __forceinline__ uint32_t kv4_key(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u << 1) | ((u >> 31) ^ 1u);
}
// The key of the extreme of four bf16 values, two to a word.
__device__ __forceinline__ uint32_t kv4_key4(uint32_t w0, uint32_t w1) {
    const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162 *>(&w0);
    const __nv_bfloat162 b = *reinterpret_cast<const __nv_bfloat162 *>(&w1);
    const float2 hi = __bfloat1622float2(__hmax2_nan(a, b)), lo = __bfloat1622float2(__hmin2_nan(a, b));
    float mx, mn;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(hi.x), "f"(hi.y));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(mn) : "f"(lo.x), "f"(lo.y));
    return kv4_key(mx >= -mn ? mx : mn);
}
__device__ __forceinline__ float kv4_scale(uint32_t key) {
    const float e = __uint_as_float((key >> 1) | ((key & 1u) ? 0u : 0x80000000u));
    return __bfloat162float(__float2bfloat16_rn(e * -0.125f));
}
// The codes of four dims under s, the first lowest: rne(x / s), clamped.  The
// quotient is x times an approximate 1 / s, corrected by its own remainder:
// where x / s is a half integer (or any fp32 number) that gives it exactly, and
// elsewhere x / s is at least 1/512 away from a tie, so the rounding is that of
// the true quotient.  Adding 1.5 2^23 + 8 rounds to the nearest even integer
// and leaves the code in the low bits; the four are joined by one multiply-add
// each, and what the constant adds up to is taken off at the end.
// Scales without a usable reciprocal (0, tiny, infinite, NaN) divide instead; a
// group with an infinity or a NaN gets codes of 8 (a NaN converts to 0) under
// an infinite or NaN scale, and reads as NaN.
__device__ __forceinline__ uint32_t kv4_pack4(const float *x, float s) {
    uint32_t w = 0;
    if (!(fabsf(s) >= 0x1p-120f && fabsf(s) < INFINITY)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = s == 0.0f ? 0 : __float2int_rn(__fdiv_rn(x[i], s));
            w |= static_cast<uint32_t>(min(max(n, -8), 7) + 8) << (4 * i);
        }
        return w;
    }
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    constexpr uint32_t kBits = 0x4b400000u;     // of 1.5 2^23
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        float q = x[i] * r;
        q = fmaf(fmaf(-q, s, x[i]), r, q);
        w = w * 16u + __float_as_uint(fminf(fmaxf(q, -8.0f), 7.0f) + (0x1.8p23f + 8.0f));
    }
    return w - kBits * 0x1111u;
}

// Stores chunk `ch` (8 dims) of row `o` of a page, and the group's scale with
// its first chunk.  `page` is the page's first byte.
template <int D>
__device__ __forceinline__ void kv4_store_chunk(uint8_t *page, bool is_v, int o, int ch,
                                                uint32_t w, float s) {
    constexpr int NG = D / kKv4Group;
    const int c = ch >> 2, t = ch & 3;
    uint8_t *scales = page + 8 * D;
    const __nv_bfloat16 sb = __float2bfloat16_rn(s);
    if (is_v) {
        uint16_t *h = reinterpret_cast<uint16_t *>(page);
        const int pair = o >> 1, r = o & 1;
        h[((pair * 8 + 2 * t) * NG + c) * 2 + r] = static_cast<uint16_t>(w);
        h[((pair * 8 + 2 * t + 1) * NG + c) * 2 + r] = static_cast<uint16_t>(w >> 16);
        if (t == 0) reinterpret_cast<__nv_bfloat16 *>(scales)[(pair * NG + c) * 2 + r] = sb;
    } else {
        reinterpret_cast<uint32_t *>(page)[o * (D / 8) + t * NG + c] = w;
        if (t == 0) reinterpret_cast<__nv_bfloat16 *>(scales)[o * NG + c] = sb;
    }
}

// The same for row o of a V page by the lanes of both rows of its pair at
// once: `mine` is this row's word of chunk ch, `theirs` the other row's; the
// even row's lane stores the words of the chunk's first four dims, the odd
// row's those of its last four.
template <int D>
__device__ __forceinline__ void kv4_store_pair(uint8_t *page, int o, int ch, uint32_t mine,
                                               uint32_t theirs, float s) {
    constexpr int NG = D / kKv4Group;
    const int c = ch >> 2, t = ch & 3, pair = o >> 1, r = o & 1;
    const uint32_t w = r ? __byte_perm(theirs, mine, 0x7632) : __byte_perm(mine, theirs, 0x5410);
    reinterpret_cast<uint32_t *>(page)[(pair * 8 + 2 * t + r) * NG + c] = w;
    if (t == 0)
        reinterpret_cast<__nv_bfloat16 *>(page + 8 * D)[(pair * NG + c) * 2 + r] =
            __float2bfloat16_rn(s);
}

}  // namespace xs
