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

// Two fp32 values in one operation.
struct F2 {
    float x, y;
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("{\n .reg .b64 p, q, s;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n"
        " mul.rn.f32x2 s, p, q;\n mov.b64 {%0, %1}, s;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("{\n .reg .b64 p, q, s;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n"
        " add.rn.f32x2 s, p, q;\n mov.b64 {%0, %1}, s;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b) {
    F2 r;
    asm("{\n .reg .b64 p, q, s;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n"
        " sub.rn.f32x2 s, p, q;\n mov.b64 {%0, %1}, s;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("{\n .reg .b64 p, q, s;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n"
        " mov.b64 s, {%6, %7};\n fma.rn.f32x2 s, p, q, s;\n mov.b64 {%0, %1}, s;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

constexpr int kKv4Group = 32;
__host__ __device__ constexpr int kv4_page_bytes(int D) { return 9 * D; }

// Keys of bf16 values, two to a word: order of magnitude first, the positive of
// two equal ones above, NaN above all.  The maximum of the keys is the key of a
// group's extreme.
__device__ __forceinline__ uint32_t kv4_keys(uint32_t w) {
    return ((w << 1) & 0xfffefffeu) | (~(w >> 15) & 0x00010001u);
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t kv4_fold(uint32_t keys) { return max(keys & 0xffffu, keys >> 16); }
// The scale of a group from its extreme's key (in the low half).
__device__ __forceinline__ float kv4_scale(uint32_t key) {
    const float e = __uint_as_float(((key >> 1) << 16) | ((key & 1u) ? 0u : 0x80000000u));
    return __bfloat162float(__float2bfloat16_rn(e * -0.125f));
}
// The codes of four dims under s[0] and of four under s[1] (the same one if
// `alike`), the first lowest: rne(x / s), clamped.  x
// times an approximate 1 / s is within 2^-19 of the quotient, which is a half
// integer or at least 1/512 away from one.  Rounded to a multiple of 2^-10 (by the
// addition of 1.5 2^13 in one multiply-add) it is exactly the half integer or
// still on its side of it, and the addition of 1.5 2^23 + 8 - 1.5 2^13, which
// is exact before its rounding, leaves the code in the low bits.  The quotient is
// at least -8 (a group's extreme is exactly that), so only the upper end is cut.  The four are joined
// by one multiply-add each, and what the constant adds up to is taken off at the end.
// Scales without a usable reciprocal (0, tiny, infinite, NaN) divide instead; a
// group with an infinity or a NaN gets codes of 8 (a NaN converts to 0) under
// an infinite or NaN scale, and reads as NaN.
__device__ __forceinline__ void kv4_pack(uint32_t *codes, const float *x, const float *s, bool alike) {
    const float lo = fminf(fabsf(s[0]), fabsf(s[1])), hi = fabsf(s[0]) + fabsf(s[1]);
    if (!(lo >= 0x1p-120f && hi < INFINITY)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            codes[u] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = s[u] == 0.0f ? 0 : __float2int_rn(__fdiv_rn(x[4 * u + i], s[u]));
                codes[u] |= static_cast<uint32_t>(min(max(n, -8), 7) + 8) << (4 * i);
            }
        }
        return;
    }
    float r[2];
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[0]) : "f"(s[0]));
    r[1] = r[0];
    if (!alike) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[1]) : "f"(s[1]));
    constexpr uint32_t kBits = 0x4b400000u;     // of 1.5 2^23
    constexpr float kFine = 0x1.8p13f, kWhole = 0x1.8p23f + 8.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 2; i >= 0; i -= 2) {
            const F2 q = fma2(F2{x[4 * u + i], x[4 * u + i + 1]}, F2{r[u], r[u]}, F2{kFine, kFine});
            const F2 n = add2(q, F2{kWhole - kFine, kWhole - kFine});
            w = w * 16u + __float_as_uint(fminf(n.y, kWhole + 7.0f));
            w = w * 16u + __float_as_uint(fminf(n.x, kWhole + 7.0f));
        }
        codes[u] = w - kBits * 0x1111u;
    }
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
