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
// where s is 0, and s is NaN where e is an infinity or NaN.  The extreme is stored exactly (n = 0), and the sign in s lets
// the one code that has no partner (-8) serve whichever side is longer.  x and
// s have 8-bit significands, so x / s is a tie or at least 1/512 away from
// one: a quotient in fp32, even an approximate one, can be rounded as the true
// one is (kv4_pack), and the codes are the same on any machine.
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
// The larger of a word's two keys, in both halves.
__device__ __forceinline__ uint32_t kv4_fold(uint32_t keys) {
    return max_u16x2(keys, __byte_perm(keys, keys, 0x1032));
}
// The bf16 scales of two groups from their extremes' keys.
__device__ __forceinline__ uint32_t kv4_scales(uint32_t keys) {
    const uint32_t e = ((keys >> 1) & 0x7fff7fffu) | (~(keys << 15) & 0x80008000u);
    const __nv_bfloat162 s = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&e),
                                     __floats2bfloat162_rn(-0.125f, -0.125f));
    return *reinterpret_cast<const uint32_t *>(&s);
}
// The codes of x[0..3] under the low scale and of x[4..7] under the high one,
// the first lowest: rne(x / s), clamped.  x times an approximate 1 / s is within
// 2^-19 of the quotient, which is a half integer or at least 1/512 away from
// one.  Rounded to a multiple of 2^-10 (by the addition of 1.5 2^13 in one
// multiply-add) it is exactly the half integer or still on its side of it, and
// the addition of 1.5 2^23 + 8 - 1.5 2^13, which is exact before its rounding,
// leaves the code in the low bits.  The quotient is at least -8 (a group's
// extreme is exactly that), so only the upper end is cut.  The four are joined by one
// multiply-add each, and what the constant adds up to is taken off at the end.
// Scales without a usable reciprocal are met first: tiny ones (whose own
// rounding may leave quotients beyond 8) and their values are lifted by 2^64;
// under 0, infinity or NaN all codes are 8, and an infinite scale becomes NaN: a
// group with an infinity or a NaN is NaN to whatever multiplies by its scale (a
// sum of n - 8 need not come out as exactly 0).
__device__ __forceinline__ void kv4_pack(uint32_t *codes, float *x, uint32_t &scales) {
    float s[2] = {__uint_as_float(scales << 16), __uint_as_float(scales & 0xffff0000u)};
    if (!(fminf(fabsf(s[0]), fabsf(s[1])) >= 0x1p-120f && fabsf(s[0]) + fabsf(s[1]) < INFINITY)) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float a = fabsf(s[u]);
            const bool none = !(a > 0.0f && a < INFINITY);
            const float lift = a < 0x1p-120f ? 0x1p64f : 1.0f;
            if (!(a < INFINITY)) scales |= u ? 0x7fff0000u : 0x7fffu;
            s[u] = none ? 1.0f : s[u] * lift;
            const float most = 8.0f * fabsf(s[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[4 * u + i] = none ? 0.0f : fminf(fmaxf(x[4 * u + i] * lift, -most), most);
        }
    }
    constexpr uint32_t kBits = 0x4b400000u;     // of 1.5 2^23
    constexpr float kFine = 0x1.8p13f, kWhole = 0x1.8p23f + 8.0f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s[u]));
        uint32_t w = 0;
#pragma unroll
        for (int i = 2; i >= 0; i -= 2) {
            const F2 q = fma2(F2{x[4 * u + i], x[4 * u + i + 1]}, F2{r, r}, F2{kFine, kFine});
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
                                                uint32_t w, uint16_t s) {
    constexpr int NG = D / kKv4Group;
    const int c = ch >> 2, t = ch & 3;
    uint8_t *scales = page + 8 * D;
    if (is_v) {
        uint16_t *h = reinterpret_cast<uint16_t *>(page);
        const int pair = o >> 1, r = o & 1;
        h[((pair * 8 + 2 * t) * NG + c) * 2 + r] = static_cast<uint16_t>(w);
        h[((pair * 8 + 2 * t + 1) * NG + c) * 2 + r] = static_cast<uint16_t>(w >> 16);
        if (t == 0) reinterpret_cast<uint16_t *>(scales)[(pair * NG + c) * 2 + r] = s;
    } else {
        reinterpret_cast<uint32_t *>(page)[o * (D / 8) + t * NG + c] = w;
        if (t == 0) reinterpret_cast<uint16_t *>(scales)[o * NG + c] = s;
    }
}

// The same for row o of a V page by the lanes of both rows of its pair at
// once: `mine` is this row's word of chunk ch, `theirs` the other row's; the
// even row's lane stores the words of the chunk's first four dims, the odd
// row's those of its last four.
template <int D>
__device__ __forceinline__ void kv4_store_pair(uint8_t *page, int o, int ch, uint32_t mine,
                                               uint32_t theirs, uint16_t s) {
    constexpr int NG = D / kKv4Group;
    const int c = ch >> 2, t = ch & 3, pair = o >> 1, r = o & 1;
    const uint32_t w = __byte_perm(mine, theirs, r ? 0x3276 : 0x5410);
    reinterpret_cast<uint32_t *>(page)[(pair * 8 + 2 * t + r) * NG + c] = w;
    if (t == 0)
        reinterpret_cast<uint16_t *>(page + 8 * D)[(pair * NG + c) * 2 + r] = s;
}

}  // namespace xs
