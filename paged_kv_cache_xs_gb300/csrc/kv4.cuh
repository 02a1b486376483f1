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
__device__ __forceinline__ float kv4_scale(uint32_t key) {
    const float e = __uint_as_float((key >> 1) | ((key & 1u) ? 0u : 0x80000000u));
    return __bfloat162float(__float2bfloat16_rn(e * -0.125f));
}
// The code of x under s.  A group with an infinity or a NaN has an infinite or
// NaN scale; its codes become 8 (a NaN converts to 0), and it reads as NaN.
__device__ __forceinline__ uint32_t kv4_code(float x, float s) {
    const int n = s == 0.0f ? 0 : __float2int_rn(__fdiv_rn(x, s));
    return static_cast<uint32_t>(min(max(n, -8), 7) + 8);
}
// Eight dims (a chunk: dims 8 ch .. 8 ch + 7) as one word, the first lowest.
__device__ __forceinline__ uint32_t kv4_pack8(const float *x, float s) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= kv4_code(x[i], s) << (4 * i);
    return w;
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

}  // namespace xs
