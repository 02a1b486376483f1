// Reading pages of the 4-bit cache back as pages of bf16 or fp32 rows: the
// attention of a prompt chunk reads them through its usual block ids (0..n-1
// of the pages written here).
//
// value = s (n - 8): an 8-bit significand times a 4-bit integer, exact in
// fp32 and rounded once to bf16.  Bound by the bytes: 9 D read and 32 D
// (bf16) written for each page and head.  (2,048 pages of 8 heads x 128: 28 us as bf16,
// a floor of 25; 97 us as fp32, a floor of 45.)
#include "kv4.cuh"

namespace xs {
namespace {

constexpr int kUnpackThreads = 256;

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t x) {
    return *reinterpret_cast<const __nv_bfloat162 *>(&x);
}
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) {
    return *reinterpret_cast<const uint32_t *>(&x);
}
// n - 8 for the low nibbles n of both halves of a word, as bf16: 0x4300 | n is
// 128 + n, and the difference is exact.
__device__ __forceinline__ uint32_t centred(uint32_t w) {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w), "r"(0x000f000fu), "r"(0x43004300u));
    return as_u32(__hsub2(as_bf162(x), as_bf162(0x43084308u)));
}
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t s) {
    return as_u32(__hmul2(as_bf162(x), as_bf162(s)));   // one rounding
}
__device__ __forceinline__ float lo_f32(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f32(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Eight values of a K row: d[j] holds n - 8 of dims j and j + 4, s2 the scale twice.
__device__ __forceinline__ void store_k(__nv_bfloat16 *p, const uint32_t *d, uint32_t s2) {
    uint32_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = times(d[j], s2);
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                   __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}
__device__ __forceinline__ void store_k(float *p, const uint32_t *d, uint32_t s2) {
    const float s = lo_f32(s2);
    reinterpret_cast<float4 *>(p)[0] =
        make_float4(lo_f32(d[0]) * s, lo_f32(d[1]) * s, lo_f32(d[2]) * s, lo_f32(d[3]) * s);
    reinterpret_cast<float4 *>(p)[1] =
        make_float4(hi_f32(d[0]) * s, hi_f32(d[1]) * s, hi_f32(d[2]) * s, hi_f32(d[3]) * s);
}
// Eight dims of two V rows, `step` elements apart: d[j] holds n - 8 of dim j of
// both, s2 their scales.
__device__ __forceinline__ void store_v(__nv_bfloat16 *p, int step, const uint32_t *d, uint32_t s2) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = times(d[j], s2);
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                   __byte_perm(v[4], v[5], 0x5410), __byte_perm(v[6], v[7], 0x5410));
    *reinterpret_cast<uint4 *>(p + step) =
        make_uint4(__byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632),
                   __byte_perm(v[4], v[5], 0x7632), __byte_perm(v[6], v[7], 0x7632));
}
__device__ __forceinline__ void store_v(float *p, int step, const uint32_t *d, uint32_t s2) {
    const float a = lo_f32(s2), b = hi_f32(s2);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t *e = d + 4 * k;
        reinterpret_cast<float4 *>(p)[k] =
            make_float4(lo_f32(e[0]) * a, lo_f32(e[1]) * a, lo_f32(e[2]) * a, lo_f32(e[3]) * a);
        reinterpret_cast<float4 *>(p + step)[k] =
            make_float4(hi_f32(e[0]) * b, hi_f32(e[1]) * b, hi_f32(e[2]) * b, hi_f32(e[3]) * b);
    }
}

// Words of a lane's 16 (D = 128) or 8 (D = 64) bytes of codes.
template <int NG> __device__ __forceinline__ void load_codes(uint32_t *w, const uint8_t *p) {
    if constexpr (NG == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    }
}

// A warp turns one page (16 rows of one head, K or V), two passes of 8 rows.
// Its loads are whole lines; its stores are 64 contiguous bytes (bf16) for
// each row and group of 32 dims.
template <typename T, int D>
__global__ void __launch_bounds__(kUnpackThreads)
    kv4_unpack_kernel(T *__restrict__ k_out, T *__restrict__ v_out,
                      const uint8_t *__restrict__ k_cache, const uint8_t *__restrict__ v_cache,
                      const int32_t *__restrict__ ids, int n, int Hkv, int64_t num_blocks,
                      int *err_flag) {
    constexpr int NG = D / kKv4Group;
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t total = static_cast<int64_t>(n) * Hkv * 2;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * (kUnpackThreads / 32);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kUnpackThreads / 32) + (threadIdx.x >> 5);
         item < total; item += stride) {
        const int64_t pv = total < (int64_t(1) << 32)
                               ? static_cast<uint32_t>(item) / static_cast<uint32_t>(Hkv)
                               : item / Hkv;                    // (page, K or V)
        const int h = static_cast<int>(item - pv * Hkv);
        const bool is_v = pv & 1;
        const int32_t blk = ids[pv >> 1];
        if (blk < 0) continue;                                  // no page here: left as it was
        if (blk >= num_blocks) {
            if (lane == 0 && h == 0) raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
            continue;
        }
        const uint8_t *page = (is_v ? v_cache : k_cache) +
                              (static_cast<int64_t>(blk) * Hkv + h) * kv4_page_bytes(D);
        if (!XS_BOUNDS((pv >> 1) < n && h >= 0 && h < Hkv, err_flag)) continue;
        T *out = (is_v ? v_out : k_out) + ((pv >> 1) * Hkv + h) * (16 * D);
        uint32_t w[2][NG];
        if (!is_v) {
            // Lane (g, t): row g (+ 8), dims 32 c + 8 t .. + 7.
            const int g = lane >> 2, t = lane & 3;
            uint16_t s[2][NG];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                load_codes<NG>(w[u], page + (g + 8 * u) * (D / 2) + t * (4 * NG));
#pragma unroll
                for (int c = 0; c < NG; ++c)
                    s[u][c] = reinterpret_cast<const uint16_t *>(page + 8 * D)[(g + 8 * u) * NG + c];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < NG; ++c) {
                    uint32_t d[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) d[j] = centred(w[u][c] >> (4 * j));
                    store_k(out + (g + 8 * u) * D + 32 * c + 8 * t, d, s[u][c] * 0x10001u);
                }
        } else {
            // Lane (i, q): dims 32 c + 8 q .. + 7 of rows 2 i and 2 i + 1.
            const int i = lane >> 2, q = lane & 3;
            uint32_t s2[NG];
            load_codes<NG>(w[0], page + i * D + (2 * q) * (4 * NG));
            load_codes<NG>(w[1], page + i * D + (2 * q + 1) * (4 * NG));
            load_codes<NG>(s2, page + 8 * D + i * (4 * NG));
#pragma unroll
            for (int c = 0; c < NG; ++c) {
                uint32_t d[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = centred(w[j >> 2][c] >> (4 * (j & 3)));
                store_v(out + 2 * i * D + 32 * c + 8 * q, D, d, s2[c]);
            }
        }
    }
}

}  // namespace
XS_DEFINE_BOUNDS_COUNTER(bounds_failures_kv4_cache)

}  // namespace xs

extern "C" int64_t xs_kv4_page_bytes(int D) {
    return D == 64 || D == 128 ? xs::kv4_page_bytes(D) : static_cast<int64_t>(XS_EUNSUPPORTED);
}

extern "C" int xs_kv4_unpack(void *k_out, void *v_out, const void *k_cache, const void *v_cache,
                             const int32_t *block_ids, int n, int Hkv, int D, int block_size,
                             int64_t num_blocks, int dtype, int *err_flag, cudaStream_t stream) {
    if (!k_out || !v_out || !k_cache || !v_cache || !block_ids) return XS_ENULL;
    if (!xs::elem_bytes(dtype)) return XS_EDTYPE;
    if (n < 0 || Hkv <= 0 || D <= 0 || block_size <= 0 || num_blocks < 0) return XS_ESHAPE;
    if ((D != 64 && D != 128) || block_size != 16) return XS_EUNSUPPORTED;
    if (!xs::aligned16(k_out) || !xs::aligned16(v_out) || !xs::aligned16(k_cache) ||
        !xs::aligned16(v_cache))
        return XS_EALIGN;
    if (n == 0) return XS_OK;
    const int64_t total = static_cast<int64_t>(n) * Hkv * 2;     // a warp each
    const int64_t want = (total + xs::kUnpackThreads / 32 - 1) / (xs::kUnpackThreads / 32);
    const int grid = static_cast<int>(want < (1 << 20) ? want : (1 << 20));
    auto kc = static_cast<const uint8_t *>(k_cache), vc = static_cast<const uint8_t *>(v_cache);
    auto go = [&](auto kernel, auto *ko, auto *vo) {
        return xs::launch_after(kernel, dim3(grid), xs::kUnpackThreads, 0, stream, 1, ko, vo, kc, vc,
                                block_ids, n, Hkv, num_blocks, err_flag);
    };
    if (dtype == XS_BF16) {
        auto *ko = static_cast<__nv_bfloat16 *>(k_out), *vo = static_cast<__nv_bfloat16 *>(v_out);
        return D == 128 ? go(xs::kv4_unpack_kernel<__nv_bfloat16, 128>, ko, vo)
                        : go(xs::kv4_unpack_kernel<__nv_bfloat16, 64>, ko, vo);
    }
    auto *ko = static_cast<float *>(k_out), *vo = static_cast<float *>(v_out);
    return D == 128 ? go(xs::kv4_unpack_kernel<float, 128>, ko, vo)
                    : go(xs::kv4_unpack_kernel<float, 64>, ko, vo);
}
