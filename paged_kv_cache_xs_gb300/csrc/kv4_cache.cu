// Reading pages of the 4-bit cache back as pages of bf16 or fp32 rows: the
// attention of a prompt chunk reads them through its usual block ids (0..n-1
// of the pages written here).
//
// value = s (n - 8): an 8-bit significand times a 4-bit integer, exact in
// fp32 and rounded once to bf16.  Bound by the bytes: 9 D read and 32 D
// (bf16) written for each page and head.
#include "kv4.cuh"

namespace xs {
namespace {

constexpr int kUnpackThreads = 256;

template <typename T> struct Store8;
template <> struct Store8<__nv_bfloat16> {
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, const float *f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Store8<float> {
    static __device__ __forceinline__ void put(float *p, const float *f) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// One thread turns one chunk of 8 dims (a word of a K page, two half words of
// a V page) into 8 values; a warp's stores are contiguous.
template <typename T, int D>
__global__ void __launch_bounds__(kUnpackThreads)
    kv4_unpack_kernel(T *__restrict__ k_out, T *__restrict__ v_out,
                      const uint8_t *__restrict__ k_cache, const uint8_t *__restrict__ v_cache,
                      const int32_t *__restrict__ ids, int n, int Hkv, int64_t num_blocks,
                      int *err_flag) {
    constexpr int NG = D / kKv4Group, kChunks = 16 * D / 8;
    const int64_t total = static_cast<int64_t>(n) * Hkv * 2 * kChunks;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += stride) {
        const int at = static_cast<int>(i % kChunks);
        const int64_t item = i / kChunks;           // ((page, K or V), head)
        const int64_t pv = item / Hkv;
        const int h = static_cast<int>(item - pv * Hkv);
        const bool is_v = pv & 1;
        const int32_t blk = ids[pv >> 1];
        if (blk < 0) continue;                      // no page here: left as it was
        if (blk >= num_blocks) {
            if (at == 0 && h == 0) raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
            continue;
        }
        const uint8_t *page = (is_v ? v_cache : k_cache) +
                              (static_cast<int64_t>(blk) * Hkv + h) * kv4_page_bytes(D);
        const __nv_bfloat16 *scales = reinterpret_cast<const __nv_bfloat16 *>(page + 8 * D);
        const int o = at / (D / 8), ch = at % (D / 8), c = ch >> 2, t = ch & 3;
        uint32_t w;
        float s;
        if (is_v) {
            const uint16_t *half = reinterpret_cast<const uint16_t *>(page);
            const int pair = o >> 1, r = o & 1;
            w = half[((pair * 8 + 2 * t) * NG + c) * 2 + r] |
                static_cast<uint32_t>(half[((pair * 8 + 2 * t + 1) * NG + c) * 2 + r]) << 16;
            s = __bfloat162float(scales[(pair * NG + c) * 2 + r]);
        } else {
            w = reinterpret_cast<const uint32_t *>(page)[o * (D / 8) + t * NG + c];
            s = __bfloat162float(scales[o * NG + c]);
        }
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = s * static_cast<float>(static_cast<int>((w >> (4 * e)) & 15) - 8);
        T *dst = (is_v ? v_out : k_out) + (((pv >> 1) * Hkv + h) * 16 + o) * D + 8 * ch;
        Store8<T>::put(dst, f);
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
    const int64_t total = static_cast<int64_t>(n) * Hkv * 2 * (2 * D);
    const int64_t want = (total + xs::kUnpackThreads - 1) / xs::kUnpackThreads;
    const int grid = static_cast<int>(want < (1 << 20) ? want : (1 << 20));
    auto kc = static_cast<const uint8_t *>(k_cache), vc = static_cast<const uint8_t *>(v_cache);
    auto go = [&](auto kernel, auto *ko, auto *vo) {
        kernel<<<grid, xs::kUnpackThreads, 0, stream>>>(ko, vo, kc, vc, block_ids, n, Hkv,
                                                        num_blocks, err_flag);
    };
    if (dtype == XS_BF16) {
        auto *ko = static_cast<__nv_bfloat16 *>(k_out), *vo = static_cast<__nv_bfloat16 *>(v_out);
        D == 128 ? go(xs::kv4_unpack_kernel<__nv_bfloat16, 128>, ko, vo)
                 : go(xs::kv4_unpack_kernel<__nv_bfloat16, 64>, ko, vo);
    } else {
        auto *ko = static_cast<float *>(k_out), *vo = static_cast<float *>(v_out);
        D == 128 ? go(xs::kv4_unpack_kernel<float, 128>, ko, vo)
                 : go(xs::kv4_unpack_kernel<float, 64>, ko, vo);
    }
    return xs::launch_status();
}
