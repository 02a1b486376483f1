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
// A row is D / 16 lanes.  Each lane holds two chunks of 8 dims that the
// rotation pairs with one another (dims 8 j.. and rotary_dim / 2 + 8 j.. of
// split halves, 16 j.. of neighbouring pairs), so the rotation needs no
// exchange and every access is 16 bytes.  Nothing is read twice but the table
// and the weights, which stay in the caches: the pass is bound by the bytes of
// the rows, or for a decode batch by the latency of length -> table -> page.
#include "kv4.cuh"

namespace xs {
namespace {

constexpr int kRopeThreads = 256;

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
    bool interleaved, kv4;
    int *err_flag;
};

// Chunk of 8 values at p (16-byte aligned) as fp32, and back.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *f) {
    unpack16(*reinterpret_cast<const uint4 *>(p), f, static_cast<__nv_bfloat16 *>(nullptr));
}
__device__ __forceinline__ void load8(const float *p, float *f) {
    unpack16(reinterpret_cast<const uint4 *>(p)[0], f, static_cast<float *>(nullptr));
    unpack16(reinterpret_cast<const uint4 *>(p)[1], f + 4, static_cast<float *>(nullptr));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float *f) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Mean of the squares of a row, of which each of its lanes holds 16 values.
template <int kLanes> __device__ __forceinline__ float mean_square(const float *x) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
    for (int m = kLanes / 2; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    return sum * (1.0f / (16 * kLanes));
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
    const int32_t blk = p.tables[t * p.max_blocks + page];
    if (blk < 0 || blk >= p.num_blocks) {
        raise_flag(err_flag, XS_FLAG_BAD_BLOCK);
        return -1;
    }
    return static_cast<int64_t>(blk) * 16 + (pos & 15);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeParams p) {
    constexpr int kLanes = D / 16;              // lanes of a row
    constexpr int kRows = 32 / kLanes;          // rows of a warp
    __shared__ uint32_t keys[kRopeThreads / 32][kRows][D / 8];
    const int lane = threadIdx.x & 31, j = lane % kLanes, warp = threadIdx.x >> 5;
    const int64_t total = static_cast<int64_t>(p.T) * p.rows_per_token;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kRopeThreads / kLanes);
    for (int64_t base = (static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + warp) * kRows;
         base < total; base += step) {
        const int64_t r = base + lane / kLanes;
        bool on = r < total;
        const int64_t t = !on ? 0
                          : total < (int64_t(1) << 32)
                              ? static_cast<uint32_t>(r) / static_cast<uint32_t>(p.rows_per_token)
                              : r / p.rows_per_token;
        const int h = static_cast<int>(on ? r - t * p.rows_per_token : 0);
        const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hkv;
        int64_t pos = 0;
        if (on) {
            if (p.lens)
                pos = static_cast<int64_t>(p.lens[t]) - 1;
            else if (p.positions)
                pos = p.positions[t];
            on = pos >= 0;
        }
        const bool turned = p.rot > 0 && !is_v;
        if (on && turned && pos >= p.max_pos) {
            if (j == 0) raise_flag(p.err_flag, XS_FLAG_BAD_LEN);
            on = false;
        }
        // The lane's two chunks, and the index of its first pair's angle.
        const bool rotates = turned && j < p.rot / 16;
        const bool split = rotates && !p.interleaved;
        const int c0 = split ? j : 2 * j, c1 = split ? p.rot / 16 + j : 2 * j + 1;
        const T *src = is_q   ? static_cast<const T *>(p.q) + t * p.q_stride + h * D
                       : is_v ? static_cast<const T *>(p.v) + t * p.v_stride + (h - p.Hq - p.Hkv) * D
                              : static_cast<const T *>(p.k) + t * p.k_stride + (h - p.Hq) * D;
        float x[16];
        if (on) {
            load8(src + 8 * c0, x);
            load8(src + 8 * c1, x + 8);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 0.0f;
        }
        const T *w = static_cast<const T *>(is_v ? nullptr : is_q ? p.q_weight : p.k_weight);
        float mean = mean_square<kLanes>(x) + p.eps;
        // Squares that leave fp32 (|x| beyond 2^60, or below 2^-50 under an eps
        // that does not cover it) are taken of x 2^-96 or x 2^96 instead.
        const float lift = mean > 0x1p125f ? 0x1p-96f : mean < 0x1p-100f ? 0x1p96f : 1.0f;
        if (__any_sync(0xffffffffu, lift != 1.0f)) {
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = x[i] * lift;
            mean = mean_square<kLanes>(y) + p.eps * lift * lift;
            if (w) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = y[i];
            }
        }
        if (on && w) {
            const float rms = rsqrtf(mean);
            float g[16];
            load8(w + 8 * c0, g);
            load8(w + 8 * c1, g + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] *= rms * g[i];
        }
        if (on && rotates) {
            float c[8], s[8];
            const float *row = p.cos_sin + pos * p.rot + 8 * j;
            load8(row, c);
            load8(row + p.rot / 2, s);
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a = x[2 * i], b = x[2 * i + 1];
                    x[2 * i] = a * c[i] - b * s[i];
                    x[2 * i + 1] = b * c[i] + a * s[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a = x[i], b = x[8 + i];
                    x[i] = a * c[i] - b * s[i];
                    x[8 + i] = b * c[i] + a * s[i];
                }
            }
        }
        if (is_q || !p.k_cache) {
            if (on) {
                T *dst = is_q ? static_cast<T *>(p.q_out) + (t * p.Hq + h) * D
                              : static_cast<T *>(p.k_out) + (t * p.Hkv + h - p.Hq) * D;
                store8(dst + 8 * c0, x);
                store8(dst + 8 * c1, x + 8);
            }
            on = false;
        }
        int64_t slot = -1;
        if (on) slot = append_slot(p, t, pos, j == 0 && !is_v ? p.err_flag : nullptr);
        const int hk = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
        const int64_t page = slot < 0 ? 0 : (slot >> 4) * p.Hkv + hk;
        const int o = static_cast<int>(slot & 15);
        if (slot >= 0 && !XS_BOUNDS(page >= 0 && page < p.num_blocks * p.Hkv, p.err_flag)) slot = -1;
        uint8_t *cache = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache);
        if (!p.kv4) {
            if (slot >= 0) {
                T *dst = reinterpret_cast<T *>(cache) + (page * 16 + o) * D;
                store8(dst + 8 * c0, x);
                store8(dst + 8 * c1, x + 8);
            }
            continue;
        }
        // 4 bits: the extremes of the row's chunks meet in shared memory (a
        // group's four chunks are not always the lanes of one row's half).
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = Elem<T>::to_f32(Elem<T>::from_f32(x[i]));
        uint32_t m0 = 0, m1 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            m0 = max(m0, kv4_key(x[i]));
            m1 = max(m1, kv4_key(x[8 + i]));
        }
        uint32_t *row_keys = keys[warp][lane / kLanes];
        __syncwarp();
        row_keys[c0] = m0;
        row_keys[c1] = m1;
        __syncwarp();
        if (slot >= 0) {
            uint8_t *dst = cache + page * kv4_page_bytes(D);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int ch = u ? c1 : c0;
                const uint32_t *k4 = row_keys + (ch & ~3);
                const float s = kv4_scale(max(max(k4[0], k4[1]), max(k4[2], k4[3])));
                kv4_store_chunk<D>(dst, is_v, o, ch, kv4_pack8(x + 8 * u, s), s);
            }
        }
    }
}

bool strided_ok(const void *ptr, int64_t stride, int eb) {
    return aligned16(ptr) && (stride * eb) % 16 == 0;
}

int launch(RopeParams &p, int D, int dtype, cudaStream_t stream) {
    p.rows_per_token = p.Hq + p.Hkv + (p.k_cache ? p.Hkv : 0);
    const int rows_per_cta = kRopeThreads / (D / 16);
    const int64_t want =
        (static_cast<int64_t>(p.T) * p.rows_per_token + rows_per_cta - 1) / rows_per_cta;
    const int grid = static_cast<int>(want < (1 << 20) ? want : (1 << 20));
    if (dtype == XS_F32) {
        if (D == 128)
            qk_norm_rope_kernel<float, 128><<<grid, kRopeThreads, 0, stream>>>(p);
        else
            qk_norm_rope_kernel<float, 64><<<grid, kRopeThreads, 0, stream>>>(p);
    } else {
        if (D == 128)
            qk_norm_rope_kernel<__nv_bfloat16, 128><<<grid, kRopeThreads, 0, stream>>>(p);
        else
            qk_norm_rope_kernel<__nv_bfloat16, 64><<<grid, kRopeThreads, 0, stream>>>(p);
    }
    return launch_status();
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
