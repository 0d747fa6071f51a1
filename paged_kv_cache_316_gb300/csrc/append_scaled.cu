// append_scaled.cu -- append of 16-bit tokens to a paged E4M3 cache that has
// one power-of-two scale for each block of tokens and head.
//
// A block's scale s' is the larger of what it had (if it holds earlier
// tokens) and the smallest 2^e under which its new values fit E4M3's range:
// with |x| <= a = m 2^x, m in [1, 2), and 448 = 1.75 * 2^8, e = x - 8 if m <=
// 1.75 and x - 7 otherwise.  New codes are rn(x / s'), earlier codes of a
// block whose scale grew rn(c s / s').
//
// The entries of one block form a run (consecutive positions); the first
// entry of a run leads it.  One warp takes one (entry, head, K or V): it
// leaves unless the entry leads, else it reads the run once for the largest
// magnitude and once to quantise.
#include <type_traits>

#include "pkv_common.cuh"

namespace pkv {

struct AppendScaledParams {
    const uint16_t *src[2];  // key, value: [nnz, H, D]
    uint8_t *cache[2];
    float *scales[2];
    int64_t nnz, page_stride, max_num_pages, scale_stride;
    const int32_t *batch_indices, *positions, *kv_indices, *kv_indptr, *kv_last_page_len;
    int B, H, D, page_shift, block_shift;
    int32_t *err;
};

constexpr int kAsWarps = 4;
constexpr int kAsMinExp = -40, kAsMaxExp = 40;

// Two finite-or-zero magnitudes (16-bit patterns without sign) of a pair.
template <typename T>
__device__ __forceinline__ uint32_t finite_mags(uint32_t w) {
    constexpr uint32_t kInf = sizeof(T) && std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
    lo = lo < kInf ? lo : 0u;
    hi = hi < kInf ? hi : 0u;
    return lo | (hi << 16);
}

template <typename T>
__device__ __forceinline__ float2 widen2(uint32_t w);
template <>
__device__ __forceinline__ float2 widen2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <>
__device__ __forceinline__ float2 widen2<__nv_bfloat16>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

// Two floats -> two E4M3 codes, a in the low byte (nearest even, saturating).
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// The scale exponent under which values up to `a` (>= 0, finite) fit.
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t u = __float_as_uint(a);
    const int x = static_cast<int>(u >> 23) - 127;
    const int e = (u & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;
    return min(max(e, kAsMinExp), kAsMaxExp);
}

template <typename T, int LAYOUT>
__global__ void __launch_bounds__(kAsWarps * 32) append_scaled_kernel(const AppendScaledParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kAsWarps + (threadIdx.x >> 5);
    const int64_t i = item / (2 * p.H);
    const int hk = static_cast<int>(item % (2 * p.H));
    if (i >= p.nnz) return;
    const int z = hk / p.H, h = hk % p.H;
    const int S = 1 << p.page_shift, G = 1 << p.block_shift;
    const int b = p.batch_indices[i], pos = p.positions[i];
    const bool first_of_all = hk == 0 && lane == 0;  // one lane reports an entry's faults
    if (b < 0 || b >= p.B) {
        if (first_of_all) set_err(p.err, PKV_DEV_ERR_BATCH);
        return;
    }
    const int page0 = p.kv_indptr[b];
    const int pages = p.kv_indptr[b + 1] - page0;
    const int64_t len = pages > 0 ? static_cast<int64_t>(pages - 1) * S + p.kv_last_page_len[b] : 0;
    if (pos < 0 || pos >= len || (pos >> p.page_shift) >= pages) {
        if (first_of_all) set_err(p.err, PKV_DEV_ERR_POS);
        return;
    }
    if (i > 0 && p.batch_indices[i - 1] == b) {
        const int before = p.positions[i - 1];
        if (before >= 0 && before >> p.block_shift == pos >> p.block_shift) {
            if (before + 1 != pos && first_of_all) set_err(p.err, PKV_DEV_ERR_POS);
            return;  // led by an earlier entry, or out of order
        }
    }
    const int64_t page = p.kv_indices[page0 + (pos >> p.page_shift)];
    if (page < 0 || page >= p.max_num_pages) {
        if (first_of_all) set_err(p.err, PKV_DEV_ERR_PAGE);
        return;
    }
    // entries i .. i + n - 1 have the positions pos, pos + 1, .. of this block
    const int slot0 = pos & (S - 1), in_block = pos & (G - 1);
    const int most = static_cast<int>(min(static_cast<int64_t>(G - in_block), min(p.nnz - i, len - pos)));
    int n = 1;
    while (n < most) {
        const int j = n + lane;
        const bool same = j < most && p.batch_indices[i + j] == b && p.positions[i + j] == pos + j;
        const unsigned m = __ballot_sync(0xffffffffu, same);
        if (m != 0xffffffffu) {
            n += __ffs(~m) - 1;
            break;
        }
        n += 32;
    }

    const int C = p.D / 8;  // 16-byte chunks of a source row
    const uint16_t *src = p.src[z] + (i * p.H + h) * static_cast<int64_t>(p.D);
    const int64_t src_row = static_cast<int64_t>(p.H) * p.D;
    uint32_t mag = 0;
    for (int q = lane; q < n * C; q += 32) {
        const uint4 v = *reinterpret_cast<const uint4 *>(src + (q / C) * src_row + (q % C) * 8);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) mag = __vmaxu2(mag, finite_mags<T>(w[k]));
    }
    mag = __vmaxu2(mag, mag >> 16) & 0xffffu;
    const float amax = widen2<T>(__reduce_max_sync(0xffffffffu, mag)).x;

    float *scale = p.scales[z] + page * p.scale_stride + (static_cast<int64_t>(h) << (p.page_shift - p.block_shift)) +
                   (slot0 >> p.block_shift);
    float s = ldexpf(1.f, scale_exponent(amax));
    float was = s;
    if (in_block > 0) {
        was = checked_scale(*scale, p.err);
        s = fmaxf(s, was);
    }
    __syncwarp();
    if (lane == 0) *scale = s;

    uint8_t *cache = p.cache[z];
    if (s > was) {  // earlier tokens of the block, rounded again under the larger scale
        const float r = was / s;
        for (int q = lane; q < in_block * C; q += 32) {
            uint8_t *at = cache + kv_row_offset<LAYOUT>(page, p.page_stride, h, slot0 - in_block + q / C, p.H, S, p.D) +
                          (q % C) * 8;
            const uint2 v = *reinterpret_cast<const uint2 *>(at);
            const uint32_t w[2] = {v.x, v.y};
            uint32_t o[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 lo = widen2<__half>(widen_e4m3x2<__half>(w[k] & 0xffffu));
                const float2 hi = widen2<__half>(widen_e4m3x2<__half>(w[k] >> 16));
                o[k] = to_e4m3x2(lo.x * r, lo.y * r) | to_e4m3x2(hi.x * r, hi.y * r) << 16;
            }
            *reinterpret_cast<uint2 *>(at) = make_uint2(o[0], o[1]);
        }
    }
    // x / s, exact as a product when s is a power of two
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
    const float inv = 1.f / s;
    for (int q = lane; q < n * C; q += 32) {
        const uint4 v = *reinterpret_cast<const uint4 *>(src + (q / C) * src_row + (q % C) * 8);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float2 f = widen2<T>(w[k]);
            f = pow2 ? make_float2(f.x * inv, f.y * inv) : make_float2(f.x / s, f.y / s);
            o[k] = to_e4m3x2(f.x, f.y);
        }
        *reinterpret_cast<uint2 *>(cache + kv_row_offset<LAYOUT>(page, p.page_stride, h, slot0 + q / C, p.H, S, p.D) +
                                   (q % C) * 8) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    }
}

}  // namespace pkv

using namespace pkv;

extern "C" int paged_append_scaled(const void *append_key, const void *append_value, int64_t nnz,
                                   const int32_t *batch_indices, const int32_t *positions, void *k_cache,
                                   void *v_cache, int64_t page_stride, int64_t max_num_pages, float *k_scales,
                                   float *v_scales, int64_t scale_page_stride, int32_t scale_block,
                                   const int32_t *kv_indices, const int32_t *kv_indptr,
                                   const int32_t *kv_last_page_len, int32_t batch_size, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t page_size, int32_t layout, int32_t dtype,
                                   int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_append_scaled");
    if (layout != PKV_NHD && layout != PKV_HND) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (nnz < 0 || batch_size < 0 || num_kv_heads <= 0 || head_dim <= 0 || max_num_pages < 0 || page_stride <= 0)
        return PKV_ERR_INVALID_ARG;
    if (head_dim % 16) return PKV_ERR_INVALID_ARG;  // 16-byte cache rows
    const int ps = ilog2_exact(page_size), bs = ilog2_exact(scale_block);
    if (ps < 3 || ps > 8) return PKV_ERR_UNSUPPORTED;
    if (bs < 3 || bs > ps) return PKV_ERR_INVALID_ARG;
    if (page_stride < static_cast<int64_t>(num_kv_heads) * page_size * head_dim || page_stride % 16 ||
        scale_page_stride < (static_cast<int64_t>(num_kv_heads) << (ps - bs)))
        return PKV_ERR_INVALID_ARG;
    if (nnz == 0) return PKV_OK;
    if (!append_key || !append_value || !batch_indices || !positions || !k_cache || !v_cache || !k_scales ||
        !v_scales || !kv_indices || !kv_indptr || !kv_last_page_len)
        return PKV_ERR_NULL;
    if (!aligned16(append_key) || !aligned16(append_value) || !aligned16(k_cache) || !aligned16(v_cache) ||
        ((reinterpret_cast<uintptr_t>(k_scales) | reinterpret_cast<uintptr_t>(v_scales)) & 3))
        return PKV_ERR_INVALID_ARG;
    const int64_t items = nnz * 2 * num_kv_heads;
    const int64_t blocks = (items + kAsWarps - 1) / kAsWarps;
    if (nnz > 0x7fffffff || blocks > 0x7fffffff) return PKV_ERR_UNSUPPORTED;

    AppendScaledParams p;
    p.src[0] = static_cast<const uint16_t *>(append_key);
    p.src[1] = static_cast<const uint16_t *>(append_value);
    p.cache[0] = static_cast<uint8_t *>(k_cache);
    p.cache[1] = static_cast<uint8_t *>(v_cache);
    p.scales[0] = k_scales;
    p.scales[1] = v_scales;
    p.nnz = nnz;
    p.page_stride = page_stride;
    p.max_num_pages = max_num_pages;
    p.scale_stride = scale_page_stride;
    p.batch_indices = batch_indices;
    p.positions = positions;
    p.kv_indices = kv_indices;
    p.kv_indptr = kv_indptr;
    p.kv_last_page_len = kv_last_page_len;
    p.B = batch_size;
    p.H = num_kv_heads;
    p.D = head_dim;
    p.page_shift = ps;
    p.block_shift = bs;
    p.err = err_word;
    auto kern = dtype == PKV_BF16
                    ? (layout == PKV_HND ? append_scaled_kernel<__nv_bfloat16, PKV_HND>
                                         : append_scaled_kernel<__nv_bfloat16, PKV_NHD>)
                    : (layout == PKV_HND ? append_scaled_kernel<__half, PKV_HND> : append_scaled_kernel<__half, PKV_NHD>);
    kern<<<static_cast<unsigned>(blocks), kAsWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
    note_launches(1);
    return launch_status();
}
