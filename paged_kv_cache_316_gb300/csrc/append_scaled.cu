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
// entry of a run leads it.  A CTA takes kAsEntries entries (fewer when there
// are few): in every warp lane j resolves entry j, so that the chain of index
// reads runs once for all of a CTA's heads, then the warps share the heads of
// K and V and take the runs that start in the CTA's entries one after another.
// A run of up to 16 rows of 128 elements stays in registers between its
// largest magnitude and its quantisation (eight 16-byte loads a lane, all in
// flight), so every new value is read once; longer runs and other widths are
// read twice, the second time from L2.
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
    int entries;  // entries a CTA takes, at most kAsEntries
    int32_t *err;
};

constexpr int kAsWarps = 8;
constexpr int kAsEntries = 16;
constexpr int kAsMinExp = -40, kAsMaxExp = 40;

// The pattern of infinity without sign: magnitudes from it on are not finite.
template <typename T>
__device__ __forceinline__ uint32_t inf_bits() {
    return std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
}
// Two finite-or-zero magnitudes (16-bit patterns without sign) of a pair.
template <typename T>
__device__ __forceinline__ uint32_t finite_mags(uint32_t w) {
    const uint32_t kInf = inf_bits<T>();
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

// Eight 16-bit values over s -> eight codes: as products with 1 / s (EXACT:
// s is a power of two), else as quotients.
template <typename T, bool EXACT>
__device__ __forceinline__ uint2 quantise8(const uint4 &v, float s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const float inv = EXACT ? __uint_as_float((254u << 23) - __float_as_uint(s)) : 0.f;
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = widen2<T>(w[k]);
        o[k] = EXACT ? to_e4m3x2(f.x * inv, f.y * inv) : to_e4m3x2(f.x / s, f.y / s);
    }
    return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

// C: 16-byte chunks of a source row (0: any, p.D / 8)
template <typename T, int LAYOUT, int C_>
__global__ void __launch_bounds__(kAsWarps * 32) append_scaled_kernel(const AppendScaledParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = 1 << p.page_shift, G = 1 << p.block_shift;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * p.entries;
    // lane j: entry i0 + j (the CTA leads the runs that start in its first
    // p.entries entries; the others tell where those runs end)
    const int64_t i = i0 + lane;
    const bool report = warp == 0 && blockIdx.y == 0 && lane < p.entries && i < p.nnz;
    int b = -1, pos = -1, most = 0;
    int64_t page = -1;
    bool leads = false;
    if (i < p.nnz) {
        b = p.batch_indices[i];
        pos = p.positions[i];
    }
    int b_before = __shfl_up_sync(0xffffffffu, b, 1), pos_before = __shfl_up_sync(0xffffffffu, pos, 1);
    if (lane == 0 && i > 0 && i < p.nnz) {
        b_before = p.batch_indices[i - 1];
        pos_before = p.positions[i - 1];
    }
    if (lane < p.entries && i < p.nnz) {
        if (b < 0 || b >= p.B) {
            if (report) set_err(p.err, PKV_DEV_ERR_BATCH);
        } else {
            const int page0 = p.kv_indptr[b];
            const int pages = p.kv_indptr[b + 1] - page0;
            const int64_t len = pages > 0 ? static_cast<int64_t>(pages - 1) * S + p.kv_last_page_len[b] : 0;
            if (pos < 0 || pos >= len || (pos >> p.page_shift) >= pages) {
                if (report) set_err(p.err, PKV_DEV_ERR_POS);
            } else if (i > 0 && b_before == b && pos_before >= 0 &&
                       pos_before >> p.block_shift == pos >> p.block_shift) {
                // led by an earlier entry, or out of order
                if (pos_before + 1 != pos && report) set_err(p.err, PKV_DEV_ERR_POS);
            } else {
                page = p.kv_indices[page0 + (pos >> p.page_shift)];
                if (page < 0 || page >= p.max_num_pages) {
                    if (report) set_err(p.err, PKV_DEV_ERR_PAGE);
                } else {
                    leads = true;
                    most = static_cast<int>(
                        min(static_cast<int64_t>(G - (pos & (G - 1))), min(p.nnz - i, len - static_cast<int64_t>(pos))));
                }
            }
        }
    }
    // entry j + 1 goes on where entry j is
    const int b_after = __shfl_down_sync(0xffffffffu, b, 1), pos_after = __shfl_down_sync(0xffffffffu, pos, 1);
    const unsigned joined = __ballot_sync(0xffffffffu, lane < 31 && b_after == b && pos_after == pos + 1);
    const int C = C_ ? C_ : p.D / 8;
    const int64_t src_row = static_cast<int64_t>(p.H) * p.D;
    for (unsigned todo = __ballot_sync(0xffffffffu, leads); todo; todo &= todo - 1) {
        const int j = __ffs(todo) - 1;
        const int rb = __shfl_sync(0xffffffffu, b, j), rpos = __shfl_sync(0xffffffffu, pos, j);
        const int rmost = __shfl_sync(0xffffffffu, most, j);
        const int64_t rpage = __shfl_sync(0xffffffffu, page, j), ri = i0 + j;
        // rows of the run: entries ri .. ri + n - 1
        int n = min(rmost, __ffs(~(joined >> j)));
        if (n < rmost && j + n == 32) {  // it goes on past the lanes' entries
            while (n < rmost) {
                const int k = n + lane;
                const bool same = k < rmost && p.batch_indices[ri + k] == rb && p.positions[ri + k] == rpos + k;
                const unsigned m = __ballot_sync(0xffffffffu, same);
                if (m != 0xffffffffu) {
                    n += __ffs(~m) - 1;
                    break;
                }
                n += 32;
            }
        }
        const int slot0 = rpos & (S - 1), in_block = rpos & (G - 1);
        for (int hk = blockIdx.y * kAsWarps + warp; hk < 2 * p.H; hk += gridDim.y * kAsWarps) {
            const int z = hk >= p.H ? 1 : 0, h = hk - z * p.H;
            const uint16_t *src = p.src[z] + (ri * p.H + h) * static_cast<int64_t>(p.D);
            uint8_t *cache = p.cache[z];
            float *scale = p.scales[z] + rpage * p.scale_stride +
                           (static_cast<int64_t>(h) << (p.page_shift - p.block_shift)) + (slot0 >> p.block_shift);
            float was = in_block > 0 ? *scale : 0.f;  // (its latency overlaps the rows')
            constexpr int kHeld = 8, kC = C_ ? C_ : 16;
            constexpr uint32_t kMag = 0x7fff7fffu;
            const bool held = C_ != 0 && n * C <= kHeld * 32;
            uint4 v[kHeld];
            uint32_t mag = 0;
            if (held) {
                // chunk q = lane + 32 k of the run: (C 16) row lane / 16 + 2 k
                const uint16_t *at = src + (lane / kC) * src_row + (lane % kC) * 8;
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    v[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (lane + 32 * k < n * kC)
                        v[k] = __ldcs(reinterpret_cast<const uint4 *>(at + static_cast<int64_t>(k * (32 / kC)) * src_row));
                }
#pragma unroll
                for (int k = 0; k < kHeld; ++k)
                    mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(v[k].x & kMag, v[k].y & kMag),
                                                 __vmaxu2(v[k].z & kMag, v[k].w & kMag)));
            } else {
                for (int q = lane; q < n * C; q += 32) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(src + (q / C) * src_row + (q % C) * 8);
                    mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(x.x & kMag, x.y & kMag), __vmaxu2(x.z & kMag, x.w & kMag)));
                }
            }
            mag = __vmaxu2(mag, mag >> 16) & 0xffffu;
            mag = __reduce_max_sync(0xffffffffu, mag);
            if (mag >= inf_bits<T>()) {  // an infinity or NaN among them: again, over the finite ones
                mag = 0;
                for (int q = lane; q < n * C; q += 32) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(src + (q / C) * src_row + (q % C) * 8);
                    mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(finite_mags<T>(x.x), finite_mags<T>(x.y)),
                                                 __vmaxu2(finite_mags<T>(x.z), finite_mags<T>(x.w))));
                }
                mag = __vmaxu2(mag, mag >> 16) & 0xffffu;
                mag = __reduce_max_sync(0xffffffffu, mag);
            }
            const float amax = widen2<T>(mag).x;
            // 2^e by its bits: e is in [-40, 40]
            float s = __uint_as_float(static_cast<uint32_t>(scale_exponent(amax) + 127) << 23);
            if (in_block > 0) {
                was = checked_scale(was, p.err);
                s = fmaxf(s, was);
            } else {
                was = s;
            }
            __syncwarp();
            if (lane == 0) *scale = s;
            if (s > was) {  // earlier tokens of the block, rounded again under the larger scale
                const float r = was / s;
                for (int q = lane; q < in_block * C; q += 32) {
                    uint8_t *at = cache +
                                  kv_row_offset<LAYOUT>(rpage, p.page_stride, h, slot0 - in_block + q / C, p.H, S, p.D) +
                                  (q % C) * 8;
                    const uint2 x = *reinterpret_cast<const uint2 *>(at);
                    const uint32_t w[2] = {x.x, x.y};
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
            const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
            uint8_t *dst = cache + kv_row_offset<LAYOUT>(rpage, p.page_stride, h, slot0, p.H, S, p.D);
            const int64_t dst_row = LAYOUT == PKV_HND ? p.D : src_row;
            if (held && pow2) {
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    if (lane + 32 * k < n * kC)
                        *reinterpret_cast<uint2 *>(dst + (lane / kC + k * (32 / kC)) * dst_row + (lane % kC) * 8) =
                            quantise8<T, true>(v[k], s);
                }
            } else {
                for (int q = lane; q < n * C; q += 32) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(src + (q / C) * src_row + (q % C) * 8);
                    *reinterpret_cast<uint2 *>(dst + (q / C) * dst_row + (q % C) * 8) =
                        pow2 ? quantise8<T, true>(x, s) : quantise8<T, false>(x, s);
                }
            }
        }
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
    if (nnz > 0x7fffffff) return PKV_ERR_UNSUPPORTED;

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
    // Entries a CTA takes: as many as leave four CTAs for every SM; with few
    // entries the heads are spread over more CTAs too.
    const int64_t want = 4LL * num_sms();
    const int64_t per = nnz / want;
    p.entries = static_cast<int>(per < 1 ? 1 : (per > kAsEntries ? kAsEntries : per));
    const int64_t gx = (nnz + p.entries - 1) / p.entries;
    const int most_y = (2 * num_kv_heads + kAsWarps - 1) / kAsWarps;
    const int64_t gy = (want + gx - 1) / gx;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy < most_y ? gy : most_y));
    auto pick = [&](auto kd, auto ka) { return head_dim == 128 ? kd : ka; };
    auto kern = dtype == PKV_BF16
                    ? (layout == PKV_HND ? pick(append_scaled_kernel<__nv_bfloat16, PKV_HND, 16>,
                                                append_scaled_kernel<__nv_bfloat16, PKV_HND, 0>)
                                         : pick(append_scaled_kernel<__nv_bfloat16, PKV_NHD, 16>,
                                                append_scaled_kernel<__nv_bfloat16, PKV_NHD, 0>))
                    : (layout == PKV_HND
                           ? pick(append_scaled_kernel<__half, PKV_HND, 16>, append_scaled_kernel<__half, PKV_HND, 0>)
                           : pick(append_scaled_kernel<__half, PKV_NHD, 16>, append_scaled_kernel<__half, PKV_NHD, 0>));
    kern<<<grid, kAsWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(p);
    note_launches(1);
    return launch_status();
}
