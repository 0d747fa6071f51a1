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
// are few): its first warp resolves them, lane j entry j, so that the chain of
// index reads runs once, and lists the runs that start there; then the warps
// share out the heads of K and V and take run after run.  A run of up to 16
// rows of 128 elements is staged through shared memory by the lanes that use
// it (cp.async, the next run in flight while one is quantised; a lane reads
// only what it copied, so no barrier is needed), so every new value is read
// once.  Longer runs and other widths are read twice, the second time from L2.
//
// HBM bounds it: two bytes read and one written an element.  Times of the call
// replayed from a graph (launched from the host a call takes 11 us at least):
// 1024 requests, 66k tokens of 32 heads: 286 us, 5.7 TB/s, 84% of the measured
// copy rate (one warp an entry and head, two reads: 1064 us; run list once per
// CTA and runs in registers: 380; staged one run ahead: 299; two ahead: 287).
// One token for each of 64 requests: 3.5 us, a launch and three dependent reads.
// Measured with blocks of 8 and 16 and 128 elements a row only.
#include <type_traits>

#include "pkv_common.cuh"

namespace pkv {

struct AppendScaledParams {
    const uint16_t *src[2];  // key, value: [nnz, H, D]
    uint8_t *cache[2];
    float *scales[2];
    int64_t nnz, page_stride, max_num_pages, scale_stride;
    int64_t kv_extent, scale_extent;  // elements a cache / scale pointer spans
    const int32_t *batch_indices, *positions, *kv_indices, *kv_indptr, *kv_last_page_len;
    int B, H, D, page_shift, block_shift;
    int entries;  // entries a CTA takes, at most kAsEntries
    int32_t *err;
};

// CTAs of 8 warps, 16 entries each.  Blocks of more than 8 tokens: two CTAs
// per SM (what three stages of 4 KB a warp leave room for; with fewer
// registers three measured slower, 328 against 299 us).  Blocks of 8: half the
// stage, four CTAs per SM (16 prompts: 23.5 us, 24.7 with three, 26.7 with two).
// 8 or 32 entries a CTA: 306 / 293 against 286 us.
constexpr int kAsWarps = 8;
constexpr int kAsEntries = 16;
constexpr int kAsCtas4 = 4;
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

// Eight 16-bit values over s -> eight codes.  kQuotient: divided out.
// kProduct (s a power of two, as a scale is unless the caller brought another
// kind): products with 1 / s in fp32, exact.  kHalf (fp16 values, s in
// [2^-15, 2^24]): the same products in fp16, two to an instruction and without
// widening; they are exact down to 2^-14, and a smaller quotient becomes code
// 0 either way (E4M3's smallest value is 2^-9); one beyond fp16's range
// becomes infinite and saturates as it does in fp32.
enum { kQuotient, kProduct, kHalf };
template <typename T, int HOW>
__device__ __forceinline__ uint2 quantise8(const uint4 &v, float s) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const float inv = HOW == kQuotient ? 0.f : __uint_as_float((254u << 23) - __float_as_uint(s));
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (HOW == kHalf) {
            const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&w[k]), __float2half2_rn(inv));
            uint16_t r;
            asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
            o[k] = r;
        } else {
            float2 f = widen2<T>(w[k]);
            f = HOW == kProduct ? __fmul2_rn(f, make_float2(inv, inv)) : make_float2(f.x / s, f.y / s);
            o[k] = to_e4m3x2(f.x, f.y);
        }
    }
    return make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
}

// One run of entries: rows ri .. ri + n - 1 of the new tokens go to the slots
// slot .. slot + n - 1 of a page, inside one block.
struct AppendRun {
    int64_t entry, page;
    int n, slot;
};

// Lane j of the CTA's first warp resolves entry i0 + j; the runs that start in
// the first p.entries of them are listed in `runs`, their number returned.
__device__ __forceinline__ int list_runs(const AppendScaledParams &p, int64_t i0, bool report, AppendRun *runs) {
    const int lane = threadIdx.x & 31;
    const int S = 1 << p.page_shift, G = 1 << p.block_shift;
    const int64_t i = i0 + lane;
    report = report && lane < p.entries;
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
    // bit j: entry j + 1 goes on where entry j is
    const int b_after = __shfl_down_sync(0xffffffffu, b, 1), pos_after = __shfl_down_sync(0xffffffffu, pos, 1);
    const unsigned joined = __ballot_sync(0xffffffffu, lane < 31 && b_after == b && pos_after == pos + 1);
    int n = min(most, __ffs(~(joined >> lane)));
    unsigned open = __ballot_sync(0xffffffffu, leads && n < most && lane + n == 32);  // goes on past the lanes
    for (; open; open &= open - 1) {
        const int j = __ffs(open) - 1;
        const int rb = __shfl_sync(0xffffffffu, b, j), rpos = __shfl_sync(0xffffffffu, pos, j);
        const int rmost = __shfl_sync(0xffffffffu, most, j);
        int m = __shfl_sync(0xffffffffu, n, j);
        while (m < rmost) {
            const int k = m + lane;
            const bool same = k < rmost && p.batch_indices[i0 + j + k] == rb && p.positions[i0 + j + k] == rpos + k;
            const unsigned all = __ballot_sync(0xffffffffu, same);
            if (all != 0xffffffffu) {
                m += __ffs(~all) - 1;
                break;
            }
            m += 32;
        }
        if (lane == j) n = m;
    }
    const unsigned leaders = __ballot_sync(0xffffffffu, leads);
    if (leads) {
        AppendRun &r = runs[__popc(leaders & ((1u << lane) - 1))];
        r.entry = i;
        r.page = page;
        r.n = n;
        r.slot = pos & (S - 1);
    }
    return __popc(leaders);
}

constexpr int kAsStages = 3;

// D128: rows of 128 elements (16 chunks of 16 bytes), short runs staged;
// else any width, p.D / 8 chunks.
template <typename T, int LAYOUT, int HELD>
__global__ void __launch_bounds__(kAsWarps * 32, HELD == 4 ? kAsCtas4 : 2) append_scaled_kernel(const AppendScaledParams p) {
    constexpr bool D128 = HELD > 0;
    constexpr int kAsHeld = D128 ? HELD : 1, kAsStage = kAsHeld * 32 * 16;  // bytes of one warp's stage
    extern __shared__ __align__(16) uint8_t stage_mem[];
    __shared__ AppendRun runs[kAsEntries];
    __shared__ int n_runs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = 1 << p.page_shift, G = 1 << p.block_shift;
    if (warp == 0) {
        const int k = list_runs(p, static_cast<int64_t>(blockIdx.x) * p.entries, blockIdx.y == 0, runs);
        if (lane == 0) n_runs = k;
    }
    __syncthreads();
    const int C = D128 ? 16 : p.D / 8;
    const int64_t src_row = static_cast<int64_t>(p.H) * p.D;
    constexpr uint32_t kMag = 0x7fff7fffu;
    uint8_t *stages = stage_mem + warp * (kAsStages * kAsStage) + lane * 16;  // chunk k at 512 k

    // the warp's items: run by run, heads hk0, hk0 + step, .. of K then V
    const int hk0 = blockIdx.y * kAsWarps + warp, step = gridDim.y * kAsWarps;
    const int total_runs = hk0 < 2 * p.H ? n_runs : 0;
    auto chunk_row = [&](int k) { return (lane >> 4) + 2 * k; };  // (D128) row of the lane's chunk k
    auto source = [&](const AppendRun &r, int hk) {
        return p.src[hk >= p.H] + (r.entry * p.H + (hk >= p.H ? hk - p.H : hk)) * static_cast<int64_t>(p.D);
    };
    auto issue = [&](int run, int hk, int st) {
        if constexpr (D128) {
            if (run < total_runs && runs[run].n <= 2 * kAsHeld) {
                const int n = runs[run].n;
                const uint16_t *at = source(runs[run], hk) + (lane >> 4) * src_row + (lane & 15) * 8;
                const uint32_t to = smem_u32(stages + st * kAsStage);
#pragma unroll
                for (int k = 0; k < kAsHeld; ++k)
                    if (chunk_row(k) < n) cp_async_16(to + 512 * k, at + 2 * k * src_row, true);
            }
            cp_async_commit();
        }
    };
    auto next = [&](int &run, int &hk) {
        hk += step;
        if (hk >= 2 * p.H) {
            ++run;
            hk = hk0;
        }
    };
    int run3 = 0, hk3 = hk0;  // the item after the ones in flight
    issue(run3, hk3, 0);
    next(run3, hk3);
    issue(run3, hk3, 1);
    next(run3, hk3);
    int st = 0;
    for (int run = 0, hk = hk0; run < total_runs;) {
        AppendRun r = runs[run];
        int n = r.n;
        const int in_block = r.slot & (G - 1);
        const int z = hk >= p.H ? 1 : 0, h = hk - z * p.H;
        float *scale = p.scales[z] + r.page * p.scale_stride + (static_cast<int64_t>(h) << (p.page_shift - p.block_shift)) +
                       (r.slot >> p.block_shift);
        const bool scale_in = dbg_in(scale - p.scales[z], 1, p.scale_extent, p.err);
        float was = in_block > 0 && scale_in ? *scale : 0.f;
        issue(run3, hk3, st == 0 ? 2 : st - 1);
        next(run3, hk3);
        const uint16_t *src = source(r, hk);
        const bool held = D128 && n <= 2 * kAsHeld;
        uint4 v[kAsHeld];
        uint32_t mag = 0;
        if (held) {
            cp_async_wait<2>();
#pragma unroll
            for (int k = 0; k < kAsHeld; ++k) {
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (chunk_row(k) < n) v[k] = *reinterpret_cast<const uint4 *>(stages + st * kAsStage + 512 * k);
                mag = __vmaxu2(mag, __vmaxu2(__vmaxu2(v[k].x & kMag, v[k].y & kMag), __vmaxu2(v[k].z & kMag, v[k].w & kMag)));
            }
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
        // 2^e by its bits: e is in [-40, 40]
        float s = __uint_as_float(static_cast<uint32_t>(scale_exponent(widen2<T>(mag).x) + 127) << 23);
        if (in_block > 0) {
            was = checked_scale(was, p.err);
            s = fmaxf(s, was);
        } else {
            was = s;
        }
        __syncwarp();
        if (lane == 0 && scale_in) *scale = s;
        if constexpr (kDebugBounds) {  // the block's rows and its scale lie in the pool (else nothing is touched)
            const int64_t row = kv_row_offset<LAYOUT>(r.page, p.page_stride, h, r.slot - in_block, p.H, S, p.D);
            const int64_t step_d = LAYOUT == PKV_HND ? p.D : src_row;
            if (!dbg_in(row, (in_block + n - 1) * step_d + p.D, p.kv_extent, p.err)) n = 0;
        }
        uint8_t *dst = p.cache[z] + kv_row_offset<LAYOUT>(r.page, p.page_stride, h, r.slot, p.H, S, p.D);
        const int64_t dst_row = LAYOUT == PKV_HND ? p.D : src_row;
        if (s > was) {  // earlier tokens of the block, rounded again under the larger scale
            const float ratio = was / s;
            for (int q = lane; q < in_block * C; q += 32) {
                uint8_t *at = dst + (q / C - in_block) * dst_row + (q % C) * 8;
                const uint2 x = *reinterpret_cast<const uint2 *>(at);
                const uint32_t w[2] = {x.x, x.y};
                uint32_t o[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 lo = widen2<__half>(widen_e4m3x2<__half>(w[k] & 0xffffu));
                    const float2 hi = widen2<__half>(widen_e4m3x2<__half>(w[k] >> 16));
                    o[k] = to_e4m3x2(lo.x * ratio, lo.y * ratio) | to_e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
                }
                *reinterpret_cast<uint2 *>(at) = make_uint2(o[0], o[1]);
            }
        }
        const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
        constexpr bool kFp16 = std::is_same<T, __half>::value;
        if (held && pow2 && (!kFp16 || (s >= 0x1p-15f && s <= 0x1p24f))) {
            uint8_t *at = dst + (lane >> 4) * dst_row + (lane & 15) * 8;
#pragma unroll
            for (int k = 0; k < kAsHeld; ++k)
                if (chunk_row(k) < n)
                    *reinterpret_cast<uint2 *>(at + 2 * k * dst_row) = quantise8<T, kFp16 ? kHalf : kProduct>(v[k], s);
        } else {
            for (int q = lane; q < n * C; q += 32) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src + (q / C) * src_row + (q % C) * 8);
                *reinterpret_cast<uint2 *>(dst + (q / C) * dst_row + (q % C) * 8) =
                    pow2 ? quantise8<T, kProduct>(x, s) : quantise8<T, kQuotient>(x, s);
            }
        }
        next(run, hk);
        st = st == 2 ? 0 : st + 1;
    }
    if constexpr (D128) cp_async_wait<0>();
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
    p.kv_extent = max_num_pages > 0
                      ? (max_num_pages - 1) * page_stride + static_cast<int64_t>(num_kv_heads) * page_size * head_dim
                      : 0;
    p.scale_extent = max_num_pages > 0
                         ? (max_num_pages - 1) * scale_page_stride + (static_cast<int64_t>(num_kv_heads) << (ps - bs))
                         : 0;
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
    // rows of 128 elements: staged runs of up to 8 rows (blocks of 8) or 16
    const int held = head_dim != 128 ? 0 : (scale_block == 8 ? 4 : 8);
    auto pick = [&](auto k8, auto k4, auto any) { return held == 8 ? k8 : (held == 4 ? k4 : any); };
    auto by_layout = [&](auto hnd, auto nhd) { return layout == PKV_HND ? hnd : nhd; };
    using B = __nv_bfloat16;
    using F = __half;
    auto kern = dtype == PKV_BF16
                    ? by_layout(pick(append_scaled_kernel<B, PKV_HND, 8>, append_scaled_kernel<B, PKV_HND, 4>,
                                     append_scaled_kernel<B, PKV_HND, 0>),
                                pick(append_scaled_kernel<B, PKV_NHD, 8>, append_scaled_kernel<B, PKV_NHD, 4>,
                                     append_scaled_kernel<B, PKV_NHD, 0>))
                    : by_layout(pick(append_scaled_kernel<F, PKV_HND, 8>, append_scaled_kernel<F, PKV_HND, 4>,
                                     append_scaled_kernel<F, PKV_HND, 0>),
                                pick(append_scaled_kernel<F, PKV_NHD, 8>, append_scaled_kernel<F, PKV_NHD, 4>,
                                     append_scaled_kernel<F, PKV_NHD, 0>));
    const size_t smem = static_cast<size_t>(kAsWarps) * kAsStages * held * 32 * 16;
    if (smem > 48 * 1024 - 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return PKV_ERR_CUDA;
    kern<<<grid, kAsWarps * 32, smem, static_cast<cudaStream_t>(stream)>>>(p);
    note_launches(1);
    return launch_status();
}
