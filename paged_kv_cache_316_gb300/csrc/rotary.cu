// rotary.cu -- what lies between the projections and the cache: an RMS norm of
// every head of queries and keys, the rotation of their pairs by the token's
// position, and the append of keys and values to their pages, in one pass
// (paged_append_rotary); the same onto rows (paged_rotary).
//
// A head row x of D elements: y = x / sqrt(mean(x^2) + eps) * w (where there
// are weights), then each rotated pair (u, v) with frequency f becomes
// m (u cos a - v sin a, v cos a + u sin a), a = position * f.  All of it in
// fp32, rounded once to the row's type.
//
// The angle is counted in turns as a 64-bit fraction: f / 2 pi becomes
// F = round(2^64 frac(f / 2 pi)), and position * F mod 2^64 is the angle less
// its whole turns without a rounding, so that an angle is as good at position
// 10^9 as at 1 (with the double's 2^-53 of a turn a step: 2^-22 of a turn
// there, where an fp32 product of position and frequency has lost all).  The
// upper 32 bits feed sincospif.
//
// A warp takes a token and a range of its heads; a lane holds 16 bytes of a
// row, so D <= 64, 128 and 256 elements take 8, 16 and 32 lanes and a warp 4,
// 2 and 1 rows at a time.  The token's cosines and sines are computed once by
// the lanes that share them out, brought to the lanes that need them through
// shared memory, and kept in registers over the token's heads.
#include "pkv_common.cuh"

namespace pkv {

struct RotaryParams {
    const uint16_t *src[3];  // query, key, value rows
    int64_t src_stride[3];   // elements from token to token
    uint16_t *dst[3];        // query rows; key / value rows or caches
    int64_t nnz;
    int Hq, Hkv, heads;      // heads: Hq + Hkv, + Hkv with values
    int D;
    // rotation
    const int32_t *rot_pos;
    const double *freq;
    int start, half;         // first rotated dimension, rotated pairs
    float magnitude;
    // norms
    const void *weight[2];   // query, key weights in the rows' type, or NULL
    float eps, inv_d;
    // pages (batch_indices NULL: keys go to rows)
    const int32_t *batch_indices, *positions, *kv_indices, *kv_indptr, *kv_last_page_len;
    int64_t page_stride, max_num_pages, kv_extent;
    int B, page_shift, layout;
    int per_warp;            // heads a warp takes of its token
    int parts;               // warps a token is divided among
    int32_t *err;
};

constexpr int kRotWarps = 8;
constexpr int kRotMaxHalf = 128;

template <typename T>
__device__ __forceinline__ float2 rot_unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 rot_unpack<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <>
__device__ __forceinline__ float2 rot_unpack<__nv_bfloat16>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}
template <typename T>
__device__ __forceinline__ void rot_unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = rot_unpack<T>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The angle of one step in 2^-64 turns.
__device__ __forceinline__ uint64_t turns_per_step(double f) {
    double t = f * 0.15915494309189535;  // 1 / (2 pi)
    t -= floor(t);
    return __double2ull_rn(t * 18446744073709551616.0);
}
// (cos, sin) of position * step, times m.
__device__ __forceinline__ float2 turned(int pos, uint64_t step, float m) {
    const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
    const float half_turns = static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * m, s * m);
}

// Element offset of head 0 of a token's row in the caches, -1 (and its error
// bit) if it has no place there.
__device__ __forceinline__ int64_t rotary_slot(const RotaryParams &p, int64_t tok, bool report) {
    const int b = p.batch_indices[tok], pos = p.positions[tok];
    if (b < 0 || b >= p.B) {
        if (report) set_err(p.err, PKV_DEV_ERR_BATCH);
        return -1;
    }
    const int S = 1 << p.page_shift;
    const int first = p.kv_indptr[b], pages = p.kv_indptr[b + 1] - first;
    const int64_t len = pages > 0 ? static_cast<int64_t>(pages - 1) * S + p.kv_last_page_len[b] : 0;
    if (pos < 0 || pos >= len || (pos >> p.page_shift) >= pages) {
        if (report) set_err(p.err, PKV_DEV_ERR_POS);
        return -1;
    }
    const int64_t page = p.kv_indices[first + (pos >> p.page_shift)];
    if (page < 0 || page >= p.max_num_pages) {
        if (report) set_err(p.err, PKV_DEV_ERR_PAGE);
        return -1;
    }
    return page * p.page_stride + static_cast<int64_t>(pos & (S - 1)) * (p.layout == PKV_HND ? p.D : p.Hkv * p.D);
}

// LPR lanes to a row; PAIRED: neighbouring elements are a pair (else element
// i of the rotated part goes with element i + half).
template <typename T, int LPR, bool PAIRED>
__global__ void __launch_bounds__(kRotWarps * 32) rotary_kernel(const RotaryParams p) {
    constexpr int RPW = 32 / LPR;               // rows a warp takes at a time
    constexpr int NF = kRotMaxHalf / 32 / (LPR == 32 ? 1 : (LPR == 16 ? 2 : 4));  // frequencies of a lane
    constexpr int NC = PAIRED ? 4 : 8;          // (cos, sin) of a lane's eight elements
    constexpr int U = 4;                        // loads in flight
    __shared__ float2 table[kRotWarps][kRotMaxHalf];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & (LPR - 1), sub = lane / LPR;  // 16-byte chunk of the row, row of the warp's
    const bool on = c * 8 < p.D;
    const int i0 = c * 8 - p.start;             // first element's place in the rotated part
    const bool rot = on && i0 >= 0 && i0 < 2 * p.half;
    const int t0 = PAIRED ? i0 >> 1 : (i0 < p.half ? i0 : i0 - p.half);  // its first table entry
    const float sign = !PAIRED && i0 < p.half ? -1.f : 1.f;
    const int mate = PAIRED || !rot ? lane : (i0 < p.half ? lane + p.half / 8 : lane - p.half / 8);
    uint64_t step[NF];
#pragma unroll
    for (int k = 0; k < NF; ++k) step[k] = lane + 32 * k < p.half ? turns_per_step(p.freq[lane + 32 * k]) : 0;
    const bool norm[2] = {p.weight[0] != nullptr, p.weight[1] != nullptr};
    float w[2][8];
#pragma unroll
    for (int z = 0; z < 2; ++z)
        if (norm[z] && on)
            rot_unpack8<T>(reinterpret_cast<const uint4 *>(p.weight[z])[c], w[z]);
        else
            for (int e = 0; e < 8; ++e) w[z][e] = 0.f;

    const int64_t tasks = p.nnz * p.parts;
    for (int64_t task = static_cast<int64_t>(blockIdx.x) * kRotWarps + warp; task < tasks;
         task += static_cast<int64_t>(gridDim.x) * kRotWarps) {
        const int64_t tok = task / p.parts;
        const int h0 = static_cast<int>(task - tok * p.parts) * p.per_warp, h1 = min(h0 + p.per_warp, p.heads);
        // which tensor a head row belongs to, and its head there
        auto tensor = [&](int h) { return h < p.Hq ? 0 : (h < p.Hq + p.Hkv ? 1 : 2); };
        auto head_in = [&](int h, int z) { return z == 0 ? h : (z == 1 ? h - p.Hq : h - p.Hq - p.Hkv); };
        uint4 raw[U];
        auto load = [&](int h) {  // rows h, h + RPW, ..
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int hh = h + k * RPW + sub;
                raw[k] = make_uint4(0u, 0u, 0u, 0u);
                if (hh < h1 && on) {
                    const int z = tensor(hh);
                    raw[k] = *reinterpret_cast<const uint4 *>(p.src[z] + tok * p.src_stride[z] +
                                                              static_cast<int64_t>(head_in(hh, z)) * p.D + c * 8);
                }
            }
        };
        load(h0);
        const int pos = p.rot_pos[tok];
#pragma unroll
        for (int k = 0; k < NF; ++k)
            if (lane + 32 * k < p.half) table[warp][lane + 32 * k] = turned(pos, step[k], p.magnitude);
        __syncwarp();
        float2 cs[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) cs[k] = rot ? table[warp][t0 + k] : make_float2(1.f, 0.f);
        __syncwarp();  // (the table is rewritten for the next token)
        int64_t slot = -1;
        if (p.batch_indices && h1 > p.Hq) slot = rotary_slot(p, tok, lane == 0 && h1 == p.heads);
        for (int h = h0; h < h1; h += U * RPW) {
            if (h != h0) load(h);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int hh = h + k * RPW + sub;
                if (h + k * RPW >= h1) break;  // (uniform: no row left for any lane)
                const bool live = hh < h1 && on;
                const int z = tensor(min(hh, h1 - 1));
                uint4 out = raw[k];
                if (__any_sync(0xffffffffu, z < 2)) {
                    float x[8];
                    rot_unpack8<T>(raw[k], x);
                    if (norm[0] || norm[1]) {
                        float ss = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                        const float inv = rsqrtf(fmaf(ss, p.inv_d, p.eps));
                        if (z < 2 && norm[z]) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] *= inv * (z ? w[1][e] : w[0][e]);
                        }
                    }
                    if constexpr (PAIRED) {
                        if (rot) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float u = x[2 * e], v = x[2 * e + 1];
                                x[2 * e] = u * cs[e].x - v * cs[e].y;
                                x[2 * e + 1] = v * cs[e].x + u * cs[e].y;
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float other = __shfl_sync(0xffffffffu, x[e], mate);
                            if (rot) x[e] = fmaf(x[e], cs[e].x, sign * other * cs[e].y);
                        }
                    }
                    if (z < 2) out = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
                }
                if (!live) continue;
                const int64_t hd = static_cast<int64_t>(head_in(hh, z));
                if (z == 0 || !p.batch_indices) {
                    const int64_t e = (tok * (z == 0 ? p.Hq : p.Hkv) + hd) * p.D + c * 8;
                    *reinterpret_cast<uint4 *>(p.dst[z] + e) = out;
                } else if (slot >= 0) {
                    const int64_t e = slot + hd * (p.layout == PKV_HND ? p.D << p.page_shift : p.D) + c * 8;
                    if (dbg_in(e, 8, p.kv_extent, p.err)) *reinterpret_cast<uint4 *>(p.dst[z] + e) = out;
                }
            }
        }
    }
}

static int check_rotary(const RotaryParams &p, int rotary_dim, int rotary_start, int dtype) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (p.nnz < 0 || p.Hq <= 0 || p.Hkv <= 0 || p.D <= 0 || rotary_dim < 0 || rotary_start < 0 ||
        rotary_start + static_cast<int64_t>(rotary_dim) > p.D || !(p.eps >= 0.f))
        return PKV_ERR_INVALID_ARG;
    if (p.D % 16 || rotary_dim % 16 || rotary_start % 8) return PKV_ERR_INVALID_ARG;
    if (p.D > 256 || p.Hq > 65536 || p.Hkv > 65536) return PKV_ERR_UNSUPPORTED;
    if (p.nnz > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    for (int z = 0; z < 3; ++z)
        if (p.src[z] && (!aligned16(p.src[z]) || p.src_stride[z] % 8 ||
                         p.src_stride[z] < static_cast<int64_t>(z == 0 ? p.Hq : p.Hkv) * p.D))
            return PKV_ERR_INVALID_ARG;
    if ((p.weight[0] && !aligned16(p.weight[0])) || (p.weight[1] && !aligned16(p.weight[1])) ||
        (reinterpret_cast<uintptr_t>(p.freq) & 7) || !aligned16(p.dst[0]) || !aligned16(p.dst[1]) || !aligned16(p.dst[2]))
        return PKV_ERR_INVALID_ARG;
    return PKV_OK;
}

template <typename T>
static int run_rotary(RotaryParams &p, bool paired, cudaStream_t st) {
    const int rows = p.D <= 64 ? 4 : (p.D <= 128 ? 2 : 1);
    // A warp takes all heads of a token where there are tokens enough for every
    // warp that fits the machine; with fewer the heads are divided, down to one
    // load of four rows a lane.
    const int64_t want = static_cast<int64_t>(num_sms()) * 4 * kRotWarps;
    const int least = 4 * rows;
    const int most_parts = (p.heads + least - 1) / least;
    int64_t parts = (want + p.nnz - 1) / p.nnz;
    if (parts > most_parts) parts = most_parts;
    p.per_warp = static_cast<int>((p.heads + parts - 1) / parts);
    p.per_warp = (p.per_warp + least - 1) / least * least;
    p.parts = (p.heads + p.per_warp - 1) / p.per_warp;
    const int64_t blocks = (p.nnz * p.parts + kRotWarps - 1) / kRotWarps;
    const int64_t most = static_cast<int64_t>(num_sms()) * 4;
    const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
    auto pick = [&](auto a, auto b) { return paired ? a : b; };
    auto kern = rows == 4 ? pick(rotary_kernel<T, 8, true>, rotary_kernel<T, 8, false>)
                          : (rows == 2 ? pick(rotary_kernel<T, 16, true>, rotary_kernel<T, 16, false>)
                                       : pick(rotary_kernel<T, 32, true>, rotary_kernel<T, 32, false>));
    kern<<<grid, kRotWarps * 32, 0, st>>>(p);
    note_launches(1);
    return launch_status();
}

}  // namespace pkv

using namespace pkv;

extern "C" int paged_rotary(const void *query, const void *key, int64_t query_stride, int64_t key_stride, int64_t nnz,
                            const int32_t *positions, const double *frequencies, int32_t rotary_dim,
                            int32_t rotary_start, int32_t interleaved, float magnitude, const void *query_weight,
                            const void *key_weight, float eps, int32_t num_qo_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t dtype, void *query_out, void *key_out, void *stream) {
    const CallRange nvtx_range("paged_rotary");
    RotaryParams p = {};
    p.src[0] = static_cast<const uint16_t *>(query);
    p.src[1] = static_cast<const uint16_t *>(key);
    p.src_stride[0] = query_stride;
    p.src_stride[1] = key_stride;
    p.dst[0] = static_cast<uint16_t *>(query_out);
    p.dst[1] = static_cast<uint16_t *>(key_out);
    p.nnz = nnz;
    p.Hq = num_qo_heads;
    p.Hkv = num_kv_heads;
    p.heads = num_qo_heads + num_kv_heads;
    p.D = head_dim;
    p.rot_pos = positions;
    p.freq = frequencies;
    p.start = rotary_start;
    p.half = rotary_dim / 2;
    p.magnitude = magnitude;
    p.weight[0] = query_weight;
    p.weight[1] = key_weight;
    p.eps = eps;
    p.inv_d = 1.f / static_cast<float>(head_dim > 0 ? head_dim : 1);
    const int rc = check_rotary(p, rotary_dim, rotary_start, dtype);
    if (rc != PKV_OK) return rc;
    if (nnz == 0) return PKV_OK;
    if (!query || !key || !positions || (rotary_dim > 0 && !frequencies) || !query_out || !key_out) return PKV_ERR_NULL;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_BF16 ? run_rotary<__nv_bfloat16>(p, interleaved != 0, st)
                             : run_rotary<__half>(p, interleaved != 0, st);
}

extern "C" int paged_append_rotary(const void *query, const void *key, const void *value, int64_t query_stride,
                                   int64_t key_stride, int64_t value_stride, int64_t nnz, const int32_t *batch_indices,
                                   const int32_t *positions, const int32_t *rotary_positions, void *k_cache,
                                   void *v_cache, int64_t page_stride, int64_t max_num_pages, const int32_t *kv_indices,
                                   const int32_t *kv_indptr, const int32_t *kv_last_page_len, int32_t batch_size,
                                   const double *frequencies, int32_t rotary_dim, int32_t rotary_start,
                                   int32_t interleaved, float magnitude, const void *query_weight,
                                   const void *key_weight, float eps, int32_t num_qo_heads, int32_t num_kv_heads,
                                   int32_t head_dim, int32_t page_size, int32_t layout, int32_t dtype, void *query_out,
                                   int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_append_rotary");
    if (layout != PKV_NHD && layout != PKV_HND) return PKV_ERR_INVALID_ARG;
    RotaryParams p = {};
    p.src[0] = static_cast<const uint16_t *>(query);
    p.src[1] = static_cast<const uint16_t *>(key);
    p.src[2] = static_cast<const uint16_t *>(value);
    p.src_stride[0] = query_stride;
    p.src_stride[1] = key_stride;
    p.src_stride[2] = value_stride;
    p.dst[0] = static_cast<uint16_t *>(query_out);
    p.dst[1] = static_cast<uint16_t *>(k_cache);
    p.dst[2] = static_cast<uint16_t *>(v_cache);
    p.nnz = nnz;
    p.Hq = num_qo_heads;
    p.Hkv = num_kv_heads;
    p.heads = num_qo_heads + 2 * num_kv_heads;
    p.D = head_dim;
    p.rot_pos = rotary_positions ? rotary_positions : positions;
    p.freq = frequencies;
    p.start = rotary_start;
    p.half = rotary_dim / 2;
    p.magnitude = magnitude;
    p.weight[0] = query_weight;
    p.weight[1] = key_weight;
    p.eps = eps;
    p.inv_d = 1.f / static_cast<float>(head_dim > 0 ? head_dim : 1);
    int rc = check_rotary(p, rotary_dim, rotary_start, dtype);
    if (rc != PKV_OK) return rc;
    if (batch_size < 0 || max_num_pages < 0 || page_stride <= 0) return PKV_ERR_INVALID_ARG;
    p.page_shift = ilog2_exact(page_size);
    if (p.page_shift < 0 || p.page_shift > 16) return PKV_ERR_UNSUPPORTED;
    const int64_t page = static_cast<int64_t>(num_kv_heads) * page_size * head_dim;
    if (page_stride < page || page_stride % 8) return PKV_ERR_INVALID_ARG;
    if (nnz == 0) return PKV_OK;
    if (!query || !key || !value || !batch_indices || !positions || !k_cache || !v_cache || !kv_indices || !kv_indptr ||
        !kv_last_page_len || (rotary_dim > 0 && !frequencies) || !query_out)
        return PKV_ERR_NULL;
    p.batch_indices = batch_indices;
    p.positions = positions;
    p.kv_indices = kv_indices;
    p.kv_indptr = kv_indptr;
    p.kv_last_page_len = kv_last_page_len;
    p.page_stride = page_stride;
    p.max_num_pages = max_num_pages;
    p.kv_extent = max_num_pages > 0 ? (max_num_pages - 1) * page_stride + page : 0;
    p.B = batch_size;
    p.layout = layout;
    p.err = err_word;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_BF16 ? run_rotary<__nv_bfloat16>(p, interleaved != 0, st)
                             : run_rotary<__half>(p, interleaved != 0, st);
}
