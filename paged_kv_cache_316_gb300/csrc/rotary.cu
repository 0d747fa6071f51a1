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
// there, where an fp32 product of position and frequency has lost all).  All 64
// bits, rounded once to fp32, feed sincospif: the sine of a small angle is as
// good in itself as that of a large one.
//
// Instruction issue bounds it before HBM does, so the work of an element is
// brought down.  A lane holds both elements of its pairs, a and b (two pieces
// of four elements half the rotated part apart, or eight neighbours), so that
//   a' = (1 / rms) (ca a - sb b),   b' = (1 / rms) (cb b + sa a),
// with the weights, cosines, sines and the magnitude folded into the four
// factors once a token: two products and a fused product an element, two
// elements to an instruction, and no exchange between lanes.  The sums of
// squares of four row groups are reduced together, a quarter of them to a
// lane.  The token's cosines and sines are computed once by the lanes that
// share them out and exchanged through shared memory.
//
// A warp takes a token and a range of its row groups, queries, keys, then
// values; D <= 64, 128 and 256 elements take 8, 16 and 32 lanes, so a group is
// 4, 2 and 1 rows, and a batch four groups.  Batches come through a ring in
// shared memory (cp.async), on into the warp's next token.
//
// Times of the call replayed from a graph (a floor of bytes at 6788 GB/s):
// 65,962 tokens of 1024 requests, 32 + 8 heads, norms: 255 us (floor 239);
// 17,664 tokens, fp16, half of each head, neighbours: 70 (64); 8,039 rows of 32
// + 32 heads of 192: 66.7 (58); 4096 tokens of a fused projection: 22 (14.8;
// its 8,192 tasks on 2,432 warps are 3.4 rounds that take the time of 4, 2.8
// us, and launch, first reads and tail are 4); 64 tokens: 4.6, seven: 3.7.
// On the way: a row's partner by shuffles and loads of four rows, 490 us for
// the first; rows through the ring one at a time, factors folded, 312; pairs in
// one lane and sums of squares reduced four at a time, loads into registers,
// 273.  More in flight is slower: 5 or 6 CTAs on an SM 254 and 307, three
// stages 255 (with 5 CTAs 261), and the second case 77 us; fewer too (3 CTAs
// 279): reads and writes of many rows at once leave DRAM's open pages.
#include "pkv_common.cuh"

namespace pkv {

struct RotaryParams {
    const uint16_t *src[3];  // query, key, value rows
    int64_t src_stride[3];   // elements from token to token
    uint16_t *dst[3];        // query rows; key / value rows or caches
    int64_t nnz;
    int Hq, Hkv;
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
    int batches[3];          // batches of kRotU row groups of each tensor
    int per_part;            // a token's batches are divided among `parts` warps
    uint32_t parts, tasks;   // tasks: tokens times parts
    int32_t *err;
};

constexpr int kRotWarps = 4, kRotCtas = 4;
constexpr int kRotU = 4;  // row groups in flight
constexpr int kRotRounds = 3;
// Stages of the ring, batches in flight less one: a batch is 2 KB a warp, 1 to
// 2 KB with one row to a group.
template <int LPR>
struct RotCfg {
    static constexpr int STAGES = LPR == 32 ? 3 : 2;
};

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
// The angle of one step in 2^-64 turns.
__device__ __forceinline__ uint64_t turns_per_step(double f) {
    double t = f * 0.15915494309189535;  // 1 / (2 pi)
    t -= floor(t);
    return __double2ull_rn(t * 18446744073709551616.0);
}
// (cos, sin) of position * step, times m.
__device__ __forceinline__ float2 turned(int pos, uint64_t step, float m) {
    const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
    const float half_turns = static_cast<float>(static_cast<int64_t>(a)) * 0x1p-63f;
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

// The sums over LPR lanes of four values a lane, as 1 / sqrt(mean + eps).
template <int LPR>
__device__ __forceinline__ void inverse_rms4(const float (&s)[4], float inv_d, float eps, float (&inv)[4]) {
    const int lane = threadIdx.x & 31;
    const bool b0 = lane & 1, b1 = lane & 2;
    // lane 0 .. 3 of four take the values 0, 2, 1, 3
    const float u = (b0 ? s[2] : s[0]) + __shfl_xor_sync(0xffffffffu, b0 ? s[0] : s[2], 1);
    const float v = (b0 ? s[3] : s[1]) + __shfl_xor_sync(0xffffffffu, b0 ? s[1] : s[3], 1);
    float q = (b1 ? v : u) + __shfl_xor_sync(0xffffffffu, b1 ? u : v, 2);
#pragma unroll
    for (int o = 4; o < LPR; o <<= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    q = rsqrtf(fmaf(q, inv_d, eps));
#pragma unroll
    for (int k = 0; k < 4; ++k) inv[k] = __shfl_sync(0xffffffffu, q, (lane & ~3) + (k >> 1) + 2 * (k & 1));
}

// LPR lanes to a row; PAIRED: neighbouring elements are a pair (else element
// i of the rotated part goes with element i + half).
template <typename T, int LPR, bool PAIRED>
__global__ void __launch_bounds__(kRotWarps * 32, kRotCtas) rotary_kernel(const __grid_constant__ RotaryParams p) {
    constexpr int RPW = 32 / LPR, STAGES = RotCfg<LPR>::STAGES;  // rows of a group; of the ring
    constexpr int NF = LPR == 32 ? 4 : (LPR == 16 ? 2 : 1);  // frequencies of a lane
    __shared__ __align__(16) float2 table[kRotWarps][32 * NF];
    __shared__ uint64_t steps[32 * NF];
    extern __shared__ __align__(16) uint4 ring_mem[];
    auto ring = reinterpret_cast<uint4(*)[STAGES][kRotU][32]>(ring_mem);
    if (threadIdx.x < p.half) steps[threadIdx.x] = turns_per_step(p.freq[threadIdx.x]);
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = lane & (LPR - 1), sub = lane / LPR;  // the lane's place in its row, its row of the group
    const bool on = c * 8 < p.D;
    const uint32_t parts = p.parts, stride = gridDim.x * kRotWarps, task0 = blockIdx.x * kRotWarps + warp;
    const int all = p.batches[0] + p.batches[1] + p.batches[2];
    // the stream of batches, STAGES - 1 of them ahead: lane by lane 16 bytes
    // of the rows, zeros for rows past the last head
    uint32_t f_task = task0, f_tok = task0 / parts;
    int f_batch = static_cast<int>(task0 - f_tok * parts) * p.per_part, f_end = min(f_batch + p.per_part, all), f_stage = 0;
    auto fetch = [&]() {
        if (f_task < p.tasks) {
            const int z = f_batch < p.batches[0] ? 0 : (f_batch < p.batches[0] + p.batches[1] ? 1 : 2);
            const int b = f_batch - (z > 0 ? p.batches[0] : 0) - (z > 1 ? p.batches[1] : 0);
            const int h0 = b * (kRotU * RPW) + sub, H = z == 0 ? p.Hq : p.Hkv;
            const uint16_t *src = p.src[z] + f_tok * p.src_stride[z] + (h0 * p.D + c * 8);
            const uint32_t to = smem_u32(&ring[warp][f_stage][0][lane]);
#pragma unroll
            for (int k = 0; k < kRotU; ++k) {
                const bool ok = on && h0 + k * RPW < H;
                cp_async_16(to + k * 512, ok ? src + k * (RPW * p.D) : p.src[0], ok);
            }
            if (++f_batch == f_end) {
                f_task += stride;
                if (f_task < p.tasks) {
                    f_tok = f_task / parts;
                    f_batch = static_cast<int>(f_task - f_tok * parts) * p.per_part;
                    f_end = min(f_batch + p.per_part, all);
                }
            }
        }
        cp_async_commit();
        f_stage = f_stage == STAGES - 1 ? 0 : f_stage + 1;
    };
#pragma unroll 1
    for (int k = 0; k < STAGES - 1; ++k) fetch();
    int stage = 0;
    // where the lane's elements are: four pairs of the rotated part (from its
    // pair t0 on), or two pieces of four outside it (so that neighbouring lanes'
    // pieces fill whole sectors)
    int at_a = c * 8, at_b = c * 8 + 4, t0 = -1;
    if constexpr (PAIRED) {
        if (c * 8 >= p.start && c * 8 < p.start + 2 * p.half) t0 = (c * 8 - p.start) >> 1;
    } else if (4 * c < p.half) {
        t0 = 4 * c;
        at_a = p.start + t0;
        at_b = at_a + p.half;
    } else {
        at_a = 4 * c - p.half;  // in the first half of what is left, and in its second
        at_b = at_a + (p.D >> 1) - p.half;
        if (at_a >= p.start) at_a += 2 * p.half;
        if (at_b >= p.start) at_b += 2 * p.half;
    }
    // the lane's pairs as (a0, a1), (a2, a3) and (b0, b1), (b2, b3)
    auto split = [](const uint2 &u, const uint2 &v, float2 (&a)[2], float2 (&b)[2]) {
        if constexpr (PAIRED) {
            const float2 w0 = rot_unpack<T>(u.x), w1 = rot_unpack<T>(u.y), w2 = rot_unpack<T>(v.x), w3 = rot_unpack<T>(v.y);
            a[0] = make_float2(w0.x, w1.x);
            b[0] = make_float2(w0.y, w1.y);
            a[1] = make_float2(w2.x, w3.x);
            b[1] = make_float2(w2.y, w3.y);
        } else {
            a[0] = rot_unpack<T>(u.x);
            a[1] = rot_unpack<T>(u.y);
            b[0] = rot_unpack<T>(v.x);
            b[1] = rot_unpack<T>(v.y);
        }
    };

    for (uint32_t task = task0; task < p.tasks; task += stride) {
        const uint32_t tok = task / parts;
        int batch = static_cast<int>(task - tok * parts) * p.per_part;
        const int end = min(batch + p.per_part, all);
        const int pos = p.rot_pos[tok];
        int64_t place = -1;
        if (p.batch_indices && end > p.batches[0]) place = rotary_slot(p, tok, lane == 0 && end == all);
        bool fresh = true;  // the token's table is yet to be written
        int first = 0;
#pragma unroll 1
        for (int z = 0; z < 3; ++z) {
            const int last = first + p.batches[z], stop = min(end, last);
            const int H = z == 0 ? p.Hq : p.Hkv;
            const bool paged = z > 0 && p.batch_indices;
            uint16_t *dst = p.dst[z] + (paged ? place : static_cast<int64_t>(tok) * H * p.D);
            const uint32_t hop = paged && p.layout == PKV_HND ? static_cast<uint32_t>(p.D) << p.page_shift : p.D;
            const bool writes = on && (!paged || place >= 0);
            const bool norm = z < 2 && p.weight[z];
            float2 ca[2], sa[2], cb[2], sb[2];
            bool ready = z == 2;
            for (; batch < stop; ++batch) {
                const int h0 = (batch - first) * kRotU * RPW + sub;
                fetch();
                cp_async_wait<STAGES - 1>();
                const uint4 *rows = ring[warp][stage][0];
                stage = stage == STAGES - 1 ? 0 : stage + 1;
                if (z == 2) {  // values: as they are, every lane its own bytes
#pragma unroll
                    for (int k = 0; k < kRotU; ++k) {
                        const uint32_t o = (h0 + k * RPW) * hop + c * 8;
                        if (writes && h0 + k * RPW < H && (!paged || dbg_in(place + o, 8, p.kv_extent, p.err)))
                            *reinterpret_cast<uint4 *>(dst + o) = rows[k * 32 + lane];
                    }
                    continue;
                }
                __syncwarp();  // every lane's copies have landed
                uint2 u[kRotU], v[kRotU];
#pragma unroll
                for (int k = 0; k < kRotU; ++k) {
                    const uint16_t *row = reinterpret_cast<const uint16_t *>(rows + k * 32 + sub * LPR);
                    u[k] = v[k] = make_uint2(0u, 0u);
                    if (on) {
                        u[k] = *reinterpret_cast<const uint2 *>(row + at_a);
                        v[k] = *reinterpret_cast<const uint2 *>(row + at_b);
                    }
                }
                __syncwarp();  // (the stage is copied over by the next fetch)
                if (!ready) {  // the factors, while the rows arrive
                    if (fresh) {
                        __syncwarp();  // (the table of the token before has been read)
#pragma unroll
                        for (int k = 0; k < NF; ++k)
                            if (lane + 32 * k < p.half) table[warp][lane + 32 * k] = turned(pos, steps[lane + 32 * k], p.magnitude);
                        __syncwarp();
                        fresh = false;
                    }
                    float2 cs[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) cs[e] = t0 >= 0 ? table[warp][t0 + e] : make_float2(1.f, 0.f);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        ca[e] = cb[e] = make_float2(cs[2 * e].x, cs[2 * e + 1].x);
                        sa[e] = make_float2(cs[2 * e].y, cs[2 * e + 1].y);
                        sb[e] = make_float2(-cs[2 * e].y, -cs[2 * e + 1].y);
                    }
                    if (norm && on) {
                        const uint16_t *w = static_cast<const uint16_t *>(p.weight[z]);
                        float2 wa[2], wb[2];
                        split(*reinterpret_cast<const uint2 *>(w + at_a), *reinterpret_cast<const uint2 *>(w + at_b), wa, wb);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            ca[e] = __fmul2_rn(ca[e], wa[e]);
                            sa[e] = __fmul2_rn(sa[e], wa[e]);
                            cb[e] = __fmul2_rn(cb[e], wb[e]);
                            sb[e] = __fmul2_rn(sb[e], wb[e]);
                        }
                    }
                    ready = true;
                }
                float inv[kRotU];
                if (norm) {
                    float ss[kRotU];
#pragma unroll
                    for (int k = 0; k < kRotU; ++k) {
                        float2 a[2], b[2];
                        split(u[k], v[k], a, b);
                        const float2 q = __ffma2_rn(b[1], b[1], __ffma2_rn(b[0], b[0], __ffma2_rn(a[1], a[1], __fmul2_rn(a[0], a[0]))));
                        ss[k] = q.x + q.y;
                    }
                    inverse_rms4<LPR>(ss, p.inv_d, p.eps, inv);
                }
#pragma unroll
                for (int k = 0; k < kRotU; ++k) {
                    float2 a[2], b[2], x[2], y[2];
                    split(u[k], v[k], a, b);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[e] = __fmul2_rn(a[e], ca[e]);
                        y[e] = __fmul2_rn(b[e], cb[e]);
                        if (t0 >= 0) {  // (outside the rotated part no product with another element)
                            x[e] = __ffma2_rn(b[e], sb[e], x[e]);
                            y[e] = __ffma2_rn(a[e], sa[e], y[e]);
                        }
                        if (norm) {
                            x[e] = __fmul2_rn(x[e], make_float2(inv[k], inv[k]));
                            y[e] = __fmul2_rn(y[e], make_float2(inv[k], inv[k]));
                        }
                    }
                    const uint32_t o = (h0 + k * RPW) * hop;
                    if (!writes || h0 + k * RPW >= H || (paged && !dbg_in(place + o, p.D, p.kv_extent, p.err))) continue;
                    if constexpr (PAIRED) {
                        *reinterpret_cast<uint4 *>(dst + o + at_a) =
                            make_uint4(pack2<T>(x[0].x, y[0].x), pack2<T>(x[0].y, y[0].y), pack2<T>(x[1].x, y[1].x),
                                       pack2<T>(x[1].y, y[1].y));
                    } else {
                        *reinterpret_cast<uint2 *>(dst + o + at_a) = make_uint2(pack2<T>(x[0].x, x[0].y), pack2<T>(x[1].x, x[1].y));
                        *reinterpret_cast<uint2 *>(dst + o + at_b) = make_uint2(pack2<T>(y[0].x, y[0].y), pack2<T>(y[1].x, y[1].y));
                    }
                }
            }
            first = last;
        }
    }
}

static int check_rotary(const RotaryParams &p, int rotary_dim, int rotary_start, int dtype) {
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (p.nnz < 0 || p.Hq <= 0 || p.Hkv <= 0 || p.D <= 0 || rotary_dim < 0 || rotary_start < 0 ||
        rotary_start + static_cast<int64_t>(rotary_dim) > p.D || !(p.eps >= 0.f))
        return PKV_ERR_INVALID_ARG;
    if (p.D % 16 || rotary_dim % 16 || rotary_start % 8) return PKV_ERR_INVALID_ARG;
    if (p.D > 256 || p.Hq > 16384 || p.Hkv > 16384) return PKV_ERR_UNSUPPORTED;
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
    const int heads = kRotU * rows;  // of a batch
    p.batches[0] = (p.Hq + heads - 1) / heads;
    p.batches[1] = (p.Hkv + heads - 1) / heads;
    p.batches[2] = p.src[2] ? p.batches[1] : 0;
    const int all = p.batches[0] + p.batches[1] + p.batches[2];
    // A token's batches are divided among warps where there are fewer than
    // kRotRounds tokens to a warp that fits the machine.
    const int64_t warps = static_cast<int64_t>(num_sms()) * kRotCtas * kRotWarps;
    int64_t parts = (warps * kRotRounds + p.nnz - 1) / p.nnz;
    if (parts > all) parts = all;
    p.per_part = static_cast<int>((all + parts - 1) / parts);
    p.parts = (all + p.per_part - 1) / p.per_part;
    p.tasks = static_cast<uint32_t>(p.nnz * p.parts);  // (several parts only where there are few tokens)
    const int64_t blocks = (static_cast<int64_t>(p.tasks) + kRotWarps - 1) / kRotWarps;
    const int64_t most = static_cast<int64_t>(num_sms()) * kRotCtas;
    const unsigned grid = static_cast<unsigned>(blocks < most ? blocks : most);
    auto pick = [&](auto a, auto b) { return paired ? a : b; };
    auto kern = rows == 4 ? pick(rotary_kernel<T, 8, true>, rotary_kernel<T, 8, false>)
                          : (rows == 2 ? pick(rotary_kernel<T, 16, true>, rotary_kernel<T, 16, false>)
                                       : pick(rotary_kernel<T, 32, true>, rotary_kernel<T, 32, false>));
    const int stages = rows == 4 ? RotCfg<8>::STAGES : (rows == 2 ? RotCfg<16>::STAGES : RotCfg<32>::STAGES);
    const int smem = kRotWarps * stages * kRotU * 512;  // (24 KB at most, beside 5 KB of tables)
    kern<<<grid, kRotWarps * 32, smem, st>>>(p);
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
    if (page > (1 << 30)) return PKV_ERR_UNSUPPORTED;  // (offsets in a page: 32 bits)
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
