// decode_split.cuh -- split-KV GQA batch decode over a paged KV cache: the
// kernels, their plan and their launch, shared by decode.cu and
// decode_window.cu.
//
// Computes what flashinfer.decode.trtllm_batch_decode_with_kv_cache
// documents (parameters query, kv_cache, workspace_buffer, block_tables,
// seq_lens, max_seq_len, bmm1_scale, bmm2_scale, window_left, sinks,
// kv_layout, q_len_per_req): for every request, kv head and split of its
// visible key range, one CTA streams the split's K/V rows through a
// cp.async ring in shared memory and keeps an online softmax; a second
// kernel merges the splits by their log-sum-exp and adds the sink term.
//
// Row packing: the group = Hqo / Hkv query heads that share a kv head and
// the Q query tokens of a request form R = group * Q rows, padded to
// 16 * MT rows of one mma.sync m16n8k16 A operand, so each K/V row read
// from HBM feeds every query row that needs it.
//
// Roundings: a weight is rounded to the MMA's 16-bit type for its product with
// V (bf16 or fp16 as the cache, fp16 over an E4M3 cache: register MMAs take
// 16-bit operands at twice TF32's rate, and V has no more bits), the output
// once at the end; scores, maxima, sums, O, the splits' partials and the LSE
// are fp32.  Against 64 bits the output is off by 1.3 times what its own
// rounding gives where the weights have its type, by no more than its own
// rounding with weights in fp16 and a bf16 output.
//
// The kernel takes two extensions (EXT; their own translation unit,
// decode_window.cu): a window that keeps the first tokens visible, and an
// E4M3 cache with a scale for each block of keys and head.  Every visible key
// is read once, so HBM bounds them: 128 requests, one token, a window of 4096
// keys and 128 first tokens over a 16-bit cache: 315 us, 97% of the measured
// copy rate.  Over an E4M3 cache, with half the bytes, the work around a key
// counts: 64 requests of up to 8192 keys, 4 rows: 98 us, 85%; 96 requests
// of 4 tokens, 32 rows: 227 us, 47%, bound by the issue of register MMAs (64
// a warp and tile, 8 cycles each) and the softmax between them with two warps
// to a scheduler.  Tried and slower: the work of all requests laid end to end
// and cut evenly (105 / 266 us: the SMs do not stream at one rate), QK of the
// next tile ahead of the softmax (249 us: a warp issues in order), QK and PV on
// tcgen05 from fp16 tiles widened in shared memory (343 us: 4,000 cycles a
// tile of fences, barriers and waits, at most two CTAs per SM by tensor
// memory), splits of half and a quarter of the length (no change).  Times of
// the call replayed from a graph.
#pragma once

#include <math.h>

#include <type_traits>

#include "pkv_common.cuh"

namespace pkv {

constexpr int kDecD = 128;                        // head_dim
constexpr int kDecTile = 64;                      // keys per pipeline stage
// Ring depth and CTAs per SM.  One row tile (up to 16 packed query rows): 3
// CTAs per SM with a 2-stage ring; more row tiles need more registers: 2
// CTAs per SM, 3 stages.  An E4M3 stage is half as large, so its ring is 4
// stages deep at the same CTA counts.
// With swapped operands (SW 8-row tiles, see the split kernel) and 32 rows the
// output takes 128 registers a lane: 2 CTAs.
template <int MT, bool KV8 = false, int SW = 0>
struct DecCfg {
    static constexpr int STAGES = KV8 ? 4 : (MT == 1 ? 2 : 3);
    static constexpr int CTAS = MT == 1 && SW < 4 ? 3 : 2;
    static constexpr int ROWS = SW == 4 ? 32 : 16 * MT;  // query rows of a CTA
};
constexpr int kDecThreads = 128;
constexpr int kDecRowBytes = kDecD * 2;           // one K or V row
constexpr int kDecTileBytes = kDecTile * kDecRowBytes;
constexpr int kDecStageBytes = 2 * kDecTileBytes; // K tile then V tile
// An E4M3 cache is staged as 128-byte rows (K then V, 8 KB each per tile),
// 16-byte chunk c of row r at chunk c ^ (r & 7), and the MMA fragments are
// widened straight from those bytes (no 16-bit copy of the tile).
constexpr int kDec8RowBytes = kDecD;
constexpr int kDec8TileBytes = kDecTile * kDec8RowBytes;
template <bool KV8>
struct DecSmem {
    static constexpr int STAGE = KV8 ? 2 * kDec8TileBytes : kDecStageBytes;  // one ring stage
};
__device__ __forceinline__ int swz8(int r, int c) { return r * kDec8RowBytes + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ float2 unpack2_bf16(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}
constexpr int kDecMinPage = 8;                    // smallest supported page size
constexpr int kDecMaxChunk = 5120;                // largest split (keys)
constexpr int kDecMaxPages = kDecMaxChunk / kDecMinPage + 2;  // page ids one split can touch

struct DecodeParams {
    const void *q;
    const void *k;
    const void *v;
    int64_t page_stride;
    int64_t max_num_pages;
    const int32_t *block_tables;
    int64_t bt_stride;
    const uint32_t *seq_lens;
    int B;
    int max_seq_len;
    float scale_log2;  // bmm1_scale * log2(e): logits in base-2 units
    // device-resident fp32 bmm1 / bmm2 scales (NULL: the host values), read
    // when the kernels run, so a captured graph follows their current value
    const float *bmm1_dev, *bmm2_dev;
    float bmm2;
    int window_left;
    const float *sinks;
    int Q, Hqo, Hkv, group, R;  // Q: query tokens per request (the largest, with cu_q)
    const int32_t *cu_q;        // [B+1] variable-length query rows, or NULL (rows b*Q + t)
    int64_t num_tokens;         // query / out rows the caller holds
    int64_t kv_extent;  // elements a cache pointer spans: (max_num_pages - 1) * page_stride + one page
    int64_t ws_rows;    // partial rows of the workspace (B * Hkv * n_split_max * R)
    int page_shift;
    int chunk;        // keys per split
    int n_split_max;  // split slots per (request, kv head) in the workspace
    void *out;
    float *lse;
    float *ws_o;      // [B][Hkv][n_split_max][R][128] normalised partial outputs
    float *ws_lse;    // [B][Hkv][n_split_max][R] partial log2-sum-exp
    int32_t *err;
    // EXT >= 1: the first keys of a request that stay visible under a window
    int first_tokens;
    // EXT == 2: scales of an E4M3 cache, [page][kv head][page_size / block]
    // with scale_stride floats from page to page, blocks of 2^block_shift keys
    const float *k_scales, *v_scales;
    int64_t scale_stride;
    int block_shift;
    int pages_cap, scales_cap;  // entries of the split's page and scale lists (shared memory)
};

// Lowest visible key `lo` of a request and how its range [lo, L) is cut into
// splits: from `first` = lo rounded down to a 64-key tile, split s covers
// keys [max(lo, first + s * chunk), min(L, first + (s + 1) * chunk)).  An
// empty request keeps one split so its rows are written.
__host__ __device__ inline void decode_split_geometry(int L, int Q, int window_left, int chunk,
                                                      int &lo, int &first, int &n_split) {
    lo = 0;
    if (window_left >= 0) {
        lo = L - Q - window_left;
        if (lo < 0) lo = 0;
    }
    first = lo & ~(kDecTile - 1);
    n_split = L <= lo ? 1 : (L - first + chunk - 1) / chunk;
}

// The same under a window that keeps the first `first_tokens` keys visible
// too.  A request's keys are then read as one run of tiles: the n_first keys
// [0, n_first) that hold the first tokens (whole 64-key tiles), then the keys
// from `first` (the window's first tile) on, `gap` = first - n_first keys
// further; split s covers [s * chunk, (s + 1) * chunk) of that run.  Where
// the first tokens reach the window, every key is visible and gap is 0.
struct DecodeRun {
    int lo;       // keys [first_tokens, lo) are visible to no query
    int n_first;  // keys of the first part of the run
    int gap;      // distance of the second part's keys from the run's index
    int n;        // length of the run
    int n_split;
};
__host__ __device__ inline DecodeRun decode_run(int L, int Q, int window_left, int first_tokens, int chunk) {
    DecodeRun r;
    r.lo = window_left >= 0 ? L - Q - window_left : 0;
    if (r.lo <= first_tokens) r.lo = 0;
    const int first = r.lo & ~(kDecTile - 1);
    r.n_first = first_tokens < first ? (first_tokens + kDecTile - 1) & ~(kDecTile - 1) : first;
    r.gap = first - r.n_first;
    r.n = L - r.gap;
    r.n_split = L <= 0 ? 1 : (r.n + chunk - 1) / chunk;
    return r;
}

// Barrier over the MT warps that share a slice of keys (warps kg*MT ..
// kg*MT + MT - 1): a warp sync for one, __syncthreads for all four, else the
// named barrier 1 + kg.
template <int MT>
__device__ __forceinline__ void key_group_sync(int kg) {
    if constexpr (MT == 1) {
        __syncwarp();
    } else if constexpr (MT * 32 == kDecThreads) {
        __syncthreads();
    } else {
        asm volatile("bar.sync %0, %1;\n" ::"r"(1 + kg), "n"(MT * 32) : "memory");
    }
}

template <typename T>
__device__ __forceinline__ void store4(T *dst, float a, float b, float c, float d) {
    uint2 v;
    v.x = pack2<T>(a, b);
    v.y = pack2<T>(c, d);
    *reinterpret_cast<uint2 *>(dst) = v;
}

// SW > 0 (an E4M3 cache and at most 8 SW query rows): the MMAs take the keys
// as their 16-row side, S^T = K Q^T and O^T = V^T P^T (see the tile loop).
// EXT: 0 all keys or a window; 1 a window and first tokens; 2 the same over
// an E4M3 cache with a scale for each block of keys and head.
template <typename T, int MT, int LAYOUT, bool KV8, int SW = 0, int EXT = 0>
__global__ void __launch_bounds__(kDecThreads, DecCfg<MT, KV8, SW>::CTAS) decode_split_kernel(const DecodeParams p) {
    constexpr bool FIRST = EXT >= 1, SCL = EXT == 2;
    static_assert(!SCL || KV8, "block scales: E4M3 cache");
    constexpr int kDecStages = DecCfg<MT, KV8, SW>::STAGES;
    constexpr int STAGE_BYTES = DecSmem<KV8>::STAGE;
    // the MMA element type: over an E4M3 cache always fp16 (E4M3 widens to
    // fp16 in one instruction; a bf16 query is brought to fp16 exactly, see
    // below)
    using TM = typename std::conditional<KV8, __half, T>::type;
    static_assert(!SW || (KV8 && MT == 1), "swapped operands: E4M3 cache, one row tile");
    constexpr int NKG = 4 / MT;          // warps that split the keys of a tile
    constexpr int KPW = kDecTile / NKG;  // keys per warp per tile
    constexpr int NT = KPW / 8;          // 8-key score tiles per warp
    constexpr int ROWS = DecCfg<MT, KV8, SW>::ROWS;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_s = smem + kDecStages * STAGE_BYTES;
    uint8_t *kvalid = q_s + ROWS * kDecRowBytes;
    float *comb_m = reinterpret_cast<float *>(kvalid + kDecStages * kDecTile);
    float *comb_l = comb_m + NKG * ROWS;
    int *pages_s = reinterpret_cast<int *>(comb_l + NKG * ROWS);  // the split's page ids
    // (SCL) the split's scales: K scale times the logit scale, V scale
    float2 *scale_s = reinterpret_cast<float2 *>(pages_s + (FIRST ? p.pages_cap : kDecMaxPages));
    const int pages_cap = FIRST ? p.pages_cap : kDecMaxPages;
    __shared__ int any_bad[4];  // per key group: a row of its slice was on a bad page

    // launched as a dependent of the stream's previous kernel (enable_pdl):
    // wait for it before reading anything it may have written
    pdl_wait();
    const int s = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int mt = warp % MT, kg = warp / MT;
    const int gtid = tid - kg * MT * 32;  // thread index within the key group
    const int kw0 = kg * KPW;             // the group's key slice of every tile
    const uint32_t L_in = p.seq_lens[b];
    const int L = L_in > static_cast<uint32_t>(p.max_seq_len) ? p.max_seq_len : static_cast<int>(L_in);
    if (L_in > static_cast<uint32_t>(p.max_seq_len) && s == 0 && kvh == 0 && threadIdx.x == 0)
        set_err(p.err, PKV_DEV_ERR_LEN);
    // this request's query tokens: Q at rows b*Q + t, or Q_b at rows
    // cu_q[b] + t (an inconsistent entry -- decreasing, longer than the
    // planned maximum, or past the caller's rows -- is flagged and skipped)
    int Q = p.Q;
    int64_t qrow0 = static_cast<int64_t>(b) * p.Q;
    if (p.cu_q) {
        const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
        Q = c1 - c0;
        qrow0 = c0;
        if (c0 < 0 || Q < 0 || Q > p.Q || c1 > p.num_tokens) {
            if (s == 0 && kvh == 0 && threadIdx.x == 0) set_err(p.err, PKV_DEV_ERR_QLEN);
            Q = 0;
        }
        if (Q == 0) return;  // uniform over the CTA: before any barrier
    }
    const int R = p.group * Q;  // query rows of this (request, kv head)
    int lo, first, n_split;
    DecodeRun run = {};
    if constexpr (FIRST) {
        run = decode_run(L, Q, p.window_left, p.first_tokens, p.chunk);
        lo = run.lo;
        first = 0;
        n_split = run.n_split;
    } else {
        decode_split_geometry(L, Q, p.window_left, p.chunk, lo, first, n_split);
    }
    if (s >= n_split) return;
    if (L < Q && s == 0 && kvh == 0 && tid == 0) set_err(p.err, PKV_DEV_ERR_QLEN);
    const int k_begin = FIRST ? s * p.chunk : max(lo, first + s * p.chunk);
    const int k_end = FIRST ? min(run.n, (s + 1) * p.chunk) : min(L, first + (s + 1) * p.chunk);
    // tiles start on 64-key boundaries (a window's first key need not): the
    // rows before k_begin are zero-filled and masked like rows past the end
    // (FIRST: k_begin and k_end count along the run, key_of gives the key)
    const int k_tile0 = k_begin & ~(kDecTile - 1);
    const int n_tiles = k_end > k_begin ? (k_end - k_tile0 + kDecTile - 1) / kDecTile : 0;
    auto key_of = [&](int v) { return FIRST && v >= run.n_first ? v + run.gap : v; };
    // keys of rows j .. j + n - 1 of a tile, all holding a key some query sees
    auto keys_in = [&](int j, int n) {
        if constexpr (FIRST) return j + n <= L && (j >= lo || j + n <= p.first_tokens);
        return j >= k_begin && j + n <= k_end;
    };

    const T *kc = static_cast<const T *>(p.k);
    const T *vc = static_cast<const T *>(p.v);
    const uint8_t *kc8 = static_cast<const uint8_t *>(p.k);  // E4M3 cache (KV8)
    const uint8_t *vc8 = static_cast<const uint8_t *>(p.v);
    const int32_t *bt = p.block_tables + static_cast<int64_t>(b) * p.bt_stride;
    const int S = 1 << p.page_shift;
    if (tid < 4) any_bad[tid] = 0;
    // page ids of the split, fetched once (coalesced) so that the per-tile
    // address computation does not wait on global memory; -1 marks an id
    // outside the pool
    // (FIRST) the split's keys of the run's first part, then of its second,
    // [a1, e1) and [a2, e2).  A page of keys that no query sees, between the
    // first tokens and the window, may be gone: its entry is not read.
    int a1 = k_begin, e1 = k_end, a2 = 0, e2 = 0;
    if constexpr (FIRST) {
        e1 = max(a1, min(k_end, run.n_first));
        a2 = max(k_begin, run.n_first) + run.gap;
        e2 = max(a2, k_end + run.gap);
    }
    auto unseen = [&](int j, int n) { return FIRST && j >= p.first_tokens && j + n <= lo; };
    const int first_page = a1 >> p.page_shift;
    const int n_pages1 = e1 > a1 ? ((e1 - 1) >> p.page_shift) - first_page + 1 : 0;
    const int first_page2 = FIRST ? a2 >> p.page_shift : 0;
    const int n_pages = n_pages1 + (FIRST && e2 > a2 ? ((e2 - 1) >> p.page_shift) - first_page2 + 1 : 0);
    // list entry of a key's page: its page index minus this base
    const int base2 = first_page2 - n_pages1;
    auto page_base = [&](int j) { return FIRST && j >= run.n_first + run.gap ? base2 : first_page; };
    for (int i = tid; i < n_pages; i += kDecThreads) {
        const int pi = i + (FIRST && i >= n_pages1 ? base2 : first_page);
        const bool in_bt = dbg_in(pi, 1, (p.max_seq_len + S - 1) >> p.page_shift, p.err);
        const bool read = in_bt && !unseen(pi << p.page_shift, S);
        int page = read ? bt[pi] : -1;
        if (read && (page < 0 || page >= p.max_num_pages)) {
            set_err(p.err, PKV_DEV_ERR_PAGE);
            page = -1;
        }
        if (dbg_in(i, 1, pages_cap, p.err)) pages_s[i] = page;
    }
    __syncthreads();

    // K and V rows of a tile.  Every key group loads (and later widens) only
    // the KPW rows of its own key slice, the only rows its warps read, so a
    // tile needs no barrier wider than the group.  16 consecutive lanes copy
    // one 256-byte row: every warp instruction moves two whole rows.  Rows
    // past the split end or on an out-of-range page are zero-filled and never
    // read from global memory; kvalid records which rows hold a key.
    // A thread's rows of a tile are RSTEP apart; when they all lie before the
    // split end on one page (the common case), the page is looked up once
    // and the row address advances by a fixed step.
    constexpr int LPR = KV8 ? 8 : 16;                 // lanes per row
    constexpr int RSTEP = MT * 32 / LPR;              // rows between a thread's rows
    constexpr int NLOAD = KPW * LPR / (MT * 32);      // rows per thread per tile
    const int64_t row_step = (LAYOUT == PKV_HND ? kDecD : static_cast<int64_t>(p.Hkv) * kDecD) * RSTEP;
    // (EXT over an E4M3 cache, 16-key slices: the common case with everything
    // but the page's and the slot's offset worked out once; kvalid of a stage
    // is rewritten only after a tile that had rows without a key)
    constexpr bool SLICE16 = EXT > 0 && SW > 0;
    const int64_t row_bytes = LAYOUT == PKV_HND ? kDecD : static_cast<int64_t>(p.Hkv) * kDecD;
    const uint8_t *lane_k = kc8 + (LAYOUT == PKV_HND ? static_cast<int64_t>(kvh) * S : static_cast<int64_t>(kvh)) * kDecD +
                            (lane >> 3) * row_bytes + (lane & 7) * 16;
    const int64_t v_from_k = vc8 - kc8;
    const uint32_t slice_even = swz8(kw0 + (lane >> 3), lane & 7), slice_odd = swz8(kw0 + (lane >> 3) + 4, lane & 7);
    uint32_t dirty = 0xffffffffu;  // bit s: kvalid of stage s may hold zeros
    auto load_tile = [&](int stage, int j0) {
        const uint32_t dst = smem_u32(smem + stage * STAGE_BYTES);
        if constexpr (SLICE16) {
            const int js = j0 + kw0, pi = (js >> p.page_shift) - page_base(j0);
            if (p.page_shift >= 4 && keys_in(js, 16) && dbg_in(pi, 1, pages_cap, p.err)) {
                const int page = pages_s[pi];
                if (page >= 0) {
                    const uint8_t *ks = lane_k + (page * p.page_stride + (js & (S - 1)) * row_bytes);
                    const uint8_t *vs = ks + v_from_k;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t o = ((k & 1) ? slice_odd : slice_even) + (k >> 1) * (8 * kDec8RowBytes);
                        const bool in = dbg_in(ks + k * row_step - kc8, 16, p.kv_extent, p.err);
                        cp_async_16(dst + o, in ? ks + k * row_step : kc8, in);
                        cp_async_16(dst + kDec8TileBytes + o, in ? vs + k * row_step : vc8, in);
                    }
                    if ((dirty >> stage) & 1u) {
                        if (lane < 16) kvalid[stage * kDecTile + kw0 + lane] = 1;
                        dirty &= ~(1u << stage);
                    }
                    return;
                }
            }
            dirty |= 1u << stage;
        }
        {
            const int r0 = kw0 + gtid / LPR, c = gtid % LPR;
            const int jA = j0 + r0, jZ = jA + (NLOAD - 1) * RSTEP;
            const int pi = (jA >> p.page_shift) - page_base(j0);
            const int page = keys_in(jA, jZ - jA + 1) && (jA >> p.page_shift) == (jZ >> p.page_shift) &&
                                     dbg_in(pi, 1, pages_cap, p.err)
                                 ? pages_s[pi]
                                 : -1;
            if (__all_sync(0xffffffffu, page >= 0)) {
                const int64_t off = kv_row_offset<LAYOUT>(page, p.page_stride, kvh, jA & (S - 1), p.Hkv, S, kDecD);
#pragma unroll
                for (int k = 0; k < NLOAD; ++k) {
                    const int r = r0 + k * RSTEP;
                    if (c == 0) kvalid[stage * kDecTile + r] = 1;
                    if constexpr (KV8) {
                        const int64_t e = off + k * row_step + c * 16;
                        const bool in = dbg_in(e, 16, p.kv_extent, p.err);
                        cp_async_16(dst + swz8(r, c), in ? kc8 + e : kc8, in);
                        cp_async_16(dst + kDec8TileBytes + swz8(r, c), in ? vc8 + e : vc8, in);
                    } else {
                        const uint32_t o = swz(r, c, kDecRowBytes);
                        const int64_t e = off + k * row_step + c * 8;
                        const bool in = dbg_in(e, 8, p.kv_extent, p.err);
                        cp_async_16(dst + o, in ? kc + e : kc, in);
                        cp_async_16(dst + kDecTileBytes + o, in ? vc + e : vc, in);
                    }
                }
                return;
            }
        }
        if constexpr (KV8) {
            // 128-byte E4M3 rows: 8 consecutive lanes copy one row
#pragma unroll
            for (int k = 0; k < KPW * 8 / (MT * 32); ++k) {
                const int idx = k * MT * 32 + gtid;
                const int r = kw0 + (idx >> 3), c = idx & 7;
                const int j = j0 + r;
                bool ok = keys_in(j, 1);
                const uint8_t *ks = kc8, *vs = vc8;
                if (ok) {
                    const int pi = (j >> p.page_shift) - page_base(j0);
                    const int page = dbg_in(pi, 1, pages_cap, p.err) ? pages_s[pi] : -1;
                    if (page < 0) {
                        ok = false;
                        any_bad[kg] = 1;
                    } else {
                        const int64_t off = kv_row_offset<LAYOUT>(page, p.page_stride, kvh, j & (S - 1), p.Hkv,
                                                                  S, kDecD) + c * 16;
                        ok = dbg_in(off, 16, p.kv_extent, p.err);
                        if (ok) {
                            ks = kc8 + off;
                            vs = vc8 + off;
                        }
                    }
                }
                if (c == 0) kvalid[stage * kDecTile + r] = ok ? 1 : 0;
                cp_async_16(dst + swz8(r, c), ks, ok);
                cp_async_16(dst + kDec8TileBytes + swz8(r, c), vs, ok);
            }
        } else {
#pragma unroll
        for (int k = 0; k < KPW * 16 / (MT * 32); ++k) {
            const int idx = k * MT * 32 + gtid;
            const int r = kw0 + (idx >> 4), c = idx & 15;
            const int j = j0 + r;
            bool ok = keys_in(j, 1);
            const T *ks = kc, *vs = vc;
            if (ok) {
                const int pi = (j >> p.page_shift) - page_base(j0);
                const int page = dbg_in(pi, 1, pages_cap, p.err) ? pages_s[pi] : -1;
                if (page < 0) {
                    ok = false;
                    any_bad[kg] = 1;
                } else {
                    const int64_t off = kv_row_offset<LAYOUT>(page, p.page_stride, kvh, j & (S - 1), p.Hkv,
                                                              S, kDecD) + c * 8;
                    ok = dbg_in(off, 8, p.kv_extent, p.err);
                    if (ok) {
                        ks = kc + off;
                        vs = vc + off;
                    }
                }
            }
            if (c == 0) kvalid[stage * kDecTile + r] = ok ? 1 : 0;
            const uint32_t o = swz(r, c, kDecRowBytes);
            cp_async_16(dst + o, ks, ok);
            cp_async_16(dst + kDecTileBytes + o, vs, ok);
        }
        }
    };

    // query rows r = t * group + i  ->  query[(b*Q + t), kvh*group + i, :]
    const T *qp = static_cast<const T *>(p.q);
    for (int idx = tid; idx < ROWS * 16; idx += kDecThreads) {
        int r = idx >> 4, c = idx & 15;
        bool ok = r < R;
        const T *src = qp;
        if (ok) {
            int t = r / p.group, i = r - t * p.group;
            const int64_t e = ((qrow0 + t) * p.Hqo + kvh * p.group + i) * kDecD + c * 8;
            ok = dbg_in(e, 8, p.num_tokens * p.Hqo * kDecD, p.err);
            if (ok) src = qp + e;
        }
        cp_async_16(smem_u32(q_s) + swz(r, c, kDecRowBytes), src, ok);
    }
    cp_async_commit();
#pragma unroll
    for (int st = 0; st < kDecStages - 1; ++st) {
        if (st < n_tiles) load_tile(st, key_of(k_tile0 + st * kDecTile));
        cp_async_commit();
    }
    float scale_log2 = p.bmm1_dev ? __ldg(p.bmm1_dev) * kLog2e : p.scale_log2;
    // (SCL) the scales of the split's blocks, while its first tiles arrive
    const int first_block = SCL ? a1 >> p.block_shift : 0;
    const int first_block2 = SCL ? a2 >> p.block_shift : 0;
    const int n_blocks1 = SCL && e1 > a1 ? ((e1 - 1) >> p.block_shift) - first_block + 1 : 0;
    const int n_blocks = SCL ? n_blocks1 + (e2 > a2 ? ((e2 - 1) >> p.block_shift) - first_block2 + 1 : 0) : 0;
    if constexpr (SCL) {
        const int per_page_shift = p.page_shift - p.block_shift;
        for (int i = tid; i < n_blocks; i += kDecThreads) {
            const int blk = i < n_blocks1 ? first_block + i : first_block2 + i - n_blocks1;
            const int pi = (blk >> per_page_shift) - (i < n_blocks1 ? first_page : base2);
            const int page = dbg_in(pi, 1, pages_cap, p.err) ? pages_s[pi] : -1;
            float2 sc = make_float2(1.f, 1.f);
            if (page >= 0 && !unseen(blk << p.block_shift, 1 << p.block_shift)) {
                const int64_t e = static_cast<int64_t>(page) * p.scale_stride + (static_cast<int64_t>(kvh) << per_page_shift) +
                                  (blk & ((1 << per_page_shift) - 1));
                sc = make_float2(checked_scale(__ldg(p.k_scales + e), p.err), checked_scale(__ldg(p.v_scales + e), p.err));
            }
            if (dbg_in(i, 1, p.scales_cap, p.err)) scale_s[i] = sc;
        }
    }
    // (K scale, V scale) of the 8 keys from j on (j a multiple of 8, in the
    // tile at j0); keys that no query sees may get any entry
    auto scales_of = [&](int j0, int j) {
        const int i = (j >> p.block_shift) - (j0 >= run.n_first + run.gap ? first_block2 - n_blocks1 : first_block);
        return scale_s[min(max(i, 0), n_blocks - 1)];
    };
    cp_async_wait<kDecStages - 1>();
    __syncthreads();

    const float bmm2 = p.bmm2_dev ? __ldg(p.bmm2_dev) : p.bmm2;
    if constexpr (KV8 && !std::is_same<T, __half>::value) {
        // bf16 query -> fp16 for the fp16 MMAs: scaled by 2^e so that the
        // largest |q| of the CTA lies in [2^14, 2^15) -- every bf16 value of
        // the rows then converts exactly unless it falls below fp16's normal
        // range, 2^29 under that largest element -- with 2^-e moved into the
        // logit scale (powers of two, exact)
        __shared__ float qmax_s[kDecThreads / 32];
        float mx = 0.f;
        for (int idx = tid; idx < ROWS * 16; idx += kDecThreads) {
            const uint4 v = *reinterpret_cast<const uint4 *>(q_s + swz(idx >> 4, idx & 15, kDecRowBytes));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2_bf16(w[i]);
                mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) qmax_s[warp] = mx;
        __syncthreads();
        mx = fmaxf(fmaxf(qmax_s[0], qmax_s[1]), fmaxf(qmax_s[2], qmax_s[3]));
        int e = 0;
        if (mx > 0.f && isfinite(mx)) {
            int ex;
            frexpf(mx, &ex);  // mx in [2^(ex-1), 2^ex)
            e = min(max(15 - ex, -100), 100);  // (beyond that the row is all but zero)
        }
        const float up = ldexpf(1.f, e);
        scale_log2 = ldexpf(scale_log2, -e);
        __syncthreads();  // every warp has its max before the tile is rewritten
        for (int idx = tid; idx < ROWS * 16; idx += kDecThreads) {
            uint4 *a = reinterpret_cast<uint4 *>(q_s + swz(idx >> 4, idx & 15, kDecRowBytes));
            const uint4 v = *a;
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2_bf16(w[i]);
                h[i] = pack2<__half>(f.x * up, f.y * up);
            }
            *a = make_uint4(h[0], h[1], h[2], h[3]);
        }
        __syncthreads();
    }

    uint32_t qa[SW ? 1 : 8][4];
    constexpr bool QSMEM = SW == 4;  // (32 rows: read per tile, the registers hold the output)
    uint32_t qb[SW && !QSMEM ? SW : 1][8][2];  // (SW) Q^T fragments of each 8-row tile
    const uint8_t *q_lane = q_s + (lane >> 2) * kDecRowBytes;
    if constexpr (QSMEM) {
    } else if constexpr (SW > 0) {
        // B operand of the swapped QK (Q^T, k = head dim, n = query row): lane
        // (g, c) holds row 8u + g, dims 32c + 4kk + {0, 1} and {2, 3} of k-step
        // kk (the permuted order of the K rows, below)
        const int gq = lane >> 2, cq = lane & 3;
#pragma unroll
        for (int u = 0; u < SW; ++u)
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const int dim = cq * 32 + kk * 4;
                const uint2 q2 =
                    *reinterpret_cast<const uint2 *>(q_s + swz(8 * u + gq, dim >> 3, kDecRowBytes) + (dim & 7) * 2);
                qb[u][kk][0] = q2.x;
                qb[u][kk][1] = q2.y;
            }
    } else if constexpr (KV8) {
        // Over an E4M3 cache the head dimension is taken in a permuted order,
        // the same for Q and K (a dot product does not depend on it): the k
        // pairs {2c, 2c+1} and {2c+8, 2c+9} of k-step kk are the dims
        // 32c + 4kk + {0,1} and {2,3}, so that one 32-bit word of a K row
        // holds both halves of a B fragment.
        const int gq = lane >> 2, cq = lane & 3;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const int dim = cq * 32 + kk * 4;
            const uint2 lo = *reinterpret_cast<const uint2 *>(q_s + swz(16 * mt + gq, dim >> 3, kDecRowBytes) +
                                                              (dim & 7) * 2);
            const uint2 hi = *reinterpret_cast<const uint2 *>(q_s + swz(16 * mt + gq + 8, dim >> 3, kDecRowBytes) +
                                                              (dim & 7) * 2);
            qa[kk][0] = lo.x;
            qa[kk][1] = hi.x;
            qa[kk][2] = lo.y;
            qa[kk][3] = hi.y;
        }
    } else {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            ldsm_x4(qa[kk], smem_u32(q_s) + swz(16 * mt + (lane & 15), 2 * kk + (lane >> 4), kDecRowBytes));
    }

    // the two rows this lane holds in every accumulator fragment
    const int r0 = 16 * mt + (lane >> 2), r1 = r0 + 8;
    const int t0 = min(r0 / p.group, Q - 1), t1 = min(r1 / p.group, Q - 1);
    const int pos0 = L - Q + t0, pos1 = L - Q + t1;
    const int lo0 = p.window_left >= 0 ? max(0, pos0 - p.window_left) : 0;
    const int lo1 = p.window_left >= 0 ? max(0, pos1 - p.window_left) : 0;
    const int lo_max = p.window_left >= 0 ? max(0, L - 1 - p.window_left) : 0;
    const int hi_min = FIRST ? L - Q : min(L - Q, k_end - 1);
    // (swapped operands: lane (g, c) holds query rows 8u + 2c and 8u + 2c + 1
    // of row tile u; (lowest key of the window, position) of every row)
    const int sr0 = 2 * (lane & 3);
    constexpr float kNoKey = -3e38f;
    __shared__ __align__(16) int2 row_bounds[SW > 0 ? ROWS : 1];
    if constexpr (SW > 0) {
        if (tid < ROWS) {
            const int pos = L - Q + min(tid / p.group, Q - 1);
            row_bounds[tid] = make_int2(p.window_left >= 0 ? max(0, pos - p.window_left) : 0, pos);
        }
        __syncthreads();
    }

    // output: n-tiles of 8 dims, or (SW) 8 m-tiles of 16 dims for each row tile
    constexpr int NO = SW ? 8 * SW : 16;
    float o[NO][4];
#pragma unroll
    for (int i = 0; i < NO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float ms[SW ? SW : 1][2], ls[SW ? SW : 1][2];  // (SW) the same for each row tile
#pragma unroll
    for (int u = 0; u < SW; ++u) {
        ms[u][0] = ms[u][1] = kNoKey;  // (finite: a masked score's distance to it is -inf)
        ls[u][0] = ls[u][1] = 0.f;
    }

    // a key at or after a row's window start, or one of the first tokens
    auto from = [&](int j, int row_lo) { return j >= row_lo || (FIRST && j < p.first_tokens); };

    // (SCL) With block scales, key j's logit is z_j = scale ks(j) <q, k_j> and
    // its weight on the stored V row is e^z_j vs(j).  The running maximum is
    // kept over z_j + log vs(j), so that P_j = e^(z_j + log vs(j) - m), the
    // weight that goes into the fp16 MMA, is at most 2^8 whatever the scales
    // are (a key whose weight times V scale is below 2^-25 of the row's largest
    // adds nothing to the output: fp16's smallest number); the denominator sums P_j / vs(j) in fp32, and m + log of that sum
    // is the log-sum-exp of the z_j.  Eight consecutive keys share a scale
    // (blocks are at least 8 keys), so a score costs one FFMA as without
    // scales and a sum term one FFMA in place of an add.
    for (int it = 0; it < n_tiles; ++it) {
        cp_async_wait<kDecStages - 2>();
        key_group_sync<MT>(kg);  // the slice landed; the group is done with the stage reloaded next
        {
            int nxt = it + kDecStages - 1;
            if (nxt < n_tiles) load_tile(nxt % kDecStages, key_of(k_tile0 + nxt * kDecTile));
            cp_async_commit();
        }
        const int stage = it % kDecStages;
        const int j0 = key_of(k_tile0 + it * kDecTile);
        const uint32_t kb = smem_u32(smem + stage * STAGE_BYTES);
        const uint32_t vb = kb + kDecTileBytes;
        const uint8_t *k8 = smem + stage * STAGE_BYTES;  // E4M3 K rows (KV8)
        const uint8_t *v8 = k8 + kDec8TileBytes;         // E4M3 V rows (KV8)

        if constexpr (SW > 0) {
            // Swapped operands for at most 8 SW query rows: S^T (the warp's 16
            // keys x 8 rows) = K Q^T and O^T (128 dims x 8 rows) += V^T P^T for
            // each 8-row tile u, so that the keys fill the MMA's 16-row side
            // and a K or V value is widened once for all row tiles.  Lane
            // (g, c) = (lane / 4, lane % 4) holds the scores of keys kw0 + g and
            // kw0 + g + 8 for query rows 8u + 2c and 8u + 2c + 1; rows at or
            // beyond R are padding that nothing reads.
            const int g = lane >> 2, c = lane & 3;
            constexpr int CH = SW <= 2 ? 2 : 1;  // MMA chains of a row tile's scores (even / odd k-steps)
            float sc[SW][CH][4];
#pragma unroll
            for (int u = 0; u < SW; ++u)
#pragma unroll
                for (int i = 0; i < CH; ++i) sc[u][i][0] = sc[u][i][1] = sc[u][i][2] = sc[u][i][3] = 0.f;
            {
                // A = K rows kw0 + g and kw0 + g + 8: the word at byte
                // 32c + 4kk of a row holds dims 32c + 4kk .. + 3, both halves
                // of the lane's A fragment of k-step kk (the permuted order
                // the Q fragments follow)
                const uint4 u0 = *reinterpret_cast<const uint4 *>(k8 + swz8(kw0 + g, 2 * c));
                const uint4 u1 = *reinterpret_cast<const uint4 *>(k8 + swz8(kw0 + g, 2 * c + 1));
                const uint4 v0 = *reinterpret_cast<const uint4 *>(k8 + swz8(kw0 + g + 8, 2 * c));
                const uint4 v1 = *reinterpret_cast<const uint4 *>(k8 + swz8(kw0 + g + 8, 2 * c + 1));
                const uint32_t wa[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
                const uint32_t wb[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t a[4] = {widen_e4m3x2<TM>(wa[kk] & 0xffffu), widen_e4m3x2<TM>(wb[kk] & 0xffffu),
                                           widen_e4m3x2<TM>(wa[kk] >> 16), widen_e4m3x2<TM>(wb[kk] >> 16)};
#pragma unroll
                    for (int u = 0; u < SW; ++u) {
                        if constexpr (QSMEM) {
                            // row 8u + g, dims 32c + 4kk .. + 3 (16-byte chunk 4c + kk / 2, swizzled by g)
                            const uint2 q2 = *reinterpret_cast<const uint2 *>(
                                q_lane + u * (8 * kDecRowBytes) + (((4 * c + (kk >> 1)) ^ g) << 4) + (kk & 1) * 8);
                            mma16816<TM>(sc[u][kk & (CH - 1)], a, q2.x, q2.y);
                        } else {
                            mma16816<TM>(sc[u][kk & (CH - 1)], a, qb[u][kk][0], qb[u][kk][1]);
                        }
                    }
                }
            }
            float kmA = scale_log2, kmB = scale_log2, lvA = 0.f, lvB = 0.f, ivA = 1.f, ivB = 1.f;
            if constexpr (SCL) {
                const float2 fA = scales_of(j0, j0 + kw0), fB = scales_of(j0, j0 + kw0 + 8);
                kmA = fA.x * scale_log2;
                kmB = fB.x * scale_log2;
                lvA = fast_log2(fA.y);
                lvB = fast_log2(fB.y);
                ivA = fast_rcp(fA.y);
                ivB = fast_rcp(fB.y);
            }
            const bool interior = !any_bad[kg] && (j0 >= lo_max || (FIRST && j0 + kDecTile <= p.first_tokens)) &&
                                  j0 + kDecTile - 1 <= hi_min;
            // element e of a row tile: key kw0 + g + 8 (e / 2), query row 8u + 2c + (e % 2)
            float sv[SW][4];
            bool higher = false;  // a score more than 2^8 above its row's maximum
#pragma unroll
            for (int u = 0; u < SW; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x0 = CH == 2 ? sc[u][0][e] + sc[u][CH - 1][e] : sc[u][0][e];
                    const float x = SCL ? fmaf(x0, e & 2 ? kmB : kmA, e & 2 ? lvB : lvA) : x0 * scale_log2;
                    sv[u][e] = x;
                }
            }
            if (!interior) {
#pragma unroll
                for (int hk = 0; hk < 2; ++hk) {
                    const int jj = kw0 + g + 8 * hk, j = j0 + jj;
                    const bool here = kvalid[stage * kDecTile + jj] != 0;
#pragma unroll
                    for (int u = 0; u < SW; ++u) {
                        const int4 b = *reinterpret_cast<const int4 *>(&row_bounds[8 * u + sr0]);
                        if (!(here && from(j, b.x) && j <= b.y)) sv[u][2 * hk] = -INFINITY;
                        if (!(here && from(j, b.z) && j <= b.w)) sv[u][2 * hk + 1] = -INFINITY;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < SW; ++u)
                higher = higher || fmaxf(sv[u][0], sv[u][2]) > ms[u][0] + 8.f || fmaxf(sv[u][1], sv[u][3]) > ms[u][1] + 8.f;
            // the running maxima rise only where a tile's exceeds them by more
            // than 8 (a factor 2^8): only then are the row maxima over the
            // warp's 16 keys (the lanes of one c) needed
            if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
                for (int u = 0; u < SW; ++u) {
                    float mx0 = fmaxf(sv[u][0], sv[u][2]), mx1 = fmaxf(sv[u][1], sv[u][3]);
#pragma unroll
                    for (int o_ = 4; o_ < 32; o_ <<= 1) {
                        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o_));
                        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o_));
                    }
                    const float mn0 = mx0 > ms[u][0] + 8.f ? mx0 : ms[u][0], mn1 = mx1 > ms[u][1] + 8.f ? mx1 : ms[u][1];
                    const float al0 = fast_exp2(ms[u][0] - mn0), al1 = fast_exp2(ms[u][1] - mn1);
                    ls[u][0] *= al0;
                    ls[u][1] *= al1;
                    ms[u][0] = mn0;
                    ms[u][1] = mn1;
#pragma unroll
                    for (int i = 8 * u; i < 8 * u + 8; ++i) {
                        o[i][0] *= al0;
                        o[i][2] *= al0;
                        o[i][1] *= al1;
                        o[i][3] *= al1;
                    }
                }
            }
            // B = P^T (k = the warp's 16 keys, n = query row): the transposes of
            // the two 8 x 8 blocks (keys x rows) of P
            uint32_t pb[SW][2];
#pragma unroll
            for (int u = 0; u < SW; ++u) {
                const float p0 = fast_exp2(sv[u][0] - ms[u][0]), p1 = fast_exp2(sv[u][1] - ms[u][1]);
                const float p2 = fast_exp2(sv[u][2] - ms[u][0]), p3 = fast_exp2(sv[u][3] - ms[u][1]);
                // (this lane's keys; summed over g at the end)
                ls[u][0] += SCL ? fmaf(p0, ivA, p2 * ivB) : p0 + p2;
                ls[u][1] += SCL ? fmaf(p1, ivA, p3 * ivB) : p1 + p3;
                pb[u][0] = transpose8x8(pack2<TM>(p0, p1));
                pb[u][1] = transpose8x8(pack2<TM>(p2, p3));
            }
            // A = V^T (m = head dim, k = key) of m-tile i: its row m is dim
            // 16 (m % 8) + 2i + m / 8, so that a lane's 16 dims of a V row are
            // one 16-byte chunk (g) and the two keys of an A register are
            // byte-interleaved from two rows
            const uint4 x0 = *reinterpret_cast<const uint4 *>(v8 + swz8(kw0 + 2 * c, g));
            const uint4 x1 = *reinterpret_cast<const uint4 *>(v8 + swz8(kw0 + 2 * c + 1, g));
            const uint4 y0 = *reinterpret_cast<const uint4 *>(v8 + swz8(kw0 + 2 * c + 8, g));
            const uint4 y1 = *reinterpret_cast<const uint4 *>(v8 + swz8(kw0 + 2 * c + 9, g));
            const uint32_t X0[4] = {x0.x, x0.y, x0.z, x0.w}, X1[4] = {x1.x, x1.y, x1.z, x1.w};
            const uint32_t Y0[4] = {y0.x, y0.y, y0.z, y0.w}, Y1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x01 = __byte_perm(X0[i], X1[i], 0x5140), x23 = __byte_perm(X0[i], X1[i], 0x7362);
                const uint32_t y01 = __byte_perm(Y0[i], Y1[i], 0x5140), y23 = __byte_perm(Y0[i], Y1[i], 0x7362);
                const uint32_t a0[4] = {widen_e4m3x2<TM>(x01 & 0xffffu), widen_e4m3x2<TM>(x01 >> 16),
                                        widen_e4m3x2<TM>(y01 & 0xffffu), widen_e4m3x2<TM>(y01 >> 16)};
                const uint32_t a1[4] = {widen_e4m3x2<TM>(x23 & 0xffffu), widen_e4m3x2<TM>(x23 >> 16),
                                        widen_e4m3x2<TM>(y23 & 0xffffu), widen_e4m3x2<TM>(y23 >> 16)};
#pragma unroll
                for (int u = 0; u < SW; ++u) {
                    mma16816<TM>(o[8 * u + 2 * i], a0, pb[u][0], pb[u][1]);
                    mma16816<TM>(o[8 * u + 2 * i + 1], a1, pb[u][0], pb[u][1]);
                }
            }
        } else {
            float sc[NT][4];
            float iv[SCL ? NT : 1];  // 1 / V scale of each 8-key score tile
#pragma unroll
            for (int i = 0; i < NT; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
            if constexpr (KV8) {
                // key kw0 + 8nt + g: its 32 bytes at dims 32c .. 32c + 31 hold the
                // B fragments of all eight k-steps (see the Q fragments)
                const int g8 = lane >> 2, c8 = lane & 3;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int row = kw0 + nt * 8 + g8;
                    const uint4 u0 = *reinterpret_cast<const uint4 *>(k8 + swz8(row, 2 * c8));
                    const uint4 u1 = *reinterpret_cast<const uint4 *>(k8 + swz8(row, 2 * c8 + 1));
                    const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma16816<TM>(sc[nt], qa[kk], widen_e4m3x2<TM>(w[kk] & 0xffffu), widen_e4m3x2<TM>(w[kk] >> 16));
                }
            } else {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
#pragma unroll
                for (int np = 0; np < NT / 2; ++np) {
                    uint32_t bf[4];
                    int key = kw0 + np * 16 + (lane & 7) + ((lane >> 4) << 3);
                    ldsm_x4(bf, kb + swz(key, 2 * kk + ((lane >> 3) & 1), kDecRowBytes));
                    mma16816<TM>(sc[2 * np], qa[kk], bf[0], bf[1]);
                    mma16816<TM>(sc[2 * np + 1], qa[kk], bf[2], bf[3]);
                }
            }
            }

            const bool interior = !any_bad[kg] && (j0 >= lo_max || (FIRST && j0 + kDecTile <= p.first_tokens)) &&
                                  j0 + kDecTile - 1 <= hi_min;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float km = scale_log2, lv = 0.f;
                if constexpr (SCL) {
                    const float2 f = scales_of(j0, j0 + kw0 + nt * 8);
                    km = f.x * scale_log2;
                    lv = fast_log2(f.y);
                    iv[nt] = fast_rcp(f.y);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = SCL ? fmaf(sc[nt][e], km, lv) : sc[nt][e] * scale_log2;
                    if (!interior) {
                        int jj = kw0 + nt * 8 + 2 * (lane & 3) + (e & 1);
                        int j = j0 + jj;
                        bool vis = kvalid[stage * kDecTile + jj] &&
                                   (e < 2 ? (from(j, lo0) && j <= pos0) : (from(j, lo1) && j <= pos1));
                        if (!vis) x = -INFINITY;
                    }
                    sc[nt][e] = x;
                }
            }
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mx0 = fmaxf(mx0, fmaxf(sc[nt][0], sc[nt][1]));
                mx1 = fmaxf(mx1, fmaxf(sc[nt][2], sc[nt][3]));
            }
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
            // the running max rises only when a tile's exceeds it by more than 8
            // (a factor 2^8; from -inf at the first key): P stays below 2^8 and
            // O is rarely rescaled
            const float mn0 = mx0 > m0 + 8.f ? mx0 : m0, mn1 = mx1 > m1 + 8.f ? mx1 : m1;
            const float base0 = mn0 == -INFINITY ? 0.f : mn0;
            const float base1 = mn1 == -INFINITY ? 0.f : mn1;
            const float al0 = fast_exp2(m0 - base0), al1 = fast_exp2(m1 - base1);
            float rs0 = 0.f, rs1 = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                sc[nt][0] = fast_exp2(sc[nt][0] - base0);
                sc[nt][1] = fast_exp2(sc[nt][1] - base0);
                sc[nt][2] = fast_exp2(sc[nt][2] - base1);
                sc[nt][3] = fast_exp2(sc[nt][3] - base1);
                if constexpr (SCL) {
                    rs0 = fmaf(sc[nt][0] + sc[nt][1], iv[nt], rs0);
                    rs1 = fmaf(sc[nt][2] + sc[nt][3], iv[nt], rs1);
                } else {
                    rs0 += sc[nt][0] + sc[nt][1];
                    rs1 += sc[nt][2] + sc[nt][3];
                }
            }
            l0 = l0 * al0 + rs0;
            l1 = l1 * al1 + rs1;
            m0 = mn0;
            m1 = mn1;
            if (__any_sync(0xffffffffu, al0 != 1.f || al1 != 1.f)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][0] *= al0;
                    o[i][1] *= al0;
                    o[i][2] *= al1;
                    o[i][3] *= al1;
                }
            }
#pragma unroll
            for (int ks = 0; ks < NT / 2; ++ks) {
                uint32_t a[4];
                a[0] = pack2<TM>(sc[2 * ks][0], sc[2 * ks][1]);
                a[1] = pack2<TM>(sc[2 * ks][2], sc[2 * ks][3]);
                a[2] = pack2<TM>(sc[2 * ks + 1][0], sc[2 * ks + 1][1]);
                a[3] = pack2<TM>(sc[2 * ks + 1][2], sc[2 * ks + 1][3]);
                if constexpr (KV8) {
                    // The output dims are permuted too: column g of n-tile nt is
                    // dim 16g + nt, so the lane's 16 bytes of the keys 2c, 2c+1,
                    // 2c+8, 2c+9 feed all 16 n-tiles, the two keys of a B
                    // register interleaved byte by byte.
                    const int g8 = lane >> 2, rb = kw0 + ks * 16 + 2 * (lane & 3);
                    const uint4 x0 = *reinterpret_cast<const uint4 *>(v8 + swz8(rb, g8));
                    const uint4 x1 = *reinterpret_cast<const uint4 *>(v8 + swz8(rb + 1, g8));
                    const uint4 y0 = *reinterpret_cast<const uint4 *>(v8 + swz8(rb + 8, g8));
                    const uint4 y1 = *reinterpret_cast<const uint4 *>(v8 + swz8(rb + 9, g8));
                    const uint32_t X0[4] = {x0.x, x0.y, x0.z, x0.w}, X1[4] = {x1.x, x1.y, x1.z, x1.w};
                    const uint32_t Y0[4] = {y0.x, y0.y, y0.z, y0.w}, Y1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t p01 = __byte_perm(X0[i], X1[i], 0x5140), p23 = __byte_perm(X0[i], X1[i], 0x7362);
                        const uint32_t q01 = __byte_perm(Y0[i], Y1[i], 0x5140), q23 = __byte_perm(Y0[i], Y1[i], 0x7362);
                        mma16816<TM>(o[4 * i], a, widen_e4m3x2<TM>(p01 & 0xffffu), widen_e4m3x2<TM>(q01 & 0xffffu));
                        mma16816<TM>(o[4 * i + 1], a, widen_e4m3x2<TM>(p01 >> 16), widen_e4m3x2<TM>(q01 >> 16));
                        mma16816<TM>(o[4 * i + 2], a, widen_e4m3x2<TM>(p23 & 0xffffu), widen_e4m3x2<TM>(q23 & 0xffffu));
                        mma16816<TM>(o[4 * i + 3], a, widen_e4m3x2<TM>(p23 >> 16), widen_e4m3x2<TM>(q23 >> 16));
                    }
                } else {
                    const int key = kw0 + ks * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
                    for (int dp = 0; dp < 8; ++dp) {
                        uint32_t vf[4];
                        ldsm_x4_t(vf, vb + swz(key, 2 * dp + (lane >> 4), kDecRowBytes));
                        mma16816<TM>(o[2 * dp], a, vf[0], vf[1]);
                        mma16816<TM>(o[2 * dp + 1], a, vf[2], vf[3]);
                    }
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    pdl_launch_dependents();  // the merge kernel may get ready; it waits for this grid

    // combine the key groups of this CTA through shared memory
    if constexpr (SW > 0) {  // a row's keys are spread over the lanes of one c
#pragma unroll
        for (int u = 0; u < SW; ++u)
#pragma unroll
            for (int o_ = 4; o_ < 32; o_ <<= 1) {
                ls[u][0] += __shfl_xor_sync(0xffffffffu, ls[u][0], o_);
                ls[u][1] += __shfl_xor_sync(0xffffffffu, ls[u][1], o_);
            }
    } else {
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    }
    float *comb_o = reinterpret_cast<float *>(smem);  // [NKG][ROWS][128]
    if constexpr (SW > 0) {
        // lane (g, c) holds rows 8u + 2c and 8u + 2c + 1 at dims 16g .. 16g + 15:
        // o[8u + i][0 / 1] at dim 16g + 2i, o[8u + i][2 / 3] at dim 16g + 2i + 1
        const int g = lane >> 2;
#pragma unroll
        for (int u = 0; u < SW; ++u) {
            const int w = kg * ROWS + 8 * u + sr0;
            float *w0 = &comb_o[w * kDecD + 16 * g], *w1 = w0 + kDecD;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = 8 * u + 2 * q;
                *reinterpret_cast<float4 *>(w0 + 4 * q) = make_float4(o[i][0], o[i][2], o[i + 1][0], o[i + 1][2]);
                *reinterpret_cast<float4 *>(w1 + 4 * q) = make_float4(o[i][1], o[i][3], o[i + 1][1], o[i + 1][3]);
            }
            if (g == 0) {
                comb_m[w] = ms[u][0] == kNoKey ? -INFINITY : ms[u][0];
                comb_l[w] = ls[u][0];
                comb_m[w + 1] = ms[u][1] == kNoKey ? -INFINITY : ms[u][1];
                comb_l[w + 1] = ls[u][1];
            }
        }
    } else if constexpr (KV8) {
        // undo the output permutation: o[nt][e] is dim 16 (2c + (e & 1)) + nt
        const int d0 = 32 * (lane & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float *w0 = &comb_o[(kg * ROWS + r0) * kDecD + d0 + 4 * i];
            float *w1 = &comb_o[(kg * ROWS + r1) * kDecD + d0 + 4 * i];
            *reinterpret_cast<float4 *>(w0) = make_float4(o[4 * i][0], o[4 * i + 1][0], o[4 * i + 2][0], o[4 * i + 3][0]);
            *reinterpret_cast<float4 *>(w0 + 16) = make_float4(o[4 * i][1], o[4 * i + 1][1], o[4 * i + 2][1], o[4 * i + 3][1]);
            *reinterpret_cast<float4 *>(w1) = make_float4(o[4 * i][2], o[4 * i + 1][2], o[4 * i + 2][2], o[4 * i + 3][2]);
            *reinterpret_cast<float4 *>(w1 + 16) = make_float4(o[4 * i][3], o[4 * i + 1][3], o[4 * i + 2][3], o[4 * i + 3][3]);
        }
    } else {
#pragma unroll
        for (int nd = 0; nd < 16; ++nd) {
            int d = nd * 8 + 2 * (lane & 3);
            *reinterpret_cast<float2 *>(&comb_o[(kg * ROWS + r0) * kDecD + d]) = make_float2(o[nd][0], o[nd][1]);
            *reinterpret_cast<float2 *>(&comb_o[(kg * ROWS + r1) * kDecD + d]) = make_float2(o[nd][2], o[nd][3]);
        }
    }
    if (SW == 0 && (lane & 3) == 0) {
        comb_m[kg * ROWS + r0] = m0;
        comb_l[kg * ROWS + r0] = l0;
        comb_m[kg * ROWS + r1] = m1;
        comb_l[kg * ROWS + r1] = l1;
    }
    __syncthreads();

    for (int idx = tid; idx < R * 32; idx += kDecThreads) {
        const int r = idx >> 5, d = (idx & 31) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int g = 0; g < NKG; ++g) M = fmaxf(M, comb_m[g * ROWS + r]);
        const float Mb = M == -INFINITY ? 0.f : M;
        float lsum = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
        for (int g = 0; g < NKG; ++g) {
            float w = fast_exp2(comb_m[g * ROWS + r] - Mb);
            lsum += w * comb_l[g * ROWS + r];
            float4 x = *reinterpret_cast<const float4 *>(&comb_o[(g * ROWS + r) * kDecD + d]);
            a0 += w * x.x;
            a1 += w * x.y;
            a2 += w * x.z;
            a3 += w * x.w;
        }
        const int t = r / p.group, i = r - t * p.group, h = kvh * p.group + i;
        if (n_split == 1) {
            float sc_o, lse_v;
            if (p.sinks) {
                const float sk = p.sinks[h] * kLog2e;
                const float Mf = fmaxf(M, sk);
                const float wk = fast_exp2(M - Mf);
                const float den = lsum * wk + fast_exp2(sk - Mf);
                sc_o = bmm2 * wk / den;
                lse_v = (Mf + fast_log2(den)) * kLn2;
            } else if (lsum > 0.f) {
                sc_o = bmm2 / lsum;
                lse_v = (M + fast_log2(lsum)) * kLn2;
            } else {
                sc_o = 0.f;
                lse_v = -INFINITY;
            }
            if (EXT && lsum != lsum) sc_o = lse_v = lsum;  // a NaN among the visible keys
            const int64_t orow = (qrow0 + t) * p.Hqo + h;
            if (dbg_in(orow * kDecD + d, 4, p.num_tokens * p.Hqo * kDecD, p.err))
                store4(static_cast<T *>(p.out) + orow * kDecD + d, a0 * sc_o, a1 * sc_o, a2 * sc_o, a3 * sc_o);
            if (p.lse && d == 0) p.lse[orow] = lse_v;
        } else {
            const int64_t prow =
                (static_cast<int64_t>(b * p.Hkv + kvh) * p.n_split_max + s) * p.R + r;
            const float inv = lsum > 0.f ? 1.f / lsum : (EXT && lsum != lsum ? lsum : 0.f);
            if (dbg_in(prow, 1, p.ws_rows, p.err)) {
                *reinterpret_cast<float4 *>(p.ws_o + prow * kDecD + d) =
                    make_float4(a0 * inv, a1 * inv, a2 * inv, a3 * inv);
                if (d == 0) p.ws_lse[prow] = lsum > 0.f ? M + fast_log2(lsum) : (EXT && lsum != lsum ? lsum : -INFINITY);
            }
        }
    }
}

// One warp per output row (b*Q + t, h): weights the split partials by
// 2^lse_s, adds the sink to the denominator, applies bmm2_scale.
template <typename T, bool FIRST = false>
__global__ void __launch_bounds__(128) decode_merge_kernel(const DecodeParams p) {
    pdl_wait();  // the split kernel's partials
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + warp;
    if (row >= static_cast<int64_t>(p.B) * p.Q * p.Hqo) return;
    const int h = static_cast<int>(row % p.Hqo);
    const int64_t bq = row / p.Hqo;
    const int t = static_cast<int>(bq % p.Q), b = static_cast<int>(bq / p.Q);
    int Q = p.Q;
    int64_t qrow0 = static_cast<int64_t>(b) * p.Q;
    if (p.cu_q) {  // the split kernel flagged inconsistent entries; skip them the same way
        const int c0 = p.cu_q[b], c1 = p.cu_q[b + 1];
        Q = c1 - c0;
        qrow0 = c0;
        if (c0 < 0 || Q < 0 || Q > p.Q || c1 > p.num_tokens) Q = 0;
    }
    if (t >= Q) return;
    const uint32_t L_in = p.seq_lens[b];
    const int L = L_in > static_cast<uint32_t>(p.max_seq_len) ? p.max_seq_len : static_cast<int>(L_in);
    int lo, first, n_split;
    if constexpr (FIRST)
        n_split = decode_run(L, Q, p.window_left, p.first_tokens, p.chunk).n_split;
    else
        decode_split_geometry(L, Q, p.window_left, p.chunk, lo, first, n_split);
    if (n_split <= 1) return;  // the split kernel wrote this row itself
    const int kvh = h / p.group;
    const int r = t * p.group + (h - kvh * p.group);
    const int64_t base = static_cast<int64_t>(b * p.Hkv + kvh) * p.n_split_max * p.R + r;
    float M = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
    if (!dbg_in(base, static_cast<int64_t>(n_split - 1) * p.R + 1, p.ws_rows, p.err) ||
        !dbg_in(n_split, 0, p.n_split_max, p.err))
        return;
    float nan = 0.f;
    for (int s = 0; s < n_split; ++s) {
        const float x = p.ws_lse[base + static_cast<int64_t>(s) * p.R];
        M = fmaxf(M, x);
        if (FIRST && x != x) nan = x;
    }
    const int d = lane * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
    if (M != -INFINITY) {
        for (int s = 0; s < n_split; ++s) {
            const int64_t prow = base + static_cast<int64_t>(s) * p.R;
            const float w = fast_exp2(p.ws_lse[prow] - M);
            const float4 x = *reinterpret_cast<const float4 *>(p.ws_o + prow * kDecD + d);
            den += w;
            acc.x += w * x.x;
            acc.y += w * x.y;
            acc.z += w * x.z;
            acc.w += w * x.w;
        }
        if (p.sinks) den += fast_exp2(p.sinks[h] * kLog2e - M);
    }
    const float bmm2 = p.bmm2_dev ? __ldg(p.bmm2_dev) : p.bmm2;
    float sc = den > 0.f ? bmm2 / den : 0.f;
    float lse_v = den > 0.f ? (M + fast_log2(den)) * kLn2 : -INFINITY;
    if (FIRST && nan != nan) sc = lse_v = nan;  // a NaN among the visible keys
    const int64_t orow = (qrow0 + t) * p.Hqo + h;
    if (!dbg_in(orow * kDecD + d, 4, p.num_tokens * p.Hqo * kDecD, p.err)) return;
    store4(static_cast<T *>(p.out) + orow * kDecD + d, acc.x * sc, acc.y * sc, acc.z * sc, acc.w * sc);
    if (p.lse && lane == 0) p.lse[orow] = lse_v;
}

struct DecodePlan {
    int R, MT, chunk, n_split_max;
    size_t ws_o_bytes, ws_bytes;
};

static int plan_decode(int B, int Q, int Hqo, int Hkv, int D, int max_seq_len, int page_size,
                       int window_left, DecodePlan &pl, bool kv8 = false, int first_tokens = 0) {
    if (B < 0 || Q < 1 || Hqo < 1 || Hkv < 1 || max_seq_len < 0 || window_left < -1 || first_tokens < 0)
        return PKV_ERR_INVALID_ARG;
    if (Hqo % Hkv) return PKV_ERR_INVALID_ARG;
    if (B > 65535 || Hkv > 65535) return PKV_ERR_UNSUPPORTED;
    if (D != kDecD) return PKV_ERR_UNSUPPORTED;
    if (ilog2_exact(page_size) < 0 || page_size < kDecMinPage || page_size > 256) return PKV_ERR_UNSUPPORTED;
    const int group = Hqo / Hkv;
    pl.R = group * Q;
    if (pl.R > 64) return PKV_ERR_UNSUPPORTED;
    pl.MT = pl.R <= 16 ? 1 : (pl.R <= 32 ? 2 : 4);
    // keys of the longest request that some query sees (the first tokens in
    // whole tiles)
    const int64_t seen = static_cast<int64_t>(window_left) + Q +
                         (static_cast<int64_t>(first_tokens) + kDecTile - 1) / kDecTile * kDecTile;
    const int64_t span = window_left >= 0 && seen < max_seq_len ? seen : max_seq_len;
    // Larger row groups write larger partials: scale the chunk with R so the
    // partial traffic stays a few percent of the K/V bytes; then shrink it
    // while the grid would leave SMs idle.
    int chunk = 128 * pl.R;
    chunk = chunk < 1024 ? 1024 : (chunk > 4096 ? 4096 : chunk);
    // an E4M3 cache moves half the bytes per key: twice the keys per split
    // keep the per-CTA set-up and partial traffic at the same share
    if (kv8) chunk = 2 * chunk > 4096 ? 4096 : 2 * chunk;
    chunk = (chunk + kDecTile - 1) / kDecTile * kDecTile;
    // a window a little longer than the chunk (its first key need not sit on
    // a tile edge: up to 63 keys more) takes one split rather than a second,
    // nearly empty one
    const int64_t span_t = window_left >= 0 ? span + kDecTile - 1 : span;
    if (window_left >= 0 && span_t > chunk && span_t <= chunk + chunk / 4 && span_t <= kDecMaxChunk)
        chunk = static_cast<int>((span_t + kDecTile - 1) / kDecTile * kDecTile);
    const int64_t want = 2LL * num_sms();
    while (chunk > 4 * kDecTile &&
           static_cast<int64_t>(B) * Hkv * ((span + chunk - 1) / chunk) < want)
        chunk = (chunk / 2 + kDecTile - 1) / kDecTile * kDecTile;  // (tile multiples)
    pl.chunk = chunk;
    int64_t ns = span > 0 ? (span_t + chunk - 1) / chunk : 1;
    if (ns > 65535) return PKV_ERR_UNSUPPORTED;
    pl.n_split_max = static_cast<int>(ns);
    if (pl.n_split_max > 1) {
        const size_t slots = static_cast<size_t>(B) * Hkv * pl.n_split_max * pl.R;
        pl.ws_o_bytes = round_up(slots * kDecD * sizeof(float), 256);
        pl.ws_bytes = pl.ws_o_bytes + round_up(slots * sizeof(float), 256);
    } else {
        pl.ws_o_bytes = pl.ws_bytes = 0;
    }
    return PKV_OK;
}

template <typename T, int MT, int LAYOUT, bool KV8, int SW = 0, int EXT = 0>
static int launch_split(const DecodeParams &p, dim3 grid, cudaStream_t st, bool pdl) {
    constexpr int ROWS = DecCfg<MT, KV8, SW>::ROWS, NKG = 4 / MT;
    constexpr int kDecStages = DecCfg<MT, KV8, SW>::STAGES;
    const size_t smem = kDecStages * DecSmem<KV8>::STAGE + ROWS * kDecRowBytes +
                        kDecStages * kDecTile + 2 * NKG * ROWS * sizeof(float) +
                        (EXT ? p.pages_cap : kDecMaxPages) * sizeof(int) +
                        (EXT == 2 ? p.scales_cap * sizeof(float2) : 0);
    auto kern = decode_split_kernel<T, MT, LAYOUT, KV8, SW, EXT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem)) != cudaSuccess)
        return PKV_ERR_CUDA;
    if (pdl) return launch_dependent(kern, grid, dim3(kDecThreads), smem, st, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    kern<<<grid, kDecThreads, smem, st>>>(p);
    return PKV_OK;
}

template <typename T, int LAYOUT, bool KV8, int EXT = 0>
static int launch_split_mt(int MT, const DecodeParams &p, dim3 grid, cudaStream_t st, bool pdl) {
    if constexpr (KV8) {
        if (p.R <= 8) return launch_split<T, 1, LAYOUT, true, 1, EXT>(p, grid, st, pdl);  // swapped operands
        if constexpr (EXT > 0) {
            if (p.R <= 16) return launch_split<T, 1, LAYOUT, true, 2, EXT>(p, grid, st, pdl);
            if (p.R <= 32) return launch_split<T, 1, LAYOUT, true, 4, EXT>(p, grid, st, pdl);
        }
    }
    if constexpr (EXT == 0 || !KV8) {
        if (MT == 1) return launch_split<T, 1, LAYOUT, KV8, 0, EXT>(p, grid, st, pdl);
        if (MT == 2) return launch_split<T, 2, LAYOUT, KV8, 0, EXT>(p, grid, st, pdl);
    }
    return launch_split<T, 4, LAYOUT, KV8, 0, EXT>(p, grid, st, pdl);
}

// The split kernel under a window with first tokens and / or over a cache
// with block scales, and its merge (instantiated in decode_window.cu).
int run_decode_ext(const DecodeParams &p, const DecodePlan &pl, int layout, bool bf16, bool kv8, bool pdl,
                   cudaStream_t st);

template <typename T>
static int run_decode(const DecodeParams &p, const DecodePlan &pl, int layout, bool kv8, bool pdl,
                      cudaStream_t st) {
    dim3 grid(pl.n_split_max, p.Hkv, p.B);
    int rc = kv8 ? (layout == PKV_HND ? launch_split_mt<T, PKV_HND, true>(pl.MT, p, grid, st, pdl)
                                      : launch_split_mt<T, PKV_NHD, true>(pl.MT, p, grid, st, pdl))
                 : (layout == PKV_HND ? launch_split_mt<T, PKV_HND, false>(pl.MT, p, grid, st, pdl)
                                      : launch_split_mt<T, PKV_NHD, false>(pl.MT, p, grid, st, pdl));
    if (rc != PKV_OK) return rc;
    int launches = 1;
    if (pl.n_split_max > 1) {
        int64_t rows = static_cast<int64_t>(p.B) * p.Q * p.Hqo;
        if (launch_dependent(decode_merge_kernel<T>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
                             st, p) != cudaSuccess)
            return PKV_ERR_CUDA;
        ++launches;
    }
    note_launches(launches);
    return launch_status();
}

}  // namespace pkv
