// shared_own.cuh -- the own keys of a shared decode: every (request, kv head)
// and split of its keys is an item of a few tiles, streamed once from HBM.
//
// Own keys are short (a few hundred beside prefixes of thousands), so what an
// item costs around its bytes counts: its length, page ids and queries, the
// latency of its first tile.  A producer warp therefore runs ahead of the items:
// it takes over the grid's CTAs that have not begun (cluster launch control),
// looks their lengths and pages up and keeps a ring of K / V tiles filled by TMA
// across item boundaries, while four warps compute.  Two CTAs per SM, 64 KB to
// 96 KB in flight each.  A TMA box is both halves of the head of up to 64 slots:
// two boxes of one half each took the copy engine almost twice as long.  The
// issue of a box takes about 200 cycles (pages of 16 slots: 8 boxes a tile), so
// that V's are another warp's.
//
// The four warps share an item.  Scores of a tile: 16 keys a warp, all R =
// group * Q rows (padded to 16 MT) as the MMA's row side; the tile's row maxima
// through shared memory; P, rounded to the caches' type, through shared memory;
// then 32 output dimensions a warp over the tile's 64 keys, so that a row's
// output needs no reduction over warps at the item's end.  Every item's rows go
// to partials, so that no item waits for the prefix, and shared_merge_kernel
// joins them with the prefix's.
//
// Alone on all SMs: 278 MB of 256 requests' 265 keys in 55 us (5.1 TB/s, 74% of
// the copy rate), 147 MB of 64 requests' 560 in 33: the first tile comes after
// 4 us (length, page ids, data), the last items end unevenly, and an item's
// claim takes 1 to 2 us.  Beside the prefix an SM streams 35 to 45 GB/s.  Items
// are cut for the caller's largest length: where it is far above the lengths,
// splits are longer than they should be and empty items are claimed one by one
// (64 requests' 560 keys beside a prefix of 8,192: 46 us for a largest of 1,019,
// 55 for 32,768, 76 for 131,072).
//
// Every wait is bounded; a warp whose wait ran out says so in the barrier that
// all four meet at next, so that they leave together, and each of the two warps
// that issue copies waits for its own to land.
#pragma once

#include "attn_tile.cuh"
#include "shared_prefix.cuh"
#include "sm103_ptx.cuh"

namespace pkv {

constexpr int kOwnTile = 64;      // keys per ring stage
constexpr int kOwnThreads = 192;  // four warps, the producer, its second for V
constexpr uint32_t kOwnBytes = kOwnTile * 256;  // a tile's K or V

template <int MT>
struct OwnCfg {
    static constexpr int ROWS = 16 * MT;
    static constexpr int STAGES = MT == 4 ? 2 : 3;
    static constexpr uint32_t Q = STAGES * 2 * kOwnBytes, P = Q + ROWS * 256, RED = P + ROWS * 128;
    static constexpr uint32_t SMEM = 1024 + RED + 8 * ROWS * 4;
};

struct OwnParams {
    PrefixWork prefix;
    const int32_t *block_tables;
    int64_t bt_stride;
    int64_t max_num_pages;
    float scale_log2;
    const float *bmm1_dev, *bmm2_dev;
    float bmm2;
    const float *sinks;
    int R, page_shift, chunk, n_split_max;
    int ratio;  // see SharedParams
    void *out;
    float *lse;
    int merge_rows;  // most rows of a warp of the merge kernel
    int32_t *err;
    unsigned long long wait_ns;
};

// K or V cache, where the prefix kernel's wide map is not possible, as a 5-D
// map (64 dimensions, slots, the two halves of a head,
// heads, pages) whose box is `rows` slots of one head: 64 dimensions of each,
// then the other 64.
inline bool own_tmap(CUtensorMap *m, const void *base, CUtensorMapDataType t, int layout, int page_size, int heads,
                     int64_t page_stride, int64_t pages, int rows) {
    const uint64_t row = layout == PKV_HND ? 256 : 256ull * heads, head = layout == PKV_HND ? 256ull * page_size : 256;
    const uint64_t dims[5] = {64, static_cast<uint64_t>(page_size), 2, static_cast<uint64_t>(heads), static_cast<uint64_t>(pages)};
    const uint64_t strides[4] = {row, 128, head, static_cast<uint64_t>(page_stride) * 2};
    const uint32_t box[5] = {64, static_cast<uint32_t>(rows), 2, 1, 1};
    return encode_tmap(m, base, t, 5, dims, strides, box);
}

__host__ __device__ inline int own_splits(int L, int chunk) { return L <= 0 ? 1 : (L + chunk - 1) / chunk; }
// Where row r of an item goes: [B][Hkv][n_split_max][R] behind the prefix's partials.
__device__ __forceinline__ uint32_t own_part(const OwnParams &p, int b, int kvh, int s, int r) {
    return p.prefix.parts + ((static_cast<uint32_t>(b) * p.prefix.Hkv + kvh) * p.n_split_max + s) * p.R + r;
}

// The rest of a row once its maximum M (base 2) and sum den are known: what the
// output is multiplied by, and its LSE.
__device__ __forceinline__ float finish_row(const OwnParams &p, int h, float M, float den, float &lse) {
    const float bmm2 = p.bmm2_dev ? __ldg(p.bmm2_dev) : p.bmm2;
    float up = 1.f;
    if (p.sinks) {
        const float sink = p.sinks[h] * kLog2e, top = fmaxf(M, sink);
        if (top != -INFINITY) {
            up = fast_exp2(M - top);
            den = den * up + fast_exp2(sink - top);
            M = top;
        }
    }
    if (den > 0.f) {
        lse = (M + fast_log2(den)) * kLn2;
        return bmm2 * up / den;
    }
    lse = den != den ? den : -INFINITY;  // a NaN among the visible keys; no key
    return den != den ? den : 0.f;
}

// What the producer says of a ring stage.
struct OwnStage {
    int b, kvh, s, L, key0;
    int first, last, end;  // of the item; end: nothing follows
    uint32_t valid[2];     // keys of the tile that exist
    int pages[8];          // of its boxes; pages[0] < 0: no key, nothing to copy
};

// Takes over a CTA of the grid that has not begun: the answer, 16 bytes, comes
// on `bar`; then its index, or false (nothing is left: ask no more).
__device__ __forceinline__ void cta_request(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(
                     answer),
                 "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool cta_answer(uint32_t answer, int &x, int &y, int &z) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .b128 h;\n .reg .pred p;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n"
        " ld.shared.b128 h, [%4];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %3, 1, 0, p;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, %2, _}, h;\n}\n"
        : "=&r"(x), "=&r"(y), "=&r"(z), "=&r"(ok)
        : "r"(answer)
        : "memory");
    return ok != 0;
}

// Barrier of the four computing warps that tells each whether all say yes.
__device__ __forceinline__ bool own_sync(bool yes) {
    uint32_t all;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, 1, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(all)
        : "r"(yes ? 1u : 0u)
        : "memory");
    return all != 0;
}

// The newest keys of a tile, of which token t sees those up to pos + t, `left`
// of the tile being the request's: the weights of hidden ones are 0, and 0 times
// a NaN or an infinity is not 0.  Values that are neither are left to the MMA;
// the others (drafts gone wrong; hardly ever one) are multiplied here for the
// rows that see them and zeroed.  A warp does its own 32 dimensions, from which
// no other reads; true if it wrote zeros.
template <typename T, int MT, typename At>
__device__ __forceinline__ bool hidden_values(uint8_t *v, const uint8_t *weights, At at, const int (&tq)[MT][2], int pos, int left,
                                              float (&o)[MT][4][4]) {
    constexpr uint32_t kExp = IsBf16<T>::value ? 0x7f80u : 0x7c00u;  // the exponent of one that is not finite
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int j0 = max(pos + 1, 0), j1 = min(left, kOwnTile);
    auto word = [&](int j, int n) { return reinterpret_cast<uint32_t *>(v + at(j, 4 * warp + n) + 4 * c); };
    auto odd = [&](uint32_t x) { return (x & kExp) == kExp; };
    bool any = false;
    for (int j = j0 + g; j < j1; j += 8)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const uint32_t x = *word(j, n);
            any |= odd(x) || odd(x >> 16);
        }
    if (!__any_sync(0xffffffffu, any)) return false;
#pragma unroll 1
    for (int j = j0; j < j1; ++j)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                if (j > pos + tq[mt][f]) continue;
                const int row = 16 * mt + g + 8 * f;
                const T w = *reinterpret_cast<const T *>(weights + row * 128 + (((j >> 3) ^ (row & 7)) << 4) + 2 * (j & 7));
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t x = *word(j, n);
                    const float2 y = unpack2<T>(x);
                    if (odd(x)) o[mt][n][2 * f] += static_cast<float>(w) * y.x;
                    if (odd(x >> 16)) o[mt][n][2 * f + 1] += static_cast<float>(w) * y.y;
                }
            }
    __syncwarp();
    for (int j = j0 + g; j < j1; j += 8)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const uint32_t x = *word(j, n);
            if (odd(x) || odd(x >> 16)) *word(j, n) = (odd(x) ? 0u : x & 0xffffu) | (odd(x >> 16) ? 0u : x & 0xffff0000u);
        }
    __syncwarp();
    return true;
}

// DRAFTS: several tokens to a request, some of whose keys the others do not see.
// (A kernel of its own for one token: the code for several, which it never
// reaches, cost the smallest call 0.4 us of 10.9.  With it, three groups of
// requests of four tokens take the 43.3 us that they took without.)
template <typename T, int MT, bool DRAFTS>
__global__ void __launch_bounds__(kOwnThreads, 2)
    shared_own_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ OwnParams p) {
    using C = OwnCfg<MT>;
    constexpr int ST = C::STAGES, ROWS = C::ROWS;
    constexpr uint32_t STAGE = 2 * kOwnBytes;  // K then V
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t ring = smem_u32(smem), q_s = ring + C::Q, p_s = ring + C::P;
    float *red_m = reinterpret_cast<float *>(smem + C::RED), *red_l = red_m + 4 * ROWS;  // [warp][row]
    __shared__ __align__(8) uint64_t bars[4 * ST + 3];
    __shared__ __align__(16) uint4 answer_s;
    __shared__ OwnStage stage_s[ST];
    __shared__ int abort_s;
    auto b_full = [&](int s) { return smem_u32(&bars[s]); };            // K has landed, or nothing follows
    auto b_vfull = [&](int s) { return smem_u32(&bars[3 * ST + s]); };  // V has landed
    auto b_empty = [&](int s) { return smem_u32(&bars[ST + s]); };
    auto b_known = [&](int s) { return smem_u32(&bars[2 * ST + s]); };  // stage_s of a tile is written
    const uint32_t b_qfull = smem_u32(&bars[4 * ST]), b_qempty = smem_u32(&bars[4 * ST + 1]),
                   b_answer = smem_u32(&bars[4 * ST + 2]), answer = smem_u32(&answer_s);
    const PrefixWork &w = p.prefix;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();  // (the merge waits for this grid's end)
    volatile int *abort_flag = &abort_s;
    const uint64_t wlim = p.wait_ns;
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(b_full(s), 1);
            mbar_init(b_empty(s), 5);
            mbar_init(b_known(s), 1);
            mbar_init(b_vfull(s), 1);
        }
        mbar_init(b_qfull, 1);
        mbar_init(b_qempty, 4);
        mbar_init(b_answer, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    __syncthreads();
    auto give_up = [&]() {
        *abort_flag = 1;
        set_err(p.err, PKV_DEV_ERR_TIMEOUT);
    };

    if (warp == 4) {
        // ---- producer: ring stage of tile i (counted over the CTA's items): i % ST
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
        const int S = 1 << p.page_shift, RB = pf_box_rows(S, kOwnTile), nbox = kOwnTile / RB;
        const int oob = max(static_cast<int>(p.max_num_pages), 1);  // past the map: zero fill
        auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, wlim));
        };
        int s = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
        uint32_t L_in = p.prefix.seq_lens[b];
        int i = 0, items = 0;       // tiles put into the ring, items with queries
        int asked = 0, heard = 0;   // CTAs asked for, answers read
        bool more = true, ok = true;
        while (more && ok) {
            const int L = static_cast<int>(min(L_in, static_cast<uint32_t>(p.prefix.max_seq_len)));
            if (s == 0 && kvh == 0 && lane == 0) {
                if (L_in > static_cast<uint32_t>(p.prefix.max_seq_len)) set_err(p.err, PKV_DEV_ERR_LEN);
                if (L < w.Q) set_err(p.err, PKV_DEV_ERR_QLEN);
            }
            const int n_split = own_splits(L, p.chunk);
            const int k0 = s * p.chunk, k1 = min(L, k0 + p.chunk);
            const int n = s >= n_split ? 0 : max(1, (k1 - k0 + kOwnTile - 1) / kOwnTile);
            const int32_t *bt = p.block_tables + static_cast<int64_t>(b) * p.bt_stride;
            // pages of 32 boxes at a time, a lane each (-1: no key), the next 32 on the way
            auto lookup = [&](int j0) {
                const int key = k0 + (j0 + lane) * RB;
                const bool read = key < k1 && dbg_in(key >> p.page_shift, 1, (p.prefix.max_seq_len + S - 1) >> p.page_shift, p.err);
                return read ? bt[key >> p.page_shift] : -1;
            };
            int pages = -1, pages_next = n > 0 ? lookup(0) : -1;
            int ns = 0, nkvh = 0, nb = 0;
            uint32_t nL = 0;
            auto ask = [&]() {
                if (lane == 0) {
                    mbar_expect_tx(b_answer, 16);
                    cta_request(answer, b_answer);
                }
                ++asked;
            };
            auto hear = [&]() {
                if (!wait(b_answer, heard & 1)) return false;
                ++heard;
                more = cta_answer(answer, ns, nkvh, nb);
                fence_proxy_async_smem();  // (before the next answer overwrites this one)
                __syncwarp();
                if (more) nL = p.prefix.seq_lens[nb];
                return true;
            };
            for (int t = 0; t < n && ok; ++t, ++i) {
                const int st = i % ST, us = i / ST, j0 = (t * nbox) & 31;
                if (j0 == 0) {
                    pages = pages_next;
                    if (pages < 0 || pages >= p.max_num_pages) {
                        if (k0 + (t * nbox + lane) * RB < k1) set_err(p.err, PKV_DEV_ERR_PAGE);
                        pages = -1;
                    }
                    if ((t * nbox + 32) * RB < k1 - k0) pages_next = lookup(t * nbox + 32);
                }
                if (us > 0 && !wait(b_empty(st), (us - 1) & 1)) {
                    ok = false;
                    break;
                }
                // The next item, asked for three tiles before this one's end:
                // the answer takes 1 to 2 us; one taken earlier could wait here
                // while other CTAs have nothing left.
                if (t == max(0, n - 3)) ask();
                const int key0 = k0 + t * kOwnTile, left = k1 - key0;
                // keys of good pages, below the end: box j covers keys [j RB, (j + 1) RB)
                uint32_t valid[2] = {0u, 0u};
                const unsigned good = (__ballot_sync(0xffffffffu, pages >= 0) >> j0) & low_bits(nbox);
                for (int j = 0; j < nbox; ++j)
                    if ((good >> j) & 1u) {
                        const uint32_t bits = low_bits(RB);
                        if (RB == 64) valid[0] = valid[1] = 0xffffffffu;
                        else valid[(j * RB) >> 5] |= bits << ((j * RB) & 31);
                    }
                valid[0] &= low_bits(left);
                valid[1] &= low_bits(left - 32);
                const bool last = t + 1 == n;
                if (lane == 0) {
                    OwnStage &x = stage_s[st];
                    x.b = b;
                    x.kvh = kvh;
                    x.s = s;
                    x.L = L;
                    x.key0 = key0;
                    x.first = t == 0;
                    x.last = last;
                    x.end = 0;
                    x.valid[0] = valid[0];
                    x.valid[1] = valid[1];
                    mbar_expect_tx(b_full(st), good ? kOwnBytes : 0u);
                }
                const int box_page = __shfl_sync(0xffffffffu, pages, (j0 + lane) & 31);
                if (lane < nbox) stage_s[st].pages[lane] = good ? (box_page < 0 ? oob : box_page) : -1;
                __syncwarp();
                if (lane == 0) mbar_arrive(b_known(st));
                if (good) {
#pragma unroll 1
                    for (int j = 0; j < nbox; ++j) {
                        int page = __shfl_sync(0xffffffffu, pages, j0 + j);
                        if (page < 0) page = oob;
                        if (lane != 0) continue;
                        const int slot = (key0 + j * RB) & (S - 1);
                        if (kDebugBounds) {
                            dbg_in(page, 1, oob + 1, p.err);
                            dbg_in(slot, RB, S, p.err);
                        }
                        const uint32_t dst = ring + st * STAGE + j * RB * 256;
                        if (p.ratio) {  // (the prefix's maps: groups of 8 slots, (page, head))
                            tma_load_5d(dst, &tm_k, b_full(st), 0, 0, 0, slot >> 3, page * p.ratio + kvh);
                        } else {
                            tma_load_5d(dst, &tm_k, b_full(st), 0, slot, 0, kvh, page);
                        }
                    }
                }
                if (t == 0) {  // the item's queries, as soon as the ones before are read
                    ok = items == 0 || wait(b_qempty, (items - 1) & 1);
                    if (lane == 0 && ok) {
                        mbar_expect_tx(b_qfull, p.R * 256);
                        for (int c = 0; c < 2; ++c)
                            tma_load_3d(q_s + c * ROWS * 128, &tm_q, b_qfull, 64 * c, kvh * w.group, b * w.Q);
                    }
                    items += ok;
                }
                if (last && ok) ok = hear();
            }
            if (!ok) break;
            if (n == 0) {
                ask();
                ok = hear();
                if (!ok) break;
            }
            s = ns;
            kvh = nkvh;
            b = nb;
            L_in = nL;
        }
        if (ok) {  // nothing follows
            const int st = i % ST, us = i / ST;
            if (us > 0 && !wait(b_empty(st), (us - 1) & 1)) {
                ok = false;
            } else if (lane == 0) {
                stage_s[st].end = 1;
                mbar_arrive(b_known(st));
                mbar_arrive(b_full(st));
            }
        }
        if (!ok && lane == 0) give_up();
        __syncwarp();
        // every copy that this warp issued and the answer land before the CTA
        // exits (the tile whose stage the end took was consumed before)
        const int open = ok ? ST - 1 : ST;
        for (int t = i > open ? i - open : 0; t < i; ++t)
            if (!mbar_wait_drain(b_full(t % ST), (t / ST) & 1) && lane == 0) set_err(p.err, PKV_DEV_ERR_TIMEOUT);
        if (items > 0 && !mbar_wait_drain(b_qfull, (items - 1) & 1) && lane == 0) set_err(p.err, PKV_DEV_ERR_TIMEOUT);
        if (heard < asked && !mbar_wait_drain(b_answer, heard & 1) && lane == 0) set_err(p.err, PKV_DEV_ERR_TIMEOUT);
    } else if (warp == 5) {
        // ---- V's copies, of the tiles that the producer announces
        const int S = 1 << p.page_shift, RB = pf_box_rows(S, kOwnTile), nbox = kOwnTile / RB;
        int i = 0;  // tiles whose V is on its way
        for (;; ++i) {
            const int st = i % ST;
            const OwnStage &x = stage_s[st];
            if (!__all_sync(0xffffffffu, mbar_wait(b_known(st), (i / ST) & 1, abort_flag, wlim))) {
                if (lane == 0 && !*abort_flag) give_up();
                break;
            }
            const bool end = x.end;
            __syncwarp();  // (all lanes have read the record; from lane 0's arrival on it may be written again)
            if (end) break;
            if (lane != 0) continue;
            mbar_expect_tx(b_vfull(st), x.pages[0] >= 0 ? kOwnBytes : 0u);
#pragma unroll 1
            for (int j = 0; j < nbox && x.pages[0] >= 0; ++j) {
                const int slot = (x.key0 + j * RB) & (S - 1), page = x.pages[j];
                const uint32_t dst = ring + st * STAGE + kOwnBytes + j * RB * 256;
                if (p.ratio) tma_load_5d(dst, &tm_v, b_vfull(st), 0, 0, 0, slot >> 3, page * p.ratio + x.kvh);
                else tma_load_5d(dst, &tm_v, b_vfull(st), 0, slot, 0, x.kvh, page);
            }
            mbar_arrive(b_empty(st));  // (stage_s may be written again)
        }
        __syncwarp();
        // V's copies land before the CTA exits: this warp waits for those that
        // it issued, and for no tile that was announced after it gave up
        for (int t = i > ST ? i - ST : 0; t < i; ++t)
            if (!mbar_wait_drain(b_vfull(t % ST), (t / ST) & 1) && lane == 0) set_err(p.err, PKV_DEV_ERR_TIMEOUT);
    } else {
        // ---- the four computing warps; lane (g, c): rows 16 mt + g and + 8
        const int g = lane >> 2, c = lane & 3;
        const float sc = p.bmm1_dev ? __ldg(p.bmm1_dev) * kLog2e : p.scale_log2;
        auto wait_warp = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, wlim));
        };
        // 16 bytes `ch` of key `row` of a tile: 2^box_shift keys (a box's, or 8),
        // 64 dimensions of each, then the other 64
        const int box_shift = p.ratio ? 3 : min(p.page_shift, 6), box_low = (1 << box_shift) - 1;
        auto at = [&](int row, int ch) {
            return static_cast<uint32_t>(((row & ~box_low) << 8) + (ch >> 3 << (box_shift + 7)) + ((row & box_low) << 7) +
                                         (((ch & 7) ^ (row & 7)) << 4));
        };
        int tq[MT][2];  // the rows' tokens
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int f = 0; f < 2; ++f) tq[mt][f] = min((16 * mt + g + 8 * f) / w.group, w.Q - 1);
        uint32_t qa[MT == 1 ? 8 : 1][4];
        float m[MT][2], l[MT][2], o[MT][4][4];
        int items = 0;
        for (int i = 0;; ++i) {
            const int st = i % ST;
            const OwnStage &x = stage_s[st];
            const uint32_t k_s = ring + st * STAGE, v_s = k_s + kOwnBytes;
            bool ok = wait_warp(b_full(st), (i / ST) & 1);
            const bool end = ok && x.end;
            float sv[MT][2][4];
            bool whole = true, hides = false;
            if (ok && !end) {
                if (x.first) {
                    ok = wait_warp(b_qfull, items & 1);
                    ++items;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        m[mt][0] = m[mt][1] = -INFINITY;
                        l[mt][0] = l[mt][1] = 0.f;
#pragma unroll
                        for (int n = 0; n < 4; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
                    }
                }
                auto q_frag = [&](uint32_t (&a)[4], int mt, int kk) {
                    const int row = 16 * mt + (lane & 15), ch = 2 * kk + (lane >> 4);
                    ldsm_x4(a, q_s + (ch >> 3) * (ROWS * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
                };
                if constexpr (MT == 1) {
                    if (x.first) {
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) q_frag(qa[kk], 0, kk);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b_qempty);
                    }
                }
                // S = Q K^T of this warp's 16 keys
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int n = 0; n < 2; ++n) sv[mt][n][0] = sv[mt][n][1] = sv[mt][n][2] = sv[mt][n][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const int row = 16 * warp + (lane >> 4) * 8 + (lane & 7), ch = 2 * kk + ((lane >> 3) & 1);
                    uint32_t kb[4];
                    ldsm_x4(kb, k_s + at(row, ch));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        if constexpr (MT == 1) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) a[e] = qa[kk][e];
                        } else {
                            q_frag(a, mt, kk);
                        }
                        mma16816<T>(sv[mt][0], a, kb[0], kb[1]);
                        mma16816<T>(sv[mt][1], a, kb[2], kb[3]);
                    }
                }
                if constexpr (MT > 1) {
                    __syncwarp();
                    if (x.last && lane == 0) mbar_arrive(b_qempty);
                }
                const uint32_t v0 = x.valid[0], v1 = x.valid[1];
                whole = (v0 & v1) == 0xffffffffu;
                if constexpr (DRAFTS) hides = x.key0 + kOwnTile - 1 > x.L - w.Q;  // keys that some tokens do not see
                const bool plain = whole && x.key0 + kOwnTile - 1 <= x.L - w.Q;
                const uint32_t mine = (warp < 2 ? v0 : v1) >> (16 * (warp & 1));  // this warp's 16 keys
                const int pos = x.L - w.Q - x.key0 - 16 * warp;                   // token 0's newest key among them
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float top = -INFINITY;
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float &z = sv[mt][n][2 * f + e];
                                const int j = 8 * n + 2 * c + e;
                                z *= sc;
                                if (!plain && (!((mine >> j) & 1u) || j > pos + tq[mt][f])) z = -INFINITY;
                                top = fmaxf(top, z);
                            }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        if (c == 0) red_m[warp * ROWS + 16 * mt + g + 8 * f] = top;
                    }
                ok = wait_warp(b_vfull(st), (i / ST) & 1);
                // values of rows without a key may be anything: zeroed, so that P = 0 cannot make 0 * NaN
                if (ok && !whole)
                    for (int q = tid; q < kOwnTile * 16; q += 128) {
                        const int row = q >> 4, ch = q & 15;
                        if (!(((row < 32 ? v0 : v1) >> (row & 31)) & 1u))
                            *reinterpret_cast<uint4 *>(smem + st * STAGE + kOwnBytes + at(row, ch)) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
            }
            if (!own_sync(ok)) {
                if (!ok) give_up();
                break;
            }
            if (end) break;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int row = 16 * mt + g + 8 * f;
                    const float top = fmaxf(fmaxf(red_m[row], red_m[ROWS + row]), fmaxf(red_m[2 * ROWS + row], red_m[3 * ROWS + row]));
                    const float now = fmaxf(m[mt][f], top), base = now == -INFINITY ? 0.f : now;
                    const float keep = fast_exp2(m[mt][f] - base);
                    m[mt][f] = now;
                    l[mt][f] *= keep;
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        o[mt][n][2 * f] *= keep;
                        o[mt][n][2 * f + 1] *= keep;
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float p0 = fast_exp2(sv[mt][n][2 * f] - base), p1 = fast_exp2(sv[mt][n][2 * f + 1] - base);
                        l[mt][f] += p0 + p1;
                        *reinterpret_cast<uint32_t *>(smem + C::P + row * 128 + (((2 * warp + n) ^ (row & 7)) << 4) + 4 * c) =
                            pack2<T>(p0, p1);
                    }
                }
            named_bar_sync(1, 128);
            bool zeroed = false;
            if constexpr (DRAFTS)
                if (hides)
                    zeroed = hidden_values<T, MT>(smem + st * STAGE + kOwnBytes, smem + C::P, at, tq, x.L - w.Q - x.key0,
                                                  x.L - x.key0, o);
            // O += P V of this warp's 32 dimensions
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                uint32_t vb[2][4];
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    const int row = 16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7), ch = 4 * warp + 2 * h2 + (lane >> 4);
                    ldsm_x4_t(vb[h2], v_s + at(row, ch));
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t a[4];
                    const int row = 16 * mt + (lane & 15), ch = 2 * kk + (lane >> 4);
                    ldsm_x4(a, p_s + row * 128 + ((ch ^ (row & 7)) << 4));
#pragma unroll
                    for (int n = 0; n < 4; ++n) mma16816<T>(o[mt][n], a, vb[n >> 1][2 * (n & 1)], vb[n >> 1][2 * (n & 1) + 1]);
                }
            }
            const bool last = x.last;
            const int b = x.b, kvh = x.kvh, s = x.s;
            if (!whole || zeroed) fence_proxy_async_smem();  // (zeros written before the next copy into the stage)
            __syncwarp();
            if (lane == 0) mbar_arrive(b_empty(st));
            if (!last) continue;

            // ---- the item's end
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    l[mt][f] += __shfl_xor_sync(0xffffffffu, l[mt][f], 1);
                    l[mt][f] += __shfl_xor_sync(0xffffffffu, l[mt][f], 2);
                    if (c == 0) red_l[warp * ROWS + 16 * mt + g + 8 * f] = l[mt][f];
                }
            named_bar_sync(1, 128);
            const int d = 32 * warp + 2 * c;  // this lane's dimensions: d + 8 n, and the next
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int r = 16 * mt + g + 8 * f;
                    const uint32_t row = own_part(p, b, kvh, s, r);
                    if (r >= p.R || !dbg_in(row, 1, w.all, p.err)) continue;
                    const float den = (red_l[r] + red_l[ROWS + r]) + (red_l[2 * ROWS + r] + red_l[3 * ROWS + r]);
                    const float inv = den > 0.f ? 1.f / den : (den != den ? den : 0.f);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        *reinterpret_cast<float2 *>(w.ws_o + static_cast<size_t>(row) * 128 + d + 8 * n) =
                            make_float2(o[mt][n][2 * f] * inv, o[mt][n][2 * f + 1] * inv);
                    if (warp == 0 && c == 0)
                        w.ws_lse[row] = den > 0.f ? m[mt][f] + fast_log2(den) : (den != den ? den : -INFINITY);
                }
        }
    }
    pdl_wait();  // whoever waits for this grid waits for the one before it too
}

// A warp for up to `merge_rows` query heads of one token and kv head in turn:
// the partials of its request's own keys and of its group's prefix, and the
// sink.  Their rows lie one behind the other in every partial: where they are
// is worked out once, a partial to a lane, and a lane takes one partial's LSE
// and weight of a row too.  (A warp to a row, everything worked out by all of
// its lanes: 23 us for 16,384 rows of 5 partials, bound by instructions.)
template <typename T>
__global__ void __launch_bounds__(128) shared_merge_kernel(const __grid_constant__ OwnParams p) {
    const PrefixWork &w = p.prefix;
    const int lane = threadIdx.x & 31, subs = (w.group + p.merge_rows - 1) / p.merge_rows;
    const uint32_t at = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (at >= w.rows / w.group * subs) return pdl_wait();  // (rows / group: tokens * Hkv)
    const uint32_t unit = at / subs;
    const int i_first = static_cast<int>(at - unit * subs) * p.merge_rows, i_end = min(i_first + p.merge_rows, w.group);
    const int token = unit / w.Hkv, kvh = unit - token * w.Hkv, b = token / w.Q, t = token - b * w.Q;
    const int n_own = own_splits(static_cast<int>(min(w.seq_lens[b], static_cast<uint32_t>(w.max_seq_len))), p.chunk);
    PrefixGroup x;
    bool bad;
    scan_prefixes(w, [](uint32_t) {}, [=](int lo, int hi, uint32_t, uint32_t) { return lo <= b && b < hi; }, x, bad);
    if (w.ctas == 0 && at == 0) report_prefixes(w, bad);  // (max_prefix 0: no kernel over the prefixes does)
    const uint32_t own0 = own_part(p, b, kvh, 0, t * w.group);
    pdl_wait();
    const PrefixParts parts = prefix_parts(w, x, w.ctas > 0 ? *w.per : 1, token, kvh);
    const int n = n_own + parts.n;
    auto place = [&](int j) { return j < n_own ? own0 + static_cast<uint32_t>(j) * p.R : parts.at(j - n_own); };
    uint32_t mine = place(lane);
    for (int i = i_first; i < i_end; ++i) {
        float M = -INFINITY, den = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; j0 < n; j0 += 32) {
            const int m = min(n - j0, 32);
            if (n > 32) mine = place(j0 + lane);
            const bool in = lane < m && dbg_in(mine + i, 1, w.all, p.err);
            const float y = in ? w.ws_lse[mine + i] : -INFINITY;
            float keep = 0.f, u = 0.f;
            for (int k0 = 0; k0 < m; k0 += 8) {  // eight partials' loads in flight together
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t row = __shfl_sync(0xffffffffu, mine, k0 + k) + i;
                    v[k] = k0 + k < m && dbg_in(row, 1, w.all, p.err)
                               ? *reinterpret_cast<const float4 *>(w.ws_o + static_cast<size_t>(row) * 128 + lane * 4)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (k0 == 0) {  // the weights of all 32
                    float now = y;
#pragma unroll
                    for (int o = 16; o; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
                    now = fmaxf(now, M);
                    const float base = now == -INFINITY ? 0.f : now;
                    keep = fast_exp2(M - base);
                    u = fast_exp2(y - base);  // (a part's NaN stays)
                    M = now;
                    float sum = u;
#pragma unroll
                    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    den = den * keep + sum;
                    acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float f = __shfl_sync(0xffffffffu, u, k0 + k);
                    acc.x += f * v[k].x;
                    acc.y += f * v[k].y;
                    acc.z += f * v[k].z;
                    acc.w += f * v[k].w;
                }
            }
        }
        const int h = kvh * w.group + i;
        const size_t row = static_cast<size_t>(token) * w.Hqo + h;
        float lse;
        const float mul = finish_row(p, h, M, den, lse);
        uint2 out;
        out.x = pack2<T>(acc.x * mul, acc.y * mul);
        out.y = pack2<T>(acc.z * mul, acc.w * mul);
        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + row * 128 + lane * 4) = out;
        if (p.lse && lane == 0) p.lse[row] = lse;
    }
}

}  // namespace pkv
