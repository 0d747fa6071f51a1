// decode_shared.cu -- decode of a batch whose requests share long prefixes:
// each group of requests has one prefix, read once for all its rows, and every
// request its own keys behind it.
//
// A row's softmax runs over two sets of keys, so it is taken over each with its
// log-sum-exp and merged: out = sum_s e^(l_s - L) o_s, L = log sum_s e^(l_s)
// (+ e^sink).  Three grids:
//   shared_prefix_kernel  the prefixes: all rows of a group that share a kv
//           head (tokens x query heads) against its keys, on tcgen05;
//   shared_own_kernel     the requests' own keys (shared_own.cuh), HBM-bound
//           streaming; it does not wait for the first grid but runs beside it;
//   shared_merge_kernel   joins the partials of both.
//
// The prefix kernel.  One CTA on each of the SMs that the prefixes' work is
// worth (prefix_steps_per_team) takes an even share of the steps (see
// shared_prefix.cuh), item by item: NB blocks of 128 rows (row = token * group
// + head; a block holds as many whole tokens as fit) and one kv head, so that
// a K / V tile in shared memory serves 128 NB rows.  Warps 0 .. 4 NB - 1 are
// the softmax, one thread a row: scores read from TMEM once, running maximum
// in base 2 that rises only where a tile's exceeds it by more than 2^8, P
// written as 16-bit pairs over the consumed scores, the A operand of the PV
// MMA, whose first half of the keys begins while the second's P is made.  Then
// a TMA warp for Q and K, the MMA warp, a TMA warp for V, and an idle one.
// With two blocks the MMAs alternate (QK_A QK_B, then PV_A(t)
// QK_A(t+1) PV_B(t) QK_B(t+1)), so that the tensor core works for one block
// while the softmax of the other runs.  The K / V ring runs on from one item
// into the next; the next Q comes as soon as the last QK has read this one.
// Every wait is bounded.
//
// A step (2 x 128 rows, 128 keys) takes 2,800 cycles, its MMAs 2,048: scores -
// maximum - exponentials - P of a row in one thread are 1,400, and two blocks
// do not hide all of it.  Tried: two threads to a row, both finding its maximum
// (290 us of the third case's prefix against 206: 96 registers a thread, and the
// maximum's work twice); the first half's P from the last tile's maximum while
// this one's is found (204, and short prefixes 2 to 5% slower); two stages of K
// (2,930 cycles, waiting for L2); P in one piece (169 us against 166 on all
// SMs); boxes of one half of the head (190 against 176).
//
// Times of the call replayed from a graph (floor of bytes at 6788 GB/s or
// operations at 1912 TFLOP/s): 64 requests behind 8,192 keys, 64 to 1024 of
// their own, 32 / 8 heads: 46 us (27); 45 requests of 4 tokens behind three
// prefixes of up to 14,309, 28 / 4 heads, fp16: 43 (10); 256 behind 32,768,
// 64 / 8 heads: 219 (145), 206 of them the prefix on 120 SMs, own keys beside
// it on 32; 4 behind 512: 11.
//
// Roundings: P to the caches' 16-bit type for its product with V, the output
// once at the end; scores, maxima, sums, O, the partials and the LSE are fp32.
#include <math.h>

#include <atomic>

#include "attn_tile.cuh"
#include "shared_own.cuh"
#include "shared_prefix.cuh"
#include "sm103_ptx.cuh"

namespace pkv {

constexpr int kShD = 128;
constexpr int kOwnItems = 5;  // own keys: items of a CTA
constexpr uint32_t kShTileBytes = kShTile * kShD * 2;  // a K or V tile, a block of Q rows
template <int NB>
struct ShCfg {
    static constexpr int SOFTMAX = 4 * NB;                        // softmax warps
    static constexpr int THREADS = 32 * (SOFTMAX + 4);
    static constexpr int KST = 3, VST = NB == 2 ? 2 : 3;          // ring stages of K and of V
    static constexpr uint32_t TMEM = NB == 2 ? 512 : 256;         // columns
    static constexpr uint32_t SMEM = 1024 + (NB + KST + VST) * kShTileBytes + 8 * (3 + 2 * (KST + VST) + 4 * NB);
};
// Two blocks: registers as in the prefill kernel (launched with 384 x 168).
constexpr int kShRegsLow = 104, kShRegsHigh = 200;

struct SharedParams {
    PrefixWork w;
    const int32_t *prefix_tables;
    int64_t pt_stride;
    int page_shift;
    int64_t max_num_pages;
    int hnd, ratio;  // ratio (WIDE): (page, head) is row page * ratio + head of the cache's map
    float scale_log2;
    const float *bmm1_dev;
    unsigned long long wait_ns;
};

// A CTA's way through its items; each warp keeps its own in shared memory, out
// of the registers that the tile loops need.
struct PrefixWalk {
    PrefixGroup x;
    int head, item, k;  // the kv head, the item of it, the segment's first step
    __device__ __forceinline__ void next(const PrefixWork &p) {  // (there is one: the team has steps left)
        k = 0;
        if (++item < x.items) return;
        item = 0;
        if (++head < p.Hkv) return;
        head = 0;
        do read_prefix_group(p, x.g + 1, x);
        while (x.items * x.nk == 0 && x.g + 1 < p.G);
    }
};

template <typename T, int NB, bool WIDE>
__global__ void __launch_bounds__(ShCfg<NB>::THREADS, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const SharedParams p) {
    using C = ShCfg<NB>;
    constexpr int KST = C::KST, VST = C::VST, SW = C::SOFTMAX, THREADS = C::THREADS;
    // a tile in shared memory: WIDE, groups of 8 keys, 64 dimensions of each
    // then the other 64; else 64 dimensions of all keys, then the other 64
    constexpr uint32_t HALF = WIDE ? 1024 : kShTileBytes / 2, GROUP8 = WIDE ? 2048 : 1024;
    constexpr uint32_t O_COL = NB * 128;  // TMEM: S of block x at 128 x, O at O_COL + 128 x
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t q_s = smem_u32(smem), k_s = q_s + NB * kShTileBytes, v_s = k_s + KST * kShTileBytes;
    uint8_t *v_gen = smem + (NB + KST) * kShTileBytes;
    const uint32_t bar0 = v_s + VST * kShTileBytes;
    const uint32_t b_qfull = bar0, b_qempty = bar0 + 8;
    auto b_kfull = [&](int s) { return bar0 + 8u * (2 + s); };
    auto b_kempty = [&](int s) { return bar0 + 8u * (2 + KST + s); };
    auto b_vfull = [&](int s) { return bar0 + 8u * (2 + 2 * KST + s); };
    auto b_vempty = [&](int s) { return bar0 + 8u * (2 + 2 * KST + VST + s); };
    auto b_sfull = [&](int x) { return bar0 + 8u * (2 + 2 * (KST + VST) + x); };
    auto b_pfull = [&](int x, int half) { return bar0 + 8u * (2 + 2 * (KST + VST) + NB + 2 * x + half); };
    auto b_odone = [&](int x) { return bar0 + 8u * (2 + 2 * (KST + VST) + 3 * NB + x); };
    const uint32_t b_drain = bar0 + 8u * (2 + 2 * (KST + VST) + 4 * NB);
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s, steps_s;
    __shared__ PrefixWalk walk_s[THREADS / 32];
    const PrefixWork &w = p.w;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the own keys' grid may start as soon as every CTA of this one has
    pdl_launch_dependents();
    if (warp == SW + 1) {
        tmem_alloc(smem_u32(&tmem_base_s), C::TMEM);
        tmem_relinquish();
        tc_fence_before();
    } else if (warp == SW) {
        if (lane == 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
            mbar_init(b_qfull, 1);
            mbar_init(b_qempty, 1);
            for (int s = 0; s < KST; ++s) {
                mbar_init(b_kfull(s), 1);
                mbar_init(b_kempty(s), 1);
            }
            for (int s = 0; s < VST; ++s) {
                mbar_init(b_vfull(s), 1);
                mbar_init(b_vempty(s), 1);
            }
            for (int x = 0; x < NB; ++x) {
                mbar_init(b_sfull(x), 1);
                mbar_init(b_pfull(x, 0), 128);
                mbar_init(b_pfull(x, 1), 128);
                mbar_init(b_odone(x), 1);
            }
            mbar_init(b_drain, 1);
            abort_s = 0;
            fence_mbar_init();
        }
    } else if (warp == 0) {
        PrefixWalk at;
        bool bad;
        const uint32_t team = blockIdx.x / w.team;
        uint32_t W = 0, per = 1, w0 = 0;
        const OwnLengths own = own_lengths(w);
        scan_prefixes(
            w,
            [&](uint32_t all) {
                W = all;
                per = prefix_steps_per_team(w, all, own);
                w0 = team * per;
            },
            [&](int, int, uint32_t first, uint32_t n) { return w0 >= first && w0 - first < n; }, at.x, bad);
        if (bad) W = 0;
        if (blockIdx.x == 0) {
            report_prefixes(w, bad);
            if (lane == 0) *w.per = per;
        }
        if (lane == 0) steps_s = w0 < W ? static_cast<int>(min(per, W - w0)) : 0;
        if (w0 < W) {
            const uint32_t item = (w0 - at.x.base) / at.x.nk;
            at.k = static_cast<int>((w0 - at.x.base) - item * at.x.nk);
            at.head = static_cast<int>(item / at.x.items);
            at.item = static_cast<int>(item - at.head * at.x.items);
            if (lane < THREADS / 32) walk_s[lane] = at;
        }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const int steps = steps_s;
    if (steps == 0) {  // uniform over the CTA
        if (warp == SW + 1) tmem_dealloc(tmem, C::TMEM);
        return;
    }
    PrefixWalk &at = walk_s[warp];
    const int member = static_cast<int>(blockIdx.x) % w.team;
    // f(the CTA's tile of the item, its first step counted over the CTA's
    // segments, its steps, the segment's number) for each item with such a tile
    auto segments = [&](auto f) {
        for (int left = steps, s0 = 0, seg = 0; left > 0;) {
            const int n = min(left, at.x.nk - at.k), tile = at.item * w.team + member;
            if (tile < at.x.tiles) {
                if (!f(tile, s0, n, seg)) return;
                s0 += n;
                ++seg;
            }
            left -= n;
            __syncwarp();
            if (left > 0 && lane == 0) at.next(w);
            __syncwarp();
        }
    };

    volatile int *abort_flag = &abort_s;
    const uint64_t wlim = p.wait_ns;
    auto give_up = [&]() {
        *abort_flag = 1;
        set_err(w.err, PKV_DEV_ERR_TIMEOUT);
    };
    // Phases, counted over all of the CTA's steps i and segments: K / V stage of
    // step i: i / KST, i / VST; sfull / pfull of a block: i; Q and odone: the segment.
    // Every wait is for the newest phase that can be pending.
    if (warp >= SW) {
        if constexpr (NB == 2) reg_dealloc<kShRegsLow>();
        if (warp == SW || warp == SW + 2) {
            // ---- TMA: Q and K (warp SW), V (warp SW + 2)
            const bool is_k = warp == SW;
            const int ST = is_k ? KST : VST;
            const bool leader = elect_one();
            const int leader_lane = __ffs(__ballot_sync(0xffffffffu, leader)) - 1;
            const CUtensorMap *tm = is_k ? &tm_k : &tm_v;
            const uint32_t base = is_k ? k_s : v_s;
            const int S = 1 << p.page_shift, RB = pf_box_rows(S, WIDE ? kOwnTile : kShTile), nbox = kShTile / RB;
            const int oob = max(static_cast<int>(p.max_num_pages), 1);  // past the map: zero fill
            int issued = 0, queries = 0;  // (leader) steps, segments with copies issued
            bool ok = true;
            segments([&](int tile, int s0, int n, int seg) {
                const int32_t *pt = p.prefix_tables + static_cast<int64_t>(at.x.g) * p.pt_stride;
                // pages of 32 boxes at a time, a lane each, the next 32 on the way
                const int key0 = at.k * kShTile, P = at.x.P, head = at.head;
                auto lookup = [&](int j0) {
                    const int key = key0 + (j0 + lane) * RB;
                    const bool read = key < P && dbg_in(key >> p.page_shift, 1, (w.max_prefix + S - 1) >> p.page_shift, w.err);
                    return read ? pt[key >> p.page_shift] : -1;
                };
                int pages = -1, pages_next = lookup(0);
                for (int t = 0; t < n; ++t) {
                    const int j0 = (t * nbox) & 31;
                    if (j0 == 0) {
                        pages = pages_next;
                        if (pages < 0 || pages >= p.max_num_pages) {
                            if (is_k && key0 + (t * nbox + lane) * RB < min(P, key0 + n * kShTile)) set_err(w.err, PKV_DEV_ERR_PAGE);
                            pages = oob;
                        }
                        if (t * nbox + 32 < n * nbox) pages_next = lookup(t * nbox + 32);
                    }
                    const int i = s0 + t, st = i % ST, us = i / ST;
                    if (leader && us > 0 && !mbar_wait(is_k ? b_kempty(st) : b_vempty(st), (us - 1) & 1, abort_flag, wlim)) {
                        give_up();
                        ok = false;
                    }
                    ok = __shfl_sync(0xffffffffu, ok, leader_lane);
                    if (!ok) return false;
                    const uint32_t full = is_k ? b_kfull(st) : b_vfull(st);
                    if (leader) mbar_expect_tx(full, kShTileBytes);
#pragma unroll 1
                    for (int b = 0; b < nbox; ++b) {
                        const int page = __shfl_sync(0xffffffffu, pages, j0 + b);
                        if (!leader) continue;
                        const int slot = (key0 + t * kShTile + b * RB) & (S - 1);
                        if (kDebugBounds) {
                            dbg_in(page, 1, oob + 1, w.err);
                            dbg_in(slot, RB, S, w.err);
                        }
                        const uint32_t dst = base + st * kShTileBytes + b * RB * (WIDE ? 256 : 128);
                        if constexpr (WIDE) {
                            tma_load_5d(dst, tm, full, 0, 0, 0, slot >> 3, page * p.ratio + head);
                        } else {
                            for (int c = 0; c < 2; ++c)
                                tma_load_4d(dst + c * HALF, tm, full, 64 * c, p.hnd ? slot : head, p.hnd ? head : slot, page);
                        }
                    }
                    if (leader) issued = i + 1;
                    if (!is_k || t > 0) continue;
                    // every block's tokens, 64 elements at a time; tokens past the
                    // last row come as zeros, ones of another group are not written out
                    if (leader && seg > 0 && !mbar_wait(b_qempty, (seg - 1) & 1, abort_flag, wlim)) {
                        give_up();
                        ok = false;
                    }
                    ok = __shfl_sync(0xffffffffu, ok, leader_lane);
                    if (!ok) return false;
                    if (!leader) continue;
                    const int tok0 = at.x.a * w.Q + tile * NB * w.tok;
                    mbar_expect_tx(b_qfull, NB * 2 * static_cast<uint32_t>(w.tok * w.group) * 128);
                    for (int x = 0; x < NB; ++x)
                        for (int c = 0; c < 2; ++c)
                            tma_load_3d(q_s + x * kShTileBytes + c * (kShTileBytes / 2), &tm_q, b_qfull, 64 * c,
                                        head * w.group, tok0 + x * w.tok);
                    queries = seg + 1;
                }
                return true;
            });
            // every copy lands before the CTA exits
            if (leader) {
                for (int t = issued > ST ? issued - ST : 0; t < issued; ++t)
                    if (!mbar_wait_drain(is_k ? b_kfull(t % ST) : b_vfull(t % ST), (t / ST) & 1))
                        set_err(w.err, PKV_DEV_ERR_TIMEOUT);
                if (queries > 0 && !mbar_wait_drain(b_qfull, (queries - 1) & 1)) set_err(w.err, PKV_DEV_ERR_TIMEOUT);
            }
            __syncwarp();
        } else if (warp == SW + 1) {
            // ---- MMA issuer: the warp runs the loop, one elected lane issues
            const bool leader = elect_one();
            auto mwait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, wlim));
            };
            auto commit = [&](uint32_t bar) {
                if (leader) umma_commit(bar);
            };
            constexpr uint32_t idesc_qk = umma_idesc(128, kShTile, IsBf16<T>::value, false);
            constexpr uint32_t idesc_pv = umma_idesc(128, kShD, IsBf16<T>::value, true);
            const uint64_t qdesc = umma_sdesc_sw128(q_s, 16, 1024), kdesc = umma_sdesc_sw128(k_s, 16, GROUP8);
            const uint64_t vdesc = umma_sdesc_sw128(v_s, HALF, GROUP8);
            auto qk = [&](int x, int i) {  // S_x = Q_x K(i)^T, 16 dimensions a step
                const uint64_t qd = qdesc + ((x * kShTileBytes) >> 4), kd = kdesc + (((i % KST) * kShTileBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < kShD / 16; ++kk) {
                    const uint32_t dim = (kk & 3) * 32, qo = (kk >> 2) * (kShTileBytes / 2) + dim, ko = (kk >> 2) * HALF + dim;
                    if (leader) umma_ss(tmem + x * 128, qd + (qo >> 4), kd + (ko >> 4), idesc_qk, kk > 0 ? 1u : 0u);
                }
                commit(b_sfull(x));
            };
            auto pv = [&](int x, int i, int half, bool more) {  // O_x (+)= P_x V(i) of 64 keys, 16 a step
                const uint64_t vd = vdesc + (((i % VST) * kShTileBytes) >> 4);
#pragma unroll
                for (int kk = half * (kShTile / 32); kk < (half + 1) * (kShTile / 32); ++kk)
                    if (leader)
                        umma_ts(tmem + O_COL + x * 128, tmem + x * 128 + 32 * (kk / 2) + 8 * (kk % 2),
                                vd + ((kk * 2 * GROUP8) >> 4), idesc_pv, more || kk > 0 ? 1u : 0u);
            };
            bool ok = true;
            segments([&](int tile, int s0, int n, int seg) {
                ok = mwait(b_qfull, seg & 1) && mwait(b_kfull(s0 % KST), (s0 / KST) & 1);
                if (!ok) return false;
                tc_fence_after();
                // (S_x is free: the PV that read P_x from it was issued before)
                for (int x = 0; x < NB; ++x) qk(x, s0);
                commit(b_kempty(s0 % KST));
                if (n == 1) commit(b_qempty);
                for (int t = 0; t < n; ++t) {
                    const int i = s0 + t;
                    const bool more = t + 1 < n;
                    ok = mwait(b_vfull(i % VST), (i / VST) & 1);
                    if (!ok) return false;
                    for (int x = 0; x < NB; ++x) {
                        for (int half = 0; half < 2; ++half) {
                            ok = mwait(b_pfull(x, half), i & 1);
                            if (!ok) return false;
                            tc_fence_after();
                            pv(x, i, half, t > 0 || half > 0);  // (a segment's first overwrites O_x, drained before its P came)
                        }
                        if (x == NB - 1) commit(b_vempty(i % VST));
                        if (!more) {
                            commit(b_odone(x));
                            continue;
                        }
                        if (x == 0) {
                            ok = mwait(b_kfull((i + 1) % KST), ((i + 1) / KST) & 1);
                            if (!ok) return false;
                            tc_fence_after();
                        }
                        qk(x, i + 1);
                    }
                    if (more) commit(b_kempty((i + 1) % KST));
                    if (t + 2 == n) commit(b_qempty);
                }
                return true;
            });
            if (!ok && leader) give_up();
            commit(b_drain);  // every MMA completes before tensor memory is freed
            if (leader && !mbar_wait_drain(b_drain, 0)) set_err(w.err, PKV_DEV_ERR_TIMEOUT);
            __syncwarp();
        }
    } else {
        // ---- softmax: block X, TMEM lane quarter warp % 4, a thread a row
        if constexpr (NB == 2) reg_alloc<kShRegsHigh>();
        const int X = warp >> 2, qd = warp & 3, r = 32 * qd + lane;
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * qd) << 16);
        const uint32_t s_addr = t_lane + X * 128, o_addr = t_lane + O_COL + X * 128;
        const float sc = p.bmm1_dev ? __ldg(p.bmm1_dev) * kLog2e : p.scale_log2;
        const bool pos_scale = sc > 0.f;  // max on raw scores, one FFMA scales and shifts
        const float2 mul = make_float2(pos_scale ? sc : 1.f, pos_scale ? sc : 1.f);
        auto wait_warp = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, wlim));
        };
        bool ok = true;
        segments([&](int tile, int s0, int n, int seg) {
            float m = -INFINITY, l = 0.f;
            const int keys = at.x.P - at.k * kShTile;  // left of the prefix
            for (int t = 0; t < n; ++t) {
                    const int i0 = s0 + t, past = keys - t * kShTile;  // keys of the tile from here on are not the prefix's
                if (!wait_warp(b_sfull(X), i0 & 1)) return ok = false;
                tc_fence_after();
                if (!pos_scale || past < kShTile) {  // rare work, rolled and out of the way
#pragma unroll 1
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t hidden = ~low_bits(past - 32 * i);
                        if (pos_scale && hidden == 0u) continue;
                        uint32_t ra[32];
                        tmem_ld32(s_addr + 32 * i, ra);
                        tmem_wait_ld_regs(ra);
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            if (!pos_scale) ra[c] = __float_as_uint(__uint_as_float(ra[c]) * sc);
                            if (hidden & (1u << c)) ra[c] = __float_as_uint(-INFINITY);
                        }
                        tmem_st32(s_addr + 32 * i, ra);
                    }
                    tmem_wait_st();
                }
                uint32_t rs[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld32(s_addr + 32 * i, rs[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_wait_ld_regs(rs[i]);  // (the first waits for all)
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t *y = &rs[i][8 * q];
                        const float a = fmax3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
                        const float b = fmax3(__uint_as_float(y[3]), __uint_as_float(y[4]), __uint_as_float(y[5]));
                        top = fmax3(top, fmaxf(a, b), fmaxf(__uint_as_float(y[6]), __uint_as_float(y[7])));
                    }
                if (pos_scale) top *= sc;
                float alpha = 1.f;
                if (top > m + 8.f) {  // (first tile: from -inf)
                    alpha = fast_exp2(m - top);
                    m = top;
                    l *= alpha;
                }
                // rows of V that are no key of the prefix may hold anything: zeroed by
                // block A, so that P = 0 there cannot produce 0 * NaN
                if (X == 0 && past < kShTile) {
                    if (!wait_warp(b_vfull(i0 % VST), (i0 / VST) & 1)) return ok = false;
                    uint8_t *vbase = v_gen + (i0 % VST) * kShTileBytes;
                    for (int q = r; q < (kShTile - past) * 16; q += 128) {
                        const int row = past + (q >> 4), c = q & 15;
                        *reinterpret_cast<uint4 *>(vbase + (c >> 3) * HALF + (row >> 3) * GROUP8 + (row & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                // O *= alpha where a maximum moved (the PV before is complete: S(t) is)
                if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < kShD / 32; ++c) {
                        uint32_t ro[32];
                        tmem_ld32(o_addr + c * 32, ro);
                        tmem_wait_ld_regs(ro);
#pragma unroll
                        for (int e = 0; e < 32; ++e) ro[e] = __float_as_uint(__uint_as_float(ro[e]) * alpha);
                        tmem_st32(o_addr + c * 32, ro);
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;
                const float2 shift = make_float2(-base, -base);
                float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t pw[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = __ffma2_rn(
                            make_float2(__uint_as_float(rs[i][2 * e]), __uint_as_float(rs[i][2 * e + 1])), mul, shift);
                        const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                        if (e & 1) lb = __fadd2_rn(lb, make_float2(p0, p1));
                        else la = __fadd2_rn(la, make_float2(p0, p1));
                        pw[e] = pack2<T>(p0, p1);
                    }
                    tmem_st16(s_addr + 32 * i, pw);
                    if (i & 1) {  // half of the keys: their product may begin
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(b_pfull(X, i >> 1));
                    }
                }
                l += (la.x + la.y) + (lb.x + lb.y);
            }
            if (!wait_warp(b_odone(X), seg & 1)) return ok = false;
            tc_fence_after();
            // the row's place in the partials, or -1 (padding, another group's)
            const int tk = r / w.group, h = r - tk * w.group, token = at.x.a * w.Q + (tile * NB + X) * w.tok + tk;
            const bool valid = tk < w.tok && token < at.x.b * w.Q;
            int64_t row = -1;
            if (valid)
                row = at.k == 0 ? static_cast<int64_t>(token) * w.Hqo + at.head * w.group + h
                                : w.rows + (static_cast<int64_t>(blockIdx.x) * NB + X) * 128 + r;
            const float inv = l > 0.f ? 1.f / l : (l != l ? l : 0.f);
            // written from accumulator fragments: four lanes write 32 bytes of a row
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {  // rows 16 (c / 2) and on, columns 64 (c % 2) and on
                uint32_t ro[32];
                tmem_ld16x256(o_addr + (static_cast<uint32_t>(16 * (c >> 1)) << 16) + 64 * (c & 1), ro);
                tmem_wait_ld_regs(ro);
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const int from = 16 * (c >> 1) + 8 * f + (lane >> 2);
                    const int64_t to = __shfl_sync(0xffffffffu, row, from);
                    const float mul = __shfl_sync(0xffffffffu, inv, from);
                    if (to < 0 || !dbg_in(to, 1, w.parts, w.err)) continue;
                    float *dst = w.ws_o + to * kShD + 64 * (c & 1) + 2 * (lane & 3);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float2 *>(dst + 8 * i) =
                            make_float2(__uint_as_float(ro[4 * i + 2 * f]) * mul, __uint_as_float(ro[4 * i + 2 * f + 1]) * mul);
                }
            }
            if (valid && dbg_in(row, 1, w.parts, w.err))
                w.ws_lse[row] = l > 0.f ? m + fast_log2(l) : (l != l ? l : -INFINITY);
            return true;
        });
        if (!ok) give_up();
        tmem_wait_st();
        tmem_wait_ld();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == SW + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
}

// K or V cache as a 5-D map (64 dimensions, 8 slots, the two halves of a head,
// groups of 8 slots, (page, head)), whose box, `rows` slots of one head, lands
// as WIDE tiles have it: one copy where cache_tmap's 64-dimension boxes take
// two.  Boxes of 16 slots: the copy engine took 1714 to 2400 cycles for a tile
// of K in 16 of those, about as long as a step's MMAs.  Where the page stride
// is no multiple of the unit that makes (page, head) one index, or the index
// passes 31 bits, wide_ratio says 0 and the kernel takes the narrow boxes.
static int wide_ratio(int layout, int S, int heads, int64_t page_stride, int64_t pages) {
    const int64_t unit = layout == PKV_HND ? static_cast<int64_t>(S) * kShD : kShD;
    const int64_t r = page_stride / unit;
    return page_stride % unit || (pages + 2) * r + heads >= (1LL << 31) ? 0 : static_cast<int>(r);
}
static bool wide_tmap(CUtensorMap *m, const void *base, CUtensorMapDataType t, int layout, int S, int heads, int ratio,
                      int64_t pages, int rows) {
    const uint64_t row = layout == PKV_HND ? 256 : 256ull * heads, unit = layout == PKV_HND ? 256ull * S : 256;
    const uint64_t dims[5] = {64, 8, 2, static_cast<uint64_t>(S / 8), static_cast<uint64_t>(pages * ratio)};
    const uint64_t strides[4] = {row, 128, 8 * row, unit};
    const uint32_t box[5] = {64, 8, 2, static_cast<uint32_t>(rows / 8), 1};
    return encode_tmap(m, base, t, 5, dims, strides, box);
}

struct SharedPlan {
    int R, MT, chunk, n_split_max;  // own keys: rows of an item, tiles of 16 of them, keys and splits
    int nb, tok, team, ctas;
    int64_t rows, parts;
    int64_t all;         // partial rows: the prefix's, then the own keys'
    size_t lse, per, bytes;  // offsets in the workspace, its size
};

// The workspace is as large as the largest call with no more of anything
// (requests, tokens, groups, keys) needs, so that one reserved for a server's
// maxima holds every smaller call; the calls themselves do not need more with
// more keys always: splits of own keys get longer, a second block of rows
// halves the tiles, teams leave CTAs out.  So the rows are counted by bounds
// that grow with each size:
//   own keys: (request, kv head) pairs times splits of c keys, c >= max(256,
//     min(X / K, 4096)) (plan_shared) with X the keys of all pairs and K =
//     10 SMs: at most a split more for each pair than X / c;
//   prefix: a CTA holds up to nb blocks of 128 rows; blocks of full tiles,
//     2 more for each group, and never more than 2 for each token or SM.
static int64_t most_partials(const SharedPlan &pl, int64_t B, int64_t Hkv, int64_t tokens, int64_t G, int64_t max_seq_len,
                             int64_t nk) {
    const int64_t sms = num_sms(), K = kOwnItems * 2 * sms, X = B * Hkv * max_seq_len;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    // (X / floor(X / K) <= K + K / 256 + 1 where X / K >= 256)
    int64_t splits = up(X, 256) < K + K / 256 + 1 ? up(X, 256) : K + K / 256 + 1;
    if (splits < up(X, 4096)) splits = up(X, 4096);
    splits += B * Hkv;
    const int64_t short_splits = B * Hkv * own_splits(static_cast<int>(max_seq_len), 256);
    if (splits > short_splits) splits = short_splits;
    int64_t blocks = up(tokens, pl.tok) + 2 * G;
    if (blocks > 2 * tokens) blocks = 2 * tokens;
    blocks = G > 0 && nk > 0 ? (blocks * Hkv * nk < 2 * sms ? blocks * Hkv * nk : 2 * sms) : 0;
    return (blocks > 0 ? pl.rows : 0) + blocks * 128 + splits * pl.R;
}

static int plan_shared(int B, int Q, int Hqo, int Hkv, int D, int G, int max_prefix, int max_seq_len, int page_size,
                       SharedPlan &pl) {
    if (B < 0 || Q < 1 || Hqo < 1 || Hkv < 1 || max_seq_len < 0 || G < 0 || max_prefix < 0 || Hqo % Hkv)
        return PKV_ERR_INVALID_ARG;
    const int group = Hqo / Hkv;
    if (B > 65535 || Hkv > 65535 || D != kShD || ilog2_exact(page_size) < 3 || page_size > 256 ||
        static_cast<int64_t>(group) * Q > 64 || max_seq_len > (1 << 30))
        return PKV_ERR_UNSUPPORTED;
    // Own keys: splits short enough that each of two CTAs per SM has several,
    // which evens out requests of different lengths, but of no fewer than 256
    // keys.
    pl.R = group * Q;
    pl.MT = pl.R <= 16 ? 1 : (pl.R <= 32 ? 2 : 4);
    const int64_t share = static_cast<int64_t>(B) * Hkv * max_seq_len / (kOwnItems * 2 * num_sms());
    const int64_t chunk = (share < 256 ? 256 : (share > 4096 ? 4096 : share)) + kOwnTile - 1;
    pl.chunk = static_cast<int>(chunk / kOwnTile * kOwnTile);
    pl.n_split_max = own_splits(max_seq_len, pl.chunk);
    if (max_prefix > (1 << 30) || static_cast<int64_t>(B) * Q * Hqo > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    pl.rows = static_cast<int64_t>(B) * Q * Hqo;
    pl.tok = 128 / group;
    const int64_t tokens = static_cast<int64_t>(B) * Q;
    // Two blocks to a CTA where the groups' rows fill more than one on average.
    pl.nb = tokens > static_cast<int64_t>(pl.tok) * (G > 0 ? G : 1) ? 2 : 1;
    // tiles of tokens, each group's last one partly filled, and their steps
    const int64_t T = static_cast<int64_t>(pl.nb) * pl.tok;
    int64_t tiles = (tokens + static_cast<int64_t>(G) * (T - 1)) / T;
    if (tiles > tokens) tiles = tokens;
    const int64_t nk = (static_cast<int64_t>(max_prefix) + kShTile - 1) / kShTile, sms = num_sms();
    if (tiles * Hkv * nk > 0x3fffffff) return PKV_ERR_UNSUPPORTED;
    // Teams pay where the tiles of a group would read more keys than L2 holds
    // at different times: 256 requests over one prefix of 134 MB, 8 tiles a kv
    // head, read 917 MB from HBM one by one and 140 MB in teams of 8.  The
    // largest team up to 16 that keeps 15/16 of the CTAs' time busy: what a
    // team's last item and the SMs beyond whole teams leave idle (of several
    // groups only the mean size is known here: half an item each is idle).
    pl.team = 1;
    const int64_t tiles_g = tiles / (G > 0 ? G : 1);
    if (static_cast<double>(nk) * kShTile * G * Hkv * kShD * 4 > 64e6)
        for (int m = 2; m <= 16 && m <= tiles_g; ++m) {
            const int64_t items2 = G == 1 ? 2 * ((tiles_g + m - 1) / m) * m : 2 * tiles_g + m - 1;
            if (2 * tiles_g * (sms / m * m) * 16 >= items2 * sms * 15) pl.team = m;
        }
    const int64_t most = tiles * Hkv * nk;  // (a CTA takes one step at least; a team is for more than that)
    pl.ctas = G > 0 && nk > 0 ? static_cast<int>((most < sms ? most : sms) / pl.team * pl.team) : 0;
    pl.parts = pl.ctas > 0 ? pl.rows + static_cast<int64_t>(pl.ctas) * pl.nb * 128 : 0;
    pl.all = pl.parts + static_cast<int64_t>(B) * Hkv * pl.n_split_max * pl.R;
    if (pl.all > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    pl.lse = static_cast<size_t>(pl.all) * kShD * sizeof(float);
    const size_t most_rows = static_cast<size_t>(most_partials(pl, B, Hkv, tokens, G, max_seq_len, nk));
    pl.per = round_up(most_rows * (kShD + 1) * sizeof(float), 256);
    pl.bytes = most_rows > 0 ? pl.per + 256 : 0;
    return PKV_OK;
}

struct SharedMaps {
    CUtensorMap q, k, v;              // the prefix kernel's: queries of a block of rows, the caches
    CUtensorMap own_q, own_k, own_v;  // the own keys': queries of a request, the caches (k and v where they are wide)
};

// The kernel's dynamic shared memory, asked for once per device (bit d of
// `set`: done on device d): a host call less in every later launch.
template <typename K>
static bool allow_smem(K kern, int bytes, std::atomic<unsigned long long> &set) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (set.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    set.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

template <typename T, int NB, bool WIDE>
static int launch_prefix(const SharedMaps &m, const SharedParams &p, dim3 grid, cudaStream_t st) {
    auto kern = shared_prefix_kernel<T, NB, WIDE>;
    static std::atomic<unsigned long long> set{0};
    if (!allow_smem(kern, static_cast<int>(ShCfg<NB>::SMEM), set)) return PKV_ERR_CUDA;
    if constexpr (NB == 2) {
        // the register split draws on what the CTA is launched with: refuse to
        // launch if the compiled kernel has fewer (setmaxnreg.inc would wait forever)
        static std::atomic<int> ok{-1};
        if (ok < 0) {
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return PKV_ERR_CUDA;
            ok = fa.numRegs * ShCfg<NB>::THREADS >= 128 * kShRegsLow + 256 * kShRegsHigh ? 1 : 0;
        }
        if (!ok) return PKV_ERR_UNSUPPORTED;
    }
    kern<<<grid, ShCfg<NB>::THREADS, ShCfg<NB>::SMEM, st>>>(m.q, m.k, m.v, p);
    return PKV_OK;
}

template <typename T, int MT, bool DRAFTS>
static int launch_own(const SharedMaps &m, const OwnParams &p, dim3 grid, cudaStream_t st) {
    auto kern = shared_own_kernel<T, MT, DRAFTS>;
    constexpr int smem = static_cast<int>(OwnCfg<MT>::SMEM);
    static std::atomic<unsigned long long> set{0};
    if (!allow_smem(kern, smem, set)) return PKV_ERR_CUDA;
    const CUtensorMap &k = p.ratio ? m.k : m.own_k, &v = p.ratio ? m.v : m.own_v;
    if (p.prefix.ctas > 0)
        return launch_dependent(kern, grid, dim3(kOwnThreads), smem, st, m.own_q, k, v, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    kern<<<grid, kOwnThreads, smem, st>>>(m.own_q, k, v, p);
    return PKV_OK;
}

template <typename T>
static int run_shared(const SharedMaps &m, const SharedParams &s, const OwnParams &p, const SharedPlan &pl, cudaStream_t st) {
    int launches = 2, rc = PKV_OK;
    if (pl.ctas > 0) {
        const dim3 grid(pl.ctas);
        rc = pl.nb == 2 ? (s.ratio ? launch_prefix<T, 2, true>(m, s, grid, st) : launch_prefix<T, 2, false>(m, s, grid, st))
                        : (s.ratio ? launch_prefix<T, 1, true>(m, s, grid, st) : launch_prefix<T, 1, false>(m, s, grid, st));
        if (rc != PKV_OK) return rc;
        ++launches;
    }
    const dim3 grid(pl.n_split_max, p.prefix.Hkv, p.prefix.B);
    if (p.prefix.Q == 1)
        rc = pl.MT == 1 ? launch_own<T, 1, false>(m, p, grid, st)
                        : (pl.MT == 2 ? launch_own<T, 2, false>(m, p, grid, st) : launch_own<T, 4, false>(m, p, grid, st));
    else
        rc = pl.MT == 1 ? launch_own<T, 1, true>(m, p, grid, st)
                        : (pl.MT == 2 ? launch_own<T, 2, true>(m, p, grid, st) : launch_own<T, 4, true>(m, p, grid, st));
    if (rc != PKV_OK) return rc;
    const int64_t warps = pl.rows / p.prefix.group * ((p.prefix.group + p.merge_rows - 1) / p.merge_rows);
    if (launch_dependent(shared_merge_kernel<T>, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, st, p) !=
        cudaSuccess)
        return PKV_ERR_CUDA;
    note_launches(launches);
    return launch_status();
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t paged_decode_shared_workspace_size(int32_t batch_size, int32_t q_len_per_req, int32_t num_qo_heads,
                                                     int32_t num_kv_heads, int32_t head_dim, int32_t num_groups,
                                                     int32_t max_prefix_len, int32_t max_seq_len, int32_t page_size) {
    SharedPlan pl;
    if (plan_shared(batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim, num_groups, max_prefix_len,
                    max_seq_len, page_size, pl) != PKV_OK)
        return 0;
    return pl.bytes;
}

extern "C" int paged_decode_shared(const void *query, const void *k_cache, const void *v_cache, int64_t page_stride,
                                   int64_t max_num_pages, void *workspace, size_t workspace_bytes,
                                   const int32_t *prefix_tables, int32_t prefix_table_stride,
                                   const int32_t *prefix_lens, const int32_t *group_indptr, int32_t num_groups,
                                   int32_t max_prefix_len, const int32_t *block_tables, int32_t block_table_stride,
                                   const uint32_t *seq_lens, int32_t batch_size, int32_t max_seq_len, float bmm1_scale,
                                   float bmm2_scale, const float *bmm1_scale_dev, const float *bmm2_scale_dev,
                                   const float *sinks, int32_t q_len_per_req, int32_t num_qo_heads,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t page_size, int32_t layout,
                                   int32_t dtype, void *out, float *lse, int32_t *err_word, void *stream) {
    const CallRange nvtx_range("paged_decode_shared");
    if (layout != PKV_NHD && layout != PKV_HND) return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    SharedPlan pl;
    const int rc = plan_shared(batch_size, q_len_per_req, num_qo_heads, num_kv_heads, head_dim, num_groups,
                               max_prefix_len, max_seq_len, page_size, pl);
    if (rc != PKV_OK) return rc;
    const int64_t page = static_cast<int64_t>(num_kv_heads) * page_size * head_dim;
    if (page_stride < page || page_stride % 8 || max_num_pages < 0 || max_num_pages > 0x7ffffffe ||
        static_cast<int64_t>(block_table_stride) * page_size < max_seq_len ||
        (num_groups > 0 && static_cast<int64_t>(prefix_table_stride) * page_size < max_prefix_len))
        return PKV_ERR_INVALID_ARG;
    if (batch_size == 0) return PKV_OK;
    if (!query || !k_cache || !v_cache || !block_tables || !seq_lens || !out || !workspace) return PKV_ERR_NULL;
    if (num_groups > 0 && (!prefix_tables || !prefix_lens || !group_indptr)) return PKV_ERR_NULL;
    if (!aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < pl.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255)) return PKV_ERR_WORKSPACE;
    char *ws = static_cast<char *>(workspace);

    SharedParams s = {};
    PrefixWork &w = s.w;
    w.group_indptr = group_indptr;
    w.prefix_lens = prefix_lens;
    w.seq_lens = seq_lens;
    w.max_seq_len = max_seq_len;
    w.G = num_groups;
    w.B = batch_size;
    w.Q = q_len_per_req;
    w.Hqo = num_qo_heads;
    w.Hkv = num_kv_heads;
    w.group = num_qo_heads / num_kv_heads;
    w.tok = pl.tok;
    w.nb = pl.nb;
    w.max_prefix = max_prefix_len;
    w.team = pl.team;
    w.ctas = pl.ctas;
    w.sms = num_sms();
    w.rows = static_cast<uint32_t>(pl.rows);
    w.parts = static_cast<uint32_t>(pl.parts);
    w.all = static_cast<uint32_t>(pl.all);
    w.ws_o = reinterpret_cast<float *>(ws);
    w.ws_lse = reinterpret_cast<float *>(ws + pl.lse);
    w.per = reinterpret_cast<uint32_t *>(ws + pl.per);
    w.err = err_word;
    s.prefix_tables = prefix_tables;
    s.pt_stride = prefix_table_stride;
    s.page_shift = ilog2_exact(page_size);
    s.max_num_pages = max_num_pages;
    s.scale_log2 = bmm1_scale * kLog2e;
    s.bmm1_dev = bmm1_scale_dev;
    s.wait_ns = wait_limit_ns();
    s.hnd = layout == PKV_HND;
    s.ratio = wide_ratio(layout, page_size, num_kv_heads, page_stride, max_num_pages);

    OwnParams d = {};
    d.prefix = w;
    d.block_tables = block_tables;
    d.bt_stride = block_table_stride;
    d.max_num_pages = max_num_pages;
    d.scale_log2 = s.scale_log2;
    d.bmm1_dev = bmm1_scale_dev;
    d.bmm2_dev = bmm2_scale_dev;
    d.bmm2 = bmm2_scale;
    d.sinks = sinks;
    d.R = pl.R;
    d.page_shift = s.page_shift;
    d.ratio = s.ratio;
    d.chunk = pl.chunk;
    d.n_split_max = pl.n_split_max;
    d.out = out;
    d.lse = lse;
    // (a warp for a row until every SM has 28 of them)
    const int64_t fill = (pl.rows + 28 * num_sms() - 1) / (28 * num_sms());
    d.merge_rows = static_cast<int>(fill < w.group ? fill : w.group);
    d.err = err_word;
    d.wait_ns = s.wait_ns;

    SharedMaps m;
    const CUtensorMapDataType t = dtype == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    // rows of queries in one box for each half of the head: (64 elements, the
    // group's heads, whole tokens)
    const uint64_t dims[3] = {kShD, static_cast<uint64_t>(num_qo_heads), static_cast<uint64_t>(batch_size) * q_len_per_req};
    const uint64_t strides[2] = {kShD * 2, static_cast<uint64_t>(num_qo_heads) * kShD * 2};
    const uint32_t heads = static_cast<uint32_t>(w.group);
    const uint32_t block[3] = {64, heads, static_cast<uint32_t>(w.tok)}, own[3] = {64, heads, static_cast<uint32_t>(w.Q)};
    const int64_t pages = max_num_pages > 0 ? max_num_pages : 1;
    const int box = pf_box_rows(page_size, kOwnTile);
    if ((pl.ctas > 0 && !encode_tmap(&m.q, query, t, 3, dims, strides, block)) ||
        !encode_tmap(&m.own_q, query, t, 3, dims, strides, own))
        return PKV_ERR_CUDA;
    if (s.ratio) {  // the same boxes for both kernels
        if (!wide_tmap(&m.k, k_cache, t, layout, page_size, num_kv_heads, s.ratio, pages, box) ||
            !wide_tmap(&m.v, v_cache, t, layout, page_size, num_kv_heads, s.ratio, pages, box))
            return PKV_ERR_CUDA;
    } else {
        const int box_p = pf_box_rows(page_size, kShTile);
        if ((pl.ctas > 0 &&
             (!cache_tmap(&m.k, k_cache, t, layout, kShD, page_size, num_kv_heads, page_stride, pages, box_p) ||
              !cache_tmap(&m.v, v_cache, t, layout, kShD, page_size, num_kv_heads, page_stride, pages, box_p))) ||
            !own_tmap(&m.own_k, k_cache, t, layout, page_size, num_kv_heads, page_stride, pages, box) ||
            !own_tmap(&m.own_v, v_cache, t, layout, page_size, num_kv_heads, page_stride, pages, box))
            return PKV_ERR_CUDA;
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_BF16 ? run_shared<__nv_bfloat16>(m, s, d, pl, st) : run_shared<__half>(m, s, d, pl, st);
}
