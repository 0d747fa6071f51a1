// decode_shared.cu -- decode of a batch whose requests share long prefixes:
// each group of requests has one prefix, read once for all its rows, and every
// request its own keys behind it.
//
// A row's softmax runs over two sets of keys, so it is taken over each with its
// log-sum-exp and merged: out = sum_s e^(l_s - L) o_s, L = log sum_s e^(l_s)
// (+ e^sink).  Three grids:
//   shared_prefix_kernel  the prefix: all rows of a group that share a kv head
//           (tokens x query heads) against a slice of its keys, on tcgen05;
//   decode_split_kernel   the requests' own keys (EXT 3), HBM-bound streaming;
//           it does not wait for the first grid but runs beside its end;
//   shared_merge_kernel   one warp a row joins the partials of both.
//
// The prefix kernel.  A CTA takes NB blocks of 128 rows (row = token * group +
// head; a block holds as many whole tokens as fit), one kv head and one slice
// of the prefix, so that a K / V tile in shared memory serves 128 NB rows.
// Warps 0 .. 4 NB - 1 are the softmax, one thread a row: scores read from TMEM
// once, running maximum in base 2 that rises only where a tile's exceeds it by
// more than 2^8, P written as 16-bit pairs over the consumed scores, the A
// operand of the PV MMA.  Then a TMA warp for Q and K, the MMA warp, a TMA warp
// for V, and an idle one.  With two blocks the MMAs alternate (QK_A QK_B, then
// PV_A(t) QK_A(t+1) PV_B(t) QK_B(t+1)), so that the tensor core works for one
// block while the softmax of the other runs.  Every wait is bounded.
//
// Roundings: P to the caches' 16-bit type for its product with V, the output
// once at the end; scores, maxima, sums, O, the partials and the LSE are fp32.
#include <math.h>

#include "attn_tile.cuh"
#include "decode_split.cuh"
#include "sm103_ptx.cuh"

namespace pkv {

constexpr int kShTile = 128;  // keys per tile
constexpr int kShD = 128;
constexpr uint32_t kShTileBytes = kShTile * kShD * 2;  // a K or V tile, a block of Q rows
template <int NB>
struct ShCfg {
    static constexpr int SOFTMAX = 4 * NB;                        // softmax warps
    static constexpr int THREADS = 32 * (SOFTMAX + 4);
    static constexpr int STAGES = NB == 2 ? 2 : 3;                // of K and of V
    static constexpr uint32_t TMEM = NB == 2 ? 512 : 256;         // columns
    static constexpr uint32_t SMEM = 1024 + (NB + 2 * STAGES) * kShTileBytes + 8 * (1 + 4 * STAGES + 3 * NB + 1);
};
// Two blocks: registers as in the prefill kernel (launched with 384 x 168).
constexpr int kShRegsLow = 104, kShRegsHigh = 200;

struct SharedParams {
    const int32_t *group_indptr, *prefix_lens, *prefix_tables;
    int64_t pt_stride;
    int G, B, Q, Hqo, Hkv, group;
    int tok;  // tokens of a block: 128 / group
    int max_prefix, page_shift, chunk, n_split;
    int64_t max_num_pages;
    float scale_log2;
    const float *bmm1_dev;
    float *ws_o;    // [n_split][rows][128], rows = B * Q * Hqo
    float *ws_lse;  // [n_split][rows], base 2
    int64_t rows;
    int32_t *err;
    unsigned long long wait_ns;
};

// The group that unit u belongs to, by one warp: unit(a, b) says how many units
// the group of requests [a, b) has, and the units of the groups are numbered in
// order.  Returns the group (its requests and first unit in a, b, u0), or -1 if
// there are fewer units or the array is not in order (*bad).
template <typename F>
__device__ __forceinline__ int find_group(const int32_t *indptr, int G, int B, int u, F unit, int &a, int &b, int &u0,
                                          bool &bad) {
    const int lane = threadIdx.x & 31;
    int found = -1, carry = 0;
    bad = false;
    for (int g0 = 0; g0 < G; g0 += 32) {
        const int g = g0 + lane;
        const int lo = g < G ? indptr[g] : 0, hi = g < G ? indptr[g + 1] : 0;
        const bool wrong = g < G && (lo < 0 || hi < lo || hi > B || (g == 0 && lo != 0));
        if (__any_sync(0xffffffffu, wrong)) bad = true;
        const int n = g < G && !wrong ? unit(lo, hi) : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const unsigned m = __ballot_sync(0xffffffffu, carry + x > u);
        if (m && found < 0) {
            const int j = __ffs(m) - 1;
            found = g0 + j;
            a = __shfl_sync(0xffffffffu, lo, j);
            b = __shfl_sync(0xffffffffu, hi, j);
            u0 = carry + __shfl_sync(0xffffffffu, x - n, j);
        }
        carry += __shfl_sync(0xffffffffu, x, 31);
    }
    return bad ? -1 : found;
}

template <typename T, int LAYOUT, int NB>
__global__ void __launch_bounds__(ShCfg<NB>::THREADS, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const SharedParams p) {
    using C = ShCfg<NB>;
    constexpr int ST = C::STAGES, SW = C::SOFTMAX;
    constexpr uint32_t O_COL = NB * 128;  // TMEM: S of block x at 128 x, O at O_COL + 128 x
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t q_s = smem_u32(smem), k_s = q_s + NB * kShTileBytes, v_s = k_s + ST * kShTileBytes;
    uint8_t *v_gen = smem + (NB + ST) * kShTileBytes;
    const uint32_t bar0 = v_s + ST * kShTileBytes;
    const uint32_t b_qfull = bar0;
    auto b_kfull = [&](int s) { return bar0 + 8u * (1 + s); };
    auto b_kempty = [&](int s) { return bar0 + 8u * (1 + ST + s); };
    auto b_vfull = [&](int s) { return bar0 + 8u * (1 + 2 * ST + s); };
    auto b_vempty = [&](int s) { return bar0 + 8u * (1 + 3 * ST + s); };
    auto b_sfull = [&](int x) { return bar0 + 8u * (1 + 4 * ST + x); };
    auto b_pfull = [&](int x) { return bar0 + 8u * (1 + 4 * ST + NB + x); };
    auto b_odone = [&](int x) { return bar0 + 8u * (1 + 4 * ST + 2 * NB + x); };
    const uint32_t b_drain = bar0 + 8u * (1 + 4 * ST + 3 * NB);
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s, where_s[4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the own keys' grid may start as soon as every CTA of this one has
    pdl_launch_dependents();
    const int kvh = blockIdx.y, split = blockIdx.z;
    if (warp == 0) {
        int a = 0, b = 0, u0 = 0;
        bool bad;
        const int g = find_group(p.group_indptr, p.G, p.B, blockIdx.x,
                                 [&](int lo, int hi) { return ((hi - lo) * p.Q + NB * p.tok - 1) / (NB * p.tok); }, a, b,
                                 u0, bad);
        int P = 0;
        if (g >= 0) {
            P = p.prefix_lens[g];
            if ((P < 0 || P > p.max_prefix) && lane == 0) set_err(p.err, PKV_DEV_ERR_LEN);
            P = min(max(P, 0), p.max_prefix);
        }
        if (bad && lane == 0) set_err(p.err, PKV_DEV_ERR_BATCH);
        if (lane == 0) {
            where_s[0] = g;
            where_s[1] = a * p.Q + (static_cast<int>(blockIdx.x) - u0) * NB * p.tok;  // first token
            where_s[2] = b * p.Q;                                                     // end of the group's tokens
            where_s[3] = P;
        }
    }
    __syncthreads();
    const int grp = where_s[0], tok0 = where_s[1], tok1 = where_s[2], P = where_s[3];
    const int k0 = split * p.chunk, k1 = min(P, k0 + p.chunk);
    if (grp < 0 || k0 >= k1) return;  // uniform over the CTA
    const int n = (k1 - k0 + kShTile - 1) / kShTile;

    if (tid == 0) {
        mbar_init(b_qfull, 1);
        for (int s = 0; s < ST; ++s) {
            mbar_init(b_kfull(s), 1);
            mbar_init(b_kempty(s), 1);
            mbar_init(b_vfull(s), 1);
            mbar_init(b_vempty(s), 1);
        }
        for (int x = 0; x < NB; ++x) {
            mbar_init(b_sfull(x), 1);
            mbar_init(b_pfull(x), 128);
            mbar_init(b_odone(x), 1);
        }
        mbar_init(b_drain, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    if (warp == SW + 1) {
        tmem_alloc(smem_u32(&tmem_base_s), C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    volatile int *abort_flag = &abort_s;
    const uint64_t wlim = p.wait_ns;
    auto give_up = [&]() {
        *abort_flag = 1;
        set_err(p.err, PKV_DEV_ERR_TIMEOUT);
    };
    // Phases: K / V stage s of tile t: t / ST; sfull / pfull of a block: t; every
    // wait is for the newest phase that can be pending.
    if (warp >= SW) {
        if constexpr (NB == 2) reg_dealloc<kShRegsLow>();
        if (warp == SW || warp == SW + 2) {
            // ---- TMA: Q and K (warp SW), V (warp SW + 2)
            const bool is_k = warp == SW;
            const bool leader = elect_one();
            const int leader_lane = __ffs(__ballot_sync(0xffffffffu, leader)) - 1;
            const CUtensorMap *tm = is_k ? &tm_k : &tm_v;
            const uint32_t base = is_k ? k_s : v_s;
            if (leader) {
                prefetch_tmap(tm);
                if (is_k) {
                    // every block's tokens, 64 elements at a time; tokens past the
                    // last row come as zeros, ones of another group are not written out
                    const uint32_t half = static_cast<uint32_t>(p.tok * p.group) * 128;
                    mbar_expect_tx(b_qfull, NB * 2 * half);
                    for (int x = 0; x < NB; ++x)
                        for (int c = 0; c < 2; ++c)
                            tma_load_3d(q_s + x * kShTileBytes + c * (kShTileBytes / 2), &tm_q, b_qfull, 64 * c,
                                        kvh * p.group, tok0 + x * p.tok);
                }
            }
            const int S = 1 << p.page_shift, RB = pf_box_rows(S, kShTile), nbox = kShTile / RB;
            const int oob = max(static_cast<int>(p.max_num_pages), 1);  // past the map: zero fill
            const int32_t *pt = p.prefix_tables + static_cast<int64_t>(grp) * p.pt_stride;
            auto lookup = [&](int t) {  // lane i < nbox: page of box i of tile t
                const int key = k0 + t * kShTile + lane * RB;
                int page = oob;
                if (lane < nbox && key < P && dbg_in(key >> p.page_shift, 1, (p.max_prefix + S - 1) >> p.page_shift, p.err)) {
                    page = pt[key >> p.page_shift];
                    if (page < 0 || page >= p.max_num_pages) {
                        if (is_k) set_err(p.err, PKV_DEV_ERR_PAGE);
                        page = oob;
                    }
                }
                return page;
            };
            bool ok = true;
            int issued = 0;  // (leader) tiles with copies issued
            int next = lookup(0);
            for (int t = 0; t < n && ok; ++t) {
                const int pg = next;
                if (t + 1 < n) next = lookup(t + 1);
                const int st = t % ST, us = t / ST;
                if (leader && us > 0 && !mbar_wait(is_k ? b_kempty(st) : b_vempty(st), (us - 1) & 1, abort_flag, wlim)) {
                    give_up();
                    ok = false;
                }
                ok = __shfl_sync(0xffffffffu, ok, leader_lane);
                if (!ok) break;
                const uint32_t full = is_k ? b_kfull(st) : b_vfull(st);
                if (leader) mbar_expect_tx(full, kShTileBytes);
#pragma unroll 1
                for (int i = 0; i < nbox; ++i) {
                    const int page = __shfl_sync(0xffffffffu, pg, i);
                    if (!leader) continue;
                    const int slot = (k0 + t * kShTile + i * RB) & (S - 1);
                    if (kDebugBounds) {
                        dbg_in(page, 1, oob + 1, p.err);
                        dbg_in(slot, RB, S, p.err);
                    }
                    for (int c = 0; c < 2; ++c)
                        tma_load_4d(base + st * kShTileBytes + c * (kShTileBytes / 2) + i * RB * 128, tm, full, 64 * c,
                                    LAYOUT == PKV_HND ? slot : kvh, LAYOUT == PKV_HND ? kvh : slot, page);
                }
                if (leader) issued = t + 1;
            }
            // every copy lands before the CTA exits
            if (leader) {
                for (int t = issued > ST ? issued - ST : 0; t < issued; ++t)
                    if (!mbar_wait_drain(is_k ? b_kfull(t % ST) : b_vfull(t % ST), (t / ST) & 1))
                        set_err(p.err, PKV_DEV_ERR_TIMEOUT);
                if (is_k && !mbar_wait_drain(b_qfull, 0)) set_err(p.err, PKV_DEV_ERR_TIMEOUT);
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
            const uint64_t qdesc = umma_sdesc_sw128(q_s, 16, 1024), kdesc = umma_sdesc_sw128(k_s, 16, 1024);
            const uint64_t vdesc = umma_sdesc_sw128(v_s, kShTileBytes / 2, 1024);
            auto qk = [&](int x, int t) {  // S_x = Q_x K(t)^T, 16 dimensions a step
                const uint64_t qd = qdesc + ((x * kShTileBytes) >> 4), kd = kdesc + (((t % ST) * kShTileBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < kShD / 16; ++kk) {
                    const uint32_t at = (kk >> 2) * (kShTileBytes / 2) + (kk & 3) * 32;
                    if (leader) umma_ss(tmem + x * 128, qd + (at >> 4), kd + (at >> 4), idesc_qk, kk > 0 ? 1u : 0u);
                }
                commit(b_sfull(x));
            };
            auto pv = [&](int x, int t) {  // O_x (+)= P_x V(t), 16 keys a step
                const uint64_t vd = vdesc + (((t % ST) * kShTileBytes) >> 4);
#pragma unroll
                for (int kk = 0; kk < kShTile / 16; ++kk)
                    if (leader)
                        umma_ts(tmem + O_COL + x * 128, tmem + x * 128 + 32 * (kk / 2) + 8 * (kk % 2),
                                vd + ((kk * 16 * 128) >> 4), idesc_pv, t > 0 || kk > 0 ? 1u : 0u);
            };
            bool ok = mwait(b_qfull, 0) && mwait(b_kfull(0), 0);
            if (ok) {
                tc_fence_after();
                for (int x = 0; x < NB; ++x) qk(x, 0);
                commit(b_kempty(0));
            }
            for (int t = 0; t < n && ok; ++t) {
                const bool more = t + 1 < n;
                ok = mwait(b_vfull(t % ST), (t / ST) & 1) &&
                     (!more || mwait(b_kfull((t + 1) % ST), ((t + 1) / ST) & 1));
                if (!ok) break;
                for (int x = 0; x < NB; ++x) {
                    ok = mwait(b_pfull(x), t & 1);
                    if (!ok) break;
                    tc_fence_after();
                    pv(x, t);
                    if (!more) commit(b_odone(x));
                    else qk(x, t + 1);
                }
                if (!ok) break;
                if (more) commit(b_kempty((t + 1) % ST));
                commit(b_vempty(t % ST));
            }
            if (!ok && leader) give_up();
            commit(b_drain);  // every MMA completes before tensor memory is freed
            if (leader && !mbar_wait_drain(b_drain, 0)) set_err(p.err, PKV_DEV_ERR_TIMEOUT);
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
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int t = 0; t < n; ++t) {
            const int past = k1 - k0 - t * kShTile;  // keys of the tile from here on are not the slice's
            if (!wait_warp(b_sfull(X), t & 1)) { ok = false; break; }
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
                    const uint32_t *w = &rs[i][8 * q];
                    const float a = fmax3(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]));
                    const float b = fmax3(__uint_as_float(w[3]), __uint_as_float(w[4]), __uint_as_float(w[5]));
                    top = fmax3(top, fmaxf(a, b), fmaxf(__uint_as_float(w[6]), __uint_as_float(w[7])));
                }
            if (pos_scale) top *= sc;
            float alpha = 1.f;
            if (top > m + 8.f) {  // (first tile: from -inf)
                alpha = fast_exp2(m - top);
                m = top;
                l *= alpha;
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
            }
            l += (la.x + la.y) + (lb.x + lb.y);
            // rows of V that are no key of the slice may hold anything: zeroed by
            // block A, so that P = 0 there cannot produce 0 * NaN
            if (X == 0 && past < kShTile) {
                if (!wait_warp(b_vfull(t % ST), (t / ST) & 1)) { ok = false; break; }
                uint8_t *vbase = v_gen + (t % ST) * kShTileBytes;
                for (int q = r; q < (kShTile - past) * 16; q += 128) {
                    const int row = past + (q >> 4), c = q & 15;
                    *reinterpret_cast<uint4 *>(vbase + (c >> 3) * (kShTileBytes / 2) + row * 128 + (c & 7) * 16) =
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
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(b_pfull(X));
        }
        if (ok && !wait_warp(b_odone(X), 0)) ok = false;
        if (ok) {
            tc_fence_after();
            // the row's place in the partials, or -1 (padding, another group's)
            const int tk = r / p.group, h = r - tk * p.group, token = tok0 + X * p.tok + tk;
            const bool valid = tk < p.tok && token < tok1;
            const int64_t row = valid ? static_cast<int64_t>(split) * p.rows + static_cast<int64_t>(token) * p.Hqo +
                                            kvh * p.group + h
                                      : -1;
            const float inv = l > 0.f ? 1.f / l : (l != l ? l : 0.f);
            int64_t quad[4];  // of the rows of this lane's four
#pragma unroll
            for (int i = 0; i < 4; ++i) quad[i] = __shfl_sync(0xffffffffu, row, (lane & ~3) + i);
#pragma unroll 1
            for (int c = 0; c < kShD / 32; ++c) {
                uint32_t ro[32];
                tmem_ld32(o_addr + c * 32, ro);
                tmem_wait_ld_regs(ro);
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {  // four lanes trade pieces: a store writes 64 bytes of a row
                    uint32_t w[4][4];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e >> 2][e & 3] = __float_as_uint(__uint_as_float(ro[16 * h2 + e]) * inv);
                    transpose4(w);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (quad[i] >= 0 && dbg_in(quad[i], 1, p.rows * p.n_split, p.err))
                            *reinterpret_cast<uint4 *>(p.ws_o + quad[i] * kShD + c * 32 + h2 * 16 + (lane & 3) * 4) =
                                make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                }
            }
            if (valid && dbg_in(row, 1, p.rows * p.n_split, p.err))
                p.ws_lse[row] = l > 0.f ? m + fast_log2(l) : (l != l ? l : -INFINITY);
        } else {
            give_up();
        }
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

// One warp per output row: the partials of its group's prefix and of its own
// keys, weighted by 2^lse, and the sink.
struct SharedMerge {
    SharedParams s;
    DecodeParams d;  // the own keys' partials, the outputs
};
template <typename T>
__global__ void __launch_bounds__(128) shared_merge_kernel(const __grid_constant__ SharedMerge mp) {
    const SharedParams &p = mp.s;
    const DecodeParams &d = mp.d;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= p.rows) return;
    const int h = static_cast<int>(row % p.Hqo), token = static_cast<int>(row / p.Hqo);
    const int b = token / p.Q, t = token - b * p.Q;
    int lo = 0, hi = 0, u0 = 0, n_prefix = 0;
    bool bad;
    const int g = find_group(p.group_indptr, p.G, p.B, b, [](int x, int y) { return y - x; }, lo, hi, u0, bad);
    if (g >= 0) n_prefix = (min(max(p.prefix_lens[g], 0), p.max_prefix) + p.chunk - 1) / p.chunk;
    const uint32_t L_in = d.seq_lens[b];
    const int L = L_in > static_cast<uint32_t>(d.max_seq_len) ? d.max_seq_len : static_cast<int>(L_in);
    int k_lo, first, n_own;
    decode_split_geometry(L, p.Q, -1, d.chunk, k_lo, first, n_own);
    const int kvh = h / p.group;
    const int64_t own = static_cast<int64_t>(b * p.Hkv + kvh) * d.n_split_max * d.R + t * p.group + (h - kvh * p.group);
    if (!dbg_in(own, static_cast<int64_t>(n_own - 1) * d.R + 1, d.ws_rows, d.err) ||
        !dbg_in(n_prefix, 0, p.n_split, d.err))
        return;
    const int n = n_prefix + n_own;
    auto lse_at = [&](int i) { return i < n_prefix ? p.ws_lse + i * p.rows + row : d.ws_lse + own + static_cast<int64_t>(i - n_prefix) * d.R; };
    auto o_at = [&](int i) {
        return i < n_prefix ? p.ws_o + (i * p.rows + row) * kShD : d.ws_o + (own + static_cast<int64_t>(i - n_prefix) * d.R) * kShD;
    };
    const float sink = d.sinks ? d.sinks[h] * kLog2e : -INFINITY;
    float M = sink, den = 0.f, nan = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += 32) {  // 32 partials at a time, a lane each for their weights
        const float x = i0 + lane < n ? *lse_at(i0 + lane) : -INFINITY;
        float top = x;
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (__any_sync(0xffffffffu, x != x)) nan = __int_as_float(0x7fc00000);
        const float mn = fmaxf(M, top);
        if (mn == -INFINITY) continue;
        const float keep = fast_exp2(M - mn), w = fast_exp2(x - mn);
        M = mn;
        den *= keep;
        acc.x *= keep;
        acc.y *= keep;
        acc.z *= keep;
        acc.w *= keep;
        const int m = min(32, n - i0);
#pragma unroll 4
        for (int i = 0; i < m; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const float4 v = *reinterpret_cast<const float4 *>(o_at(i0 + i) + lane * 4);
            den += wi;
            acc.x += wi * v.x;
            acc.y += wi * v.y;
            acc.z += wi * v.z;
            acc.w += wi * v.w;
        }
    }
    if (d.sinks && M != -INFINITY) den += fast_exp2(sink - M);
    const float bmm2 = d.bmm2_dev ? __ldg(d.bmm2_dev) : d.bmm2;
    float sc = den > 0.f ? bmm2 / den : 0.f;
    float lse_v = den > 0.f ? (M + fast_log2(den)) * kLn2 : -INFINITY;
    if (nan != nan) sc = lse_v = nan;  // a NaN among the visible keys
    store4(static_cast<T *>(d.out) + row * kShD + lane * 4, acc.x * sc, acc.y * sc, acc.z * sc, acc.w * sc);
    if (d.lse && lane == 0) d.lse[row] = lse_v;
}

struct SharedPlan {
    DecodePlan own;
    int nb, tok, tiles, chunk, n_split;
    int64_t rows;
    size_t prefix_o, prefix_lse, own_o, own_lse, bytes;  // offsets in the workspace
};

static int plan_shared(int B, int Q, int Hqo, int Hkv, int D, int G, int max_prefix, int max_seq_len, int page_size,
                       SharedPlan &pl) {
    if (G < 0 || max_prefix < 0) return PKV_ERR_INVALID_ARG;
    const int rc = plan_decode(B, Q, Hqo, Hkv, D, max_seq_len, page_size, -1, pl.own);
    if (rc != PKV_OK) return rc;
    const int group = Hqo / Hkv;
    if (max_prefix > (1 << 30) || static_cast<int64_t>(B) * Q * Hqo > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    pl.rows = static_cast<int64_t>(B) * Q * Hqo;
    pl.tok = 128 / group;
    const int64_t tokens = static_cast<int64_t>(B) * Q;
    // Two blocks to a CTA where the groups' rows fill more than one on average.
    pl.nb = tokens > static_cast<int64_t>(pl.tok) * (G > 0 ? G : 1) ? 2 : 1;
    // tiles of tokens, each group's last one partly filled
    const int64_t T = static_cast<int64_t>(pl.nb) * pl.tok;
    int64_t tiles = (tokens + static_cast<int64_t>(G) * (T - 1)) / T;
    if (tiles > tokens) tiles = tokens;
    if (tiles > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    pl.tiles = static_cast<int>(tiles);
    // Slices of the prefix: what the rounds of CTAs take, in tiles of 128 keys,
    // a CTA's start and end counted as four, and the partials that a slice adds
    // (8.5 MB of them, written and read, as one).
    const int64_t all = (static_cast<int64_t>(max_prefix) + kShTile - 1) / kShTile;
    const int64_t sms = num_sms(), items = tiles * Hkv;
    int64_t best = 1;
    double least = 0;
    for (int64_t ns = 1; ns <= all && ns <= 128; ++ns) {
        const int64_t per = (all + ns - 1) / ns;
        if ((all + per - 1) / per != ns) continue;  // (fewer slices do the same)
        const double cost = static_cast<double>((items * ns + sms - 1) / sms) * static_cast<double>(per + 4) +
                            static_cast<double>(ns) * static_cast<double>(pl.rows) * 1024 / 8.5e6;
        if (ns == 1 || cost < least) {
            least = cost;
            best = ns;
        }
    }
    pl.n_split = static_cast<int>(best);
    pl.chunk = all > 0 ? static_cast<int>((all + best - 1) / best) * kShTile : kShTile;
    const size_t slots = static_cast<size_t>(B) * Hkv * pl.own.n_split_max * pl.own.R;
    size_t at = 0;
    pl.prefix_o = at;
    at += round_up(static_cast<size_t>(pl.n_split) * pl.rows * kShD * sizeof(float), 256);
    pl.prefix_lse = at;
    at += round_up(static_cast<size_t>(pl.n_split) * pl.rows * sizeof(float), 256);
    pl.own_o = at;
    at += round_up(slots * kShD * sizeof(float), 256);
    pl.own_lse = at;
    at += round_up(slots * sizeof(float), 256);
    pl.bytes = at;
    return PKV_OK;
}

template <typename T, int LAYOUT, int NB>
static int launch_prefix(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const SharedParams &p,
                         dim3 grid, cudaStream_t st) {
    auto kern = shared_prefix_kernel<T, LAYOUT, NB>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(ShCfg<NB>::SMEM)) !=
        cudaSuccess)
        return PKV_ERR_CUDA;
    if constexpr (NB == 2) {
        // the register split draws on what the CTA is launched with: refuse to
        // launch if the compiled kernel has fewer (setmaxnreg.inc would wait forever)
        static int ok = -1;
        if (ok < 0) {
            cudaFuncAttributes fa;
            if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return PKV_ERR_CUDA;
            ok = fa.numRegs * ShCfg<NB>::THREADS >= 128 * kShRegsLow + 256 * kShRegsHigh ? 1 : 0;
        }
        if (!ok) return PKV_ERR_UNSUPPORTED;
    }
    kern<<<grid, ShCfg<NB>::THREADS, ShCfg<NB>::SMEM, st>>>(tq, tk, tv, p);
    return PKV_OK;
}

template <typename T>
static int run_shared(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const SharedParams &s,
                      const DecodeParams &d, const SharedPlan &pl, int layout, cudaStream_t st) {
    const bool hnd = layout == PKV_HND, prefix = s.max_prefix > 0 && s.G > 0;
    int launches = 2;
    if (prefix) {
        const dim3 grid(pl.tiles, s.Hkv, pl.n_split);
        const int rc = pl.nb == 2 ? (hnd ? launch_prefix<T, PKV_HND, 2>(tq, tk, tv, s, grid, st)
                                         : launch_prefix<T, PKV_NHD, 2>(tq, tk, tv, s, grid, st))
                                  : (hnd ? launch_prefix<T, PKV_HND, 1>(tq, tk, tv, s, grid, st)
                                         : launch_prefix<T, PKV_NHD, 1>(tq, tk, tv, s, grid, st));
        if (rc != PKV_OK) return rc;
        ++launches;
    }
    const dim3 grid(pl.own.n_split_max, s.Hkv, s.B);
    const int rc = hnd ? launch_split_mt<T, PKV_HND, false, 3>(pl.own.MT, d, grid, st, prefix)
                       : launch_split_mt<T, PKV_NHD, false, 3>(pl.own.MT, d, grid, st, prefix);
    if (rc != PKV_OK) return rc;
    SharedMerge m{s, d};
    if (launch_dependent(shared_merge_kernel<T>, dim3(static_cast<unsigned>((s.rows + 3) / 4)), dim3(128), 0, st, m) !=
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
    s.group_indptr = group_indptr;
    s.prefix_lens = prefix_lens;
    s.prefix_tables = prefix_tables;
    s.pt_stride = prefix_table_stride;
    s.G = num_groups;
    s.B = batch_size;
    s.Q = q_len_per_req;
    s.Hqo = num_qo_heads;
    s.Hkv = num_kv_heads;
    s.group = num_qo_heads / num_kv_heads;
    s.tok = pl.tok;
    s.max_prefix = max_prefix_len;
    s.page_shift = ilog2_exact(page_size);
    s.chunk = pl.chunk;
    s.n_split = pl.n_split;
    s.max_num_pages = max_num_pages;
    s.scale_log2 = bmm1_scale * kLog2e;
    s.bmm1_dev = bmm1_scale_dev;
    s.ws_o = reinterpret_cast<float *>(ws + pl.prefix_o);
    s.ws_lse = reinterpret_cast<float *>(ws + pl.prefix_lse);
    s.rows = pl.rows;
    s.err = err_word;
    s.wait_ns = wait_limit_ns();

    DecodeParams d = {};
    d.q = query;
    d.k = k_cache;
    d.v = v_cache;
    d.page_stride = page_stride;
    d.max_num_pages = max_num_pages;
    d.block_tables = block_tables;
    d.bt_stride = block_table_stride;
    d.seq_lens = seq_lens;
    d.B = batch_size;
    d.max_seq_len = max_seq_len;
    d.scale_log2 = bmm1_scale * kLog2e;
    d.bmm1_dev = bmm1_scale_dev;
    d.bmm2_dev = bmm2_scale_dev;
    d.bmm2 = bmm2_scale;
    d.window_left = -1;
    d.sinks = sinks;
    d.Q = q_len_per_req;
    d.Hqo = num_qo_heads;
    d.Hkv = num_kv_heads;
    d.group = s.group;
    d.R = pl.own.R;
    d.num_tokens = static_cast<int64_t>(batch_size) * q_len_per_req;
    d.kv_extent = max_num_pages > 0 ? (max_num_pages - 1) * page_stride + page : 0;
    d.ws_rows = static_cast<int64_t>(batch_size) * num_kv_heads * pl.own.n_split_max * pl.own.R;
    d.page_shift = s.page_shift;
    d.chunk = pl.own.chunk;
    d.n_split_max = pl.own.n_split_max;
    d.out = out;
    d.lse = lse;
    d.ws_o = reinterpret_cast<float *>(ws + pl.own_o);
    d.ws_lse = reinterpret_cast<float *>(ws + pl.own_lse);
    d.err = err_word;

    CUtensorMap tq, tk, tv;
    if (num_groups > 0 && max_prefix_len > 0) {
        const CUtensorMapDataType t = dtype == PKV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        // a block of rows in one box for each half of the head: (64 elements,
        // the group's heads, whole tokens)
        const uint64_t dims[3] = {kShD, static_cast<uint64_t>(num_qo_heads), static_cast<uint64_t>(d.num_tokens)};
        const uint64_t strides[2] = {kShD * 2, static_cast<uint64_t>(num_qo_heads) * kShD * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(s.group), static_cast<uint32_t>(s.tok)};
        const int rows = pf_box_rows(page_size, kShTile);
        const int64_t pages = max_num_pages > 0 ? max_num_pages : 1;
        if (!encode_tmap(&tq, query, t, 3, dims, strides, box) ||
            !cache_tmap(&tk, k_cache, t, layout, kShD, page_size, num_kv_heads, page_stride, pages, rows) ||
            !cache_tmap(&tv, v_cache, t, layout, kShD, page_size, num_kv_heads, page_stride, pages, rows))
            return PKV_ERR_CUDA;
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == PKV_BF16 ? run_shared<__nv_bfloat16>(tq, tk, tv, s, d, pl, layout, st)
                             : run_shared<__half>(tq, tk, tv, s, d, pl, layout, st);
}
