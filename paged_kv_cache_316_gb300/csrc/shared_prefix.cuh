// shared_prefix.cuh -- how the prefixes of a shared decode are cut into work
// and where the partial results of a row lie: the part that the prefix kernel
// (decode_shared.cu) and the kernels that join its partials agree on.
//
// Work.  CTAs come in teams of `team` neighbours (1 where nothing is won, see
// plan_shared).  An item is `team` tiles of a group's tokens (a tile: nb blocks
// of `tok` tokens), one for each member, at one kv head; it takes nk =
// ceil(prefix / 128) steps, a step being a tile of 128 keys, which the members
// read at about the same time: from HBM once.  The items of all groups laid
// end to end (by group, kv head, tiles of tokens) are W steps, of which team c
// takes [c per, (c + 1) per): the lengths and sizes are read on the device, so
// that the cut is even whatever they are, and every kernel that needs it works
// it out again.  A CTA's run through one item is a segment; only its first can
// begin inside an item.
//
// Partials: one array of fp32 output rows and one of base-2 LSEs.  Row (token,
// head) of the segment that begins the item: index token * Hqo + head; of a
// segment that continues it: rows + (cta * nb + block) * 128 + row of the
// block; then, from `parts` on, those of the own keys (shared_own.cuh).
#pragma once

#include "pkv_common.cuh"

namespace pkv {

constexpr int kShTile = 128;  // keys per step
constexpr float kShCtaSteps = 5.f;  // what a CTA of the prefix kernel costs beside its steps

struct PrefixWork {
    const int32_t *group_indptr, *prefix_lens;
    const uint32_t *seq_lens;  // own keys
    int max_seq_len;
    int G, B, Q, Hqo, Hkv, group;
    int tok, nb;  // tokens of a block (128 / group), blocks of an item
    int max_prefix;
    int team, ctas;  // ctas: a multiple of team
    int sms;
    uint32_t rows;   // B * Q * Hqo
    uint32_t parts;  // rows + ctas * nb * 128 (0 without a prefix)
    uint32_t all;    // parts and the own keys' rows
    float *ws_o;     // [all][128]
    float *ws_lse;   // [all]
    uint32_t *per;   // prefix_steps_per_team, for the kernel that joins
    int32_t *err;
};

// One group: its requests [a, b), its prefix of P keys in nk steps, its tiles
// of tokens and items at a kv head, and the number of its first step.
struct PrefixGroup {
    int g, a, b, P, nk, tiles, items;
    uint32_t base;
};

__device__ __forceinline__ void read_prefix_group(const PrefixWork &p, int g, PrefixGroup &x) {
    x.g = g;
    x.a = p.group_indptr[g];
    x.b = p.group_indptr[g + 1];
    x.P = min(max(p.prefix_lens[g], 0), p.max_prefix);
    x.nk = (x.P + kShTile - 1) / kShTile;
    const int T = p.nb * p.tok;
    x.tiles = ((x.b - x.a) * p.Q + T - 1) / T;
    x.items = (x.tiles + p.team - 1) / p.team;
}

// All groups, by one warp: calls total(W), then finds the group for which
// match(a, b, first step, steps) holds (g = -1: none).  Where group_indptr is
// not in order no group has work (*bad).  Up to 32 groups are read once, more
// of them twice.
template <typename G, typename F>
__device__ __forceinline__ void scan_prefixes(const PrefixWork &p, G total, F match, PrefixGroup &found, bool &bad) {
    const int lane = threadIdx.x & 31;
    found.g = -1;
    bad = false;
    PrefixGroup x = {};
    uint32_t n = 0, sum = 0;  // steps of this lane's group; of it and the lanes before
    for (int pass = p.G <= 32 ? 1 : 0; pass < 2; ++pass) {
        uint32_t carry = 0;
        for (int g0 = 0; g0 < p.G; g0 += 32) {
            const int g = g0 + lane;
            bool wrong = false;
            if (g < p.G) {
                read_prefix_group(p, g, x);
                wrong = x.a < 0 || x.b < x.a || x.b > p.B || (g == 0 && x.a != 0);
            }
            if (__any_sync(0xffffffffu, wrong)) bad = true;
            if (bad) break;
            sum = n = g < p.G ? static_cast<uint32_t>(x.items) * p.Hkv * x.nk : 0u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
            if (p.G <= 32) total(all);
            if (pass == 1) {
                const unsigned m = __ballot_sync(0xffffffffu, g < p.G && match(x.a, x.b, carry + sum - n, n));
                if (m && found.g < 0) {
                    const int j = __ffs(m) - 1;
                    found.g = g0 + j;
                    found.a = __shfl_sync(0xffffffffu, x.a, j);
                    found.b = __shfl_sync(0xffffffffu, x.b, j);
                    found.P = __shfl_sync(0xffffffffu, x.P, j);
                    found.nk = __shfl_sync(0xffffffffu, x.nk, j);
                    found.tiles = __shfl_sync(0xffffffffu, x.tiles, j);
                    found.items = __shfl_sync(0xffffffffu, x.items, j);
                    found.base = carry + __shfl_sync(0xffffffffu, sum - n, j);
                }
            }
            carry += all;
        }
        if (bad) {
            found.g = -1;
            return;
        }
        if (pass == 0) total(carry);
    }
}

// What is wrong with the groups, into the error word, by one warp.
__device__ __forceinline__ void report_prefixes(const PrefixWork &p, bool bad) {
    const int lane = threadIdx.x & 31;
    if (bad && lane == 0) set_err(p.err, PKV_DEV_ERR_BATCH);
    for (int g = lane; g < p.G && !bad; g += 32)
        if (p.prefix_lens[g] < 0 || p.prefix_lens[g] > p.max_prefix) set_err(p.err, PKV_DEV_ERR_LEN);
}

// Steps of a team, by one warp.  N CTAs take C + W / N steps' time each (C =
// kShCtaSteps), and the other SMs stream own keys meanwhile, which cost one SM A
// steps: both are done at the same time T, and S SMs busy until then, if
//   T = C + W / N,  S T = C N + W + A,  so  C N^2 + (W + A - C S) N - W S = 0
// (W the CTAs' steps; N = S without own keys).  A: 128 own keys of a head are
// streamed in about a step; of more than 256 requests, 256 spread evenly over
// the batch stand for all.  So few steps that half of the SMs have one each are
// not put together.  Every CTA of the prefix kernel works it out alike; the
// kernel that joins reads it.
// Against all SMs for the prefix first: 220 us for 226 (256 requests behind
// 32,768 keys), 46 for 50 (64 behind 8,192), 42.5 for 45 (45 of 4 tokens in
// three groups); A from 0.8 to 1 of this the same, from 0.7 or 1.5 slower.
// The lengths are fetched first, beside the groups that W is found from.
struct OwnLengths {
    uint32_t x[8];  // of n = min(B, 256) requests, the (lane + 32 i)-th of them
    float each;     // requests that one stands for, B / n
};
__device__ __forceinline__ OwnLengths own_lengths(const PrefixWork &p) {
    const int lane = threadIdx.x & 31, n = min(p.B, 256);
    OwnLengths r;
    r.each = p.B > 256 ? static_cast<float>(p.B) / 256.f : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = lane + 32 * i, b = p.B > 256 ? (k * p.B) >> 8 : k;  // (k B / n; B < 2^16)
        r.x[i] = k < n ? p.seq_lens[b] : 0u;
    }
    return r;
}
__device__ __forceinline__ uint32_t prefix_steps_per_team(const PrefixWork &p, uint32_t W, const OwnLengths &own) {
    const uint32_t least = (W + p.ctas / p.team - 1) / (p.ctas / p.team);
    const uint64_t w = static_cast<uint64_t>(W) * p.team;
    if (2 * w <= static_cast<uint32_t>(p.sms)) return max(least, 1u);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += static_cast<float>(min(own.x[i], static_cast<uint32_t>(p.max_seq_len)));
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float A = sum * own.each * static_cast<float>(p.Hkv) / kShTile, S = static_cast<float>(p.sms), steps = static_cast<float>(w);
    const float half = 0.5f * (steps + A - kShCtaSteps * S);
    const float N = (sqrtf(half * half + kShCtaSteps * steps * S) - half) / kShCtaSteps;
    const uint32_t teams = max(1u, min(static_cast<uint32_t>(N), static_cast<uint32_t>(p.ctas)) / p.team);
    return max(least, (W + teams - 1) / teams);
}

// The partials of a token's rows at one kv head: the first at `row` (of the
// kv head's first query head), n in all, the others at extra + i * step.
struct PrefixParts {
    int n;
    uint32_t row, extra, step;
    __device__ __forceinline__ uint32_t at(int i) const { return i == 0 ? row : extra + static_cast<uint32_t>(i) * step; }
};
__device__ __forceinline__ PrefixParts prefix_parts(const PrefixWork &p, const PrefixGroup &x, uint32_t per, int token, int kvh) {
    PrefixParts r;
    r.n = 0;
    r.row = static_cast<uint32_t>(token) * p.Hqo + kvh * p.group;
    r.extra = 0;
    r.step = p.team * p.nb * 128;
    if (x.g < 0 || x.nk == 0) return r;
    const int T = p.nb * p.tok, tk = token - x.a * p.Q, tile = tk / T, in = tk - tile * T, block = in / p.tok;
    const int item = tile / p.team, member = tile - item * p.team;
    const uint32_t s0 = x.base + (static_cast<uint32_t>(kvh) * x.items + item) * x.nk, c0 = s0 / per;
    r.n = static_cast<int>((s0 + x.nk - 1) / per - c0) + 1;
    r.extra = p.rows + ((c0 * p.team + member) * p.nb + block) * 128 + (in - block * p.tok) * p.group;
    return r;
}

}  // namespace pkv
