// merge_states.cu -- attention over separate parts of the keys, merged: with
// (o_i, l_i) the output and log-sum-exp over part i,
//   L = log sum e^(l_i),  out = sum e^(l_i - L) o_i.
// A part in which a row sees nothing has l_i = -inf and counts for nothing,
// whatever its o_i holds; a row that sees nothing anywhere gets 0 and -inf.
//
// One pass: a lane holds 16 bytes of a row of every part and keeps the running
// maximum and sum of the softmax over the parts in fp32; the result is rounded
// once.  All lanes of a row are in one warp, so that a result may replace the
// part it was made from.  HBM bounds it.
#include "pkv_common.cuh"

namespace pkv {

constexpr int kMergeMax = PKV_MERGE_MAX_STATES;
struct MergeParams {
    const uint16_t *o[kMergeMax];
    const float *lse[kMergeMax];
    int n;
    int64_t rows;
    int chunks, lanes_shift;  // 16-byte chunks of a row; log2 of the lanes it takes
    uint16_t *out;
    float *out_lse;
};

template <typename T>
__device__ __forceinline__ float2 merge_unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 merge_unpack<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <>
__device__ __forceinline__ float2 merge_unpack<__nv_bfloat16>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

constexpr int kMergeThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) merge_states_kernel(const __grid_constant__ MergeParams p) {
    const int64_t thread = static_cast<int64_t>(blockIdx.x) * kMergeThreads + threadIdx.x;
    const int64_t row = thread >> p.lanes_shift;
    const int c = static_cast<int>(thread) & ((1 << p.lanes_shift) - 1);
    const bool on = row < p.rows && c < p.chunks;
    float m = -INFINITY, total = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    constexpr int kBatch = 4;
    for (int i0 = 0; i0 < p.n; i0 += kBatch) {
        float l[kBatch];
        uint4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            l[k] = -INFINITY;
            x[k] = make_uint4(0u, 0u, 0u, 0u);
            if (on && i0 + k < p.n) {
                l[k] = p.lse[i0 + k][row];
                x[k] = *reinterpret_cast<const uint4 *>(p.o[i0 + k] + (row * p.chunks + c) * 8);
            }
        }
        const float mn = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), m);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float keep = fast_exp2((m - base) * kLog2e);
        total *= keep;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= keep;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            // -1: nothing is seen.  (A weight that is 0 by underflow counts: a NaN
            // in its part stays one in any order of the parts.)
            const float w = l[k] == -INFINITY ? -1.f : fast_exp2((l[k] - base) * kLog2e);
            if (!(w < 0.f)) {
                total += w;
                const uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = merge_unpack<T>(v[e]);
                    acc[2 * e] = fmaf(w, f.x, acc[2 * e]);
                    acc[2 * e + 1] = fmaf(w, f.y, acc[2 * e + 1]);
                }
            }
        }
        m = mn;
    }
    __syncwarp();  // every lane of the row has read its parts
    if (!on) return;
    const float inv = total != 0.f ? 1.f / total : 0.f;
    *reinterpret_cast<uint4 *>(p.out + (row * p.chunks + c) * 8) =
        make_uint4(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv),
                   pack2<T>(acc[4] * inv, acc[5] * inv), pack2<T>(acc[6] * inv, acc[7] * inv));
    if (c == 0) p.out_lse[row] = total != 0.f ? m + logf(total) : -INFINITY;
}

}  // namespace pkv

using namespace pkv;

extern "C" int paged_merge_states(const void *const *outs, const float *const *lses, int32_t num_states, int64_t rows,
                                  int32_t head_dim, int32_t dtype, void *out, float *lse, void *stream) {
    const CallRange nvtx_range("paged_merge_states");
    if (dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_INVALID_ARG;
    if (num_states < 1 || rows < 0 || head_dim <= 0 || head_dim % 8) return PKV_ERR_INVALID_ARG;
    if (num_states > kMergeMax || head_dim > 256) return PKV_ERR_UNSUPPORTED;
    if (rows == 0) return PKV_OK;
    if (!outs || !lses || !out || !lse) return PKV_ERR_NULL;
    MergeParams p = {};
    for (int i = 0; i < num_states; ++i) {
        if (!outs[i] || !lses[i]) return PKV_ERR_NULL;
        if (!aligned16(outs[i]) || (reinterpret_cast<uintptr_t>(lses[i]) & 3)) return PKV_ERR_INVALID_ARG;
        p.o[i] = static_cast<const uint16_t *>(outs[i]);
        p.lse[i] = lses[i];
    }
    if (!aligned16(out) || (reinterpret_cast<uintptr_t>(lse) & 3)) return PKV_ERR_INVALID_ARG;
    p.n = num_states;
    p.rows = rows;
    p.chunks = head_dim / 8;
    while ((1 << p.lanes_shift) < p.chunks) ++p.lanes_shift;
    p.out = static_cast<uint16_t *>(out);
    p.out_lse = lse;
    const int64_t blocks = ((rows << p.lanes_shift) + kMergeThreads - 1) / kMergeThreads;
    if (blocks > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == PKV_BF16)
        merge_states_kernel<__nv_bfloat16><<<static_cast<unsigned>(blocks), kMergeThreads, 0, st>>>(p);
    else
        merge_states_kernel<__half><<<static_cast<unsigned>(blocks), kMergeThreads, 0, st>>>(p);
    note_launches(1);
    return launch_status();
}
