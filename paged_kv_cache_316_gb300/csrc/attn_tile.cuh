// attn_tile.cuh -- pieces shared by the tcgen05 attention kernels: the tensor
// map of a paged cache, and what a softmax thread does with its row.
#pragma once

#include "pkv_common.cuh"
#include "sm103_ptx.cuh"

namespace pkv {

// Rows per TMA box: pages, or parts of pages of the largest power of two
// dividing BN, so that no box crosses a page and the boxes tile a key tile.
__host__ __device__ __forceinline__ int pf_box_rows(int page_size, int bn) {
    const int p2 = bn & -bn;
    return page_size < p2 ? page_size : p2;
}

template <typename T>
struct IsBf16 {
    static constexpr bool value = false;
};
template <>
struct IsBf16<__nv_bfloat16> {
    static constexpr bool value = true;
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// max of three floats in one instruction
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The n low bits set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// 4 x 4 transpose of 16-byte pieces over four neighbouring lanes: piece i of
// lane q becomes what was piece q of lane i.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d <= 2; d *= 2) {
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & d) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[i][e] : w[i + d][e], d);
                w[i][e] = up ? got : w[i][e];
                w[i + d][e] = up ? w[i + d][e] : got;
            }
        }
    }
}

// Wait for this thread's tensor-memory loads, with the 32 destination
// registers as operands so that no use of them can be scheduled before it.
__device__ __forceinline__ void tmem_wait_ld_regs(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]),
                   "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]),
                   "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// K or V cache as a 4-D tensor map whose box is one 128-byte d-atom (64
// 16-bit or 128 one-byte elements, es bytes each) of `rows` consecutive
// slots of one (page, kv head).
inline bool cache_tmap(CUtensorMap *m, const void *base, CUtensorMapDataType dt, int layout, int d,
                       int page_size, int num_kv_heads, int64_t page_stride, int64_t num_pages,
                       int rows, int es = 2) {
    uint64_t dims[4], strides[3];
    uint32_t box[4];
    dims[0] = d;
    box[0] = 128 / es;
    strides[0] = static_cast<uint64_t>(d) * es;
    if (layout == PKV_HND) {
        dims[1] = page_size;
        dims[2] = num_kv_heads;
        strides[1] = static_cast<uint64_t>(page_size) * d * es;
        box[1] = rows;
        box[2] = 1;
    } else {
        dims[1] = num_kv_heads;
        dims[2] = page_size;
        strides[1] = static_cast<uint64_t>(num_kv_heads) * d * es;
        box[1] = 1;
        box[2] = rows;
    }
    dims[3] = static_cast<uint64_t>(num_pages);
    strides[2] = static_cast<uint64_t>(page_stride) * es;
    box[3] = 1;
    return encode_tmap(m, base, dt, 4, dims, strides, box);
}

}  // namespace pkv
