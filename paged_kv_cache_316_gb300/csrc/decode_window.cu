// decode_window.cu -- the decode kernels for a sliding window that keeps a few
// first tokens visible, and for an E4M3 cache with a scale for each block of
// keys and head (the kernels are in decode_split.cuh, EXT 1 and 2).
#include "decode_split.cuh"

namespace pkv {

template <typename T>
static int run_ext(const DecodeParams &p, const DecodePlan &pl, int layout, bool kv8, bool pdl, cudaStream_t st) {
    dim3 grid(pl.n_split_max, p.Hkv, p.B);
    const bool hnd = layout == PKV_HND;
    int rc;
    if (p.k_scales)
        rc = hnd ? launch_split_mt<T, PKV_HND, true, 2>(pl.MT, p, grid, st, pdl)
                 : launch_split_mt<T, PKV_NHD, true, 2>(pl.MT, p, grid, st, pdl);
    else if (kv8)
        rc = hnd ? launch_split_mt<T, PKV_HND, true, 1>(pl.MT, p, grid, st, pdl)
                 : launch_split_mt<T, PKV_NHD, true, 1>(pl.MT, p, grid, st, pdl);
    else
        rc = hnd ? launch_split_mt<T, PKV_HND, false, 1>(pl.MT, p, grid, st, pdl)
                 : launch_split_mt<T, PKV_NHD, false, 1>(pl.MT, p, grid, st, pdl);
    if (rc != PKV_OK) return rc;
    int launches = 1;
    if (pl.n_split_max > 1) {
        const int64_t rows = static_cast<int64_t>(p.B) * p.Q * p.Hqo;
        if (launch_dependent(decode_merge_kernel<T, true>, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0,
                             st, p) != cudaSuccess)
            return PKV_ERR_CUDA;
        ++launches;
    }
    note_launches(launches);
    return launch_status();
}

int run_decode_ext(const DecodeParams &p, const DecodePlan &pl, int layout, bool bf16, bool kv8, bool pdl,
                   cudaStream_t st) {
    return bf16 ? run_ext<__nv_bfloat16>(p, pl, layout, kv8, pdl, st) : run_ext<__half>(p, pl, layout, kv8, pdl, st);
}

}  // namespace pkv
