// Attention of one new token per sequence over its whole paged cache (shadowkv_paged_attention): the kernels of
// paged_attn.cuh for bf16, e5m2 and fp32, with and without weights.
#include "paged_attn.cuh"

namespace skv {

int paged_attn_ctas(int dtype, int d, int nsm) { return nsm * occ_of(dtype, d); }

int launch_paged_attn(int dtype, int d, const PagedAttnParams& p, int ncta, cudaStream_t s) {
    if (dtype == SKV_F32) return d == 64 ? launch_f32<64, false>(p, ncta, s) : launch_f32<128, false>(p, ncta, s);
    if (dtype == SKV_FP8)
        return d == 64 ? launch_pa<TileTC<64, Holds::kE5M2>, 64, false, 8>(p, ncta, s)
                       : launch_pa<TileTC<128, Holds::kE5M2>, 128, false, 8>(p, ncta, s);
    return d == 64 ? launch_pa<TileTC<64, Holds::kBf16>, 64, false, 8>(p, ncta, s)
                   : launch_pa<TileTC<128, Holds::kBf16>, 128, false, 8>(p, ncta, s);
}

cudaError_t paged_attn_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
