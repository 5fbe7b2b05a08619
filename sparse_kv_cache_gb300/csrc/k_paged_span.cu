// Attention of one new token per sequence over the rows that a window and the first rows leave, and over caches of
// e4m3 codes (shadowkv_paged_attention_ext): the kernels of paged_attn.cuh for all types, without weights.
#include "paged_attn.cuh"

namespace skv {

int launch_paged_span(int dtype, int d, const PagedAttnParams& p, int ncta, cudaStream_t s) {
    if (dtype == SKV_F32) return d == 64 ? launch_f32<64, true>(p, ncta, s) : launch_f32<128, true>(p, ncta, s);
    if (dtype == SKV_FP8)
        return d == 64 ? launch_pa<TileTC<64, Holds::kE5M2, true>, 64, false, 8>(p, ncta, s)
                       : launch_pa<TileTC<128, Holds::kE5M2, true>, 128, false, 8>(p, ncta, s);
    return d == 64 ? launch_pa<TileTC<64, Holds::kBf16, true>, 64, false, 8>(p, ncta, s)
                   : launch_pa<TileTC<128, Holds::kBf16, true>, 128, false, 8>(p, ncta, s);
}

int launch_paged_codes(int d, const PagedCodesParams& p, int ncta, cudaStream_t s) {
    return d == 64 ? launch_pa<TileTC<64, Holds::kE4M3, true>, 64, false, 8>(p, ncta, s)
                   : launch_pa<TileTC<128, Holds::kE4M3, true>, 128, false, 8>(p, ncta, s);
}

cudaError_t paged_span_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
