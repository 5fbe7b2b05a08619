// Norm, rotation and cache append of queries and keys (shadowkv_qk_norm_rope).
//
// Per head x of a token: y = x / sqrt(mean(x^2) + eps) * w, then the pairs (y_i, y_{i + rd/2})
// turn by position * base^(-2i/rd).  Each element is read once and written once (a key twice
// where it is handed on and appended), so memory bounds a prompt and launch latency a decode step.
//
// A row (one head of one token) belongs to d/16 lanes.  Lane c < rd/16 holds the elements
// 8c .. 8c+7 of the first half and their partners behind rd/2, so the rotation needs no exchange
// between lanes; lanes behind hold 16 consecutive elements that pass through.  Only the sum of
// squares crosses lanes.  The cos and sin of a token's rd/2 angles are formed once per token by
// rd/2 threads and shared by all of its heads.
//
// Angles: position * theta_i in turns is kept in 64-bit fixed point, where whole turns fall off
// the top by themselves, so the reduction is exact for every int32 position; the 32 leading bits
// of the remaining turn, as a fraction of pi, go to sincospi (error below 2^-23 of a half turn).
#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kNrThreads = 256;
constexpr int kNrMaxTok = 16;     // tokens per CTA at most

// 16 elements of a row: 8 at o1, 8 at o2
template <typename T>
__device__ __forceinline__ void load16(const T* p, int o1, int o2, float (&a)[8], float (&z)[8]) {
    load8(p + o1, a);
    load8(p + o2, z);
}

template <typename T, int D, bool kE5M2>
__global__ void __launch_bounds__(kNrThreads) k_norm_rope(const __grid_constant__ NormRopeParams p) {
    constexpr int kLanes = D / 16;                  // lanes of a row
    constexpr int kRows = kNrThreads / kLanes;      // rows in flight
    __shared__ float s_cos[kNrMaxTok * D / 2], s_sin[kNrMaxTok * D / 2];
    __shared__ int s_pos[kNrMaxTok];

    const int tid = threadIdx.x, c = tid % kLanes, half = p.rd / 2;
    const int t0 = blockIdx.x * p.per_cta, nt = min(p.per_cta, p.tokens - t0);
    if (tid < nt) s_pos[tid] = __ldg(p.positions + t0 + tid);
    for (int i = tid; i < nt * half; i += kNrThreads) {
        const int t = i / half, f = i % half;
        const int pos = __ldg(p.positions + t0 + t);
        const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.turn[f];
        float sn, cs;
        sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &sn, &cs);
        s_cos[t * (D / 2) + f] = cs;
        s_sin[t * (D / 2) + f] = sn;
    }
    __syncthreads();

    const bool turns = c < p.rd / 16;
    const int o1 = turns ? 8 * c : p.rd + 16 * (c - p.rd / 16);
    const int o2 = turns ? half + 8 * c : o1 + 8;
    const bool cache = p.c.k != nullptr;
    const int per_tok = p.nq + p.c.H * (cache ? 2 : 1);
    const int rows = nt * per_tok;

    // the loop bound is uniform in the CTA, so every lane takes part in the shuffles
    for (int r0 = 0; r0 < rows; r0 += kRows) {
        const int r = r0 + tid / kLanes;
        const bool live = r < rows;
        const int t = live ? r / per_tok : 0, j = live ? r % per_tok : 0;
        const int pos = s_pos[t], tok = t0 + t;
        const bool on = live && pos >= 0;
        const bool is_q = j < p.nq, is_k = !is_q && j < p.nq + p.c.H;
        const int h = is_q ? j : is_k ? j - p.nq : j - p.nq - p.c.H;
        float a[8], z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = z[i] = 0.f;
        if (on) {
            const T* src = is_q   ? static_cast<const T*>(p.q) + tok * p.q_tok + h * p.q_head
                           : is_k ? static_cast<const T*>(p.k) + tok * p.k_tok + h * p.k_head
                                  : static_cast<const T*>(p.v) + tok * p.v_tok + h * p.v_head;
            load16(src, o1, o2, a, z);
        }
        const T* w = static_cast<const T*>(is_q ? p.qw : is_k ? p.kw : nullptr);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(z[i], z[i], ss));
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!on) continue;
        if (w) {
            const float rs = rsqrtf(ss * (1.f / D) + p.eps);
            float wa[8], wz[8];
            load16(w, o1, o2, wa, wz);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a[i] *= rs * wa[i];
                z[i] *= rs * wz[i];
            }
        }
        if (turns && (is_q || is_k)) {
            const float* cs = s_cos + t * (D / 2) + 8 * c;
            const float* sn = s_sin + t * (D / 2) + 8 * c;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = a[i], y = z[i];
                a[i] = fmaf(x, cs[i], -(y * sn[i]));
                z[i] = fmaf(y, cs[i], x * sn[i]);
            }
        }
        if (is_q) {
            T* dst = static_cast<T*>(p.qo) + tok * p.qo_tok + h * p.qo_head;
            store8(dst + o1, a);
            store8(dst + o2, z);
            continue;
        }
        if (is_k && p.ko) {
            T* dst = static_cast<T*>(p.ko) + tok * p.ko_tok + h * p.ko_head;
            store8(dst + o1, a);
            store8(dst + o2, z);
        }
        if (!cache) continue;
        const int sq = __ldg(p.seq + tok), at = __ldg(p.index + tok);
        if (sq < 0) continue;
        if (sq >= p.c.batch || at < 0 || at >= p.c.cap) {
            set_err(g_err, DEV_ERR_BOUNDS, 701);
            continue;
        }
        const int page = page_of(p.c, sq, at, g_err, 702);
        if (page < 0) continue;
        const int off = at & ((1 << p.c.lg) - 1);
        if (is_k) {
            T* dst = static_cast<T*>(p.c.k) + page * p.c.k_page + h * p.c.k_head + off * p.c.k_row;
            store8(dst + o1, a);
            store8(dst + o2, z);
            const int64_t row = (static_cast<int64_t>(sq) * p.c.H + h) * p.row_pitch + at;
            if (c == 0 && p.row_position) p.row_position[row] = pos;
            if (c == 0 && p.row_weight) p.row_weight[row] = 0.f;
        } else if (kE5M2) {
            uint8_t* dst = static_cast<uint8_t*>(p.c.v) + page * p.c.v_page + h * p.c.v_head + off * p.c.v_row;
            uint32_t wd[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float* x = i < 2 ? a : z;
                const int b = (i & 1) * 4;
                wd[i] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    wd[i] |= static_cast<uint32_t>(from_f<__nv_fp8_e5m2>(x[b + e]).__x) << (8 * e);
            }
            *reinterpret_cast<uint2*>(dst + o1) = make_uint2(wd[0], wd[1]);
            *reinterpret_cast<uint2*>(dst + o2) = make_uint2(wd[2], wd[3]);
        } else {
            T* dst = static_cast<T*>(p.c.v) + page * p.c.v_page + h * p.c.v_head + off * p.c.v_row;
            store8(dst + o1, a);
            store8(dst + o2, z);
        }
    }
}

template <typename T, int D, bool kE5M2>
static int launch_nr(NormRopeParams p, cudaStream_t s) {
    // tokens per CTA: enough rows for every lane group of the CTA
    const int per_tok = p.nq + p.c.H * (p.c.k ? 2 : 1);
    const int rows = kNrThreads / (D / 16);
    p.per_cta = rows / per_tok < 1 ? 1 : rows / per_tok > kNrMaxTok ? kNrMaxTok : rows / per_tok;
    const int grid = (p.tokens + p.per_cta - 1) / p.per_cta;
    k_norm_rope<T, D, kE5M2><<<grid, kNrThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_norm_rope(int dtype, int d, const NormRopeParams& p, cudaStream_t s) {
    if (dtype == SKV_F32) return d == 64 ? launch_nr<float, 64, false>(p, s) : launch_nr<float, 128, false>(p, s);
    if (dtype == SKV_FP8 && p.c.k)
        return d == 64 ? launch_nr<__nv_bfloat16, 64, true>(p, s) : launch_nr<__nv_bfloat16, 128, true>(p, s);
    return d == 64 ? launch_nr<__nv_bfloat16, 64, false>(p, s) : launch_nr<__nv_bfloat16, 128, false>(p, s);
}

cudaError_t norm_rope_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
