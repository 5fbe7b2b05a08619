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

// 16 elements of a row as they lie in memory: 8 at o1, 8 at o2
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> { uint4 a, z; };
template <> struct Raw<float> { float4 a0, a1, z0, z1; };

__device__ __forceinline__ void fetch(Raw<__nv_bfloat16>& r, const __nv_bfloat16* p, int o1, int o2) {
    r.a = *reinterpret_cast<const uint4*>(p + o1);
    r.z = *reinterpret_cast<const uint4*>(p + o2);
}
__device__ __forceinline__ void fetch(Raw<float>& r, const float* p, int o1, int o2) {
    r.a0 = reinterpret_cast<const float4*>(p + o1)[0];
    r.a1 = reinterpret_cast<const float4*>(p + o1)[1];
    r.z0 = reinterpret_cast<const float4*>(p + o2)[0];
    r.z1 = reinterpret_cast<const float4*>(p + o2)[1];
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&a)[8], float (&z)[8]) {
    load8(reinterpret_cast<const __nv_bfloat16*>(&r.a), a);
    load8(reinterpret_cast<const __nv_bfloat16*>(&r.z), z);
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&a)[8], float (&z)[8]) {
    a[0] = r.a0.x; a[1] = r.a0.y; a[2] = r.a0.z; a[3] = r.a0.w;
    a[4] = r.a1.x; a[5] = r.a1.y; a[6] = r.a1.z; a[7] = r.a1.w;
    z[0] = r.z0.x; z[1] = r.z0.y; z[2] = r.z0.z; z[3] = r.z0.w;
    z[4] = r.z1.x; z[5] = r.z1.y; z[6] = r.z1.z; z[7] = r.z1.w;
}

// Which row of the CTA's tokens a lane group holds: head j of token t (q heads, then k, then v).
struct Row {
    int t, j;
    __device__ __forceinline__ void step(int rows, int per_tok) {
        j += rows;
        while (j >= per_tok) {
            j -= per_tok;
            ++t;
        }
    }
};

template <typename T, int D, bool kE5M2>
__global__ void __launch_bounds__(kNrThreads) k_norm_rope(const __grid_constant__ NormRopeParams p) {
    constexpr int kLanes = D / 16;                  // lanes of a row
    constexpr int kRows = kNrThreads / kLanes;      // rows side by side
    constexpr int kDeep = sizeof(T) == 2 ? 4 : 2;   // rows of a thread whose loads are in flight at once
    __shared__ __align__(16) float s_cos[kNrMaxTok * D / 2], s_sin[kNrMaxTok * D / 2];

    const int tid = threadIdx.x, c = tid % kLanes, half = p.rd / 2;
    const int t0 = blockIdx.x * p.per_cta, nt = min(p.per_cta, p.tokens - t0);
    const bool cache = p.c.k != nullptr;
    const int per_tok = p.nq + p.c.H * (cache ? 2 : 1);
    const bool turns = c < p.rd / 16;
    const int o1 = turns ? 8 * c : p.rd + 16 * (c - p.rd / 16);
    const int o2 = turns ? half + 8 * c : o1 + 8;

    Row at{0, 0};
    at.step(tid / kLanes, per_tok);
    bool first = true;
    // the loop bound is uniform in the CTA, so every lane takes part in the shuffles
    for (int r0 = 0; r0 < nt * per_tok; r0 += kRows * kDeep) {
        Raw<T> raw[kDeep];
        Row rows[kDeep];
        int pos[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            rows[i] = at;
            at.step(kRows, per_tok);
            pos[i] = rows[i].t < nt ? __ldg(p.positions + t0 + rows[i].t) : -1;
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int tok = t0 + rows[i].t, j = rows[i].j;
            const T* src = j < p.nq ? static_cast<const T*>(p.q) + tok * p.q_tok + j * p.q_head
                           : j < p.nq + p.c.H ? static_cast<const T*>(p.k) + tok * p.k_tok + (j - p.nq) * p.k_head
                                              : static_cast<const T*>(p.v) + tok * p.v_tok + (j - p.nq - p.c.H) * p.v_head;
            raw[i] = Raw<T>{};
            if (pos[i] >= 0) fetch(raw[i], src, o1, o2);
        }
        if (first) {       // the angles, while the first rows are on their way
            first = false;
            for (int i = tid; i < nt * half; i += kNrThreads) {
                const int t = i / half, f = i % half;
                const uint64_t turned = static_cast<uint64_t>(static_cast<int64_t>(__ldg(p.positions + t0 + t))) * p.turn[f];
                float sn, cs;
                sincospif(static_cast<float>(static_cast<int32_t>(turned >> 32)) * 0x1p-31f, &sn, &cs);
                s_cos[t * (D / 2) + f] = cs;
                s_sin[t * (D / 2) + f] = sn;
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int t = rows[i].t, tok = t0 + t, j = rows[i].j;
            const bool is_q = j < p.nq, is_k = !is_q && j < p.nq + p.c.H;
            float a[8], z[8];
            widen(raw[i], a, z);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(z[e], z[e], ss));
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (pos[i] < 0) continue;
            const T* w = static_cast<const T*>(is_q ? p.qw : is_k ? p.kw : nullptr);
            if (w) {
                const float rs = rsqrtf(ss * (1.f / D) + p.eps);
                Raw<T> wr;
                float wa[8], wz[8];
                fetch(wr, w, o1, o2);
                widen(wr, wa, wz);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    a[e] *= rs * wa[e];
                    z[e] *= rs * wz[e];
                }
            }
            if (turns && (is_q || is_k)) {
                const float* cs = s_cos + t * (D / 2) + 8 * c;
                const float* sn = s_sin + t * (D / 2) + 8 * c;
                float cv[8], sv[8];
                load8(cs, cv);
                load8(sn, sv);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = a[e], y = z[e];
                    a[e] = fmaf(x, cv[e], -(y * sv[e]));
                    z[e] = fmaf(y, cv[e], x * sv[e]);
                }
            }
            if (is_q) {
                T* dst = static_cast<T*>(p.qo) + tok * p.qo_tok + j * p.qo_head;
                store8(dst + o1, a);
                store8(dst + o2, z);
                continue;
            }
            const int h = is_k ? j - p.nq : j - p.nq - p.c.H;
            if (is_k && p.ko) {
                T* dst = static_cast<T*>(p.ko) + tok * p.ko_tok + h * p.ko_head;
                store8(dst + o1, a);
                store8(dst + o2, z);
            }
            if (!cache) continue;
            const int sq = __ldg(p.seq + tok), row = __ldg(p.index + tok);
            if (sq < 0) continue;
            if (sq >= p.c.batch || row < 0 || row >= p.c.cap) {
                set_err(g_err, DEV_ERR_BOUNDS, 701);
                continue;
            }
            const int page = page_of(p.c, sq, row, g_err, 702);
            if (page < 0) continue;
            const int off = row & ((1 << p.c.lg) - 1);
            if (is_k) {
                T* dst = static_cast<T*>(p.c.k) + page * p.c.k_page + h * p.c.k_head + off * p.c.k_row;
                store8(dst + o1, a);
                store8(dst + o2, z);
                const int64_t held = (static_cast<int64_t>(sq) * p.c.H + h) * p.row_pitch + row;
                if (c == 0 && p.row_position) p.row_position[held] = pos[i];
                if (c == 0 && p.row_weight) p.row_weight[held] = 0.f;
            } else if (kE5M2) {
                uint8_t* dst = static_cast<uint8_t*>(p.c.v) + page * p.c.v_page + h * p.c.v_head + off * p.c.v_row;
                uint32_t wd[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    wd[e / 4] |= static_cast<uint32_t>(from_f<__nv_fp8_e5m2>(a[e]).__x) << (8 * (e % 4));
                    wd[2 + e / 4] |= static_cast<uint32_t>(from_f<__nv_fp8_e5m2>(z[e]).__x) << (8 * (e % 4));
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
}

template <typename T, int D, bool kE5M2>
static int launch_nr(NormRopeParams p, int nsm, cudaStream_t s) {
    const int per_tok = p.nq + p.c.H * (p.c.k ? 2 : 1);
    constexpr int kRows = kNrThreads / (D / 16);
    // one token per CTA while that leaves SMs idle (a decode step), else enough for four rows per
    // lane group, whose loads then overlap
    int per = 1;
    if (p.tokens > 4 * nsm) per = (4 * kRows + per_tok / 2) / per_tok;
    p.per_cta = per < 1 ? 1 : per > kNrMaxTok ? kNrMaxTok : per;
    const int grid = (p.tokens + p.per_cta - 1) / p.per_cta;
    k_norm_rope<T, D, kE5M2><<<grid, kNrThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int launch_norm_rope(int dtype, int d, const NormRopeParams& p, int nsm, cudaStream_t s) {
    if (dtype == SKV_F32) return d == 64 ? launch_nr<float, 64, false>(p, nsm, s) : launch_nr<float, 128, false>(p, nsm, s);
    if (dtype == SKV_FP8 && p.c.k)
        return d == 64 ? launch_nr<__nv_bfloat16, 64, true>(p, nsm, s) : launch_nr<__nv_bfloat16, 128, true>(p, nsm, s);
    return d == 64 ? launch_nr<__nv_bfloat16, 64, false>(p, nsm, s) : launch_nr<__nv_bfloat16, 128, false>(p, nsm, s);
}

cudaError_t norm_rope_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
