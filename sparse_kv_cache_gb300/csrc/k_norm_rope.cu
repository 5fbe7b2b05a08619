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
//
// Measured back to back: 32K tokens of 32 + 2 x 8 heads, d = 128, 140 us, 6.2 TB/s of a copy's 6.7;
// 5105 tokens of 16 + 2 x 2 heads with e5m2 values 14.5 us (51 MB: latency of one wave of CTAs, four rounds of
// loads one after the other in each); a decode step of 8 tokens 3.2 us.
#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kNrThreads = 128;
constexpr int max_tokens(int d) { return 2048 / d; }     // of a CTA, for their angles' 8 KB of shared memory

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

__device__ __forceinline__ void put(__nv_bfloat16* p, int o1, int o2, const Raw<__nv_bfloat16>& r) {
    *reinterpret_cast<uint4*>(p + o1) = r.a;
    *reinterpret_cast<uint4*>(p + o2) = r.z;
}
__device__ __forceinline__ void put(float* p, int o1, int o2, const Raw<float>& r) {
    reinterpret_cast<float4*>(p + o1)[0] = r.a0;
    reinterpret_cast<float4*>(p + o1)[1] = r.a1;
    reinterpret_cast<float4*>(p + o2)[0] = r.z0;
    reinterpret_cast<float4*>(p + o2)[1] = r.z1;
}

template <typename T, int D, bool kE5M2, int kOcc>      // kOcc: CTAs per SM
__global__ void __launch_bounds__(kNrThreads, kOcc) k_norm_rope(const __grid_constant__ NormRopeParams p) {
    constexpr int kLanes = D / 16;                  // lanes of a row
    constexpr int kDeep = sizeof(T) == 2 ? 3 : 2;   // rows of a thread whose loads are in flight at once
    __shared__ __align__(16) float s_cos[max_tokens(D) * D / 2], s_sin[max_tokens(D) * D / 2];

    begin_call();
    // p.groups lane groups share a token; group g of it takes the heads g, g + groups, ... of q, and
    // likewise of k and v together
    const int tid = threadIdx.x, c = tid % kLanes, half = p.rd / 2;
    const int per_cta = kNrThreads / kLanes / p.groups;
    const int t0 = blockIdx.x * per_cta, nt = min(per_cta, p.tokens - t0);
    const int t = tid / kLanes / p.groups, g = tid / kLanes % p.groups;
    const int64_t tok = t0 + t;
    const int pos = t < nt ? p.positions[tok] : -1;
    const bool cache = p.c.k != nullptr;
    const int H = p.c.H, n_kv = cache ? 2 * H : H;
    const int q_slots = (p.nq + p.groups - 1) / p.groups, slots = q_slots + (n_kv + p.groups - 1) / p.groups;
    const bool turns = c < p.rd / 16;
    const int o1 = turns ? 8 * c : p.rd + 16 * (c - p.rd / 16);
    const int o2 = turns ? half + 8 * c : o1 + 8;
    const T* q = static_cast<const T*>(p.q) + tok * p.q_tok;
    const T* k = static_cast<const T*>(p.k) + tok * p.k_tok;
    const T* v = static_cast<const T*>(p.v) + tok * p.v_tok;

    // where the token's rows go in the cache: asked for early, needed late
    int seq = -1, row = 0;
    if (cache && pos >= 0) {
        seq = p.seq[tok];
        row = p.index[tok];
    }
    float cs[8] = {}, sn[8] = {};
    int page = -1;
    for (int s0 = 0; s0 < slots; s0 += kDeep) {       // uniform: every lane takes part in the shuffles
        // (asked for before the position is known: a padding token's rows are there to be read too)
        Raw<T> raw[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            raw[i] = Raw<T>{};
            const int s = s0 + i;
            if (s < q_slots) {
                const int h = s * p.groups + g;
                if (t < nt && h < p.nq) fetch(raw[i], q + h * p.q_head, o1, o2);
            } else if (s < slots) {
                const int h = (s - q_slots) * p.groups + g;
                if (t < nt && h < n_kv) fetch(raw[i], h < H ? k + h * p.k_head : v + (h - H) * p.v_head, o1, o2);
            }
        }
        if (s0 == 0) {     // the angles, while the first rows are on their way
            for (int i = tid; i < nt * half; i += kNrThreads) {
                const int a = i / half, f = i % half;
                const uint64_t turned = static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + a])) * p.turn[f];
                float y, x;
                sincospif(static_cast<float>(static_cast<int32_t>(turned >> 32)) * 0x1p-31f, &y, &x);
                s_cos[a * (D / 2) + f] = x;
                s_sin[a * (D / 2) + f] = y;
            }
            if (seq >= 0) {
                if (seq >= p.c.batch || row < 0 || row >= p.c.cap) set_err(g_err, DEV_ERR_BOUNDS, 701);
                else page = page_of(p.c, seq, row, g_err, 702);
            }
            __syncthreads();
            if (turns) {
                load8(s_cos + t * (D / 2) + 8 * c, cs);
                load8(s_sin + t * (D / 2) + 8 * c, sn);
            }
        }
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
            const int s = s0 + i;
            if (s >= slots) break;
            const bool is_q = s < q_slots;
            const int h = (is_q ? s : s - q_slots) * p.groups + g;
            const bool is_v = !is_q && h >= H, live = pos >= 0 && h < (is_q ? p.nq : n_kv);
            float a[8], z[8];
            widen(raw[i], a, z);
            const T* w = static_cast<const T*>(is_q ? p.qw : p.kw);
            if (w) {       // uniform
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(z[e], z[e], ss));
#pragma unroll
                for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
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
            if (turns) {     // (a turn by nothing would not do: an infinite partner times a sine of 0 is NaN)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = a[e], y = z[e];
                    a[e] = fmaf(x, cs[e], -(y * sn[e]));
                    z[e] = fmaf(y, cs[e], x * sn[e]);
                }
            }
            if (!live) continue;
            if (is_q) {
                T* dst = static_cast<T*>(p.qo) + tok * p.qo_tok + h * p.qo_head;
                store8(dst + o1, a);
                store8(dst + o2, z);
                continue;
            }
            const int off = row & ((1 << p.c.lg) - 1);
            if (!is_v) {
                if (p.ko) {
                    T* dst = static_cast<T*>(p.ko) + tok * p.ko_tok + h * p.ko_head;
                    store8(dst + o1, a);
                    store8(dst + o2, z);
                }
                if (page < 0) continue;
                T* dst = static_cast<T*>(p.c.k) + page * p.c.k_page + h * p.c.k_head + off * p.c.k_row;
                store8(dst + o1, a);
                store8(dst + o2, z);
                const int64_t held = (static_cast<int64_t>(seq) * H + h) * p.row_pitch + row;
                if (c == 0 && p.row_position) p.row_position[held] = pos;
                if (c == 0 && p.row_weight) p.row_weight[held] = 0.f;
            } else if (page >= 0) {
                const int64_t at = page * p.c.v_page + (h - H) * p.c.v_head + off * p.c.v_row;
                if (kE5M2) {
                    uint8_t* dst = static_cast<uint8_t*>(p.c.v) + at;
                    widen(raw[i], a, z);
                    uint32_t wd[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        wd[e / 4] |= static_cast<uint32_t>(from_f<__nv_fp8_e5m2>(a[e]).__x) << (8 * (e % 4));
                        wd[2 + e / 4] |= static_cast<uint32_t>(from_f<__nv_fp8_e5m2>(z[e]).__x) << (8 * (e % 4));
                    }
                    *reinterpret_cast<uint2*>(dst + o1) = make_uint2(wd[0], wd[1]);
                    *reinterpret_cast<uint2*>(dst + o2) = make_uint2(wd[2], wd[3]);
                } else {
                    put(static_cast<T*>(p.c.v) + at, o1, o2, raw[i]);
                }
            }
        }
    }
}

template <typename T, int D, bool kE5M2>
static int launch_nr(NormRopeParams p, int nsm, cudaStream_t s) {
    constexpr int kRows = kNrThreads / (D / 16);
    const int n_kv = p.c.H * (p.c.k ? 2 : 1);
    // Lane groups per token: all of a CTA's, or fewer as long as that leaves four CTAs per SM.  Then the
    // number that leaves the fewest groups without a head, and of equals the largest whose threads
    // have ten rows of a token (whose angles they hold), or the smallest (32K tokens of 32 + 2 x 8
    // heads, four groups: 141 us, two 143, eight 151; 5K tokens of 16 + 2 x 2 heads, two groups: 14.7 us,
    // four 16.2).
    auto slots_of = [&](int g) { return (p.nq + g - 1) / g + (n_kv + g - 1) / g; };
    p.groups = kRows;
    static_assert(kRows <= max_tokens(D), "a CTA has the angles' room for a token per lane group");
    for (int g = kRows / 2; g >= 1 && p.tokens / (kRows / g) >= 4 * nsm; g /= 2) {
        const int spent = slots_of(g) * g, had = slots_of(p.groups) * p.groups;
        if (spent < had || (spent == had && slots_of(p.groups) < 10)) p.groups = g;
    }
    const int per = kRows / p.groups, grid = (p.tokens - 1) / per + 1;
    // Five CTAs per SM have the registers to keep their rows' loads in flight, seven take fewer waves (and spill
    // 8 bytes in bf16, 48 with e5m2 values, 56 in fp32): a wave of seven takes 1.2 times as long as one of five
    // (fp32: 1.45).  5105 tokens of 16 + 2 x 2 heads 14.2
    // us with five, 19.7 with seven; 32K of 32 + 2 x 8 150 and 140, 4096 26.7 and 22.3, 3000 16.7 and 20.1.
    const int w5 = (grid + 5 * nsm - 1) / (5 * nsm), w7 = (grid + 7 * nsm - 1) / (7 * nsm);
    const bool seven = sizeof(T) == 2 ? 6 * w7 < 5 * w5 : 3 * w7 < 2 * w5;
    auto kernel = seven ? k_norm_rope<T, D, kE5M2, 7> : k_norm_rope<T, D, kE5M2, 5>;
    // (a step's attention follows at once; a prompt is better off with the driver's split, 140 us against 141)
    return launch_first(kernel, grid, kNrThreads, 0, 1, w5 == 1 ? kCarve : 0, s, p) == cudaSuccess ? 0 : -1;
}

int launch_norm_rope(int dtype, int d, const NormRopeParams& p, int nsm, cudaStream_t s) {
    if (dtype == SKV_F32) return d == 64 ? launch_nr<float, 64, false>(p, nsm, s) : launch_nr<float, 128, false>(p, nsm, s);
    if (dtype == SKV_FP8 && p.c.k)
        return d == 64 ? launch_nr<__nv_bfloat16, 64, true>(p, nsm, s) : launch_nr<__nv_bfloat16, 128, true>(p, nsm, s);
    return d == 64 ? launch_nr<__nv_bfloat16, 64, false>(p, nsm, s) : launch_nr<__nv_bfloat16, 128, false>(p, nsm, s);
}

cudaError_t norm_rope_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
