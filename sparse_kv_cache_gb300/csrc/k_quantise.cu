// Rows of an 8-bit paged cache: written (shadowkv_paged_quantise) and read back (shadowkv_paged_dequantise).
//
// A value is code * scale: an e4m3 code (1 sign, 4 exponent and 3 mantissa bits, bias 7, largest 448) and an
// fp32 scale of its block (2^lgb rows of a page) and head.  Scales are powers of two, 2^e with the smallest
// e >= -100 that brings the block's largest finite |x| to 448 at most: codes have a floating point of their
// own, so a finer scale would gain less than one bit at the bottom of their range, and with these a
// product and a quotient by a scale are exact, a code is x rounded once, and rows that are rounded again when
// a later row of their block is larger lose nothing but what falls below the smallest code.
//
// Both are bound by memory: 3 bytes (bf16) or 5 (fp32) per element.
#include <math_constants.h>

#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

// two floats as e4m3 codes, nearest even (the lower byte is the first; NaN is 0x7f)
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ------------------------------------------------------------------ writing

constexpr int kQzWarps = 8;
constexpr int kQzRows = 16;       // rows of a warp

// a lane's eight elements of a row, as they come
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const uint4*>(p); }
    __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
        v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
        v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
    }
    // the largest magnitude with those before it (NaN is passed over)
    __device__ __forceinline__ float most(float m) const {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
        const __nv_bfloat162 x = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])), __hmax2(__habs2(h[2]), __habs2(h[3])));
        return fmaxf(m, fmaxf(__low2float(x), __high2float(x)));
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* p) {
        a = static_cast<const float4*>(p)[0];
        b = static_cast<const float4*>(p)[1];
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void floats(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ float most(float m) const {
        const float x = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w)));
        const float y = fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w)));
        return fmaxf(m, fmaxf(x, y));
    }
};
__device__ __forceinline__ float finite_or(float x, float other) {
    return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u ? other : x;
}

// 2^e of a block whose largest finite magnitude is m: 448 = 1.75 * 2^8, so e is m's exponent less 8, and one
// more where its mantissa is above 1.75 (which the sum carries into the exponent)
__device__ __forceinline__ float block_scale(float m) {
    const int e = static_cast<int>((__float_as_uint(m) + 0x1FFFFFu) >> 23) - 8;
    return __uint_as_float(static_cast<uint32_t>(max(e, 27)) << 23);
}

// A unit is a block that gets new rows, of one head, of keys or of values; its rows lie in the registers of
// one warp or several (block / 16).  Which blocks those are only the device knows: sequence b has
// (start[b] >> lgb) + 2b slots before its own, which leaves every sequence room for the blocks that its
// tokens can touch, and a slot without a block ends at once.  (32K tokens, blocks of 64: two slots of 514.)
// A prompt of 32K tokens in bf16 36.4 us, 5.5 TB/s (three CTAs to an SM 40), in fp32 4.4 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kQzWarps, sizeof(T) == 4 ? 3 : 4) k_quantise(const __grid_constant__ QuantParams p) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes, kSteps = kQzRows / kPer;
    __shared__ float s_most[kQzWarps];
    begin_call();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int W = p.lgb > 4 ? 1 << (p.lgb - 4) : 1;                 // warps of a unit
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kQzWarps / W) + warp / W;
    const int64_t per_slot = 2 * p.c.H;
    const int64_t slot = unit / per_slot;
    const int h = static_cast<int>(unit % per_slot) >> 1;
    const bool values = unit & 1;
    // (there are more threads than sequences: 64 for each at least)
    const int64_t thread = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (thread < p.c.batch) check_sequence(p.c, p.start, p.tokens, static_cast<int>(thread), g_err, 814);
    int row0 = 0, from = 0, to = 0, len = 0, tok = 0, page = -1;
    if (slot < p.slots) {
        const int b = find_sequence(p.start, p.c.batch, slot, [&](int s, int i) { return (s >> p.lgb) + 2 * static_cast<int64_t>(i); });
        const int t0 = __ldcg(p.start + b), t1 = __ldcg(p.start + b + 1);
        len = rows_of(p.c, b, g_err, 811);
        if (t0 < 0 || t1 > p.tokens || t1 < t0 || t1 - t0 > p.c.cap - len) set_err(g_err, DEV_ERR_BOUNDS, 812);
        if (t0 >= 0 && t1 <= p.tokens && t0 < t1) {
            const int64_t skip = slot - ((t0 >> p.lgb) + 2 * static_cast<int64_t>(b)), blk = (len >> p.lgb) + skip;
            const int n = min(t1 - t0, p.c.cap - len);
            // (a place before the first sequence's has no block: tokens before start[0] are of no sequence)
            if (skip >= 0 && blk << p.lgb < len + n) {
                row0 = static_cast<int>(blk) << p.lgb;
                from = max(row0, len);
                to = min(row0 + (1 << p.lgb), len + n);
                tok = t0 + from - len;
                page = page_of(p.c, b, row0, g_err, 813);
                if (page < 0) to = from;
            }
        }
    }
    const bool live = from < to;
    const int at = row0 & ((1 << p.c.lg) - 1);                      // the block's first row in its page
    const int sub = lane / kLanes, dim = 8 * (lane % kLanes);
    const int first = row0 + (warp % W) * kQzRows + sub;            // this lane's rows: first + step * kPer
    const int64_t x_tok = values ? p.v_tok : p.k_tok;
    const T* x = static_cast<const T*>(values ? p.v : p.k) + h * (values ? p.v_head : p.k_head) + dim;
    float* scale = (values ? p.v_scale : p.k_scale) +
                   (static_cast<int64_t>(page) * p.c.H + h) * (1 << (p.c.lg - p.lgb)) + (at >> p.lgb);
    const bool joins = live && row0 < len;
    const float old = joins ? __ldcg(scale) : 0.f;
    Eight<T> in[kSteps];
    float m = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int row = first + s * kPer;
        in[s].clear();
        if (row >= from && row < to) in[s].load(x + (tok + (row - from)) * x_tok);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) m = in[s].most(m);
    // infinities have no code but NaN's, and no part in the scale
    const bool wild = __any_sync(0xffffffffu, m == CUDART_INF_F);
    if (wild) {
        m = 0.f;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            float v[8];
            in[s].floats(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(finite_or(v[i], 0.f)));
        }
    }
    m = warp_max(m);
    if (W > 1) {
        if (lane == 0) s_most[warp] = m;
        __syncthreads();
        for (int w = 0; w < W; ++w) m = fmaxf(m, s_most[warp / W * W + w]);
    }
    if (!live) return;
    const float size = joins ? fmaxf(block_scale(m), old) : block_scale(m);
    uint8_t* out = (values ? static_cast<uint8_t*>(p.c.v) + page * p.c.v_page + h * p.c.v_head
                           : static_cast<uint8_t*>(p.c.k) + page * p.c.k_page + h * p.c.k_head) + dim;
    const int64_t pitch = values ? p.c.v_row : p.c.k_row;
    const float inv = 1.f / size;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int row = first + s * kPer;
        if (row < from || row >= to) continue;
        float v[8];
        in[s].floats(v);
        if (wild) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = finite_or(v[i], CUDART_NAN_F);
        }
        *reinterpret_cast<uint2*>(out + (at + row - row0) * pitch) =
            make_uint2(e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16,
                       e4m3x2(v[4] * inv, v[5] * inv) | e4m3x2(v[6] * inv, v[7] * inv) << 16);
    }
    if (joins && size != old) {
        // held codes of this warp's rows, to the new scale
        const float by = old / size;
        for (int s = 0; s < kSteps; ++s) {
            const int row = first + s * kPer;
            if (row >= len || row >= row0 + (1 << p.lgb)) break;
            uint2* held = reinterpret_cast<uint2*>(out + (at + row - row0) * pitch);
            const uint2 w = __ldcg(held);
            auto again = [&](uint32_t four) {
                const float2 a = from_e4m3x2(four & 0xFFFF), b = from_e4m3x2(four >> 16);
                return e4m3x2(a.x * by, a.y * by) | e4m3x2(b.x * by, b.y * by) << 16;
            };
            *held = make_uint2(again(w.x), again(w.y));
        }
    }
    if (warp % W == 0 && lane == 0) *scale = size;
}

// ------------------------------------------------------------------ reading back

constexpr int kDqWarps = 8;
constexpr int kDqTokens = 32;

// A CTA takes 32 tokens, a warp of it all their rows of one head, of keys or of values: 4 KB, all asked for before
// any is converted.  Four 32K contexts in bf16 131 us, 6.2 TB/s (with 16 codes to a lane, whose result is two stores of
// every other 16 bytes, 147; with several heads to a warp, the next one's loads during this one's stores, 180).
template <typename T, int D>
__global__ void __launch_bounds__(32 * kDqWarps) k_dequantise(const __grid_constant__ DequantParams p) {
    constexpr int kEach = 16 / sizeof(T);       // codes of a lane: 16 bytes of the result, side by side
    constexpr int kLanes = D / kEach, kPer = 32 / kLanes, kSteps = kDqTokens / kPer;
    __shared__ int s_page[kDqTokens], s_at[kDqTokens];
    begin_call();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t0 = blockIdx.x * kDqTokens;
    if (warp == 0) {
        const int t = t0 + lane;
        int b = find_sequence(p.start, p.c.batch, t0, [](int s, int) { return static_cast<int64_t>(s); });
        // the sequences that begin behind it, 32 at a time (start[batch] begins none)
        for (int base = b + 1; base < p.c.batch; base += 32) {
            const int mine = base + lane < p.c.batch ? __ldcg(p.start + base + lane) : INT32_MAX;
            for (int j = 0; j < 32; ++j) b += __shfl_sync(0xffffffffu, mine, j) <= t;
            if (__shfl_sync(0xffffffffu, mine, 31) > t0 + 31) break;
        }
        int page = -1, at = 0;
        if (t < p.tokens) {
            const int s0 = __ldcg(p.start + b), s1 = __ldcg(p.start + b + 1), first = __ldcg(p.first + b);
            const int n = rows_of(p.c, b, g_err, 821);
            if (first < 0 || s0 < 0 || s1 < s0 || s1 > p.tokens) {
                set_err(g_err, DEV_ERR_BOUNDS, 822);
            } else if (t >= s0 && t < s1 && first < n && t - s0 < n - first) {
                at = first + (t - s0);
                page = page_of(p.c, b, at, g_err, 823);
            }
        }
        s_page[lane] = page;
        s_at[lane] = at & ((1 << p.c.lg) - 1);
    } else if (warp == 1 && blockIdx.y == 0) {
        for (int64_t b = t0 + lane; b < p.c.batch; b += static_cast<int64_t>(gridDim.x) * kDqTokens) {
            check_sequence(p.c, p.start, p.tokens, static_cast<int>(b), g_err, 824);
            if (__ldcg(p.first + b) < 0) set_err(g_err, DEV_ERR_BOUNDS, 824);
        }
    }
    __syncthreads();
    const int what = blockIdx.y * kDqWarps + warp;
    if (what >= 2 * p.c.H) return;
    const int h = what >> 1;
    const bool values = what & 1;
    const int sub = lane / kLanes, dim = kEach * (lane % kLanes);
    const uint8_t* pool = static_cast<const uint8_t*>(values ? p.c.v : p.c.k) + h * (values ? p.c.v_head : p.c.k_head) + dim;
    const int64_t pg = values ? p.c.v_page : p.c.k_page, pitch = values ? p.c.v_row : p.c.k_row;
    const float* scale = (values ? p.v_scale : p.k_scale) + static_cast<int64_t>(h) * (1 << (p.c.lg - p.lgb));
    T* out = static_cast<T*>(values ? p.v : p.k) + h * (values ? p.v_head : p.k_head) + dim;
    const int64_t o_tok = values ? p.v_tok : p.k_tok;
    uint32_t w[kSteps][kEach / 4];
    float f[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i = s * kPer + sub;
        const int64_t page = s_page[i];
        if (page < 0) continue;
        const uint8_t* src = pool + page * pg + s_at[i] * pitch;
        if constexpr (kEach == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(src);
            w[s][0] = x.x;
            w[s][1] = x.y;
        } else {
            w[s][0] = *reinterpret_cast<const uint32_t*>(src);
        }
        f[s] = __ldcg(scale + page * p.c.H * (1 << (p.c.lg - p.lgb)) + (s_at[i] >> p.lgb));
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i = s * kPer + sub;
        if (s_page[i] < 0) continue;
        float v[kEach];
#pragma unroll
        for (int e = 0; e < kEach; e += 2) {
            const float2 x = from_e4m3x2(e & 2 ? w[s][e / 4] >> 16 : w[s][e / 4] & 0xFFFF);
            v[e] = x.x * f[s];
            v[e + 1] = x.y * f[s];
        }
        T* dst = out + (t0 + i) * o_tok;
        if constexpr (kEach == 8) store8(dst, v);
        else *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// ------------------------------------------------------------------ launches

int64_t quantise_slots(int tokens, int batch, int lgb) { return (tokens >> lgb) + 2 * static_cast<int64_t>(batch); }

int launch_quantise(int dtype, int d, const QuantParams& p, cudaStream_t s) {
    const int W = p.lgb > 4 ? 1 << (p.lgb - 4) : 1;
    const int64_t units = p.slots * 2 * p.c.H, per = kQzWarps / W, grid = (units + per - 1) / per;
    auto kernel = dtype == SKV_F32 ? (d == 64 ? k_quantise<float, 64> : k_quantise<float, 128>)
                                   : (d == 64 ? k_quantise<__nv_bfloat16, 64> : k_quantise<__nv_bfloat16, 128>);
    return launch_first(kernel, static_cast<unsigned>(grid), 32 * kQzWarps, 0, 1, 0, s, p) == cudaSuccess ? 0 : -1;
}

int launch_dequantise(int dtype, int d, const DequantParams& p, cudaStream_t s) {
    const dim3 grid((p.tokens + kDqTokens - 1) / kDqTokens, (2 * p.c.H + kDqWarps - 1) / kDqWarps);
    auto kernel = dtype == SKV_F32 ? (d == 64 ? k_dequantise<float, 64> : k_dequantise<float, 128>)
                                   : (d == 64 ? k_dequantise<__nv_bfloat16, 64> : k_dequantise<__nv_bfloat16, 128>);
    return launch_first(kernel, grid, 32 * kDqWarps, 0, 1, 0, s, p) == cudaSuccess ? 0 : -1;
}

cudaError_t quantise_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
