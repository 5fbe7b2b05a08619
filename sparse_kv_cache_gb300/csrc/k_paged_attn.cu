// Attention of one new token per sequence over its paged cache (shadowkv_paged_attention).
//
// out = softmax(scale q.K^T).V for the G query heads of every unit (a sequence's KV head), in one
// pass over the unit's rows with a running base and sum of the softmax.  Each cached byte is read
// once and takes part in G products per element, 2G flops per byte in bf16, so memory bounds it.
//
// Work split.  The rows of all units form one sequence of 64-row blocks; CTA i of n takes the
// blocks [i T / n, (i + 1) T / n), whatever units they belong to, so every SM gets the same
// share of any mix of lengths and the host need not know them (a captured graph replays with new
// lengths).  A unit that lies in one CTA's range is finished there; the shares of the others go
// to the CTA's two records (its first and its last unit), and k_paged_merge, a programmatic
// dependent, joins them in order.
//
// bf16 and e5m2: the four warps of a CTA take 16 rows each at a time, with no shared memory in
// the loop.  S^T = K.Q^T has the rows in the 16-wide dimension of m16n8k16 and the heads in the
// 8-wide one, so up to eight heads waste nothing; its operands come straight from 16-byte global
// loads, because a dot product may take its terms in any order as long as both operands agree.
// O^T = V^T.P^T takes pairs of rows interleaved by byte permutes, again from 16-byte loads, and
// P^T is S^T's accumulator passed through movmatrix.  The tensor cores are busy for less than a
// tenth of the time that the loads take, so the warp-level instruction suffices: tcgen05 would
// put both operands and the accumulator through shared and tensor memory first.
//
// fp32 takes the same split with products on the CUDA cores: a half-warp per row, four rows'
// sums joined by a transposing reduction.
#include <math_constants.h>

#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kPaThreads = 128;
constexpr int kPaWarps = kPaThreads / 32;
constexpr int kPaTile = 16;                       // rows of a warp's step
constexpr int kPaBlock = kPaTile * kPaWarps;      // rows of a CTA's step
constexpr int kPaHeads = 8;                       // heads of an accumulator
constexpr float kPaSlack = 8.f;                   // the base moves when a score passes it by 2^8

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 or 8 bytes read once (not kept in L1), zeros where `in` is false
__device__ __forceinline__ uint4 ld_stream(const void* p, bool in) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(static_cast<int>(in)));
    return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p, bool in) {
    uint2 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n\t}"
        : "=&r"(v.x), "=&r"(v.y)
        : "l"(p), "r"(static_cast<int>(in)));
    return v;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// ------------------------------------------------------------------ the split of the work

__device__ __forceinline__ int blocks_of(int n) { return (n + kPaBlock - 1) / kPaBlock; }

// Where block x of the launch lies: its sequence, KV head, and block of the unit.
struct Place {
    int64_t total;    // blocks of all units
    int64_t n;        // CTAs that have work
    int64_t first;    // first block of the sequence in the launch
    int b, rows, nb;  // sequence, its rows, blocks per unit of it
};
struct PlanSmem {
    int64_t warp_sum[kPaWarps];
    int64_t first;
    int b, rows;
};

// Every thread sums a run of sequences; the thread whose run holds CTA i's first block finds it.
__device__ __forceinline__ Place plan(const PagedView& c, int64_t i, int64_t ctas, PlanSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (c.batch + kPaThreads - 1) / kPaThreads;
    const int s0 = min(tid * per, c.batch), s1 = min(s0 + per, c.batch);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) mine += blocks_of(rows_of(c, s, g_err, 711));
    int64_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += x;
    }
    if (lane == 31) sm.warp_sum[warp] = run;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) {
        if (w < warp) before += sm.warp_sum[w];
        all += sm.warp_sum[w];
    }
    Place pl;
    pl.total = all * c.H;
    pl.n = min(ctas, pl.total);
    int64_t at = (before + run - mine) * c.H;
    if (i < pl.n) {
        const int64_t x = i * pl.total / pl.n;
        if (x >= at && x < at + mine * c.H) {
            for (int s = s0; s < s1; ++s) {
                const int rows = rows_of(c, s, g_err, 711);
                const int64_t size = static_cast<int64_t>(blocks_of(rows)) * c.H;
                if (x < at + size) {
                    sm.first = at;
                    sm.b = s;
                    sm.rows = rows;
                    break;
                }
                at += size;
            }
        }
    }
    __syncthreads();
    pl.first = sm.first;
    pl.b = sm.b;
    pl.rows = sm.rows;
    pl.nb = i < pl.n ? blocks_of(pl.rows) : 1;
    return pl;
}

// The next sequence after b that has rows.
__device__ __forceinline__ void next_rows(const PagedView& c, int& b, int& rows) {
    do rows = ++b < c.batch ? rows_of(c, b, g_err, 711) : -1;
    while (rows == 0);
}

// ------------------------------------------------------------------ a warp's share of a unit

// What the four warps hand to the join: O [warp][head][d] unnormalised, base and sum per head.
// Heads lie in two planes by parity with a pitch of d + 2, so that the accumulators' pairs of
// dimensions go to distinct banks.
template <int D>
struct JoinSmem {
    float o[kPaWarps][2][kPaHeads / 2][D + 2];
    float m[kPaWarps][kPaHeads], l[kPaWarps][kPaHeads];
};

// Page ids of a warp's coming tiles: lane j holds those of tile j of the current 32.
struct PageIds {
    int a, b;    // of the tile's first and last eight rows
};

// tile t of the warp covers rows row0 + t * kPaBlock ..+15 of sequence b
__device__ __forceinline__ PageIds page_ids(const PagedView& c, int b, int row, int end) {
    PageIds id{-1, -1};
    if (row < end) {
        id.a = page_of(c, b, row, g_err, 712);
        id.b = c.lg > 3 ? id.a : row + 8 < end ? page_of(c, b, row + 8, g_err, 712) : -1;
    }
    return id;
}

template <int D, bool kE5M2>
struct TileTC {
    static constexpr int kKV = D / 32;                     // 16-byte words of a key row per lane
    static constexpr int kVV = kE5M2 ? 1 : D / 64;         // words of a value row per lane
    static constexpr float kBaseShift = kE5M2 ? 7.f : 0.f; // keeps small fp16 probabilities normal: p <= 2^15
    uint4 q[kKV];
    float o[D / 16][4];
    float m0, m1, l0, l1;                                  // heads 2c and 2c + 1

    __device__ __forceinline__ void load_q(const PagedAttnParams& p, int b, int h, float*) {
        const int g = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_seq + (h * p.G + g) * p.q_head + c * 8;
#pragma unroll
        for (int j = 0; j < kKV; ++j)
            q[j] = g < p.G ? __ldg(reinterpret_cast<const uint4*>(src + 32 * j)) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -CUDART_INF_F;
        l0 = l1 = 0.f;
    }
    struct Keys { uint4 a[kKV], b[kKV]; };                 // row r and row r + 8
    struct Values { uint4 v[4][kVV]; };                    // rows 2c, 2c + 1, 2c + 8, 2c + 9

    __device__ __forceinline__ void load_k(const PagedAttnParams& p, int h, int row, int end, int ida, int idb, Keys& k) {
        const int r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3, mask = (1 << p.c.lg) - 1;
        const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.c.k) + h * p.c.k_head + c * 8;
        const __nv_bfloat16* pa = base + ida * p.c.k_page + ((row + r) & mask) * p.c.k_row;
        const __nv_bfloat16* pb = base + idb * p.c.k_page + ((row + 8 + r) & mask) * p.c.k_row;
        const bool ia = ida >= 0 && row + r < end, ib = idb >= 0 && row + 8 + r < end;
#pragma unroll
        for (int j = 0; j < kKV; ++j) {
            k.a[j] = ld_stream(pa + 32 * j, ia);
            k.b[j] = ld_stream(pb + 32 * j, ib);
        }
    }
    __device__ __forceinline__ void load_v(const PagedAttnParams& p, int h, int row, int end, int ida, int idb, Values& v) {
        const int r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3, mask = (1 << p.c.lg) - 1;
        constexpr int es = kE5M2 ? 1 : 2, lane_bytes = kE5M2 ? D / 8 : 16;
        const uint8_t* base = static_cast<const uint8_t*>(p.c.v) + h * p.c.v_head * es + r * lane_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = row + 2 * c + (i & 1) + (i >> 1) * 8, id = i < 2 ? ida : idb;
            const uint8_t* src = base + (id * p.c.v_page + (t & mask) * p.c.v_row) * es;
            const bool in = id >= 0 && t < end;
#pragma unroll
            for (int j = 0; j < kVV; ++j) {
                if (kE5M2 && D == 64) {
                    const uint2 x = ld_stream8(src, in);
                    v.v[i][j] = make_uint4(x.x, x.y, 0, 0);
                } else {
                    v.v[i][j] = ld_stream(src + 128 * j, in);
                }
            }
        }
    }
    // scores of the tile's rows: s[0], s[1] row r, s[2], s[3] row r + 8, heads 2c and 2c + 1
    __device__ __forceinline__ void scores(const Keys& k, float (&s)[4]) {
        s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
        for (int j = 0; j < kKV; ++j) {
            mma_bf16(s, k.a[j].x, k.b[j].x, k.a[j].y, k.b[j].y, q[j].x, q[j].y);
            mma_bf16(s, k.a[j].z, k.b[j].z, k.a[j].w, k.b[j].w, q[j].z, q[j].w);
        }
    }
    // raw products kept for the weights: z [row][Gp]
    __device__ __forceinline__ void keep(const PagedAttnParams& p, float* z, int row, int end, int ida, int idb,
                                         const float (&s)[4]) {
        const int r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
        if (2 * c >= p.G) return;
        if (row + r < end)
            *reinterpret_cast<float2*>(z + static_cast<int64_t>(row + r) * p.Gp + 2 * c) =
                ida >= 0 ? make_float2(s[0], s[1]) : make_float2(-CUDART_INF_F, -CUDART_INF_F);
        if (row + 8 + r < end)
            *reinterpret_cast<float2*>(z + static_cast<int64_t>(row + 8 + r) * p.Gp + 2 * c) =
                idb >= 0 ? make_float2(s[2], s[3]) : make_float2(-CUDART_INF_F, -CUDART_INF_F);
    }
    // probabilities against the running base; returns P^T as the second product's operand
    __device__ __forceinline__ void softmax(float scale, int row, int end, int ida, int idb, const float (&s)[4], uint32_t& b0,
                                            uint32_t& b1) {
        const int r = (threadIdx.x & 31) >> 2;
        // scores in powers of two, -inf for an absent row (whatever the sign of the scale)
        const bool ia = ida >= 0 && row + r < end, ib = idb >= 0 && row + 8 + r < end;
        float x0 = ia ? s[0] * scale : -CUDART_INF_F, x1 = ia ? s[1] * scale : -CUDART_INF_F;
        float x2 = ib ? s[2] * scale : -CUDART_INF_F, x3 = ib ? s[3] * scale : -CUDART_INF_F;
        float t0 = fmaxf(x0, x2), t1 = fmaxf(x1, x3);
        if (__any_sync(0xffffffffu, t0 > m0 + kPaSlack || t1 > m1 + kPaSlack)) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, x));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, x));
            }
            t0 = fmaxf(t0, m0);
            t1 = fmaxf(t1, m1);
            const float w0 = m0 == -CUDART_INF_F ? 0.f : exp2_fast(m0 - t0);
            const float w1 = m1 == -CUDART_INF_F ? 0.f : exp2_fast(m1 - t1);
            m0 = t0;
            m1 = t1;
            l0 *= w0;
            l1 *= w1;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                o[i][0] *= w0;
                o[i][1] *= w1;
                o[i][2] *= w0;
                o[i][3] *= w1;
            }
        }
        const float n0 = m0 == -CUDART_INF_F ? 0.f : m0 - kBaseShift, n1 = m1 == -CUDART_INF_F ? 0.f : m1 - kBaseShift;
        x0 = ia ? exp2_fast(fmaf(s[0], scale, -n0)) : 0.f;
        x1 = ia ? exp2_fast(fmaf(s[1], scale, -n1)) : 0.f;
        x2 = ib ? exp2_fast(fmaf(s[2], scale, -n0)) : 0.f;
        x3 = ib ? exp2_fast(fmaf(s[3], scale, -n1)) : 0.f;
        l0 += x0 + x2;
        l1 += x1 + x3;
        // rounded to the values' type for the tensor cores (half a step, 2^-9 of a bf16
        // probability and 2^-12 of an fp16 one, unbiased); the sums keep the fp32 ones
        if (kE5M2) {
            const __half2 lo = __floats2half2_rn(x0, x1), hi = __floats2half2_rn(x2, x3);
            b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
            b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi));
        } else {
            b0 = transpose8x8(pack_bf16x2(x0, x1));
            b1 = transpose8x8(pack_bf16x2(x2, x3));
        }
    }
    __device__ __forceinline__ void values(const Values& v, uint32_t b0, uint32_t b1) {
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            if (kE5M2) {
                // tile t: dimensions 2t and 2t + 1 of the lane's; a byte becomes the upper half of an fp16
                const uint32_t sel = (t & 1) ? 0x7362 : 0x5140;
                const uint32_t lo = __byte_perm(word(v.v[0][0], t >> 1), word(v.v[1][0], t >> 1), sel);
                const uint32_t hi = __byte_perm(word(v.v[2][0], t >> 1), word(v.v[3][0], t >> 1), sel);
                mma_f16(o[t], __byte_perm(lo, 0, 0x1404), __byte_perm(lo, 0, 0x3424), __byte_perm(hi, 0, 0x1404),
                        __byte_perm(hi, 0, 0x3424), b0, b1);
            } else {
                const uint32_t a = word(v.v[0][t >> 2], t & 3), b = word(v.v[1][t >> 2], t & 3);
                const uint32_t c = word(v.v[2][t >> 2], t & 3), d = word(v.v[3][t >> 2], t & 3);
                mma_bf16(o[t], __byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x5410),
                         __byte_perm(c, d, 0x7632), b0, b1);
            }
        }
    }
    // first of the two dimensions of accumulator t that lane group r holds
    __device__ __forceinline__ static int dim_of(int t, int r) {
        return kE5M2 ? (D / 8) * r + 2 * t : 64 * (t >> 2) + 8 * r + 2 * (t & 3);
    }
    __device__ __forceinline__ void hand_over(JoinSmem<D>& js) {
        const int warp = threadIdx.x >> 5, r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, x);
            l1 += __shfl_xor_sync(0xffffffffu, l1, x);
        }
        if (r == 0) {
            js.m[warp][2 * c] = m0 - kBaseShift;
            js.m[warp][2 * c + 1] = m1 - kBaseShift;
            js.l[warp][2 * c] = l0;
            js.l[warp][2 * c + 1] = l1;
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            *reinterpret_cast<float2*>(&js.o[warp][0][c][dim_of(t, r)]) = make_float2(o[t][0], o[t][2]);
            *reinterpret_cast<float2*>(&js.o[warp][1][c][dim_of(t, r)]) = make_float2(o[t][1], o[t][3]);
        }
    }
    // rows [row0, end) of the unit, 16 at row0 + t * kPaBlock
    __device__ __forceinline__ void share(const PagedAttnParams& p, int b, int h, int row0, int end, float* z) {
        const int lane = threadIdx.x & 31;
        if (row0 >= end) return;
        PageIds now = page_ids(p.c, b, row0 + lane * kPaBlock, end), next = now;
        int t = 0;
        Keys k;
        Values v;
        int ida = __shfl_sync(0xffffffffu, now.a, 0), idb = __shfl_sync(0xffffffffu, now.b, 0);
        load_k(p, h, row0, end, ida, idb, k);
        load_v(p, h, row0, end, ida, idb, v);
        if (row0 + 32 * kPaBlock < end) next = page_ids(p.c, b, row0 + (32 + lane) * kPaBlock, end);
        for (int row = row0; row < end; row += kPaBlock) {
            float s[4];
            scores(k, s);
            const int was_a = ida, was_b = idb;
            const bool more = row + kPaBlock < end;
            if (more) {
                if (++t == 32) {
                    t = 0;
                    now = next;
                    if (row + 33 * kPaBlock < end) next = page_ids(p.c, b, row + (33 + lane) * kPaBlock, end);
                }
                ida = __shfl_sync(0xffffffffu, now.a, t);
                idb = __shfl_sync(0xffffffffu, now.b, t);
                load_k(p, h, row + kPaBlock, end, ida, idb, k);
            }
            if (z) keep(p, z, row, end, was_a, was_b, s);
            uint32_t b0, b1;
            softmax(p.scale_log2, row, end, was_a, was_b, s, b0, b1);
            values(v, b0, b1);
            if (more) load_v(p, h, row + kPaBlock, end, ida, idb, v);
        }
    }
};

// fp32: a half-warp per eight rows, lane hl holding the dimensions 4 hl + 64 j
template <int D, int G>
struct TileF32 {
    static constexpr int kV = D / 64;      // float4 of a row per lane
    float o[G][4 * kV];
    float m[G], l[G];
    const float* sq;                       // [G][D] queries in shared memory

    __device__ __forceinline__ void load_q(const PagedAttnParams& p, int b, int h, float* s_q) {
        __syncthreads();
        for (int i = threadIdx.x; i < G * D; i += kPaThreads) {
            const int g = i / D;
            s_q[i] = g < p.G ? __ldg(static_cast<const float*>(p.q) + b * p.q_seq + (h * p.G + g) * p.q_head + i % D) : 0.f;
        }
        __syncthreads();
        sq = s_q;
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            m[g] = -CUDART_INF_F;
            l[g] = 0.f;
#pragma unroll
            for (int i = 0; i < 4 * kV; ++i) o[g][i] = 0.f;
        }
    }
    __device__ __forceinline__ void load(const float* base, int64_t page, int64_t pitch, int mask, int row, int end, int id,
                                         float (&x)[8][4 * kV]) {
        const int hl = threadIdx.x & 15;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* src = base + id * page + ((row + i) & mask) * pitch + 4 * hl;
            const bool in = id >= 0 && row + i < end;
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const uint4 w = ld_stream(src + 64 * j, in);
                x[i][4 * j] = __uint_as_float(w.x);
                x[i][4 * j + 1] = __uint_as_float(w.y);
                x[i][4 * j + 2] = __uint_as_float(w.z);
                x[i][4 * j + 3] = __uint_as_float(w.w);
            }
        }
    }
    __device__ __forceinline__ void share(const PagedAttnParams& p, int b, int h, int row0, int end, float* z) {
        const int lane = threadIdx.x & 31, hl = lane & 15, half = lane >> 4, mask = (1 << p.c.lg) - 1;
        const float* kb = static_cast<const float*>(p.c.k) + h * p.c.k_head;
        const float* vb = static_cast<const float*>(p.c.v) + h * p.c.v_head;
        PageIds now{-1, -1};
        int t = 32;
        for (int row = row0; row < end; row += kPaBlock, ++t) {
            if (t == 32) {
                t = 0;
                now = page_ids(p.c, b, row + lane * kPaBlock, end);
            }
            const int ida = __shfl_sync(0xffffffffu, now.a, t), idb = __shfl_sync(0xffffffffu, now.b, t);
            const int id = half ? idb : ida, mine = row + 8 * half;      // this half-warp's eight rows
            float x[8][4 * kV];
            load(kb, p.c.k_page, p.c.k_row, mask, mine, end, id, x);
            const bool in = id >= 0 && mine + (hl >> 1) < end;
            float s[G];
            bool up = false;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) a[i] = 0.f;
#pragma unroll
                for (int j = 0; j < kV; ++j) {
                    const float4 qv = *reinterpret_cast<const float4*>(sq + g * D + 64 * j + 4 * hl);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] = fmaf(x[i][4 * j], qv.x, a[i]);
                        a[i] = fmaf(x[i][4 * j + 1], qv.y, a[i]);
                        a[i] = fmaf(x[i][4 * j + 2], qv.z, a[i]);
                        a[i] = fmaf(x[i][4 * j + 3], qv.w, a[i]);
                    }
                }
                s[g] = transpose_reduce8(a, hl);
                if (z && (hl & 1) == 0 && mine + (hl >> 1) < end && g < p.G)
                    z[static_cast<int64_t>(mine + (hl >> 1)) * p.Gp + g] = in ? s[g] : -CUDART_INF_F;
                up = up || (in && s[g] * p.scale_log2 > m[g] + kPaSlack);
            }
            load(vb, p.c.v_page, p.c.v_row, mask, mine, end, id, x);
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float top = fmaxf(m[g], warp_max(in ? s[g] * p.scale_log2 : -CUDART_INF_F));
                    const float w = m[g] == -CUDART_INF_F ? 0.f : exp2_fast(m[g] - top);
                    m[g] = top;
                    l[g] *= w;
#pragma unroll
                    for (int i = 0; i < 4 * kV; ++i) o[g][i] *= w;
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const float pr = in ? exp2_fast(fmaf(s[g], p.scale_log2, m[g] == -CUDART_INF_F ? 0.f : -m[g])) : 0.f;
                l[g] += pr;                     // every row is held by two lanes: halved at the end
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w = __shfl_sync(0xffffffffu, pr, 16 * half + 2 * i);
#pragma unroll
                    for (int j = 0; j < 4 * kV; ++j) o[g][j] = fmaf(w, x[i][j], o[g][j]);
                }
            }
        }
    }
    __device__ __forceinline__ void hand_over(JoinSmem<D>& js) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hl = lane & 15;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float sum = 0.5f * warp_sum(l[g]);
            if (lane == 0) {
                js.m[warp][g] = m[g];
                js.l[warp][g] = sum;
            }
#pragma unroll
            for (int i = 0; i < 4 * kV; ++i) {
                const float x = o[g][i] + __shfl_xor_sync(0xffffffffu, o[g][i], 16);
                if (lane < 16) js.o[warp][g & 1][g >> 1][64 * (i / 4) + 4 * hl + i % 4] = x;
            }
        }
    }
};

// ------------------------------------------------------------------ the kernels

__device__ __forceinline__ void store_out(const PagedAttnParams& p, bool f32, int b, int h, int g, int dim, float x) {
    const int64_t at = b * p.o_seq + (h * p.G + g) * p.o_head + dim;
    if (f32) static_cast<float*>(p.out)[at] = x;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(x);
}
// base + log2(sum) as a natural logarithm; -inf for a unit of no rows
__device__ __forceinline__ float ln_of(float m, float l) { return l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.693147180559945309f; }

template <class Tile, int D, bool kF32, int kOcc>
__global__ void __launch_bounds__(kPaThreads, kOcc) k_paged_attn(const __grid_constant__ PagedAttnParams p) {
    __shared__ PlanSmem s_plan;
    __shared__ __align__(16) JoinSmem<D> js;
    __shared__ __align__(16) float s_q[kF32 ? kPaHeads * D : 4];
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t ctas = gridDim.x, me = blockIdx.x;
    const Place pl = plan(p.c, me, ctas, s_plan);

    const bool work = me < pl.n;
    const int64_t w0 = work ? me * pl.total / pl.n : 0, w1 = work ? (me + 1) * pl.total / pl.n : 0;
    int b = pl.b, rows = pl.rows, nb = pl.nb;
    int h = work ? static_cast<int>((w0 - pl.first) / nb) : 0;
    int64_t unit0 = pl.first + static_cast<int64_t>(h) * nb;     // first block of the unit
    if (tid == 0) {
        Joint j{-1, 0, 0, 0};
        if (work && unit0 < w0 && unit0 + nb <= w1) {
            const int64_t from = ((unit0 + 1) * pl.n - 1) / pl.total;      // the CTA whose range holds block unit0
            j = Joint{static_cast<int>(from), b, h, from * pl.total / pl.n == unit0 ? 0 : 1};
        }
        p.joint[me] = j;
    }
    Tile tile;
    for (int64_t cur = w0; cur < w1;) {
        const int blk = static_cast<int>(cur - unit0);
        const int64_t stop = min(w1, unit0 + nb);
        const int first = blk * kPaBlock, end = static_cast<int>(min(static_cast<int64_t>(rows), (stop - unit0) * kPaBlock));
        tile.load_q(p, b, h, s_q);
        tile.reset();
        const int64_t u = static_cast<int64_t>(b) * p.c.H + h;
        float* z = p.z ? p.z + u * p.c.cap * p.Gp : nullptr;
        tile.share(p, b, h, first + warp * kPaTile, end, z);
        tile.hand_over(js);
        __syncthreads();
        // join the warps: thread = dimension (and every other head where d is 64)
        const bool alone = cur == unit0 && stop == unit0 + nb;
        float* rec = p.rec + (me * 2 + (cur == w0 ? 0 : 1)) * p.G * (D + 2);
        for (int g = tid / D; g < p.G; g += kPaThreads / D) {
            const int dim = tid % D;
            float m = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kPaWarps; ++w) m = fmaxf(m, js.m[w][g]);
            float l = 0.f, x = 0.f;
#pragma unroll
            for (int w = 0; w < kPaWarps; ++w) {
                const float f = js.m[w][g] == -CUDART_INF_F && !(js.l[w][g] != js.l[w][g]) ? 0.f : exp2_fast(js.m[w][g] - m);
                l = fmaf(js.l[w][g], f, l);
                x = fmaf(js.o[w][g & 1][g >> 1][dim], f, x);
            }
            if (alone) {
                store_out(p, kF32, b, h, g, dim, l == 0.f ? 0.f : x / l);
                if (dim == 0) {
                    if (p.lse) p.lse[static_cast<int64_t>(b) * p.n_q + h * p.G + g] = ln_of(m, l);
                    if (p.stat) p.stat[u * p.G + g] = make_float2(m, l == 0.f ? 0.f : 1.f / l);
                }
            } else {
                rec[g * (D + 2) + dim] = x;
                if (dim == 0) *reinterpret_cast<float2*>(rec + g * (D + 2) + D) = make_float2(m, l);
            }
        }
        __syncthreads();
        cur = stop;
        if (cur >= w1) break;
        unit0 += nb;
        if (++h == p.c.H) {      // the next sequence that has rows
            h = 0;
            next_rows(p.c, b, rows);
            if (rows < 0) break;     // the lengths changed under the call
            nb = blocks_of(rows);
        }
    }
    // sequences of no rows
    for (int e = blockIdx.x; e < p.c.batch; e += gridDim.x)
        if (rows_of(p.c, e, g_err, 711) == 0) {
            for (int i = tid; i < p.n_q * D; i += kPaThreads) store_out(p, kF32, e, 0, i / D, i % D, 0.f);
            if (p.lse)
                for (int i = tid; i < p.n_q; i += kPaThreads) p.lse[static_cast<int64_t>(e) * p.n_q + i] = -CUDART_INF_F;
        }
}

// Joins the records of the units that lie in more than one CTA's range: CTA (i, g) those of head
// g of the unit that ends in CTA i's range and began before it (p.joint[i] says which, if any).
// Lanes hold four dimensions each; warps (half-warps where d is 64) take the contributors in turn.
constexpr int kPaMost = 512;      // contributors at most

template <int D, bool kF32>
__global__ void __launch_bounds__(kPaThreads) k_paged_merge(const __grid_constant__ PagedAttnParams p) {
    constexpr int kLanes = D / 4, kWays = kPaThreads / kLanes;
    __shared__ float s_f[kPaMost], s_red[kPaWarps], s_sum[kPaWarps];
    __shared__ __align__(16) float s_x[kWays][D];
    pdl_trigger();
    // every CTA waits for the grid before, so that this grid's end stands for both
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.y, me = blockIdx.x;
    const int4 raw = __ldcg(reinterpret_cast<const int4*>(p.joint) + me);
    const Joint j{raw.x, raw.y, raw.z, raw.w};
    if (j.from < 0) return;
    const int n = me - j.from + 1;
    const int64_t pitch = p.G * (D + 2);
    // contributor i's record: slot 0, but the unit began inside the first one's range
    auto rec_of = [&](int i) { return p.rec + (static_cast<int64_t>(j.from + i) * 2 + (i == 0 ? j.slot : 0)) * pitch + g * (D + 2); };
    float m = -CUDART_INF_F;
    for (int i = tid; i < n; i += kPaThreads) m = fmaxf(m, __ldcg(rec_of(i) + D));
    m = warp_max(m);
    if (lane == 0) s_red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) m = fmaxf(m, s_red[w]);
    float l = 0.f;
    for (int i = tid; i < n; i += kPaThreads) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(rec_of(i) + D));
        const float f = ml.x == -CUDART_INF_F && !(ml.y != ml.y) ? 0.f : exp2_fast(ml.x - m);
        s_f[i] = f;
        l = fmaf(ml.y, f, l);
    }
    l = warp_sum(l);
    if (lane == 0) s_sum[warp] = l;
    __syncthreads();
    l = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
    const int dim = 4 * (tid % kLanes), way = tid / kLanes;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = way; i < n; i += kWays) {
        const float* r = rec_of(i) + dim;
        const float2 a = __ldcg(reinterpret_cast<const float2*>(r)), b = __ldcg(reinterpret_cast<const float2*>(r + 2));
        const float f = s_f[i];
        x[0] = fmaf(a.x, f, x[0]);
        x[1] = fmaf(a.y, f, x[1]);
        x[2] = fmaf(b.x, f, x[2]);
        x[3] = fmaf(b.y, f, x[3]);
    }
    *reinterpret_cast<float4*>(&s_x[way][dim]) = make_float4(x[0], x[1], x[2], x[3]);
    __syncthreads();
    if (tid < D) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWays; ++w) sum += s_x[w][tid];
        store_out(p, kF32, j.b, j.h, g, tid, l == 0.f ? 0.f : sum / l);
    }
    if (tid == 0) {
        if (p.lse) p.lse[static_cast<int64_t>(j.b) * p.n_q + j.h * p.G + g] = ln_of(m, l);
        if (p.stat) p.stat[(static_cast<int64_t>(j.b) * p.c.H + j.h) * p.G + g] = make_float2(m, l == 0.f ? 0.f : 1.f / l);
    }
}

// Four rows per thread and turn: their products are loaded before any of them is used.
template <int Gp>
__device__ __forceinline__ void weigh_rows_of(const PagedAttnParams& p, int64_t u, int first, int end) {
    const float* z = p.z + u * p.c.cap * Gp;
    const float* in = p.weight + u * p.row_pitch;
    float* out = p.weight_out + u * p.row_pitch;
    float base[Gp], inv[Gp];
#pragma unroll
    for (int g = 0; g < Gp; ++g) {
        const float2 st = g < p.G ? __ldcg(p.stat + u * p.G + g) : make_float2(0.f, 0.f);
        base[g] = st.x;
        inv[g] = st.y;
    }
    for (int i0 = first + threadIdx.x; i0 < end; i0 += 4 * kPaThreads) {
        float2 x[4][Gp / 2];
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + r * kPaThreads;
            if (i >= end) continue;
            w[r] = in[i];
#pragma unroll
            for (int g = 0; g < Gp / 2; ++g) x[r][g] = __ldcg(reinterpret_cast<const float2*>(z + static_cast<int64_t>(i) * Gp) + g);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + r * kPaThreads;
            if (i >= end) continue;
            float sum = 0.f;
#pragma unroll
            for (int g = 0; g < Gp; ++g) {
                const float v = g & 1 ? x[r][g / 2].y : x[r][g / 2].x;
                // an absent row's product is -inf and adds nothing
                if (g < p.G && v != -CUDART_INF_F) sum += exp2_fast(fmaf(v, p.scale_log2, -base[g])) * inv[g];
            }
            out[i] = w[r] + sum;
        }
    }
}
__device__ __forceinline__ void weigh_rows(const PagedAttnParams& p, int64_t u, int first, int end) {
    if (p.Gp == 2) weigh_rows_of<2>(p, u, first, end);
    else if (p.Gp == 4) weigh_rows_of<4>(p, u, first, end);
    else if (p.Gp == 6) weigh_rows_of<6>(p, u, first, end);
    else weigh_rows_of<8>(p, u, first, end);
}

// weight_out = weight + sum over the heads of exp2(z scale - base) / sum, over the same split
__global__ void __launch_bounds__(kPaThreads) k_paged_weigh(const __grid_constant__ PagedAttnParams p) {
    __shared__ PlanSmem s_plan;
    const int tid = threadIdx.x;
    const int64_t ctas = gridDim.x, me = blockIdx.x;
    const Place pl = plan(p.c, me, ctas, s_plan);
    pdl_wait();
    if (me >= pl.n) return;
    const int64_t w0 = me * pl.total / pl.n, w1 = (me + 1) * pl.total / pl.n;
    int b = pl.b, rows = pl.rows, nb = pl.nb;
    int h = static_cast<int>((w0 - pl.first) / nb);
    int64_t unit0 = pl.first + static_cast<int64_t>(h) * nb;
    for (int64_t cur = w0; cur < w1;) {
        const int64_t stop = min(w1, unit0 + nb);
        const int first = static_cast<int>(cur - unit0) * kPaBlock;
        const int end = static_cast<int>(min(static_cast<int64_t>(rows), (stop - unit0) * kPaBlock));
        const int64_t u = static_cast<int64_t>(b) * p.c.H + h;
        weigh_rows(p, u, first, end);
        cur = stop;
        if (cur >= w1) break;
        unit0 += nb;
        if (++h == p.c.H) {
            h = 0;
            next_rows(p.c, b, rows);
            if (rows < 0) break;     // the lengths changed under the call
            nb = blocks_of(rows);
        }
    }
}

// ------------------------------------------------------------------ launches

constexpr int kOccTC = 3, kOccF32 = 2;     // CTAs per SM
constexpr int kWeighOcc = 3;               // CTAs of k_paged_weigh per CTA of k_paged_attn

int paged_attn_ctas(int dtype, int nsm) { return nsm * (dtype == SKV_F32 ? kOccF32 : kOccTC); }

template <class Tile, int D, bool kF32, int kOcc>
static int launch_pa(const PagedAttnParams& p, int ncta, cudaStream_t s) {
    // no more CTAs than there can be blocks of rows
    const int64_t most = static_cast<int64_t>(p.c.batch) * p.c.H * ((p.c.cap + kPaBlock - 1) / kPaBlock);
    const int n = most < ncta ? static_cast<int>(most) : ncta;
    k_paged_attn<Tile, D, kF32, kOcc><<<n, kPaThreads, 0, s>>>(p);
    if (launch_pdl(k_paged_merge<D, kF32>, dim3(n, p.G), dim3(kPaThreads), 0, s, p) != cudaSuccess) return -1;
    if (p.weight_out) {
        const int64_t wide = kWeighOcc * static_cast<int64_t>(ncta);
        const int nw = static_cast<int>(most < wide ? most : wide);
        if (launch_pdl(k_paged_weigh, dim3(nw), dim3(kPaThreads), 0, s, p) != cudaSuccess) return -1;
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}
template <int D>
static int launch_f32(const PagedAttnParams& p, int ncta, cudaStream_t s) {
    if (p.G <= 1) return launch_pa<TileF32<D, 1>, D, true, kOccF32>(p, ncta, s);
    if (p.G <= 2) return launch_pa<TileF32<D, 2>, D, true, kOccF32>(p, ncta, s);
    if (p.G <= 4) return launch_pa<TileF32<D, 4>, D, true, kOccF32>(p, ncta, s);
    return launch_pa<TileF32<D, 8>, D, true, kOccF32>(p, ncta, s);
}

int launch_paged_attn(int dtype, int d, const PagedAttnParams& p, int ncta, cudaStream_t s) {
    if (dtype == SKV_F32) return d == 64 ? launch_f32<64>(p, ncta, s) : launch_f32<128>(p, ncta, s);
    if (dtype == SKV_FP8)
        return d == 64 ? launch_pa<TileTC<64, true>, 64, false, kOccTC>(p, ncta, s)
                       : launch_pa<TileTC<128, true>, 128, false, kOccTC>(p, ncta, s);
    return d == 64 ? launch_pa<TileTC<64, false>, 64, false, kOccTC>(p, ncta, s)
                   : launch_pa<TileTC<128, false>, 128, false, kOccTC>(p, ncta, s);
}

cudaError_t paged_attn_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
