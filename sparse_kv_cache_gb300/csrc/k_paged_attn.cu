// Attention of one new token per sequence over its paged cache (shadowkv_paged_attention).
//
// out = softmax(scale q.K^T).V for the G query heads of every unit (a sequence's KV head), in one
// pass over the unit's rows with a running base and sum of the softmax.  Each cached byte is read
// once and takes part in G products per element, 2G flops per byte in bf16, so memory bounds it.
//
// Work split.  The rows of all units form one sequence of 16-row tiles; CTA i of n takes the tiles
// [i T / n, (i + 1) T / n), whatever units they belong to, and each of its four warps a quarter of
// them.  So every SM gets the same share of any mix of lengths, and the host need not know them (a
// captured graph replays with new lengths).  Warps work on their own, with no barrier between
// them, and finish the units that lie in their quarter whole.  The other shares are joined twice, each
// time in order: those of a CTA's warps through shared memory, and those of several CTAs by
// k_paged_merge, a programmatic dependent, from the CTAs' two records (of their first and last unit).
//
// bf16 and e5m2: no shared memory in the loop.  S^T = K.Q^T has the rows in the 16-wide dimension
// of m16n8k16 and the heads in the 8-wide one, so up to eight heads waste nothing; its operands
// come straight from 16-byte global loads, because a dot product may take its terms in any order
// as long as both operands agree.  O^T = V^T.P^T takes pairs of rows interleaved by byte
// permutes, again from 16-byte loads, and P^T is S^T's accumulator passed through movmatrix.  The
// tensor cores are busy for less than a tenth of the time that the loads take, so the warp-level
// instruction suffices: tcgen05 would put both operands and the accumulator through shared and
// tensor memory first.
//
// fp32 takes the same split with products on the CUDA cores: a half-warp per eight rows, their sums
// joined by a transposing reduction.
//
// Measured back to back (8 KV heads of 4 query heads, d = 128, each row's bytes once over the time;
// a copy runs at 6.7 TB/s): 8 x 128K rows in bf16 600 to 609 us by box, 7.1 TB/s; 4 x 32K rows 88.7 us, 6.1
// TB/s; 8 ragged sequences of up to 64K rows with e5m2 values 139 us, 6.2 TB/s; 192 of 0 to 611 rows (4
// KV heads of 8) 30.6 us, 4.0 TB/s, a CTA per unit whose start and end are latency; 4096 of 0 to 30 rows (2
// of 4) 31.0 us against 11.6 of their bytes; one sequence of 1013 rows 6.4 us, all of it latency (13 in a
// table for 128K rows, by whose width the form is chosen).
#include <math_constants.h>

#include <atomic>

#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kPaThreads = 128;
static_assert(kPaThreads == 32 * kPaWarps, "");
constexpr int kPaTile = 16;                       // rows of a warp's step
constexpr float kPaSlack = 8.f;                   // the base moves when a score passes it by 2^8
// Values are multiplied by p.down of a probability that is not normalised yet, 2^-8 over the rows that a
// sequence has room for: with the slack they then add up to 1 at most, so no sum of values passes the
// largest value, which may be the type's.  (Of a table for 128K rows, 2^-25: products of values below 2^-101
// lose bits at fp32's smallest.  In the exponent it would cost all probabilities 2^-20 of themselves.)

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
        "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(static_cast<int>(in)));
    return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p, bool in) {
    uint2 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
        "@p ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n\t}"
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
__device__ __forceinline__ float4 ld_cluster_v4f(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// the upper halves of two floats
__device__ __forceinline__ uint32_t cut_bf16x2(float lo, float hi) {
    return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// ------------------------------------------------------------------ the split of the work

template <int R = kPaTile>
__device__ __forceinline__ int tiles_of(int n) { return (n + R - 1) / R; }

// What CTA `me` of `ctas` takes of the tiles of R rows, and where its W parts begin.  Little work goes to the
// fewest CTAs whose parts average no more than kPaLeast tiles (so that beyond one CTA's they average more
// than half of it): with less, joining the shares takes longer than forming them (one unit of 32K rows: 17.4
// us with four, 19.2 with two, 23.2 with one).  The tiles of fp32 take longer, and so may come one by one.
constexpr int kPaLeast = 4;

template <int W>
struct PlanSmem {
    int64_t warp_sum[kPaWarps];
    int64_t at[W];       // first tile of the sequence that part starts in
    int b[W], rows[W];   // that sequence and its rows
};
template <int W>
struct Plan {
    int64_t total, n;    // tiles of all units; CTAs that have work
    int64_t lo, hi;      // tiles of this CTA (lo == hi: none)
    __device__ __forceinline__ int64_t start(int64_t i) const { return i * total / n; }
    __device__ __forceinline__ int64_t holder(int64_t x) const { return ((x + 1) * n - 1) / total; }   // of tile x
    __device__ __forceinline__ int64_t part(int w) const { return lo + w * (hi - lo) / W; }
};

// Each warp takes a quarter of the sequences, 32 at a time, and its lane j keeps the sum of the j-th run of
// them; the warp whose runs hold a part's first tile looks through that run.  A part whose sequence is not
// found (the lengths changed under the call) has no rows.
template <int W, int R, int kLeast>
__device__ __forceinline__ Plan<W> make_plan(const PagedView& c, int64_t me, int64_t ctas, PlanSmem<W>& sm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int steps = (c.batch + 32 * kPaWarps - 1) / (32 * kPaWarps), run_steps = (steps + 31) / 32;
    const int s0 = warp * steps * 32 + lane;
    constexpr int kDeep = 4;       // steps whose loads are in flight together
    int64_t mine = 0;
    int first = 0;
    for (int j0 = 0; j0 < steps; j0 += kDeep) {
        int n[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int s = s0 + 32 * (j0 + k);
            n[k] = j0 + k < steps && s < c.batch ? __ldcg(c.lens + s) : 0;
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            n[k] = rows_in(c, n[k], g_err, 711);
            const uint32_t sum = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(tiles_of<R>(n[k])));
            if (lane == (j0 + k) / run_steps) mine += sum;
        }
        if (j0 == 0) first = n[0];
    }
    if (tid < W) sm.rows[tid] = 0;
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
    Plan<W> pl;
    pl.total = all * c.H;
    pl.n = min(ctas, (pl.total + kLeast * W - 1) / (kLeast * W));
    pl.lo = me < pl.n ? pl.start(me) : 0;
    pl.hi = me < pl.n ? pl.start(me + 1) : 0;
    const int64_t begin = (before + run - mine) * c.H, stop = begin + mine * c.H;
    int held = 0, rows = first;                // the warp's step whose lengths the lanes have
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int64_t x = pl.part(w);
        const uint32_t who = __ballot_sync(0xffffffffu, pl.lo < pl.hi && x >= begin && x < stop);
        if (!who) continue;
        const int owner = __ffs(who) - 1;
        int64_t at = __shfl_sync(0xffffffffu, begin, owner);
        for (int j = owner * run_steps; j < steps; ++j) {
            const int s = s0 + 32 * j;
            if (j != held) {
                rows = s < c.batch ? rows_of(c, s, g_err, 711) : 0;
                held = j;
            }
            const uint32_t size = tiles_of<R>(rows);
            uint32_t upto = size;              // (32 sequences have 2^31 tiles at most)
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const int64_t end = at + static_cast<int64_t>(upto) * c.H, from = end - static_cast<int64_t>(size) * c.H;
            if (__any_sync(0xffffffffu, x < end)) {
                if (x >= from && x < end) {
                    sm.at[w] = from;
                    sm.b[w] = s;
                    sm.rows[w] = rows;
                }
                break;
            }
            at = __shfl_sync(0xffffffffu, end, 31);
        }
    }
    __syncthreads();
    return pl;
}

// A part's way through the units: its current unit, and the unit's first tile in the launch.
template <int R>
struct Walk {
    int b, h, rows, nt;
    int64_t unit0;
    __device__ __forceinline__ void enter(int seq, int n, int64_t at, int64_t x) {
        b = seq;
        rows = n;
        nt = tiles_of<R>(n);
        h = static_cast<int>((x - at) / nt);
        unit0 = at + static_cast<int64_t>(h) * nt;
    }
    // the next unit that has rows; false if there is none (the lengths changed under the call)
    __device__ __forceinline__ bool next(const PagedView& c) {
        unit0 += nt;
        if (++h < c.H) return true;
        h = 0;
        const int lane = threadIdx.x & 31;
        for (int s = b + 1; s < c.batch; s += 32) {
            const int n = s + lane < c.batch ? rows_of(c, s + lane, g_err, 711) : 0;
            const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
            if (!some) continue;
            const int at = __ffs(some) - 1;
            b = s + at;
            rows = __shfl_sync(0xffffffffu, n, at);
            nt = tiles_of<R>(rows);
            return true;
        }
        return false;
    }
};

// ------------------------------------------------------------------ a warp's share of a unit

__device__ __forceinline__ void store_out(const PagedAttnParams& p, bool f32, int b, int h, int g, int dim, float x) {
    const int64_t at = b * p.o_seq + (h * p.G + g) * p.o_head + dim;
    if (f32) static_cast<float*>(p.out)[at] = x;
    else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(x);
}
// base + log2(sum) as a natural logarithm; -inf for a unit of no rows
__device__ __forceinline__ float ln_of(float m, float l) { return l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.693147180559945309f; }

// four consecutive dimensions of a head
template <bool kF32>
__device__ __forceinline__ void store4(const PagedAttnParams& p, int b, int h, int g, int dim, const float (&x)[4]) {
    const int64_t at = b * p.o_seq + (h * p.G + g) * p.o_head + dim;
    if (kF32) *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(x[0], x[1], x[2], x[3]);
    else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) =
            make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// What goes with head g of a unit beside its output.
__device__ __forceinline__ void note(const PagedAttnParams& p, int b, int h, int g, float m, float l) {
    if (p.lse) p.lse[static_cast<int64_t>(b) * p.n_q + h * p.G + g] = ln_of(m, l);
    if (p.stat) p.stat[(static_cast<int64_t>(b) * p.c.H + h) * p.G + g] = make_float2(m, l == 0.f ? 0.f : 1.f / l);
}

// The shares that a CTA's warps leave for the join: two per warp, of its first and its last unit.
// O is not normalised; heads lie d + 4 apart, so that the lanes' 16-byte writes spread over the banks.
// b < 0: none; whether it holds the unit's first and last tile, and the CTA's first
struct ShareOf { int b, h; bool begins, ends, first; };
struct Run { int b, h, from, last; bool whole, first; };      // consecutive shares of one unit
template <int D, int G>
struct JoinSmem {
    float o[2 * kPaWarps][G][D + 4];
    float m[2 * kPaWarps][G], l[2 * kPaWarps][G], w[2 * kPaWarps][G];
    ShareOf of[2 * kPaWarps];
    Run run[2 * kPaWarps];
    int runs;
};
// weight of a share of base x and sum l against the base m of all
__device__ __forceinline__ float share_weight(float x, float l, float m) {
    return x == -CUDART_INF_F && !(l != l) ? 0.f : exp2_fast(x - m);
}

// A running sum of thousands of terms loses more by its roundings (the tensor cores cut off what does
// not fit) than its terms are off by.  So every 32 tiles a warp adds its sums to ones held in shared
// memory, in the place of its last share, and begins again at zero; what is held goes by the base that
// it was formed with.  (One warp over 128K rows of values 1, then -1: off by 1.7e-4 without, where all other
// roundings may make 7e-5.  8 x 128K rows take 0.2 % longer for it.)
struct HoldNone { __device__ __forceinline__ void operator()() const {} };     // a warp of few tiles

// Page ids of a warp's coming tiles: lane j holds those of tile j of the current 32.
struct PageIds {
    int a, b;    // of the tile's first and last eight rows
};

__device__ __forceinline__ PageIds page_ids(const PagedView& c, int b, int row, int end) {
    PageIds id{-1, -1};
    if (row < end) {
        id.a = page_of(c, b, row, g_err, 712);
        id.b = c.lg > 3 ? id.a : row + 8 < end ? page_of(c, b, row + 8, g_err, 712) : -1;
    }
    return id;
}

// A warp's rows of one unit: rows [row, end) of head h of sequence b, and the page ids of the first 32
// tiles.
struct Piece {
    int b, h, row, end;
    PageIds ids;
    __device__ __forceinline__ void ask(const PagedView& c) { ids = page_ids(c, b, row + (threadIdx.x & 31) * kPaTile, end); }
};
// The pieces of a warp's tiles, one after the other: all but the first begin with their unit's first
// tile, all but the last end with its last.  The lengths of 32 sequences are held by the lanes, so
// that going on to the next takes no load.
struct Pieces {
    int b, h, left, base, lens;
    bool begins, ends;      // whether the first piece does, and the last one
    __device__ __forceinline__ void fetch(const PagedView& c) {
        const int s = base + (threadIdx.x & 31);
        lens = s < c.batch ? rows_of(c, s, g_err, 711) : 0;
    }
    // the first: tiles from x on, `tiles` of them, x in the sequence `seq` whose first tile is `at`
    __device__ __forceinline__ Piece first(const PagedView& c, int seq, int rows, int64_t at, int64_t x, int64_t tiles) {
        const int nt = tiles_of(rows);
        const int skip = static_cast<int>((x - at) % nt), take = static_cast<int>(min(tiles, static_cast<int64_t>(nt - skip)));
        b = base = seq;
        h = static_cast<int>((x - at) / nt);
        left = static_cast<int>(tiles - take);
        begins = skip == 0;
        ends = skip + take == nt;
        if (left > 0) fetch(c);
        Piece q{b, h, skip * kPaTile, min(rows, (skip + take) * kPaTile), {-1, -1}};
        q.ask(c);
        return q;
    }
    __device__ __forceinline__ bool next(const PagedView& c, Piece& q) {
        if (left <= 0) return false;
        if (++h == c.H) {
            h = 0;
            uint32_t some = __ballot_sync(0xffffffffu, lens > 0) & ~((2u << (b - base)) - 1);
            while (!some) {
                base += 32;
                if (base >= c.batch) return false;      // the lengths changed under the call
                fetch(c);
                some = __ballot_sync(0xffffffffu, lens > 0);
            }
            b = base + __ffs(some) - 1;
        }
        const int rows = __shfl_sync(0xffffffffu, lens, b - base), nt = tiles_of(rows), take = min(left, nt);
        left -= take;
        ends = take == nt;
        q = Piece{b, h, 0, min(rows, take * kPaTile), {-1, -1}};
        q.ask(c);
        return true;
    }
};

// The product that scores -infinity: what is kept for an absent row, which adds no weight.
__device__ __forceinline__ float no_product(const PagedAttnParams& p) { return copysignf(CUDART_INF_F, -p.scale_log2); }

// Where the products q.k of a tile's rows are kept for the weights, [row][Gp]: nowhere, in the
// workspace, or in the warp's part of shared memory.
struct KeepNone {
    static constexpr bool on = false;
    __device__ __forceinline__ float* operator()(int, int, int) const { return nullptr; }
};
struct KeepGlobal {
    static constexpr bool on = true;
    const PagedAttnParams& p;
    __device__ __forceinline__ float* operator()(int b, int h, int row) const {
        return p.z + ((static_cast<int64_t>(b) * p.c.H + h) * p.c.cap + row) * p.Gp;
    }
};
struct KeepShared {
    static constexpr bool on = true;
    float* z;
    int row0, Gp;
    __device__ __forceinline__ float* operator()(int, int, int row) const { return z + (row - row0) * Gp; }
};

template <int D, bool kE5M2>
struct TileTC {
    static constexpr int kKV = D / 32;                     // 16-byte words of a key row per lane
    static constexpr int kVV = kE5M2 ? 1 : D / 64;         // words of a value row per lane
    // fp16 probabilities: up to 2^15, the more of the small ones are normal (2^30 e5m2 values fit into a sum)
    static constexpr float kBaseShift = kE5M2 ? 7.f : 0.f;
    static constexpr bool kLow = !kE5M2;                   // whether p.down is in the sums of values
    uint4 q[kKV];
    float o[D / 16][4];
    float m0, m1, l0, l1;                                  // heads 2c and 2c + 1
    bool held;                                             // whether the unit has held sums

    __device__ __forceinline__ void load_q(const PagedAttnParams& p, int b, int h) {
        const int g = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + b * p.q_seq + (h * p.G + g) * p.q_head + c * 8;
#pragma unroll
        for (int j = 0; j < kKV; ++j)
            q[j] = g < p.G ? *reinterpret_cast<const uint4*>(src + 32 * j) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -CUDART_INF_F;
        l0 = l1 = 0.f;
        held = false;
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
    // raw products kept for the weights, z [row][Gp] from the tile's first row on
    __device__ __forceinline__ void keep(const PagedAttnParams& p, float* z, int row, int end, int ida, int idb,
                                         const float (&s)[4]) {
        const int r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
        if (2 * c >= p.G) return;
        const float none = no_product(p);
        if (row + r < end)
            *reinterpret_cast<float2*>(z + r * p.Gp + 2 * c) =
                ida >= 0 ? make_float2(s[0], s[1]) : make_float2(none, none);
        if (row + 8 + r < end)
            *reinterpret_cast<float2*>(z + (8 + r) * p.Gp + 2 * c) =
                idb >= 0 ? make_float2(s[2], s[3]) : make_float2(none, none);
    }
    // probabilities against the running base; returns P^T as the second product's operand, b, and what
    // its rounding to bf16 left, r
    __device__ __forceinline__ void softmax(float scale, int row, int end, int ida, int idb, const float (&s)[4], float down,
                                            uint32_t& b0, uint32_t& b1, uint32_t& r0, uint32_t& r1) {
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
        // The values' type for the tensor cores: fp16 (off by 2^-11 at most), or bf16 as the sum of two
        // terms (2^-16; one term alone, 2^-8, moved the result as much as its own rounding, and two cost
        // 0.4 % of 8 x 128K rows' time and 1 % of 192 short sequences').  Both terms are above zero where the
        // probability is, or an infinite value would meet a zero or a negative term and give NaN: the first is
        // cut off a little below it, not rounded.  The sums keep the fp32 ones.
        if (kE5M2) {
            const __half2 lo = __floats2half2_rn(x0, x1), hi = __floats2half2_rn(x2, x3);
            b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&lo));
            b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&hi));
        } else {
            const float below = down * (1.f - 0x1p-20f);
            const uint32_t h0 = cut_bf16x2(x0 * below, x1 * below), h1 = cut_bf16x2(x2 * below, x3 * below);
            b0 = transpose8x8(h0);
            b1 = transpose8x8(h1);
            r0 = transpose8x8(pack_bf16x2(fmaf(x0, down, -bf16lo(h0)), fmaf(x1, down, -bf16hi(h0))));
            r1 = transpose8x8(pack_bf16x2(fmaf(x2, down, -bf16lo(h1)), fmaf(x3, down, -bf16hi(h1))));
        }
    }
    __device__ __forceinline__ void values(const Values& v, uint32_t b0, uint32_t b1, uint32_t r0, uint32_t r1) {
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
                const uint32_t e0 = __byte_perm(a, b, 0x5410), e1 = __byte_perm(a, b, 0x7632);
                const uint32_t e2 = __byte_perm(c, d, 0x5410), e3 = __byte_perm(c, d, 0x7632);
                mma_bf16(o[t], e0, e1, e2, e3, b0, b1);
                mma_bf16(o[t], e0, e1, e2, e3, r0, r1);
            }
        }
    }
    // The lane's accumulators are runs of consecutive dimensions (accumulator t holds a pair for
    // each of two heads): two runs of 8 with bf16 values, one of D / 8 with e5m2 ones.
    static constexpr int kRun = kE5M2 ? D / 8 : 8;
    __device__ __forceinline__ static int dim_of(int r, int t) { return kE5M2 ? kRun * r + 2 * t : 64 * (t / 4) + 8 * r; }
    // adds what is held in a slot to the sums
    __device__ __forceinline__ void take(const JoinSmem<D, 8>& js, int slot) {
        const int r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float l = js.l[slot][2 * c + e], w = share_weight(js.m[slot][2 * c + e], l, e ? m1 : m0);
            if (r == 0) (e ? l1 : l0) = fmaf(l, w, e ? l1 : l0);
#pragma unroll
            for (int t = 0; t < D / 16; t += 4) {
                float x[8];
                load8(&js.o[slot][2 * c + e][dim_of(r, t)], x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[t + i][e] = fmaf(x[2 * i], w, o[t + i][e]);
                    o[t + i][2 + e] = fmaf(x[2 * i + 1], w, o[t + i][2 + e]);
                }
            }
        }
        __syncwarp();      // the slot may be written again
    }
    // adds the sums to what is held and begins again at zero
    __device__ __forceinline__ void hold(JoinSmem<D, 8>& js, int slot) {
        const int r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, x);
            l1 += __shfl_xor_sync(0xffffffffu, l1, x);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int g = 2 * c + e;
            float l = e ? l1 : l0, w = 0.f;
            if (held) {
                w = share_weight(js.m[slot][g], js.l[slot][g], e ? m1 : m0);
                l = fmaf(js.l[slot][g], w, l);
            }
            __syncwarp();
            if (r == 0) {
                js.m[slot][g] = e ? m1 : m0;
                js.l[slot][g] = l;
            }
#pragma unroll
            for (int t = 0; t < D / 16; t += 4) {
                float x[8] = {};
                if (held) load8(&js.o[slot][g][dim_of(r, t)], x);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = fmaf(x[2 * i], w, o[t + i][e]);
                    x[2 * i + 1] = fmaf(x[2 * i + 1], w, o[t + i][2 + e]);
                    o[t + i][e] = o[t + i][2 + e] = 0.f;
                }
                store8(&js.o[slot][g][dim_of(r, t)], x);
            }
        }
        l0 = l1 = 0.f;
        held = true;
        __syncwarp();
    }
    // writes the unit's result, or this share of it for the join
    __device__ __forceinline__ void finish(const PagedAttnParams& p, int b, int h, bool alone, JoinSmem<D, 8>& js, int slot,
                                           int from) {
        const int r = (threadIdx.x & 31) >> 2, c = threadIdx.x & 3;
        if (held) take(js, from);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, x);
            l1 += __shfl_xor_sync(0xffffffffu, l1, x);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int g = 2 * c + e;
            if (g >= p.G) continue;
            const float m = (e ? m1 : m0) - kBaseShift, l = e ? l1 : l0;
            const float inv = !alone ? 1.f : l == 0.f ? 0.f : 1.f / (l * p.down);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + b * p.o_seq + (h * p.G + g) * p.o_head;
#pragma unroll
            for (int t = 0; t < D / 16; t += 4) {
                const int dim = dim_of(r, t);
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[2 * i] = o[t + i][e] * inv;
                    x[2 * i + 1] = o[t + i][2 + e] * inv;
                }
                if (alone) store8(out + dim, x);
                else store8(&js.o[slot][g][dim], x);
            }
            if (r == 0) {
                if (alone) {
                    note(p, b, h, g, m, l);
                } else {
                    js.m[slot][g] = m;
                    js.l[slot][g] = l;
                }
            }
        }
    }
    // The pieces from `cur` on, as one stream of tiles: the first loads of the next piece are on their
    // way before this one is done with.  next(piece) gives the following one; done(piece, whether there is
    // another) hands over; put_by() holds the sums.
    template <class Keep, class Hold, class Next, class Done>
    __device__ __forceinline__ void stream(const PagedAttnParams& p, Piece cur, float*, Keep z, Hold put_by, Next next,
                                           Done done) {
        const int lane = threadIdx.x & 31;
        Piece then;
        bool more = next(then);
        PageIds ids = cur.ids, later = ids;
        if (cur.row + 32 * kPaTile < cur.end) later = page_ids(p.c, cur.b, cur.row + (32 + lane) * kPaTile, cur.end);
        int t = 0;
        Keys k;
        Values v;
        int ida = __shfl_sync(0xffffffffu, ids.a, 0), idb = __shfl_sync(0xffffffffu, ids.b, 0);
        load_q(p, cur.b, cur.h);
        load_k(p, cur.h, cur.row, cur.end, ida, idb, k);
        load_v(p, cur.h, cur.row, cur.end, ida, idb, v);
        reset();
        for (;;) {
            float s[4];
            scores(k, s);
            const int was_a = ida, was_b = idb, row = cur.row;
            const bool last = row + kPaTile >= cur.end;
            if (!last) {
                if (++t == 32) {
                    t = 0;
                    ids = later;
                    if (row + 33 * kPaTile < cur.end) later = page_ids(p.c, cur.b, row + (33 + lane) * kPaTile, cur.end);
                }
                ida = __shfl_sync(0xffffffffu, ids.a, t);
                idb = __shfl_sync(0xffffffffu, ids.b, t);
                load_k(p, cur.h, row + kPaTile, cur.end, ida, idb, k);
            } else if (more) {
                ida = __shfl_sync(0xffffffffu, then.ids.a, 0);
                idb = __shfl_sync(0xffffffffu, then.ids.b, 0);
                load_q(p, then.b, then.h);
                load_k(p, then.h, 0, then.end, ida, idb, k);
            }
            if (Keep::on) keep(p, z(cur.b, cur.h, row), row, cur.end, was_a, was_b, s);
            uint32_t b0, b1, r0 = 0, r1 = 0;
            softmax(p.scale_log2, row, cur.end, was_a, was_b, s, p.down, b0, b1, r0, r1);
            values(v, b0, b1, r0, r1);
            if (!last) {
                if (t == 0) put_by();
                load_v(p, cur.h, row + kPaTile, cur.end, ida, idb, v);
                cur.row = row + kPaTile;
                continue;
            }
            if (more) load_v(p, then.h, 0, then.end, ida, idb, v);
            done(cur, more);
            if (!more) break;
            reset();
            cur = then;
            ids = cur.ids;
            t = 0;
            if (cur.row + 32 * kPaTile < cur.end) later = page_ids(p.c, cur.b, cur.row + (32 + lane) * kPaTile, cur.end);
            more = next(then);
        }
    }
};

// fp32: a half-warp per eight rows, lane hl holding the dimensions 4 hl + 64 j
template <int D, int G>
struct TileF32 {
    static constexpr int kV = D / 64;      // float4 of a row per lane
    static constexpr bool kLow = true;     // whether p.down is in the sums of values
    float o[G][4 * kV];
    float m[G], l[G];
    bool held;                             // whether the unit has held sums
    const float* sq;                       // [G][D + 4] the warp's queries in shared memory

    __device__ __forceinline__ void load_q(const PagedAttnParams& p, int b, int h, float* s_q) {
        __syncwarp();
        for (int i = threadIdx.x & 31; i < G * D; i += 32) {
            const int g = i / D;
            s_q[g * (D + 4) + i % D] = g < p.G ? static_cast<const float*>(p.q)[b * p.q_seq + (h * p.G + g) * p.q_head + i % D] : 0.f;
        }
        __syncwarp();
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
        held = false;
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
    template <class Keep, class Hold>
    __device__ __forceinline__ void share(const PagedAttnParams& p, const Piece& piece, const Keep& z, Hold put_by) {
        const int b = piece.b, h = piece.h, row0 = piece.row, end = piece.end;
        const int lane = threadIdx.x & 31, hl = lane & 15, half = lane >> 4, mask = (1 << p.c.lg) - 1;
        const float* kb = static_cast<const float*>(p.c.k) + h * p.c.k_head;
        const float* vb = static_cast<const float*>(p.c.v) + h * p.c.v_head;
        // the keys of the next tile and the values of this one are on their way during the scores, where
        // registers allow it (all but eight heads of 128 dimensions)
        constexpr bool kAhead = G * kV < 16;
        PageIds now = piece.ids;
        int t = 0;
        auto id_of = [&](int at) {
            const int ida = __shfl_sync(0xffffffffu, now.a, at), idb = __shfl_sync(0xffffffffu, now.b, at);
            return half ? idb : ida;
        };
        int id = id_of(0);
        float x[8][4 * kV], v[8][4 * kV];
        if (kAhead) load(kb, p.c.k_page, p.c.k_row, mask, row0 + 8 * half, end, id, x);
        for (int row = row0; row < end; row += kPaTile) {
            const int mine = row + 8 * half;      // this half-warp's eight rows
            if (kAhead) load(vb, p.c.v_page, p.c.v_row, mask, mine, end, id, v);
            else load(kb, p.c.k_page, p.c.k_row, mask, mine, end, id, x);
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
                    const float4 qv = *reinterpret_cast<const float4*>(sq + g * (D + 4) + 64 * j + 4 * hl);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] = fmaf(x[i][4 * j], qv.x, a[i]);
                        a[i] = fmaf(x[i][4 * j + 1], qv.y, a[i]);
                        a[i] = fmaf(x[i][4 * j + 2], qv.z, a[i]);
                        a[i] = fmaf(x[i][4 * j + 3], qv.w, a[i]);
                    }
                }
                s[g] = transpose_reduce8(a, hl);
                if (Keep::on && (hl & 1) == 0 && mine + (hl >> 1) < end && g < p.G)
                    z(b, h, mine + (hl >> 1))[g] = in ? s[g] : no_product(p);
                up = up || (in && s[g] * p.scale_log2 > m[g] + kPaSlack);
            }
            if (!kAhead) load(vb, p.c.v_page, p.c.v_row, mask, mine, end, id, v);
            if (row + kPaTile < end) {
                if (++t == 32) {
                    t = 0;
                    now = page_ids(p.c, b, row + (1 + lane) * kPaTile, end);
                }
                id = id_of(t);
                if (kAhead) load(kb, p.c.k_page, p.c.k_row, mask, mine + kPaTile, end, id, x);
            }
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
                const float down = pr * p.down;
                l[g] += pr;                     // every row is held by two lanes: halved at the end
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w = __shfl_sync(0xffffffffu, down, 16 * half + 2 * i);
#pragma unroll
                    for (int j = 0; j < 4 * kV; ++j) o[g][j] = fmaf(w, v[i][j], o[g][j]);
                }
            }
            if (t == 0 && row + kPaTile < end) put_by();
        }
    }
    template <class Keep, class Hold, class Next, class Done>
    __device__ __forceinline__ void stream(const PagedAttnParams& p, Piece cur, float* s_q, Keep z, Hold put_by, Next next,
                                           Done done) {
        for (bool more = true; more;) {
            load_q(p, cur.b, cur.h, s_q);
            reset();
            share(p, cur, z, put_by);
            Piece then = cur;
            more = next(then);
            done(cur, more);
            cur = then;
        }
    }
    // adds what is held in a slot to the sums: the first half-warp's, and every lane's half of the rows' sum
    __device__ __forceinline__ void take(const JoinSmem<D, G>& js, int slot) {
        const int lane = threadIdx.x & 31, hl = lane & 15;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float w = share_weight(js.m[slot][g], js.l[slot][g], m[g]);
            if (lane == 0) l[g] = fmaf(2.f * js.l[slot][g], w, l[g]);
            if (lane >= 16) continue;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(&js.o[slot][g][64 * i + 4 * hl]);
                o[g][4 * i] = fmaf(x.x, w, o[g][4 * i]);
                o[g][4 * i + 1] = fmaf(x.y, w, o[g][4 * i + 1]);
                o[g][4 * i + 2] = fmaf(x.z, w, o[g][4 * i + 2]);
                o[g][4 * i + 3] = fmaf(x.w, w, o[g][4 * i + 3]);
            }
        }
        __syncwarp();      // the slot may be written again
    }
    // the sums of both half-warps, of head g into a slot
    __device__ __forceinline__ void put(JoinSmem<D, G>& js, int slot, int g, float sum, const float (&x)[4 * kV]) const {
        const int lane = threadIdx.x & 31, hl = lane & 15;
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                *reinterpret_cast<float4*>(&js.o[slot][g][64 * i + 4 * hl]) =
                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        }
        if (lane == 0) {
            js.m[slot][g] = m[g];
            js.l[slot][g] = sum;
        }
    }
    // holds the sums so far and begins again at zero
    __device__ __forceinline__ void hold(JoinSmem<D, G>& js, int slot) {
        if (held) take(js, slot);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float x[4 * kV];
            const float sum = 0.5f * warp_sum(l[g]);
#pragma unroll
            for (int i = 0; i < 4 * kV; ++i) {
                x[i] = o[g][i] + __shfl_xor_sync(0xffffffffu, o[g][i], 16);
                o[g][i] = 0.f;
            }
            put(js, slot, g, sum, x);
            l[g] = 0.f;
        }
        held = true;
        __syncwarp();
    }
    __device__ __forceinline__ void finish(const PagedAttnParams& p, int b, int h, bool alone, JoinSmem<D, G>& js, int slot,
                                           int from) {
        const int lane = threadIdx.x & 31, hl = lane & 15;
        __syncwarp();      // no lane reads the queries any more
        if (held) take(js, from);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float sum = 0.5f * warp_sum(l[g]);
            float x[4 * kV];
#pragma unroll
            for (int i = 0; i < 4 * kV; ++i) x[i] = o[g][i] + __shfl_xor_sync(0xffffffffu, o[g][i], 16);
            if (g >= p.G) continue;
            if (!alone) {
                put(js, slot, g, sum, x);
                continue;
            }
            const float inv = sum == 0.f ? 0.f : 1.f / (sum * p.down);
            float* dst = static_cast<float*>(p.out) + b * p.o_seq + (h * p.G + g) * p.o_head;
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < kV; ++i)
                    *reinterpret_cast<float4*>(dst + 64 * i + 4 * hl) =
                        make_float4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
            }
            if (lane == 0) note(p, b, h, g, m[g], sum);
        }
    }
};

// ------------------------------------------------------------------ the kernels

// Joins the shares of a CTA's warps: each run of shares of one unit, in order, becomes the unit's
// result or one of the CTA's records.
template <int D, bool kF32, int G>
__device__ __forceinline__ void join_shares(const PagedAttnParams& p, JoinSmem<D, G>& js) {
    constexpr int kShares = 2 * kPaWarps;
    const int tid = threadIdx.x;
    if (tid < 32) {            // lane e looks at share e: which run it belongs to, where that ends
        const ShareOf f = tid < kShares ? js.of[tid] : ShareOf{-1, 0, false, false, false};
        const uint32_t some = __ballot_sync(0xffffffffu, f.b >= 0);
        const uint32_t before = some & ((1u << tid) - 1);
        const int prev = before ? 31 - __clz(before) : 0;
        const int pb = __shfl_sync(0xffffffffu, f.b, prev), ph = __shfl_sync(0xffffffffu, f.h, prev);
        const bool starts = f.b >= 0 && !(before && pb == f.b && ph == f.h);
        const uint32_t heads = __ballot_sync(0xffffffffu, starts);
        const uint32_t later = heads & ~((2u << tid) - 1);
        const uint32_t mine = some & ~((1u << tid) - 1) & (later ? (later & -later) - 1 : ~0u);
        const int last = mine ? 31 - __clz(mine) : 0;
        const bool ends = __shfl_sync(0xffffffffu, static_cast<int>(f.ends), last);
        if (starts) js.run[__popc(heads & ((1u << tid) - 1))] = Run{f.b, f.h, tid, last, f.begins && ends, f.first};
        if (tid == 0) js.runs = __popc(heads);
    }
    __syncthreads();
    const int runs = js.runs;
    // a share's weight against its run, and the run's base and sum (thread = run, head)
    if (tid < runs * G && tid % G < p.G) {
        const Run r = js.run[tid / G];
        const int g = tid % G;
        float m = -CUDART_INF_F, l = 0.f;
        for (int e = r.from; e <= r.last; ++e)
            if (js.of[e].b >= 0) m = fmaxf(m, js.m[e][g]);
        for (int e = r.from; e <= r.last; ++e)
            if (js.of[e].b >= 0) l = fmaf(js.l[e][g], share_weight(js.m[e][g], js.l[e][g], m), l);
        const float scale = !r.whole ? 1.f : l == 0.f ? 0.f : 1.f / (l * p.down);
        for (int e = r.from; e <= r.last; ++e)
            js.w[e][g] = js.of[e].b >= 0 ? share_weight(js.m[e][g], js.l[e][g], m) * scale : -1.f;
        if (r.whole) note(p, r.b, r.h, g, m, l);
        else p.rec_stat[(static_cast<int64_t>(blockIdx.x) * 2 + (r.first ? 0 : 1)) * p.G + g] = make_float2(m, l);
    }
    __syncthreads();
    for (int i = 0; i < runs; ++i) {
        const Run r = js.run[i];
        float* rec = p.rec + (static_cast<int64_t>(blockIdx.x) * 2 + (r.first ? 0 : 1)) * p.G * D;
        for (int k = tid; k < p.G * (D / 4); k += kPaThreads) {
            const int g = k / (D / 4), dim = 4 * (k % (D / 4));
            float x[4] = {0.f, 0.f, 0.f, 0.f};
            for (int e = r.from; e <= r.last; ++e) {
                const float w = js.w[e][g];
                if (w < 0.f) continue;         // no share
                const float4 v = *reinterpret_cast<const float4*>(&js.o[e][g][dim]);
                x[0] = fmaf(v.x, w, x[0]);
                x[1] = fmaf(v.y, w, x[1]);
                x[2] = fmaf(v.z, w, x[2]);
                x[3] = fmaf(v.w, w, x[3]);
            }
            if (!r.whole) {
                *reinterpret_cast<float4*>(rec + g * D + dim) = make_float4(x[0], x[1], x[2], x[3]);
            } else {
                store4<kF32>(p, r.b, r.h, g, dim, x);
            }
        }
    }
}

template <class Tile, int D, bool kF32, int G, int kOcc, bool kKeep>
__global__ void __launch_bounds__(kPaThreads, kOcc) k_paged_attn(const __grid_constant__ PagedAttnParams p) {
    extern __shared__ __align__(16) float s_q[];       // fp32: [warps][G][D + 4] their queries
    __shared__ PlanSmem<kPaWarps> s_plan;
    __shared__ __align__(16) JoinSmem<D, G> js;
    begin_call();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, me = blockIdx.x;
    const Plan<kPaWarps> pl = make_plan<kPaWarps, kPaTile, kF32 ? 1 : kPaLeast>(p.c, me, gridDim.x, s_plan);
    const int64_t w0 = pl.part(warp), w1 = pl.part(warp + 1);
    if (lane == 0) js.of[2 * warp].b = js.of[2 * warp + 1].b = -1;
    __syncwarp();
    if (w0 < w1 && s_plan.rows[warp] > 0) {
        Pieces pieces;
        const Piece head = pieces.first(p.c, s_plan.b[warp], s_plan.rows[warp], s_plan.at[warp], w0, w1 - w0);
        Tile tile;
        bool first = true;
        auto put_by = [&] { tile.hold(js, 2 * warp + 1); };
        auto next = [&](Piece& q) { return pieces.next(p.c, q); };
        auto done = [&](const Piece& q, bool more) {
            const int slot = 2 * warp + (first ? 0 : 1);
            const bool begins = !first || pieces.begins, ends = more || pieces.ends;
            tile.finish(p, q.b, q.h, begins && ends, js, slot, 2 * warp + 1);
            if (!(begins && ends) && lane == 0) js.of[slot] = ShareOf{q.b, q.h, begins, ends, first && w0 == pl.lo};
            first = false;
        };
        float* queries = s_q + warp * G * (D + 4);
        if constexpr (kKeep) tile.stream(p, head, queries, KeepGlobal{p}, put_by, next, done);
        else tile.stream(p, head, queries, KeepNone{}, put_by, next, done);
    }
    // a unit that ends in this CTA and began before it
    if (tid == 0) {
        Joint joint{-1, 0, 0, 0};
        if (pl.lo < pl.hi && s_plan.rows[0] > 0) {
            Walk<kPaTile> at;
            at.enter(s_plan.b[0], s_plan.rows[0], s_plan.at[0], pl.lo);
            if (at.unit0 < pl.lo && at.unit0 + at.nt <= pl.hi) {
                const int64_t from = pl.holder(at.unit0);
                joint = Joint{static_cast<int>(from), at.b, at.h, pl.start(from) == at.unit0 ? 0 : 1};
            }
        }
        p.joint[me] = joint;
    }
    __syncthreads();
    join_shares<D, kF32, G>(p, js);
    // sequences of no rows
    for (int e = blockIdx.x; e < p.c.batch; e += gridDim.x)
        if (rows_of(p.c, e, g_err, 711) == 0) {
            for (int i = tid; i < p.n_q * D; i += kPaThreads) store_out(p, kF32, e, 0, i / D, i % D, 0.f);
            if (p.lse)
                for (int i = tid; i < p.n_q; i += kPaThreads) p.lse[static_cast<int64_t>(e) * p.n_q + i] = -CUDART_INF_F;
        }
}

// Short sequences, where the latency of a step counts (one sequence of 1013 rows: 6.4 us against 9.6 in the
// general form, four of 4096 rows 16.5 against 20.4): a cluster of CTAs per unit, or one CTA where units are
// many, whose warps share its rows evenly.  No search for the place, no records and no second kernel:
// each CTA joins its warps' shares, and the cluster joins the CTAs' through distributed shared memory.  The
// products for the weights stay in shared memory until the sums are known.
// Tiles of a warp of a unit's longest possible sequence:
__host__ __device__ __forceinline__ int cluster_tiles(int cap, int ranks) {
    const int parts = ranks * kPaWarps;
    return ((cap + kPaTile - 1) / kPaTile + parts - 1) / parts;
}
template <class Tile, int D, bool kF32, int G, int kOcc, bool kKeep>
__global__ void __launch_bounds__(kPaThreads, kOcc) k_paged_cluster(const __grid_constant__ PagedAttnParams p, int ranks) {
    extern __shared__ __align__(16) float s_z[];        // [warps][rows of a warp at most][Gp]
    __shared__ __align__(16) JoinSmem<D, G> js;
    begin_call();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u = blockIdx.x / ranks, rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int b = u / p.c.H, h = u % p.c.H;
    const int rows = rows_of(p.c, b, g_err, 711);
    const int nt = tiles_of(rows), parts = ranks * kPaWarps, part = rank * kPaWarps + warp;
    const int t0 = static_cast<int>(static_cast<int64_t>(nt) * part / parts);
    const int t1 = static_cast<int>(static_cast<int64_t>(nt) * (part + 1) / parts);
    float* my_z = s_z + warp * cluster_tiles(p.c.cap, ranks) * kPaTile * (kKeep ? p.Gp : 0);
    Tile tile;
    auto hand_over = [&](const Piece&, bool) { tile.finish(p, b, h, false, js, 2 * warp, 0); };
    const int piece_row = t0 * kPaTile, piece_end = t0 < t1 ? min(rows, t1 * kPaTile) : piece_row;
    Piece piece{b, h, piece_row, piece_end, {-1, -1}};
    if (t0 < t1) {
        piece.ask(p.c);
        float* queries = js.o[2 * warp + 1][0];
        auto none = [](Piece&) { return false; };
        // (at most kOneWaveTiles tiles: none of them fills a row of page ids)
        if constexpr (kKeep) tile.stream(p, piece, queries, KeepShared{my_z, piece.row, p.Gp}, HoldNone{}, none, hand_over);
        else tile.stream(p, piece, queries, KeepNone{}, HoldNone{}, none, hand_over);
    } else {
        tile.reset();
        hand_over(piece, false);
    }
    __syncthreads();
    // the CTA's share, in slot 1: of the four warps' in order
    if (tid < G && tid < p.G) {
        float m = -CUDART_INF_F, l = 0.f;
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w) m = fmaxf(m, js.m[2 * w][tid]);
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w) {
            const float f = share_weight(js.m[2 * w][tid], js.l[2 * w][tid], m);
            js.w[w][tid] = f;
            l = fmaf(js.l[2 * w][tid], f, l);
        }
        js.m[1][tid] = m;
        js.l[1][tid] = l;
    }
    __syncthreads();
    for (int k = tid; k < p.G * (D / 4); k += kPaThreads) {
        const int g = k / (D / 4), dim = 4 * (k % (D / 4));
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kPaWarps; ++w) {
            const float f = js.w[w][g];
            const float4 v = *reinterpret_cast<const float4*>(&js.o[2 * w][g][dim]);
            x[0] = fmaf(v.x, f, x[0]);
            x[1] = fmaf(v.y, f, x[1]);
            x[2] = fmaf(v.z, f, x[2]);
            x[3] = fmaf(v.w, f, x[3]);
        }
        *reinterpret_cast<float4*>(&js.o[1][g][dim]) = make_float4(x[0], x[1], x[2], x[3]);
    }
    if (ranks > 1) cluster_sync_all();
    else __syncthreads();
    // every CTA of the cluster writes a part of the result
    for (int k = tid * ranks + rank; k < p.G * (D / 4); k += kPaThreads * ranks) {
        const int g = k / (D / 4), dim = 4 * (k % (D / 4));
        float m = -CUDART_INF_F, l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < ranks; ++r) m = fmaxf(m, ranks > 1 ? ld_cluster_f32(cluster_addr(&js.m[1][g], r)) : js.m[1][g]);
        for (int r = 0; r < ranks; ++r) {
            float rm, rl;
            float4 v;
            if (ranks > 1) {
                rm = ld_cluster_f32(cluster_addr(&js.m[1][g], r));
                rl = ld_cluster_f32(cluster_addr(&js.l[1][g], r));
                v = ld_cluster_v4f(cluster_addr(&js.o[1][g][dim], r));
            } else {
                rm = js.m[1][g];
                rl = js.l[1][g];
                v = *reinterpret_cast<const float4*>(&js.o[1][g][dim]);
            }
            const float f = share_weight(rm, rl, m);
            l = fmaf(rl, f, l);
            x[0] = fmaf(v.x, f, x[0]);
            x[1] = fmaf(v.y, f, x[1]);
            x[2] = fmaf(v.z, f, x[2]);
            x[3] = fmaf(v.w, f, x[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = l == 0.f ? 0.f : x[e] / (l * p.down);
        store4<kF32>(p, b, h, g, dim, x);
        if (dim == 0) note(p, b, h, g, m, l);
    }
    if (kKeep) {
        // the unit's base and 1 / sum per head, then the weights of the warp's own rows
        __shared__ float2 s_stat[G];
        if (tid < G && tid < p.G) {
            float m = -CUDART_INF_F, l = 0.f;
            for (int r = 0; r < ranks; ++r) m = fmaxf(m, ranks > 1 ? ld_cluster_f32(cluster_addr(&js.m[1][tid], r)) : js.m[1][tid]);
            for (int r = 0; r < ranks; ++r) {
                const float rm = ranks > 1 ? ld_cluster_f32(cluster_addr(&js.m[1][tid], r)) : js.m[1][tid];
                const float rl = ranks > 1 ? ld_cluster_f32(cluster_addr(&js.l[1][tid], r)) : js.l[1][tid];
                l = fmaf(rl, share_weight(rm, rl, m), l);
            }
            s_stat[tid] = make_float2(m, l == 0.f ? 0.f : 1.f / l);
        }
        __syncthreads();
        const float* in = p.weight + u * p.row_pitch;
        float* out = p.weight_out + u * p.row_pitch;
        const float none = no_product(p);
        for (int i = piece_row + lane; i < piece_end; i += 32) {
            float sum = 0.f;
            for (int g = 0; g < p.G; ++g) {
                const float x = my_z[(i - piece_row) * p.Gp + g];
                if (x != none) sum += exp2_fast(fmaf(x, p.scale_log2, -s_stat[g].x)) * s_stat[g].y;
            }
            out[i] = in[i] + sum;
        }
    }
    if (ranks > 1) cluster_sync_all();       // no CTA leaves while another reads its share
}

// Joins the records of the units that lie in more than one CTA's range: row i of the grid those of
// the unit that ends in CTA i's range and began before it (p.joint says which, if any).  The grid's
// y dimension deals the heads out.
constexpr int kPaMost = 640;      // shares of a unit at most (CTAs of the attention)
constexpr int kPaFew = 8;         // shares that a thread joins by itself

// Few shares: a thread holds four dimensions of one head, and forms the weights for itself.
template <int D, bool kF32>
__device__ __forceinline__ void merge_few(const PagedAttnParams& p, const Joint& j, int n) {
    for (int k = threadIdx.x + blockIdx.y * kPaThreads; k < p.G * (D / 4); k += gridDim.y * kPaThreads) {
        const int g = k / (D / 4), dim = 4 * (k % (D / 4));
        float2 ml[kPaFew];
        float4 v[kPaFew];
#pragma unroll
        for (int i = 0; i < kPaFew; ++i) {
            ml[i] = make_float2(-CUDART_INF_F, 0.f);
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) {
                const int64_t rec = (static_cast<int64_t>(j.from + i) * 2 + (i == 0 ? j.slot : 0)) * p.G + g;
                ml[i] = __ldcg(p.rec_stat + rec);
                v[i] = __ldcg(reinterpret_cast<const float4*>(p.rec + rec * D + dim));
            }
        }
        float m = -CUDART_INF_F, l = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kPaFew; ++i) m = fmaxf(m, ml[i].x);
#pragma unroll
        for (int i = 0; i < kPaFew; ++i) {
            if (i >= n) break;
            const float f = share_weight(ml[i].x, ml[i].y, m);
            l = fmaf(ml[i].y, f, l);
            x[0] = fmaf(v[i].x, f, x[0]);
            x[1] = fmaf(v[i].y, f, x[1]);
            x[2] = fmaf(v[i].z, f, x[2]);
            x[3] = fmaf(v[i].w, f, x[3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = l == 0.f ? 0.f : x[e] / (l * p.down);
        store4<kF32>(p, j.b, j.h, g, dim, x);
        if (dim == 0) note(p, j.b, j.h, g, m, l);
    }
}

// More: the CTA forms the weights of one head, lanes hold four dimensions, and warps (half-warps
// where d is 64) take the shares in turn.
template <int D>
struct MergeSmem {
    float f[kPaMost], red[kPaWarps], sum[kPaWarps];
    __align__(16) float x[kPaThreads / (D / 4)][D];
};
template <int D, bool kF32>
__device__ __forceinline__ void merge_many(const PagedAttnParams& p, const Joint& j, int n, int g, MergeSmem<D>& sm) {
    constexpr int kLanes = D / 4, kWays = kPaThreads / kLanes, kEach = kPaMost / kPaThreads;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // share i: slot 0, but the unit began inside the first CTA's range
    auto rec_of = [&](int i) -> int64_t {
        return (static_cast<int64_t>(j.from + i) * 2 + (i == 0 ? j.slot : 0)) * p.G + g;
    };
    float2 ml[kEach];
    float m = -CUDART_INF_F;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = tid + e * kPaThreads;
        ml[e] = i < n ? __ldcg(p.rec_stat + rec_of(i)) : make_float2(-CUDART_INF_F, 0.f);
        m = fmaxf(m, ml[e].x);
    }
    // the first shares are on their way while the weights form
    constexpr int kAhead = 8;
    const int dim = 4 * (tid % kLanes), way = tid / kLanes;
    auto fetch = [&](int i) {
        return i < n ? __ldcg(reinterpret_cast<const float4*>(p.rec + rec_of(i) * D + dim)) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 a[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) a[e] = fetch(way + e * kWays);
    m = warp_max(m);
    if (lane == 0) sm.red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPaWarps; ++w) m = fmaxf(m, sm.red[w]);
    float l = 0.f;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int i = tid + e * kPaThreads;
        const float f = share_weight(ml[e].x, ml[e].y, m);
        if (i < n) sm.f[i] = f;
        l = fmaf(ml[e].y, f, l);
    }
    l = warp_sum(l);
    if (lane == 0) sm.sum[warp] = l;
    __syncthreads();
    l = sm.sum[0] + sm.sum[1] + sm.sum[2] + sm.sum[3];
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = way; i < n; i += kAhead * kWays) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            if (i + e * kWays >= n) break;
            const float f = sm.f[i + e * kWays];
            x[0] = fmaf(a[e].x, f, x[0]);
            x[1] = fmaf(a[e].y, f, x[1]);
            x[2] = fmaf(a[e].z, f, x[2]);
            x[3] = fmaf(a[e].w, f, x[3]);
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) a[e] = fetch(i + (kAhead + e) * kWays);
    }
    *reinterpret_cast<float4*>(&sm.x[way][dim]) = make_float4(x[0], x[1], x[2], x[3]);
    __syncthreads();
    if (tid < D) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWays; ++w) sum += sm.x[w][tid];
        store_out(p, kF32, j.b, j.h, g, tid, l == 0.f ? 0.f : sum / (l * p.down));
    }
    if (tid == 0) note(p, j.b, j.h, g, m, l);
    __syncthreads();
}

template <int D, bool kF32>
__global__ void __launch_bounds__(kPaThreads) k_paged_merge(const __grid_constant__ PagedAttnParams p) {
    __shared__ MergeSmem<D> sm;
    // every CTA waits for the grid before, so that this grid's end stands for both; what comes after is
    // let in then (let in before, the next call's CTAs held the registers that this grid's wanted: 47 us
    // against 34 for 192 short sequences)
    pdl_wait();
    pdl_trigger();
    const int me = blockIdx.x;
    const int4 raw = __ldcg(reinterpret_cast<const int4*>(p.joint) + me);
    const Joint j{raw.x, raw.y, raw.z, raw.w};
    if (j.from < 0) return;
    const int n = me - j.from + 1;
    if (n <= kPaFew) {
        merge_few<D, kF32>(p, j, n);
        return;
    }
    for (int g = blockIdx.y; g < p.G; g += gridDim.y) merge_many<D, kF32>(p, j, n, g, sm);
}

// Rows per thread and turn, whose products are loaded before any of them is used: four, or two of
// more than four heads.
constexpr int kWeighRows = 1024;      // rows of a CTA's step: eight per thread

template <int Gp>
__device__ __forceinline__ void weigh_rows(const PagedAttnParams& p, int64_t u, int first, int end) {
    const float* z = p.z + u * p.c.cap * Gp;
    const float* in = p.weight + u * p.row_pitch;
    float* out = p.weight_out + u * p.row_pitch;
    const float none = no_product(p);
    float base[Gp], inv[Gp];
#pragma unroll
    for (int g = 0; g < Gp; ++g) {
        const float2 st = g < p.G ? __ldcg(p.stat + u * p.G + g) : make_float2(0.f, 0.f);
        base[g] = st.x;
        inv[g] = st.y;
    }
    constexpr int kTurn = Gp <= 4 ? 4 : 2;
    for (int i0 = first + threadIdx.x; i0 < end; i0 += kTurn * kPaThreads) {
        float2 x[kTurn][Gp / 2];
        float w[kTurn];
#pragma unroll
        for (int r = 0; r < kTurn; ++r) {
            const int i = i0 + r * kPaThreads;
            if (i >= end) continue;
            w[r] = in[i];
#pragma unroll
            for (int g = 0; g < Gp / 2; ++g) x[r][g] = __ldcg(reinterpret_cast<const float2*>(z + static_cast<int64_t>(i) * Gp) + g);
        }
#pragma unroll
        for (int r = 0; r < kTurn; ++r) {
            const int i = i0 + r * kPaThreads;
            if (i >= end) continue;
            float sum = 0.f;
#pragma unroll
            for (int g = 0; g < Gp; ++g) {
                const float v = g & 1 ? x[r][g / 2].y : x[r][g / 2].x;
                if (g < p.G && v != none) sum += exp2_fast(fmaf(v, p.scale_log2, -base[g])) * inv[g];
            }
            out[i] = w[r] + sum;
        }
    }
}
// weight_out = weight + sum over the heads of exp2(z scale - base) / sum, in steps of kWeighRows rows.
// Memory bounds it: 4 bytes in and out and the products per row; 1.4M rows of four heads in 10 us.
constexpr int kWeighOcc = 8;          // CTAs per SM
template <int Gp>
__global__ void __launch_bounds__(kPaThreads, kWeighOcc) k_paged_weigh(const __grid_constant__ PagedAttnParams p) {
    __shared__ PlanSmem<1> s_plan;
    // the lengths were there before the call began; the rest comes from the grids before
    const Plan<1> pl = make_plan<1, kWeighRows, 1>(p.c, blockIdx.x, gridDim.x, s_plan);
    pdl_wait();
    if (pl.lo == pl.hi || s_plan.rows[0] == 0) return;
    int64_t cur = pl.lo;
    Walk<kWeighRows> at;
    at.enter(s_plan.b[0], s_plan.rows[0], s_plan.at[0], cur);
    while (cur < pl.hi) {
        const int first = static_cast<int>(cur - at.unit0) * kWeighRows;
        weigh_rows<Gp>(p, static_cast<int64_t>(at.b) * p.c.H + at.h, first, min(at.rows, first + kWeighRows));
        if (++cur == at.unit0 + at.nt && cur < pl.hi && !at.next(p.c)) break;
    }
}

// ------------------------------------------------------------------ launches

// CTAs per SM, by the registers that 128 and 64 dimensions need.  (64 dimensions: 64 ragged units of up to
// 64K rows with e5m2 values 78 us with four, 89 with three; 32 of 16K rows in bf16 31.7 and 32.7; fp32, 32
// of 16K rows of four heads 51 with three, 57 with two, of eight 72 and 80; 128 dimensions and four heads
// 105 and 87.)  Short sequences in fp32 take two all the same (three of 4099 rows of 2 x 8 heads, 64
// dimensions, 14.6 us against 15.7).
constexpr int occ_of(bool f32, int d) { return (f32 ? 2 : 3) + (d == 64 ? 1 : 0); }

int paged_attn_ctas(int dtype, int d, int nsm) { return nsm * occ_of(dtype == SKV_F32, d); }

// Clusters of `ranks` CTAs that the device holds at once, asked for once per kernel: those of four and
// more do not fill every GPC (of 152 SMs with three CTAs each 110 of four, 51 of eight, 21 of 16).
constexpr int kClusterTiles = 8, kUnitTiles = 12, kOneWaveTiles = 16;
// shared memory of a cluster form's kernel: all of a kind are allowed the most, whatever one takes (calls of
// several host threads would set each other's limit)
constexpr int z_bytes(int tiles, int Gp) { return kPaWarps * tiles * kPaTile * Gp * 4; }
template <class Kernel>
static bool allow(Kernel kernel, int ranks, int smem) {
    return (ranks <= 8 || cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) &&
           (!smem || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, z_bytes(kOneWaveTiles, 8)) == cudaSuccess);
}
// shared memory of an SM that holds kOcc CTAs of a cluster form's kernel, and the split to ask for
template <int D, int G, int kOcc>
constexpr int shared_bytes(int smem) { return kOcc * (static_cast<int>(sizeof(JoinSmem<D, G>) + G * sizeof(float2)) + 1024 + smem); }
constexpr int carve_of(int bytes) {
    const int percent = (bytes * 100 + kSmShared - 1) / kSmShared;
    return percent < kCarve ? kCarve : percent > 100 ? 100 : percent;
}
template <class Tile, int D, bool kF32, int G, int kOcc, bool kKeep>
static int clusters_held(int ranks) {
    static std::atomic<int> known[17];
    int n = known[ranks].load(std::memory_order_relaxed) - 1;
    if (n >= 0) return n;
    auto kernel = k_paged_cluster<Tile, D, kF32, G, kOcc, kKeep>;
    const int smem = kKeep ? z_bytes(kClusterTiles, 8) : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks);
    cfg.blockDim = dim3(kPaThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    attr[1].val.sharedMemCarveout = carve_of(shared_bytes<D, G, kOcc>(smem));
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (!allow(kernel, ranks, smem) || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    known[ranks].store(n + 1, std::memory_order_relaxed);
    return n;
}

// CTAs of a unit's cluster, or 0: the general form.  The cluster form serves a step whose units leave
// SMs idle, whose clusters all run at once and whose longest possible sequence takes a warp no more than
// kClusterTiles tiles (with twice as many, 8 units of 16K rows took 25.0 us against the general form's
// 21.0, 64 ragged ones of 4000 rows 25.0 against 21.1; with two clusters left over, 112 of 2000 rows took
// 32.3 against 26.9, ragged 18.0 against 20.5, where 108 take 21.2 against 26.5), and one whose units,
// a CTA each, are up to three times as many as the CTAs that the device holds (fp32: twice), with at most
// kUnitTiles tiles for a warp, or kOneWaveTiles where they fill the device once.  (Ragged bf16 units of up
// to 250 rows: 460 of them 9.6 us against 18.0, 1368 23.6 against 25.6, 2000 32.1 against 31.6.  Of up to
// 611 rows: 300 16.8 against 18.5, 768 28.6 against 29.6; of 1000 300 24.7 against 22.6, 452 27.1 against
// 28.2, and 37.7 against 44.7 of 1000 each.  Units of one length lose where a few are left over: 460 of 750
// rows 41.6 against 36.5, 912 57.4 against 59.8.  fp32, 600 ragged ones of 250 rows 27.0 against 33.5; 912
// of exactly 250 54.4 against 44.7.)
// The products that are kept for the weights take shared memory, and with it an SM's L1 through which the
// loads go: a unit has a CTA only where that leaves kLeastL1 of it.  (452 units with eight heads of 128
// dimensions, weighed, in CTAs against the general form: of 600 rows, 181 KB an SM, 29.4 us against 43.3; of
// 1000, 206 KB, 57.4 against 60.9, but 440 ragged ones 47.3 against 38.9.)
constexpr int kLeastL1 = 32 << 10;
template <class Tile, int D, bool kF32, int G, int kOcc, bool kKeep>
static int cluster_ranks(const PagedAttnParams& p, int ncta) {
    const int64_t U = static_cast<int64_t>(p.c.batch) * p.c.H, tiles = (p.c.cap + kPaTile - 1) / kPaTile;
    int ranks = 1;
    while (ranks < 16 && tiles > ranks * kPaWarps && 2 * U * ranks <= ncta &&
           U <= clusters_held<Tile, D, kF32, G, kOcc, kKeep>(2 * ranks))
        ranks *= 2;
    if (ranks == 1) {
        const int tiles_most = U <= ncta && 4 * U >= 3 * static_cast<int64_t>(ncta) ? kOneWaveTiles : kUnitTiles;
        const int mine = cluster_tiles(p.c.cap, 1);
        if (U > (kF32 ? 2 : 3) * static_cast<int64_t>(ncta) || mine > tiles_most) return 0;
        return !kKeep || shared_bytes<D, G, kOcc>(z_bytes(mine, p.Gp)) <= kSmShared - kLeastL1 ? 1 : 0;
    }
    return cluster_tiles(p.c.cap, ranks) <= kClusterTiles ? ranks : 0;
}

template <class Tile, int D, bool kF32, int G, int kOcc, bool kKeep>
static int launch_cluster(const PagedAttnParams& p, int ranks, cudaStream_t s) {
    auto kernel = k_paged_cluster<Tile, D, kF32, G, kOcc, kKeep>;
    const int smem = kKeep ? z_bytes(cluster_tiles(p.c.cap, ranks), p.Gp) : 0;
    if (!allow(kernel, ranks, smem)) return -1;
    const int carve = carve_of(shared_bytes<D, G, kOcc>(smem));
    return launch_first(kernel, static_cast<unsigned>(p.c.batch) * p.c.H * ranks, kPaThreads, smem, ranks, carve, s, p, ranks) ==
                   cudaSuccess
               ? 0
               : -1;
}

template <class Tile, int D, bool kF32, int G>
static int launch_pa(PagedAttnParams p, int ncta, cudaStream_t s) {
    int bits = static_cast<int>(kPaSlack);
    while (Tile::kLow && p.c.cap > 1 << (bits - static_cast<int>(kPaSlack))) ++bits;
    p.down = Tile::kLow ? 1.f / static_cast<float>(int64_t(1) << bits) : 1.f;
    constexpr int kOcc = occ_of(kF32, D), kOccShort = kF32 ? 2 : kOcc;
    const int held = ncta / kOcc * kOccShort;
    if (p.weight_out) {
        if (const int ranks = cluster_ranks<Tile, D, kF32, G, kOccShort, true>(p, held))
            return launch_cluster<Tile, D, kF32, G, kOccShort, true>(p, ranks, s);
    } else if (const int ranks = cluster_ranks<Tile, D, kF32, G, kOccShort, false>(p, held)) {
        return launch_cluster<Tile, D, kF32, G, kOccShort, false>(p, ranks, s);
    }
    // no more CTAs than there can be tiles for their warps
    const int64_t tiles = static_cast<int64_t>(p.c.batch) * p.c.H * ((p.c.cap + kPaTile - 1) / kPaTile);
    constexpr int kMin = (kF32 ? 1 : kPaLeast) * kPaWarps;
    const int64_t most = (tiles + kMin - 1) / kMin;
    const int n = most < ncta ? static_cast<int>(most) : ncta;
    auto kernel = p.weight_out ? k_paged_attn<Tile, D, kF32, G, kOcc, true> : k_paged_attn<Tile, D, kF32, G, kOcc, false>;
    const int smem = kF32 ? kPaWarps * G * (D + 4) * 4 : 0;
    // (eight heads of 128 dimensions take more than a kernel has without asking)
    if (kF32 && G * D >= 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return -1;
    if (launch_first(kernel, n, kPaThreads, smem, 1, kCarve, s, p) != cudaSuccess) return -1;
    // a CTA per head where units are few and so have many shares; one for all heads where they are many
    const int heads = p.c.batch * static_cast<int64_t>(p.c.H) * 4 >= n ? 1 : p.G;
    if (launch_first(k_paged_merge<D, kF32>, dim3(n, heads), kPaThreads, 0, 1, kCarve, s, p) != cudaSuccess) return -1;
    if (p.weight_out) {
        const int64_t blocks = static_cast<int64_t>(p.c.batch) * p.c.H * ((p.c.cap + kWeighRows - 1) / kWeighRows);
        const int64_t wide = static_cast<int64_t>(kWeighOcc) * (ncta / kOcc);
        const int nw = static_cast<int>(blocks < wide ? blocks : wide);
        auto weigh = p.Gp == 2 ? k_paged_weigh<2> : p.Gp == 4 ? k_paged_weigh<4> : p.Gp == 6 ? k_paged_weigh<6> : k_paged_weigh<8>;
        if (launch_first(weigh, nw, kPaThreads, 0, 1, kCarve, s, p) != cudaSuccess) return -1;
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}
template <int D>
static int launch_f32(const PagedAttnParams& p, int ncta, cudaStream_t s) {
    if (p.G <= 1) return launch_pa<TileF32<D, 1>, D, true, 1>(p, ncta, s);
    if (p.G <= 2) return launch_pa<TileF32<D, 2>, D, true, 2>(p, ncta, s);
    if (p.G <= 4) return launch_pa<TileF32<D, 4>, D, true, 4>(p, ncta, s);
    return launch_pa<TileF32<D, 8>, D, true, 8>(p, ncta, s);
}

int launch_paged_attn(int dtype, int d, const PagedAttnParams& p, int ncta, cudaStream_t s) {
    if (dtype == SKV_F32) return d == 64 ? launch_f32<64>(p, ncta, s) : launch_f32<128>(p, ncta, s);
    if (dtype == SKV_FP8)
        return d == 64 ? launch_pa<TileTC<64, true>, 64, false, 8>(p, ncta, s)
                       : launch_pa<TileTC<128, true>, 128, false, 8>(p, ncta, s);
    return d == 64 ? launch_pa<TileTC<64, false>, 64, false, 8>(p, ncta, s)
                   : launch_pa<TileTC<128, false>, 128, false, 8>(p, ncta, s);
}

cudaError_t paged_attn_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
