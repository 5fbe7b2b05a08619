// Eviction from a paged cache by accumulated attention weight (shadowkv_paged_evict).
//
// Per unit (a sequence's KV head) of n rows and a budget of M < n: the M largest keys stay, where
// a row's key is its weight as an ordered integer, and the largest integer for protected rows (the
// most recent positions and the first ones).  The kept rows at M and behind fill the given-up rows
// below M, so sources and destinations are disjoint, only the rows that have to move are moved, and
// a unit that is one row over its budget moves at most one row instead of shifting the rest.
//
// k_evict_select finds the M-th largest key by a radix search of 11, 5, 11 and 5 bits (integer
// counts in shared memory, so the order of the atomics does not show) and writes both lists in
// ascending row order.  A unit belongs to a cluster of 1 to 8 CTAs, each with a contiguous slice of
// the rows, each warp with a contiguous part of the slice; counts are joined through distributed
// shared memory.  The upper halves of a slice's keys stay in shared memory, and the lower ones too
// where there is room; else the weights are read again for lanes that hold a row whose upper half
// equals the threshold's.  k_evict_move, a programmatic dependent, copies the rows.
#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvStep = 256;                   // rows of a warp's step, eight per lane
constexpr int kEvGrain = kEvStep * kEvWarps;   // a slice is a multiple of this many rows
constexpr int kEvBins = 2048;
constexpr int kEvKeys = 11 * kEvGrain;         // rows of a slice held in shared memory at most (88 KB: two CTAs per SM)
constexpr int kEvHist = 2 * kEvBins + 64;      // counts of the four passes

// weights in the order of unsigned integers: -0 counts as 0, a NaN lies above +inf
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void sync_all(int ranks) {
    if (ranks > 1) cluster_sync_all();
    else __syncthreads();
}

// eight consecutive 32-bit values from row s on, `fill` from row `end` on
template <typename T>
__device__ __forceinline__ void load_rows(const T* p, int s, int end, bool vec, T fill, T (&x)[8]) {
    if (vec && s + 8 <= end) {
        const int4 a = __ldg(reinterpret_cast<const int4*>(p + s)), b = __ldg(reinterpret_cast<const int4*>(p + s) + 1);
        const int v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = *reinterpret_cast<const T*>(&v[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = s + e < end ? __ldg(p + s + e) : fill;
    }
}

__device__ __forceinline__ int excl_scan(int x, int lane) {
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += v;
    }
    return y - x;
}

__global__ void __launch_bounds__(kEvThreads, 2) k_evict_select(const __grid_constant__ EvictParams p, int ranks,
                                                                 int key_cap, int low_cap) {
    extern __shared__ __align__(16) int sm[];
    int* s_hist = sm;                                                  // [kEvHist]
    uint16_t* s_key = reinterpret_cast<uint16_t*>(sm + kEvHist);      // [key_cap] upper halves of the keys
    uint16_t* s_low = s_key + key_cap;                                 // [low_cap] lower halves
    __shared__ int s_scan[kEvWarps], s_bin[3], s_maxes[kEvWarps], s_max;
    __shared__ int s_cnt[4][kEvWarps], s_tot[4];
    __shared__ int s_tie[kEvWarps], s_hole[kEvWarps], s_src[kEvWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u = blockIdx.x / ranks, rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int b = u / p.c.H;
    const int n = rows_of(p.c, b, g_err, 721);
    const int M = p.budget;
    pdl_trigger();
    const int64_t base = static_cast<int64_t>(u) * p.row_pitch;
    const float* w_in = p.weight + base;
    const int32_t* p_in = p.position + base;
    const bool vec = ((reinterpret_cast<uintptr_t>(w_in) | reinterpret_cast<uintptr_t>(p_in)) & 15) == 0;
    const bool copy_w = p.weight_out != p.weight, copy_p = p.position_out != p.position;
    const int64_t slice = (static_cast<int64_t>(n) + ranks - 1) / ranks;
    const int per = static_cast<int>((slice + kEvGrain - 1) / kEvGrain) * kEvStep;        // rows of a warp
    const int64_t lo64 = (static_cast<int64_t>(rank) * kEvWarps + warp) * per;
    const int lo = static_cast<int>(min(lo64, static_cast<int64_t>(n)));
    const int hi = static_cast<int>(min(lo64 + per, static_cast<int64_t>(n)));
    if (rank == 0 && tid == 0 && u % p.c.H == 0) p.new_len[b] = min(n, M);
    if (n <= M) {      // the whole cluster: nothing is given up
        if (rank == 0 && tid == 0) p.count[u] = 0;
        for (int i = lo + lane; i < hi; i += 32) {
            if (copy_w) p.weight_out[base + i] = w_in[i];
            if (copy_p) p.position_out[base + i] = p_in[i];
        }
        return;
    }

    for (int i = tid; i < kEvHist; i += kEvThreads) s_hist[i] = 0;
    // ---- the unit's last position
    int last = INT_MIN;
#pragma unroll 4
    for (int r0 = lo; r0 < hi; r0 += kEvStep) {
        int pos[8];
        load_rows<int>(p_in, r0 + 8 * lane, hi, vec, INT_MIN, pos);
#pragma unroll
        for (int e = 0; e < 8; ++e) last = max(last, pos[e]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
    if (lane == 0) s_maxes[warp] = last;
    __syncthreads();
    if (warp == 0) {
        int x = s_maxes[lane % kEvWarps];
#pragma unroll
        for (int o = 16; o; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (lane == 0) s_max = x;
    }
    sync_all(ranks);
    last = s_max;
    for (int r = 0; r < ranks; ++r)
        if (r != rank) last = max(last, ld_cluster_s32(cluster_addr(&s_max, r)));
    const int64_t safe_from = static_cast<int64_t>(last) - p.recent;

    const bool held = per * kEvWarps <= key_cap, held_low = per * kEvWarps <= low_cap;
    uint16_t *my = s_key + warp * per, *my_low = s_low + warp * per;
    auto key_of = [&](float w, int pos) -> uint32_t {
        return (pos > safe_from || pos < p.sink) ? 0xFFFFFFFFu : weight_key(w);
    };
    // the lane's eight keys from row s on
    auto make = [&](int s, uint32_t (&t)[8]) {
        float w[8];
        int pos[8];
        load_rows<float>(w_in, s, hi, vec, 0.f, w);
        load_rows<int>(p_in, s, hi, vec, 0, pos);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = key_of(w[e], pos[e]);
    };
    auto pick = [](const uint16_t* from, uint32_t (&t)[8]) {
        const uint4 v = *reinterpret_cast<const uint4*>(from);
        t[0] = v.x & 0xFFFF; t[1] = v.x >> 16; t[2] = v.y & 0xFFFF; t[3] = v.y >> 16;
        t[4] = v.z & 0xFFFF; t[5] = v.z >> 16; t[6] = v.w & 0xFFFF; t[7] = v.w >> 16;
    };
    // their upper halves, and their lower ones
    auto upper = [&](int s, uint32_t (&t)[8]) {
        if (held) {
            pick(my + (s - lo), t);
        } else {
            make(s, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] >>= 16;
        }
    };
    auto lower = [&](int s, uint32_t (&t)[8]) {
        if (held_low) {
            pick(my_low + (s - lo), t);
        } else {
            make(s, t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] &= 0xFFFF;
        }
    };
    // of the eight rows from s on: bits of those below x
    auto bits_below = [](int s, int x) -> uint32_t { return x <= s ? 0u : x - s >= 8 ? 0xFFu : (1u << (x - s)) - 1; };

    // ---- the M-th largest key, from the top; bits 31..21, 20..16, 15..5, 4..0
    uint32_t prefix = 0, T = 0;
    int need = M, ties = 0;
    bool whole = false;        // every key from T + 1 on stays, no ties
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 16 : pass == 2 ? 5 : 0, bins = (pass & 1) ? 32 : kEvBins;
        int* hist = s_hist + (pass == 0 ? 0 : pass == 1 ? 2 * kEvBins : pass == 2 ? kEvBins : 2 * kEvBins + 32);
        for (int r0 = lo; r0 < hi; r0 += kEvStep) {
            const int s = r0 + 8 * lane;
            const uint32_t in = bits_below(s, hi);
            uint32_t t[8];
            if (pass == 0) {
                make(s, t);
                auto pair = [&](int e, int sh) { return ((t[e] >> sh) & 0xFFFF) | ((t[e + 1] >> sh) << 16); };
                if (held)
                    *reinterpret_cast<uint4*>(my + (s - lo)) = make_uint4(pair(0, 16), pair(2, 16), pair(4, 16), pair(6, 16));
                if (held_low)
                    *reinterpret_cast<uint4*>(my_low + (s - lo)) = make_uint4(pair(0, 0), pair(2, 0), pair(4, 0), pair(6, 0));
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((in >> e) & 1) atomicAdd(hist + (t[e] >> 21), 1);
                continue;
            }
            upper(s, t);
            if (pass == 1) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((in >> e) & 1 && (t[e] >> 5) == prefix) atomicAdd(hist + (t[e] & 31), 1);
                continue;
            }
            uint32_t same = 0, l[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) same |= (t[e] == (pass == 2 ? prefix : prefix >> 11) ? 1u : 0u) << e;
            same &= in;
            if (!same) continue;
            lower(s, l);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (!((same >> e) & 1)) continue;
                if (pass == 2) atomicAdd(hist + (l[e] >> 5), 1);
                else if ((l[e] >> 5) == (prefix & (kEvBins - 1))) atomicAdd(hist + (l[e] & 31), 1);
            }
        }
        sync_all(ranks);
        // counts from the top: thread t holds four bins, the uppermost first
        int cnt[4] = {0, 0, 0, 0};
        const int top = bins - 1 - 4 * tid;
        if (top >= 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) cnt[e] = hist[top - e];
            for (int r = 0; r < ranks; ++r)
                if (r != rank) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) cnt[e] += ld_cluster_s32(cluster_addr(hist + top - e, r));
                }
        }
        const int mine = cnt[0] + cnt[1] + cnt[2] + cnt[3];
        int above = excl_scan(mine, lane);
        if (lane == 31) s_scan[warp] = above + mine;
        __syncthreads();
        above += __reduce_add_sync(0xffffffffu, lane < warp ? s_scan[lane % kEvWarps] : 0);
        if (above < need && above + mine >= need) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (above < need && above + cnt[e] >= need) {
                    s_bin[0] = top - e;
                    s_bin[1] = above;
                    s_bin[2] = cnt[e];
                }
                above += cnt[e];
            }
        }
        __syncthreads();
        const int inside = s_bin[2];
        need -= s_bin[1];
        prefix = (prefix << ((pass & 1) ? 5 : 11)) | static_cast<uint32_t>(s_bin[0]);
        if (inside == need && prefix != 0) {          // the whole bin stays
            T = (prefix << shift) - 1;
            whole = true;
            break;
        }
    }
    if (!whole) {
        T = prefix;
        ties = need;           // this many rows of key T stay, the lowest ones
    }
    const uint32_t T16 = T >> 16;
    const bool upper_alone = whole && (T & 0xFFFFu) == 0xFFFFu;     // no key of upper half T16 stays
    // which of the lane's eight rows from s on lie above the threshold, and which on it
    auto grade = [&](int s, uint32_t& gt, uint32_t& tie) {
        uint32_t t[8], l[8], same = 0;
        upper(s, t);
        gt = tie = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            gt |= (t[e] > T16 ? 1u : 0u) << e;
            same |= (t[e] == T16 ? 1u : 0u) << e;
        }
        const uint32_t in = bits_below(s, hi);
        gt &= in;
        same &= in;
        if (!same || upper_alone) return;
        lower(s, l);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!((same >> e) & 1)) continue;
            if (l[e] > (T & 0xFFFFu)) gt |= 1u << e;
            else if (l[e] == (T & 0xFFFFu) && !whole) tie |= 1u << e;
        }
    };

    // ---- rows of each kind per warp: given up and tied below M, kept for sure and tied behind
    int n_low = 0, n_tl = 0, n_gt = 0, n_th = 0;
    for (int r0 = lo; r0 < hi; r0 += kEvStep) {
        const int s = r0 + 8 * lane;
        uint32_t gt, tie;
        grade(s, gt, tie);
        const uint32_t in = bits_below(s, hi), low = bits_below(s, M);
        n_low += __popc(in & low & ~(gt | tie));
        n_tl += __popc(low & tie);
        n_gt += __popc(~low & gt);
        n_th += __popc(~low & tie);
    }
    n_low = __reduce_add_sync(0xffffffffu, n_low);
    n_tl = __reduce_add_sync(0xffffffffu, n_tl);
    n_gt = __reduce_add_sync(0xffffffffu, n_gt);
    n_th = __reduce_add_sync(0xffffffffu, n_th);
    if (lane == 0) {
        s_cnt[0][warp] = n_low;
        s_cnt[1][warp] = n_tl;
        s_cnt[2][warp] = n_gt;
        s_cnt[3][warp] = n_th;
    }
    __syncthreads();
    if (warp < 4) {
        const int x = __reduce_add_sync(0xffffffffu, lane < kEvWarps ? s_cnt[warp][lane] : 0);
        if (lane == 0) s_tot[warp] = x;
    }
    sync_all(ranks);
    if (warp == 0) {
        // what lies in the slices before this one (rows below M come first in every slice)
        int tie0 = 0, hole0 = 0, src0 = 0;
        for (int r = 0; r < rank; ++r) {
            const int a = ld_cluster_s32(cluster_addr(&s_tot[0], r)), tl = ld_cluster_s32(cluster_addr(&s_tot[1], r));
            const int g = ld_cluster_s32(cluster_addr(&s_tot[2], r)), th = ld_cluster_s32(cluster_addr(&s_tot[3], r));
            const int left = max(0, ties - tie0), kl = min(tl, left), kh = min(th, left - kl);
            hole0 += a + tl - kl;
            src0 += g + kh;
            tie0 += tl + th;
        }
        const int w = lane % kEvWarps;
        const bool own = lane < kEvWarps;
        const int a = own ? s_cnt[0][w] : 0, tl = own ? s_cnt[1][w] : 0, g = own ? s_cnt[2][w] : 0, th = own ? s_cnt[3][w] : 0;
        const int t0 = tie0 + excl_scan(tl + th, lane);
        const int left = max(0, ties - t0), kl = min(tl, left), kh = min(th, left - kl);
        const int holes = a + tl - kl, srcs = g + kh;
        const int h0 = hole0 + excl_scan(holes, lane), s0 = src0 + excl_scan(srcs, lane);
        if (own) {
            s_tie[w] = t0;
            s_hole[w] = h0;
            s_src[w] = s0;
        }
        if (rank == ranks - 1 && lane == kEvWarps - 1) p.count[u] = s0 + srcs;
    }
    sync_all(ranks);       // and no CTA leaves while another reads its counts
    int tie_at = s_tie[warp], hole_at = s_hole[warp], src_at = s_src[warp];
    int32_t* to = p.to + static_cast<int64_t>(u) * p.list_cap;
    int32_t* of = p.of + static_cast<int64_t>(u) * p.list_cap;
    for (int r0 = lo; r0 < hi; r0 += kEvStep) {
        const int s = r0 + 8 * lane;
        uint32_t kept, tie;
        grade(s, kept, tie);
        if (__any_sync(0xffffffffu, tie)) {
            int t = tie_at + excl_scan(__popc(tie), lane);
            tie_at += __reduce_add_sync(0xffffffffu, __popc(tie));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if ((tie >> e) & 1) {
                    if (t < ties) kept |= 1u << e;
                    ++t;
                }
        }
        const uint32_t in = bits_below(s, hi), low = bits_below(s, M);
        const uint32_t hole = in & low & ~kept, src = kept & ~low;
        if (!__any_sync(0xffffffffu, hole | src | (kept & low))) continue;
        const int both = __popc(hole) | __popc(src) << 16;       // at most 256 of each
        const int at = excl_scan(both, lane);
        const int all = __reduce_add_sync(0xffffffffu, both);
        int ha = hole_at + (at & 0xFFFF), sa = src_at + (at >> 16);
        hole_at += all & 0xFFFF;
        src_at += all >> 16;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if ((hole >> e) & 1) {
                if (ha < p.list_cap) to[ha] = s + e;
                ++ha;
            }
            if ((src >> e) & 1) {
                if (sa < p.list_cap) of[sa] = s + e;
                ++sa;
            }
            if ((kept & low) >> e & 1) {
                if (copy_w) p.weight_out[base + s + e] = w_in[s + e];
                if (copy_p) p.position_out[base + s + e] = p_in[s + e];
            }
        }
    }
}

constexpr int kMvThreads = 256;
constexpr int kMvPairs = 4;        // rows per warp and round

__global__ void __launch_bounds__(kMvThreads) k_evict_move(const __grid_constant__ EvictParams p, int parts) {
    pdl_wait();
    const int u = blockIdx.x / parts, part = blockIdx.x % parts, b = u / p.c.H, h = u % p.c.H;
    const int lane = threadIdx.x & 31;
    if (h == 0 && part == 0 && threadIdx.x == 0) p.lens_out[b] = p.new_len[b];
    const int cnt = min(p.count[u], p.list_cap);
    const int64_t base = static_cast<int64_t>(u) * p.row_pitch;
    const int32_t* to = p.to + static_cast<int64_t>(u) * p.list_cap;
    const int32_t* of = p.of + static_cast<int64_t>(u) * p.list_cap;
    const int step = parts * (kMvThreads / 32) * kMvPairs;
    const int kw = p.d * p.es / 16, vw = p.d * p.es_v / 16, mask = (1 << p.c.lg) - 1;
    uint8_t* kp = static_cast<uint8_t*>(p.c.k) + h * p.c.k_head * p.es;
    uint8_t* vp = static_cast<uint8_t*>(p.c.v) + h * p.c.v_head * p.es_v;
    for (int i0 = (part * (kMvThreads / 32) + (threadIdx.x >> 5)) * kMvPairs; i0 < cnt; i0 += step) {
        // lane j < kMvPairs looks pair j up
        int64_t kd = -1, ks = 0, vd = 0, vs = 0;
        if (lane < kMvPairs && i0 + lane < cnt) {
            const int d = to[i0 + lane], s = of[i0 + lane];
            const int pd = page_of(p.c, b, d, g_err, 722), ps = page_of(p.c, b, s, g_err, 723);
            p.weight_out[base + d] = p.weight[base + s];
            p.position_out[base + d] = p.position[base + s];
            if (pd >= 0 && ps >= 0) {
                kd = (pd * p.c.k_page + (d & mask) * p.c.k_row) * p.es;
                ks = (ps * p.c.k_page + (s & mask) * p.c.k_row) * p.es;
                vd = (pd * p.c.v_page + (d & mask) * p.c.v_row) * p.es_v;
                vs = (ps * p.c.v_page + (s & mask) * p.c.v_row) * p.es_v;
            }
        }
        // 16-byte words of the key and value rows, lane-strided
        for (int w = lane; w < ((kw + vw + 31) & ~31); w += 32) {
            uint4 x[kMvPairs];
#pragma unroll
            for (int j = 0; j < kMvPairs; ++j) {
                const int64_t d = __shfl_sync(0xffffffffu, kd, j), s = __shfl_sync(0xffffffffu, ks, j);
                const int64_t sv = __shfl_sync(0xffffffffu, vs, j);
                if (d >= 0 && w < kw + vw)
                    x[j] = __ldg(reinterpret_cast<const uint4*>(w < kw ? kp + s : vp + sv) + (w < kw ? w : w - kw));
            }
#pragma unroll
            for (int j = 0; j < kMvPairs; ++j) {
                const int64_t d = __shfl_sync(0xffffffffu, kd, j), dv = __shfl_sync(0xffffffffu, vd, j);
                if (d >= 0 && w < kw + vw)
                    *(reinterpret_cast<uint4*>(w < kw ? kp + d : vp + dv) + (w < kw ? w : w - kw)) = x[j];
            }
        }
    }
}

int launch_evict(const EvictParams& p, int nsm, cudaStream_t s) {
    const int U = p.c.batch * p.c.H;
    // CTAs per unit: as many as the device holds at once (two per SM), and no fewer than the keys
    // need to stay in shared memory; a slice of under one grain (4096 rows) would leave warps idle
    int ranks = 1;
    while (ranks < 8 && p.c.cap > ranks * kEvGrain && (U * ranks <= nsm || p.c.cap / ranks > kEvKeys)) ranks *= 2;
    const int64_t slice = (static_cast<int64_t>(p.c.cap) + ranks - 1) / ranks;
    const int64_t keys = (slice + kEvGrain - 1) / kEvGrain * kEvGrain;
    const int key_cap = static_cast<int>(keys < kEvKeys ? keys : kEvKeys);
    const int low_cap = 2 * key_cap <= kEvKeys ? key_cap : 0;
    const int smem = kEvHist * 4 + (key_cap + low_cap) * 2;
    if (cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvHist * 4 + kEvKeys * 2) !=
        cudaSuccess)
        return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(U) * ranks);
    cfg.blockDim = dim3(kEvThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, k_evict_select, p, ranks, key_cap, low_cap) != cudaSuccess) return -1;
    // CTAs per unit for the rows that move
    const int rows = (kMvThreads / 32) * kMvPairs;
    int64_t parts = (static_cast<int64_t>(p.list_cap) + rows - 1) / rows;
    const int64_t most = (16 * nsm + U - 1) / U;
    if (parts > most) parts = most;
    if (launch_pdl(k_evict_move, dim3(static_cast<unsigned>(parts * U)), dim3(kMvThreads), 0, s, p,
                   static_cast<int>(parts)) != cudaSuccess)
        return -1;
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

cudaError_t evict_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
