// Eviction from a paged cache by accumulated attention weight (shadowkv_paged_evict).
//
// Per unit (a sequence's KV head) of n rows and a budget of M < n: the M largest keys stay, where
// a row's key is its weight as an ordered integer, and the largest integer for protected rows (the
// most recent positions and the first ones).  The kept rows at M and behind fill the given-up rows
// below M, so sources and destinations are disjoint, only the rows that have to move are moved, and
// a unit that is one row over its budget moves at most one row instead of shifting the rest.
//
// k_evict_select finds the M-th largest key by a radix search of 11, 11 and 10 bits (integer
// counts in shared memory, so the order of the atomics does not show) and writes both lists in
// ascending row order.  A unit belongs to a cluster of 1 to 8 CTAs, each with a contiguous slice
// of the rows whose keys stay in its shared memory; counts are joined through distributed shared
// memory.  k_evict_move, a programmatic dependent, copies the rows.
#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048;
constexpr int kEvKeys = 40960;                 // keys of a slice held in shared memory at most (160 KB)

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

__global__ void __launch_bounds__(kEvThreads, 1) k_evict_select(const __grid_constant__ EvictParams p, int ranks,
                                                              int key_cap) {
    extern __shared__ __align__(16) uint32_t sm[];
    int* s_hist = reinterpret_cast<int*>(sm);                // [3][kEvBins]
    uint32_t* s_key = sm + 3 * kEvBins;                      // [key_cap]
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
    const bool copy_w = p.weight_out != p.weight, copy_p = p.position_out != p.position;
    // slices are whole multiples of 32 rows per warp
    const int per = (static_cast<int>((static_cast<int64_t>(n) + ranks - 1) / ranks) + kEvThreads - 1) / kEvThreads * 32;
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

    for (int i = tid; i < 3 * kEvBins; i += kEvThreads) s_hist[i] = 0;
    // ---- the unit's last position
    int last = INT_MIN;
    for (int i = lo + lane; i < hi; i += 32) last = max(last, __ldg(p_in + i));
#pragma unroll
    for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
    if (lane == 0) s_maxes[warp] = last;
    __syncthreads();
    if (warp == 0) {
        int x = s_maxes[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (lane == 0) s_max = x;
    }
    sync_all(ranks);
    last = s_max;
    for (int r = 0; r < ranks; ++r)
        if (r != rank) last = max(last, ld_cluster_s32(cluster_addr(&s_max, r)));
    const int64_t safe_from = static_cast<int64_t>(last) - p.recent;

    const bool held = per * kEvWarps <= key_cap;
    uint32_t* my = s_key + warp * per;
    auto make = [&](int i) -> uint32_t {
        const int pos = __ldg(p_in + i);
        return (pos > safe_from || pos < p.sink) ? 0xFFFFFFFFu : weight_key(__ldg(w_in + i));
    };
    auto key = [&](int i) -> uint32_t { return held ? my[i - lo] : make(i); };

    // ---- the M-th largest key, from the top
    uint32_t prefix = 0, T = 0;
    int need = M, ties = 0;
    bool whole = false;        // every key from T + 1 on stays, no ties
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        int* hist = s_hist + pass * kEvBins;
        for (int i = lo + lane; i < hi; i += 32) {
            uint32_t k;
            if (pass == 0) {
                k = make(i);
                if (held) my[i - lo] = k;
            } else {
                k = key(i);
                if ((k >> (shift + bits)) != prefix) continue;
            }
            atomicAdd(hist + ((k >> shift) & ((1u << bits) - 1)), 1);
        }
        sync_all(ranks);
        // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t
        int c0 = hist[kEvBins - 1 - 2 * tid], c1 = hist[kEvBins - 2 - 2 * tid];
        for (int r = 0; r < ranks; ++r)
            if (r != rank) {
                c0 += ld_cluster_s32(cluster_addr(hist + kEvBins - 1 - 2 * tid, r));
                c1 += ld_cluster_s32(cluster_addr(hist + kEvBins - 2 - 2 * tid, r));
            }
        int sum = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) s_scan[warp] = sum;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += s_scan[w];
        const int above = before + sum - c0 - c1;     // keys in the bins above this thread's two
        if (above < need && above + c0 + c1 >= need) {
            const bool first = above + c0 >= need;
            s_bin[0] = first ? kEvBins - 1 - 2 * tid : kEvBins - 2 - 2 * tid;
            s_bin[1] = first ? above : above + c0;
            s_bin[2] = first ? c0 : c1;
        }
        __syncthreads();
        const int bin = s_bin[0], inside = s_bin[2];
        need -= s_bin[1];
        prefix = (prefix << bits) | static_cast<uint32_t>(bin);
        __syncthreads();
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

    // ---- rows of each kind per warp: given up and tied below M, kept for sure and tied behind
    int n_low = 0, n_tl = 0, n_gt = 0, n_th = 0;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < hi;
        const uint32_t k = in ? key(i) : 0;
        const bool tie = in && !whole && k == T, gt = in && k > T;
        n_low += __popc(__ballot_sync(0xffffffffu, in && i < M && !gt && !tie));
        n_tl += __popc(__ballot_sync(0xffffffffu, i < M && tie));
        n_gt += __popc(__ballot_sync(0xffffffffu, i >= M && gt));
        n_th += __popc(__ballot_sync(0xffffffffu, i >= M && tie));
    }
    if (lane == 0) {
        s_cnt[0][warp] = n_low;
        s_cnt[1][warp] = n_tl;
        s_cnt[2][warp] = n_gt;
        s_cnt[3][warp] = n_th;
    }
    __syncthreads();
    if (warp < 4) {
        const int x = warp_sum_i(s_cnt[warp][lane]);
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
        const int a = s_cnt[0][lane], tl = s_cnt[1][lane], g = s_cnt[2][lane], th = s_cnt[3][lane];
        auto excl = [&](int x) {
            int y = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += v;
            }
            return y - x;
        };
        const int t0 = tie0 + excl(tl + th);
        const int left = max(0, ties - t0), kl = min(tl, left), kh = min(th, left - kl);
        const int holes = a + tl - kl, srcs = g + kh;
        s_tie[lane] = t0;
        s_hole[lane] = hole0 + excl(holes);
        const int s0 = src0 + excl(srcs);
        s_src[lane] = s0;
        if (rank == ranks - 1 && lane == 31) p.count[u] = s0 + srcs;
    }
    sync_all(ranks);       // and no CTA leaves while another reads its counts
    int tie_at = s_tie[warp], hole_at = s_hole[warp], src_at = s_src[warp];
    int32_t* to = p.to + static_cast<int64_t>(u) * p.list_cap;
    int32_t* of = p.of + static_cast<int64_t>(u) * p.list_cap;
    const uint32_t below = (1u << lane) - 1;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < hi;
        const uint32_t k = in ? key(i) : 0;
        const bool tie = in && !whole && k == T;
        const uint32_t tb = __ballot_sync(0xffffffffu, tie);
        const bool kept = in && ((k > T) || (tie && tie_at + __popc(tb & below) < ties));
        tie_at += __popc(tb);
        const uint32_t hb = __ballot_sync(0xffffffffu, in && i < M && !kept);
        const uint32_t sb = __ballot_sync(0xffffffffu, i >= M && kept);
        if (in && i < M && !kept) {
            const int at = hole_at + __popc(hb & below);
            if (at < p.list_cap) to[at] = i;
        }
        if (i >= M && kept) {
            const int at = src_at + __popc(sb & below);
            if (at < p.list_cap) of[at] = i;
        }
        if (i < M && kept) {
            if (copy_w) p.weight_out[base + i] = w_in[i];
            if (copy_p) p.position_out[base + i] = p_in[i];
        }
        hole_at += __popc(hb);
        src_at += __popc(sb);
    }
}

constexpr int kMvThreads = 256;
constexpr int kMvPairs = 8;        // rows per warp and round

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
    // CTAs per unit: as many as keep the device's SMs busy, and no fewer than the keys need to
    // stay in shared memory; a slice of under 4096 rows does not pay for the cluster's barriers
    int ranks = 1;
    while (ranks < 8 && p.c.cap / ranks > 4096 && (U * ranks * 2 <= nsm || p.c.cap / ranks > kEvKeys)) ranks *= 2;
    const int64_t slice = (static_cast<int64_t>(p.c.cap) + ranks - 1) / ranks;
    const int64_t keys = (slice + kEvThreads - 1) / kEvThreads * kEvThreads;
    const int key_cap = static_cast<int>(keys < kEvKeys ? keys : kEvKeys);
    const int smem = (3 * kEvBins + key_cap) * 4;
    if (cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
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
    if (cudaLaunchKernelEx(&cfg, k_evict_select, p, ranks, key_cap) != cudaSuccess) return -1;
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
