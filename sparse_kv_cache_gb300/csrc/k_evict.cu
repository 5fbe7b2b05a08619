// Eviction from a paged cache by accumulated attention weight (shadowkv_paged_evict).
//
// Per unit (a sequence's KV head) of n rows and a budget of M < n: the M largest keys stay, where
// a row's key is its weight as an ordered integer, and the largest integer for protected rows (the
// most recent positions and the first ones).  The kept rows at M and behind fill the given-up rows
// below M, so sources and destinations are disjoint, only the rows that have to move are moved, and
// a unit that is one row over its budget moves at most one row instead of shifting the rest.
//
// k_evict finds the M-th largest key by a radix search of 11, 5, 11 and 5 bits (integer counts in
// shared memory, so the order of the atomics does not show) and writes both lists in ascending row
// order.  A unit belongs to a cluster of 1 to 8 CTAs, each with a contiguous slice of the rows, each
// warp with a contiguous part of the slice; counts are joined through distributed shared memory.  The
// upper halves of a slice's keys stay in shared memory, and the lower ones too where there is room;
// else the weights are read again for lanes that hold a row whose upper half equals the threshold's.
// Once the 11 uppermost bits of the threshold are known, a warp whose rows all lie behind the budget
// keeps a list of those that can still stay -- of a long prompt a few in a hundred -- and goes on with
// that.  Where only a few rows of a unit can move (decode steps), its cluster moves them itself; else
// k_evict_move, a programmatic dependent, does with all of the device (154K rows of 64 long units:
// 63 us in all against 68).
//
// Measured back to back, 8 KV heads, d = 128, bf16: 8 ragged sequences of up to 128K rows down to 2464,
// 154K rows moved, 62 us -- 36 for the search, bound by the latency of its phases, 27 for the moves,
// 5.9 TB/s; 64 units of 2081 rows down to 2080 12 us, all of it latency.
#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kEvWide = 512, kEvNarrow = 128;  // threads of a CTA: two per SM, or eight (six where they hold 4096 keys)
constexpr int kEvStep = 256;                   // rows of a warp's step, eight per lane
constexpr int kEvBins = 2048;
constexpr int grain_of(int threads) { return kEvStep * (threads / 32); }     // a slice is a multiple of this many rows
constexpr int kEvKeys = 11 * grain_of(kEvWide);   // halves of keys held in shared memory at most (88 KB: two CTAs per SM)

// Rows of a unit that its own cluster moves, at most.  Of 2048 rows + 256, 64 units take 14.6 us with one
// kernel and 15.9 with two, + 512 19.1 and 20.5, + 952 29.4 and 24.0; 8 units, whose clusters leave most of the
// device idle, lose 0.8 us at + 512 (16.1 and 15.3).
constexpr int kEvFew = 512;
constexpr int kEvShort = 4096;                 // room of a sequence that narrow CTAs serve, at most
constexpr int kEvHist = 2 * kEvBins + 64;      // counts of the four passes

// weights in the order of unsigned integers: -0 counts as 0, a NaN lies above +inf
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xFFFFFFFEu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sync_all(int ranks) {
    if (ranks > 1) cluster_sync_all();
    else __syncthreads();
}

// Eight consecutive weights and positions from row s on.  s is a multiple of 8 below the unit's
// rows, and a sequence's room is one too, so rows that are read beyond its last lie in its room.
struct Rows8 { float4 w0, w1; int4 p0, p1; };
__device__ __forceinline__ void load_rows(const float* w, const int32_t* p, int s, Rows8& r) {
    r.w0 = reinterpret_cast<const float4*>(w + s)[0];
    r.w1 = reinterpret_cast<const float4*>(w + s)[1];
    r.p0 = reinterpret_cast<const int4*>(p + s)[0];
    r.p1 = reinterpret_cast<const int4*>(p + s)[1];
}
// Their keys: the largest for a protected row.
struct Protect {
    int from, sink;    // positions above from are recent, those below sink are first ones
    __device__ __forceinline__ uint32_t key(float w, int pos) const {
        return (pos > from || pos < sink) ? 0xFFFFFFFFu : weight_key(w);
    }
};
__device__ __forceinline__ void keys_of(const Protect& pr, const Rows8& r, uint32_t (&t)[8]) {
    t[0] = pr.key(r.w0.x, r.p0.x); t[1] = pr.key(r.w0.y, r.p0.y); t[2] = pr.key(r.w0.z, r.p0.z); t[3] = pr.key(r.w0.w, r.p0.w);
    t[4] = pr.key(r.w1.x, r.p1.x); t[5] = pr.key(r.w1.y, r.p1.y); t[6] = pr.key(r.w1.z, r.p1.z); t[7] = pr.key(r.w1.w, r.p1.w);
}
// eight upper (sh 16) or lower (sh 0) halves of keys in 16 bytes
__device__ __forceinline__ uint4 halves(const uint32_t (&t)[8], int sh) {
    auto pair = [&](int e) { return ((t[e] >> sh) & 0xFFFF) | ((t[e + 1] >> sh) << 16); };
    return make_uint4(pair(0), pair(2), pair(4), pair(6));
}
// the same from the weights, where the keys are not held (kept out of line: seldom called)
__device__ __noinline__ uint4 remade(const float* w, const int32_t* p, int s, Protect pr, int sh) {
    Rows8 r;
    load_rows(w, p, s, r);
    uint32_t t[8];
    keys_of(pr, r, t);
    return halves(t, sh);
}
// the first `count` of eight elements
template <typename T4, typename T>
__device__ __forceinline__ void copy_below(T* out, const T4& a, const T4& b, int count) {
    if (count >= 8) {
        reinterpret_cast<T4*>(out)[0] = a;
        reinterpret_cast<T4*>(out)[1] = b;
    } else if (count > 0) {
        const T x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < count) out[e] = x[e];
    }
}
// bits of the halves that f holds for
template <typename F>
__device__ __forceinline__ uint32_t mark(const uint4& v, F f) {
    return (f(v.x & 0xFFFF) ? 1u : 0u) | (f(v.x >> 16) ? 2u : 0u) | (f(v.y & 0xFFFF) ? 4u : 0u) | (f(v.y >> 16) ? 8u : 0u) |
           (f(v.z & 0xFFFF) ? 16u : 0u) | (f(v.z >> 16) ? 32u : 0u) | (f(v.w & 0xFFFF) ? 64u : 0u) | (f(v.w >> 16) ? 128u : 0u);
}
__device__ __forceinline__ uint32_t half_of(const uint4& v, int e) {
    const uint32_t x = e < 4 ? (e < 2 ? v.x : v.y) : (e < 6 ? v.z : v.w);
    return (e & 1) ? x >> 16 : x & 0xFFFF;
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

// Moves the unit's listed rows of which this is warp `warp` of `warps`: a lane of the warp looks each up,
// then their 16-byte words, four rows' at a time in flight (eight: 68 us, two: 65, against 63).
__device__ __forceinline__ void move_rows(const EvictParams& p, int u, int moves, int warp, int warps) {
    constexpr int kTurn = 32, kFlight = 4;
    const int lane = threadIdx.x & 31, b = u / p.c.H, h = u % p.c.H;
    const int64_t base = static_cast<int64_t>(u) * p.row_pitch;
    const int32_t* to = p.to + static_cast<int64_t>(u) * p.list_cap;
    const int32_t* of = p.of + static_cast<int64_t>(u) * p.list_cap;
    const int kw = p.d * p.es / 16, words = kw + p.d * p.es_v / 16, mask = (1 << p.c.lg) - 1;
    uint8_t* kp = static_cast<uint8_t*>(p.c.k) + h * p.c.k_head * p.es;
    uint8_t* vp = static_cast<uint8_t*>(p.c.v) + h * p.c.v_head * p.es_v;
#pragma unroll 1
    for (int i0 = warp * kTurn; i0 < moves; i0 += warps * kTurn) {
        int pd = -1, ps = -1, d = 0, s = 0;
        if (i0 + lane < moves) {
            d = __ldcg(to + i0 + lane);
            s = __ldcg(of + i0 + lane);
            if (d < 0 || d >= p.c.cap || s < 0 || s >= p.c.cap) {     // the lengths changed under the call
                set_err(g_err, DEV_ERR_BOUNDS, 724);
            } else {
                pd = page_of(p.c, b, d, g_err, 722);
                ps = page_of(p.c, b, s, g_err, 723);
                if (pd >= 0 && ps >= 0) {
                    p.weight_out[base + d] = p.weight[base + s];
                    p.position_out[base + d] = p.position[base + s];
                } else {       // the place keeps the row that was given up there
                    pd = -1;
                }
                d &= mask;
                s &= mask;
            }
        }
        const int rows = min(kTurn, moves - i0);
#pragma unroll 1
        for (int w = lane; w < ((words + 31) & ~31); w += 32) {      // words of a key row and its value row
            const bool key = w < kw;
            uint8_t* pool = (key ? kp : vp) + (key ? w : w - kw) * 16;
            const int64_t page = (key ? p.c.k_page : p.c.v_page) * (key ? p.es : p.es_v);
            const int64_t row = (key ? p.c.k_row : p.c.v_row) * (key ? p.es : p.es_v);
#pragma unroll 1
            for (int j0 = 0; j0 < rows; j0 += kFlight) {
                uint4 x[kFlight];
                int64_t dst[kFlight];
#pragma unroll
                for (int j = 0; j < kFlight; ++j) {
                    const int to_page = __shfl_sync(0xffffffffu, pd, j0 + j), of_page = __shfl_sync(0xffffffffu, ps, j0 + j);
                    const int to_row = __shfl_sync(0xffffffffu, d, j0 + j), of_row = __shfl_sync(0xffffffffu, s, j0 + j);
                    dst[j] = to_page >= 0 && w < words ? to_page * page + to_row * row : -1;
                    if (dst[j] >= 0) x[j] = *reinterpret_cast<const uint4*>(pool + of_page * page + of_row * row);
                }
#pragma unroll
                for (int j = 0; j < kFlight; ++j)
                    if (dst[j] >= 0) *reinterpret_cast<uint4*>(pool + dst[j]) = x[j];
            }
        }
    }
}

template <int kThreads, bool kMove>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) k_evict(const __grid_constant__ EvictParams p, int ranks,
                                                                 int key_cap, int low_cap) {
    constexpr int kWarps = kThreads / 32, kGrain = grain_of(kThreads), kEach = kEvBins / kThreads;     // bins per thread
    static_assert(kEach * kThreads == kEvBins && kEach % 4 == 0 && kWarps >= 4 && kWarps <= 32, "");
    extern __shared__ __align__(16) int sm[];
    int* s_hist = sm;                                                  // [kEvHist]
    uint16_t* s_key = reinterpret_cast<uint16_t*>(sm + kEvHist);      // [key_cap] upper halves of the keys
    uint16_t* s_low = s_key + key_cap;                                 // [low_cap] lower halves
    __shared__ int s_scan[kWarps], s_bin[3], s_maxes[kWarps], s_max;
    __shared__ int s_cnt[4][kWarps], s_tot[4];
    __shared__ int s_tie[kWarps], s_hole[kWarps], s_src[kWarps], s_moves;

    begin_call();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int u = blockIdx.x / ranks, rank = ranks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int b = u / p.c.H;
    const int n = rows_of(p.c, b, g_err, 721);
    const int M = p.budget;
    const int64_t base = static_cast<int64_t>(u) * p.row_pitch;
    const float* w_in = p.weight + base;
    const int32_t* p_in = p.position + base;
    const bool copy_w = p.weight_out != p.weight, copy_p = p.position_out != p.position;
    const int64_t slice = (static_cast<int64_t>(n) + ranks - 1) / ranks;
    const int per = static_cast<int>((slice + kGrain - 1) / kGrain) * kEvStep;        // rows of a warp
    const int64_t lo64 = (static_cast<int64_t>(rank) * kWarps + warp) * per;
    const int lo = static_cast<int>(min(lo64, static_cast<int64_t>(n)));
    const int hi = static_cast<int>(min(lo64 + per, static_cast<int64_t>(n)));
    // (the other heads' CTAs may not have read a length that is to be updated in place: it goes by new_len)
    if (rank == 0 && tid == 0 && u % p.c.H == 0) (p.lens_out == p.c.lens ? p.new_len : p.lens_out)[b] = min(n, M);
    if (n <= M) {      // the whole cluster: nothing is given up
        if (!kMove && rank == 0 && tid == 0) p.count[u] = 0;
        for (int i = lo + lane; i < hi; i += 32) {
            if (copy_w) p.weight_out[base + i] = w_in[i];
            if (copy_p) p.position_out[base + i] = p_in[i];
        }
        return;
    }

    for (int i = tid; i < kEvHist; i += kThreads) s_hist[i] = 0;
    // ---- the unit's last position
    int last = INT_MIN;
    constexpr int kDeep = 4;       // steps whose loads are in flight together
    for (int r0 = lo; r0 < hi; r0 += kDeep * kEvStep) {
        int4 pos[kDeep][2];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int s = r0 + k * kEvStep + 8 * lane;
            pos[k][0] = pos[k][1] = make_int4(INT_MIN, INT_MIN, INT_MIN, INT_MIN);
            if (s < hi) {
                pos[k][0] = reinterpret_cast<const int4*>(p_in + s)[0];
                pos[k][1] = reinterpret_cast<const int4*>(p_in + s)[1];
            }
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int left = hi - (r0 + k * kEvStep + 8 * lane);      // of the lane's eight rows, those below hi
            const int4 a = pos[k][0], b = pos[k][1];
            if (left >= 8) {
                last = max(last, max(max(max(a.x, a.y), max(a.z, a.w)), max(max(b.x, b.y), max(b.z, b.w))));
            } else {
                const int v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                for (int e = 0; e < 7; ++e) last = e < left ? max(last, v[e]) : last;
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
    if (lane == 0) s_maxes[warp] = last;
    __syncthreads();
    if (warp == 0) {
        int x = s_maxes[lane % kWarps];
#pragma unroll
        for (int o = 16; o; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        if (lane == 0) s_max = x;
    }
    sync_all(ranks);
    last = s_max;
    for (int r = 0; r < ranks; ++r)
        if (r != rank) last = max(last, ld_cluster_s32(cluster_addr(&s_max, r)));
    const Protect pr{static_cast<int>(max(static_cast<int64_t>(last) - p.recent, static_cast<int64_t>(-1))), p.sink};

    const bool held = per * kWarps <= key_cap, held_low = (warp + 1) * per <= low_cap;
    uint16_t *my = s_key + warp * per, *my_low = s_low + warp * per;
    // halves of the lane's eight keys from row s on
    auto upper = [&](int s) { return held ? *reinterpret_cast<const uint4*>(my + (s - lo)) : remade(w_in, p_in, s, pr, 16); };
    auto lower = [&](int s) { return held_low ? *reinterpret_cast<const uint4*>(my_low + (s - lo)) : remade(w_in, p_in, s, pr, 0); };
    // of the eight rows from s on: bits of those below x
    auto bits_below = [](int s, int x) -> uint32_t { return x <= s ? 0u : x - s >= 8 ? 0xFFu : (1u << (x - s)) - 1; };

    // the warp's list, where it has one: offsets of its rows from lo, and their keys
    int listed = -1;
    uint32_t* my_list = nullptr;

    // ---- the M-th largest key, from the top; bits 31..21, 20..16, 15..5, 4..0
    uint32_t prefix = 0, T = 0;
    int need = M, ties = 0;
    bool whole = false;        // every key from T + 1 on stays, no ties
    Rows8 r;
    if (lo + 8 * lane < hi) load_rows(w_in, p_in, lo + 8 * lane, r);
    for (int r0 = lo; r0 < hi; r0 += kEvStep) {
        const int s = r0 + 8 * lane;
        Rows8 next;
        if (s + kEvStep < hi) load_rows(w_in, p_in, s + kEvStep, next);       // the next step's, early
        if (s < hi) {
            const uint32_t in = bits_below(s, hi);
            uint32_t t[8];
            keys_of(pr, r, t);
            if (held) *reinterpret_cast<uint4*>(my + (s - lo)) = halves(t, 16);
            if (held_low) *reinterpret_cast<uint4*>(my_low + (s - lo)) = halves(t, 0);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if ((in >> e) & 1) atomicAdd(s_hist + (t[e] >> 21), 1);
            // the rows below the budget go to buffers of their own now; those given up are written over by
            // the rows that move there
            if (copy_w) copy_below<float4>(p.weight_out + base + s, r.w0, r.w1, M - s);
            if (copy_p) copy_below<int4>(p.position_out + base + s, r.p0, r.p1, M - s);
        }
        r = next;
    }
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 16 : pass == 2 ? 5 : 0, bins = (pass & 1) ? 32 : kEvBins;
        int* hist = s_hist + (pass == 0 ? 0 : pass == 1 ? 2 * kEvBins : pass == 2 ? kEvBins : 2 * kEvBins + 32);
        if (pass > 0 && listed >= 0) {
            for (int e = lane; e < listed; e += 32) {
                const uint32_t k = my_list[e];
                if ((k >> (shift + ((pass & 1) ? 5 : 11))) == prefix) atomicAdd(hist + ((k >> shift) & (bins - 1)), 1);
            }
        } else if (pass > 0) {
#pragma unroll 1
            for (int s = lo + 8 * lane; s < hi; s += kEvStep) {
                const uint4 up = upper(s);
                uint32_t same = bits_below(s, hi);
                if (pass == 1) same &= mark(up, [&](uint32_t t) { return (t >> 5) == prefix; });
                else same &= mark(up, [&](uint32_t t) { return t == (pass == 2 ? prefix : prefix >> 11); });
                if (!same) continue;
                const uint4 low = pass == 1 ? up : lower(s);
                for (; same; same &= same - 1) {
                    const uint32_t l = half_of(low, __ffs(same) - 1);
                    if (pass == 2) atomicAdd(hist + (l >> 5), 1);
                    else if (pass == 1 || (l >> 5) == (prefix & (kEvBins - 1))) atomicAdd(hist + (l & 31), 1);
                }
            }
        }
        sync_all(ranks);
        // counts from the top: thread t holds kEach bins, the uppermost first
        int cnt[kEach], mine = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) cnt[e] = 0;
        const int top = bins - 1 - kEach * tid;
        if (top >= 0) {
#pragma unroll
            for (int e = 0; e < kEach; e += 4) {
                const int4 own = *reinterpret_cast<const int4*>(hist + top - 3 - e);
                cnt[e] = own.w, cnt[e + 1] = own.z, cnt[e + 2] = own.y, cnt[e + 3] = own.x;
                for (int r = 0; r < ranks; ++r)
                    if (r != rank) {
                        const int4 v = ld_cluster_v4(cluster_addr(hist + top - 3 - e, r));
                        cnt[e] += v.w, cnt[e + 1] += v.z, cnt[e + 2] += v.y, cnt[e + 3] += v.x;
                    }
                mine += cnt[e] + cnt[e + 1] + cnt[e + 2] + cnt[e + 3];
            }
        }
        int above = excl_scan(mine, lane);
        if (lane == 31) s_scan[warp] = above + mine;
        __syncthreads();
        above += __reduce_add_sync(0xffffffffu, lane < warp ? s_scan[lane % kWarps] : 0);
        if (above < need && above + mine >= need) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
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
        // Of the unit's rows, M - need + inside have uppermost bits that reach the threshold's.  Where
        // those are few, a warp behind the budget lists its own: an offset of two bytes where their keys
        // were, and a key of four, in the two bytes that each of its rows has.
        if (pass == 0 && held && lo >= M && hi > lo && 4 * static_cast<int64_t>(M - need + inside) <= n) {
            listed = 0;
            bool room = true;
#pragma unroll 1
            for (int r0 = lo; r0 < hi && room; r0 += kEvStep) {       // offsets go where keys were read already
                const int s = r0 + 8 * lane;
                uint32_t some = 0;
                if (s < hi) some = mark(upper(s), [&](uint32_t t) { return (t >> 5) >= prefix; }) & bits_below(s, hi);
                int at = excl_scan(__popc(some), lane);
                const int all = __shfl_sync(0xffffffffu, at + __popc(some), 31);
                at += listed;
                listed += all;
                room = 3 * listed <= per;
                __syncwarp();
                for (; some && room; some &= some - 1) my[at++] = static_cast<uint16_t>(s + __ffs(some) - 1 - lo);
                __syncwarp();
            }
            if (room) {
                my_list = reinterpret_cast<uint32_t*>(my + per) - listed;
                for (int e = lane; e < listed; e += 32) {
                    const int row = lo + my[e];
                    my_list[e] = pr.key(w_in[row], p_in[row]);
                }
            } else {            // they crowd in this warp's rows: its keys again
                listed = -1;
#pragma unroll 1
                for (int s = lo + 8 * lane; s < hi; s += kEvStep)
                    *reinterpret_cast<uint4*>(my + (s - lo)) = remade(w_in, p_in, s, pr, 16);
            }
            __syncwarp();
        }
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
        gt = tie = 0;
        if (s >= hi) return;
        const uint4 up = upper(s);
        const uint32_t in = bits_below(s, hi), t16 = T16, t0 = T & 0xFFFFu;
        gt = in & mark(up, [&](uint32_t t) { return t > t16; });
        uint32_t same = in & mark(up, [&](uint32_t t) { return t == t16; });
        if (!same || upper_alone) return;
        const uint4 low = lower(s);
        for (; same; same &= same - 1) {
            const int e = __ffs(same) - 1;
            const uint32_t l = half_of(low, e);
            if (l > t0) gt |= 1u << e;
            else if (l == t0 && !whole) tie |= 1u << e;
        }
    };

    // ---- twice over the rows: count those of each kind per warp (given up and tied below M, kept for
    // sure and tied behind), and once it is known where each warp's begin in the lists, write them
    int n_low = 0, n_tl = 0, n_gt = 0, n_th = 0, tie_at = 0, hole_at = 0, src_at = 0;
    int32_t* to = p.to + static_cast<int64_t>(u) * p.list_cap;
    int32_t* of = p.of + static_cast<int64_t>(u) * p.list_cap;
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        for (int e0 = 0; e0 < listed; e0 += 32) {
            const bool in = e0 + lane < listed;
            const uint32_t k = in ? my_list[e0 + lane] : 0, below = (1u << lane) - 1;
            const bool tie = in && !whole && k == T;
            const uint32_t tb = __ballot_sync(0xffffffffu, tie);
            if (turn == 0) {
                n_gt += in && k > T ? 1 : 0;
                n_th += tie ? 1 : 0;
                continue;
            }
            const bool kept = in && (k > T || (tie && tie_at + __popc(tb & below) < ties));
            const uint32_t kb = __ballot_sync(0xffffffffu, kept);
            const int at = src_at + __popc(kb & below);
            if (kept && at < p.list_cap) of[at] = lo + my[e0 + lane];
            tie_at += __popc(tb);
            src_at += __popc(kb);
        }
#pragma unroll 1
        for (int r0 = listed < 0 ? lo : hi; r0 < hi; r0 += kEvStep) {
            const int s = r0 + 8 * lane;
            uint32_t kept, tie;
            grade(s, kept, tie);
            const uint32_t in = bits_below(s, hi), low = bits_below(s, M);
            if (turn == 0) {
                n_low += __popc(in & low & ~(kept | tie));
                n_tl += __popc(low & tie);
                n_gt += __popc(~low & kept);
                n_th += __popc(~low & tie);
                continue;
            }
            if (__any_sync(0xffffffffu, tie)) {
                int t = tie_at + excl_scan(__popc(tie), lane);
                tie_at += __reduce_add_sync(0xffffffffu, __popc(tie));
                for (; tie; tie &= tie - 1, ++t)
                    if (t < ties) kept |= tie & (0 - tie);
            }
            uint32_t hole = in & low & ~kept, src = kept & ~low;
            if (__any_sync(0xffffffffu, hole | src)) {
                const int both = __popc(hole) | __popc(src) << 16;       // at most 256 of each
                const int at = excl_scan(both, lane);
                const int all = __reduce_add_sync(0xffffffffu, both);
                int ha = hole_at + (at & 0xFFFF), sa = src_at + (at >> 16);
                hole_at += all & 0xFFFF;
                src_at += all >> 16;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int at_e = ha + __popc(hole & ((1u << e) - 1));
                    if (((hole >> e) & 1) && at_e < p.list_cap) to[at_e] = s + e;
                }
                for (; src; src &= src - 1, ++sa)
                    if (sa < p.list_cap) of[sa] = s + __ffs(src) - 1;
            }
        }
        if (turn == 1) break;
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
            const int x = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_cnt[warp][lane] : 0);
            if (lane == 0) s_tot[warp] = x;
        }
        sync_all(ranks);
        if (warp == 0) {
            // what lies in the slices before this one, and in all (rows below M come first in every slice)
            int tie0 = 0, hole0 = 0, src0 = 0, tie_sum = 0, hole_sum = 0, src_sum = 0;
            for (int r = 0; r < ranks; ++r) {
                if (r == rank) tie0 = tie_sum, hole0 = hole_sum, src0 = src_sum;
                int v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = r == rank ? s_tot[e] : ld_cluster_s32(cluster_addr(&s_tot[e], r));
                const int left = max(0, ties - tie_sum), kl = min(v[1], left), kh = min(v[3], left - kl);
                hole_sum += v[0] + v[1] - kl;
                src_sum += v[2] + kh;
                tie_sum += v[1] + v[3];
            }
            if (lane == 0) s_moves = min(min(hole_sum, src_sum), p.list_cap);
            const int w = lane % kWarps;
            const bool own = lane < kWarps;
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
        }
        sync_all(ranks);       // nor does a CTA leave while another reads its counts
        tie_at = s_tie[warp];
        hole_at = s_hole[warp];
        src_at = s_src[warp];
    }

    if (kMove) {
        sync_all(ranks);       // the lists are whole
        move_rows(p, u, s_moves, rank * kWarps + warp, ranks * kWarps);
    } else if (rank == 0 && tid == 0) {
        p.count[u] = s_moves;
    }
}

constexpr int kMvThreads = 128;
__global__ void __launch_bounds__(kMvThreads) k_evict_move(const __grid_constant__ EvictParams p, int parts) {
    pdl_wait();
    const int u = blockIdx.x / parts, part = blockIdx.x % parts;
    if (p.lens_out == p.c.lens && u % p.c.H == 0 && part == 0 && threadIdx.x == 0) p.lens_out[u / p.c.H] = p.new_len[u / p.c.H];
    move_rows(p, u, min(p.count[u], p.list_cap), part * (kMvThreads / 32) + (threadIdx.x >> 5), parts * (kMvThreads / 32));
}

__global__ void k_evict_lens(const __grid_constant__ EvictParams p) {
    pdl_wait();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < p.c.batch) p.lens_out[b] = __ldcg(p.new_len + b);
}

int launch_evict(const EvictParams& p, int nsm, cudaStream_t s) {
    const int U = p.c.batch * p.c.H;
    // Many short units of which few rows can move go to narrow CTAs, of which an SM holds eight, or as their
    // keys take 25 to 33 KB in rooms of 2048 to 4096 rows, eight to six (2048 units of 501 rows, one of them
    // given up: 29.4 us against 79.9; of 2049 rows: 55.0 against 98.0; but 66.6 against 61.1 for 320 units of
    // 3000 rows with 952 given up).  The others go to as many CTAs as the
    // device holds at once (two per SM), and no fewer than the keys need to stay in shared memory.  A
    // slice of under one grain would leave warps idle.
    const bool few = p.list_cap <= kEvFew, narrow = few && U > 2 * nsm && p.c.cap <= kEvShort;
    const int threads = narrow ? kEvNarrow : kEvWide, grain = grain_of(threads);
    int ranks = 1;
    while (!narrow && ranks < 8 && p.c.cap > ranks * grain && (U * ranks <= nsm || p.c.cap / ranks > kEvKeys)) ranks *= 2;
    const int64_t slice = (static_cast<int64_t>(p.c.cap) + ranks - 1) / ranks;
    const int64_t keys = (slice + grain - 1) / grain * grain;
    const int key_cap = static_cast<int>(keys < kEvKeys ? keys : kEvKeys);
    // the lower halves only where a slice is short: what they take of shared memory is taken from L1
    // (128K rows: 68 us with the upper halves alone, 79 with some of the lower ones)
    const int low_cap = 2 * key_cap <= kEvKeys ? key_cap : 0;
    const int smem = kEvHist * 4 + (key_cap + low_cap) * 2;
    auto kernel = narrow ? k_evict<kEvNarrow, true> : few ? k_evict<kEvWide, true> : k_evict<kEvWide, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvHist * 4 + kEvKeys * 2) != cudaSuccess ||
        launch_first(kernel, static_cast<unsigned>(U) * ranks, threads, smem, ranks, 0, s, p, ranks, key_cap, low_cap) !=
            cudaSuccess)
        return -1;
    cudaError_t e = cudaSuccess;
    if (!few) {
        // CTAs per unit for the rows that move
        const int rows = kMvThreads;
        int64_t parts = (static_cast<int64_t>(p.list_cap) + rows - 1) / rows;
        const int64_t most = (16 * nsm + U - 1) / U;
        if (parts > most) parts = most;
        e = launch_pdl(k_evict_move, dim3(static_cast<unsigned>(parts * U)), dim3(kMvThreads), 0, s, p, static_cast<int>(parts));
    } else if (p.lens_out == p.c.lens) {
        e = launch_pdl(k_evict_lens, dim3((p.c.batch + 127) / 128), dim3(128), 0, s, p);
    }
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? 0 : -1;
}

cudaError_t evict_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
