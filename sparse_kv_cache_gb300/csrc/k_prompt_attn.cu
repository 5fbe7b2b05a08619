// Attention of many new tokens per sequence over its paged cache (shadowkv_paged_prompt_attention): bf16, causal, whole
// or through a window with first rows.
//
// out = softmax(scale q.K^T).V, row r seeing rows j <= r with (window) j > r - window or j < sink.  4 d flops
// for every (token, query head, row seen): the fifth-generation tensor cores bound it where tokens are many, memory
// where they are few.
//
// A CTA takes 256 query rows of one KV head -- 2 x tq tokens times its G query heads, two halves of 128 rows with an
// accumulator each -- and walks the tiles of 128 rows that any of them sees.  Both halves use each tile of keys
// and values: with one half the L2 would have to deliver 64 bytes per clock to every SM, more than it has.
//   8 warps      a thread per query row: scores from tensor memory into registers, softmax, P back
//   one          page ids, TMA of queries, keys and values (pages are boxes of a tensor map)
//   one          S = Q.K^T (both operands in shared memory), O += P.V (P in tensor memory, V as it lies in the
//                pages: its dimension is the one along the rows of a page, so the operand is MN-major)
//   two          values of tiles at an edge: rows that no query sees become zeros, and whether an element that is
//                not finite is among the others, which must not meet a probability of zero
// While one half's warps form its probabilities, the tensor cores have the other half's two products.  Few tokens take
// one half and two CTAs to an SM; few units a part of their tiles each, joined by k_prompt_merge.
//
// The tensor memory holds S of both halves and O of both, 512 columns; P takes the place of its S.  A half's
// products are issued in the order P(j).V, Q.K(j+1): they execute in that order, so what says that the second
// is done says it of the first too, and a thread that has the scores of tile j + 1 may rescale O.
//
// Probabilities are rounded to bf16 once, off by 2^-9 of each on average: as far as the result's own rounding moves it
// (two terms would double the second product).  They are 2^-8 over the table's rows of a probability that is not
// normalised, in the exponent, so that no sum of values passes the type's largest; O and the sums of
// probabilities, in fp32, take the same factor, and it cancels.
//
// Measured (8 KV heads of 4 query heads, d = 128; cuBLAS reaches 1900 TFLOP/s in bursts, 1695 for seconds under the power
// limit): a prompt of 32K tokens 6.3 to 6.4 ms by machine, 1365 to 1397 TFLOP/s; through a window of 4096 1.70 ms, 1215; 4 prompts
// of 4096 463 us, 1187; chunks of 13K tokens in all through a window of 1024 302 us, of 10.5 tiles a unit with three at an
// edge; d = 64, 16K tokens 1.37 ms, 804; 8 drafts of 5 tokens over up to 4099 rows 23.5 us.  A half's tile takes its softmax
// about 1690 clocks with 128 dimensions and 1700 with 64 (128 columns in 4 of them each at the exponential unit, 32 a clock to an
// SM) and its products 1024 and 512, which the other half's overlap.  No unit is full (tensor cores 54 % and issue slots 35 %
// of the cycles of 8192 tokens): the chain softmax, P.V, Q.K of each half bounds it.
// Tried: two threads to a row (7.1 ms for 32K: 20 warps to issue for), the first half of P handed over early (no
// difference), six warps to look at values (505 us for the 4 prompts, 483 then: they wait at the others' cost), CTAs that go
// through many units (517 us, 483 then: what a unit's start and end take is hidden, but the units fall unevenly).
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

namespace skv {

static __device__ int g_err[2];

constexpr int kPrTile = 128;                   // rows of a tile of keys
constexpr int kPrHalf = 128;                   // query rows of an accumulator
constexpr float kPrSlack = 8.f;                // the base moves when a score passes it by 2^8
constexpr int kPrStages = 2;                   // tiles of keys, and of values, on their way or in use, at most
constexpr int kPrHold = 1024;                  // tiles after which sums are put by, a power of two
constexpr int kPrMaxSlots = 160;               // places for units that are taken in parts
constexpr int kPrMaxParts = 64;                // of a unit

// One thread of the warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}
// D[tmem] (+)= A[tmem] * B[smem], A 128 x 16 bf16 packed in pairs
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// An operand that is stored along its M or N dimension, 128-byte swizzle: rows of 64 elements, one per k, in
// groups of eight (1024 bytes apart); the next 64 elements lie `next` bytes away.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr, uint32_t next) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(next >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
constexpr uint32_t kBIsMN = 1u << 16;          // instruction descriptor: B is stored along N

#define PR_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define PR_F8(c, v, i) c(v[i]), c(v[i + 1]), c(v[i + 2]), c(v[i + 3]), c(v[i + 4]), c(v[i + 5]), c(v[i + 6]), c(v[i + 7])
#define PR_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
// Columns of this thread's lane, there when the function returns (the wait is in the same statement, so that nothing
// that uses them can come before it).
__device__ __forceinline__ void tmem_get32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : PR_R8(r, 0), PR_R8(r, 8), PR_R8(r, 16), PR_R8(r, 24)
        : "r"(taddr)
        : "memory");
}
// The same in steps: asked for, waited for (tmem_ld_wait), and marked as there, before which nothing uses them.
__device__ __forceinline__ void tmem_ask32(uint32_t taddr, float* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : PR_F8("=f", r, 0), PR_F8("=f", r, 8), PR_F8("=f", r, 16), PR_F8("=f", r, 24)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_have32(float* r) {
    asm volatile("" : PR_F8("+f", r, 0), PR_F8("+f", r, 8), PR_F8("+f", r, 16), PR_F8("+f", r, 24));
}
// two fp32 products and sums, or sums, in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ uint32_t tmem_get1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(taddr) : "memory");
    return r;
}
__device__ __forceinline__ void tmem_put32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::PR_W8(r, 0), PR_W8(r, 8), PR_W8(r, 16), PR_W8(r, 24),
        "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::PR_W8(r, 0), PR_W8(r, 8),
        "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ what a CTA does

// The unit of a CTA: tokens `tok` .. of the call, at rows row0 .. of sequence b; its tiles are positions
// lo .. hi of the list [0, ts), [tw, ..) of tiles.
struct PrUnit {
    int b, h, tok, ntok, row0, ts, tw, lo, hi;
    __device__ __forceinline__ int tile(int pos) const { return pos < ts ? pos : tw + (pos - ts); }
};
// Rows that the tokens first .. last of a sequence see.
struct PrSees {
    int first, last, window, sink;      // window 0: all up to one's own
    // whether some of them sees one of the rows a .. z, and whether all of them see all those rows
    __device__ __forceinline__ bool any(int a, int z) const {
        return a <= last && (window == 0 || a < sink || z > first - window);
    }
    __device__ __forceinline__ bool all(int a, int z) const {
        return z <= first && (window == 0 || a > last - window || z < sink);
    }
};
__device__ __forceinline__ PrSees sees(const PromptParams& p, const PrUnit& u, int half) {
    const int from = half * p.tq, to = min(u.ntok, from + p.tq);       // tokens of the unit: half 2 is both
    return half == 2 ? PrSees{u.row0, u.row0 + u.ntok - 1, p.c.window, p.c.sink}
                     : PrSees{u.row0 + from, u.row0 + to - 1, p.c.window, p.c.sink};
}
// The tiles of which some tokens see all rows: up to `upto`, and of those from `from` on or up to `sink`.
struct PrWhole {
    int upto, from, sink;
    __device__ __forceinline__ bool has(int tile) const { return tile <= upto && (tile >= from || tile <= sink); }
};
__device__ __forceinline__ PrWhole whole(const PrSees& s) {
    // of tile t, rows 128 t .. 128 t + 127: the last is no later than the first token's own, the first within the last
    // token's window (shifts round down)
    return PrWhole{(s.first - (kPrTile - 1)) >> 7, s.window ? ((s.last - s.window) >> 7) + 1 : INT32_MIN, (s.sink - kPrTile) >> 7};
}

// The place of a sequence's first unit: from there on places are its, and have units as long as there are tokens.
__device__ __forceinline__ int first_place(const PromptParams& p, int start, int b) { return start / p.unit_tokens + b; }
// The unit `skip` places behind sequence b's first one, with all its tiles; ntok 0 if there is none.  The sequence has
// tokens t0 .. t1 and `len` rows.
__device__ __forceinline__ PrUnit unit_at(const PromptParams& p, int64_t skip, int b, int t0, int t1, int len) {
    PrUnit u{};
    u.b = b;
    if (t0 < 0 || t1 < t0 || t1 > p.tokens) {
        set_err(g_err, DEV_ERR_BOUNDS, 913);
        return u;
    }
    skip *= p.unit_tokens;
    if (skip < 0 || skip >= t1 - t0) return u;
    u.tok = t0 + static_cast<int>(skip);
    u.ntok = min(p.unit_tokens, t1 - u.tok);
    u.row0 = len - (t1 - u.tok);
    // tiles: those of the first rows, then from the first token's window to the last token
    const int last = u.row0 + u.ntok - 1;
    if (last >= 0) {
        const int upto = last / kPrTile;
        u.tw = p.c.window ? max(0, u.row0 - p.c.window + 1) / kPrTile : 0;
        u.ts = p.c.window ? min(u.tw, (p.c.sink + kPrTile - 1) / kPrTile) : 0;
        u.hi = u.ts + upto - u.tw + 1;
    }
    return u;
}
// By one warp: which unit a block has.
__device__ __forceinline__ PrUnit find_unit(const PromptParams& p, int64_t block) {
    // the last tokens of a sequence see most: their units start first
    const int64_t place = p.slots - 1 - block / p.c.H;
    const int b = find_sequence(p.start, p.c.batch, place, [&](int s, int i) { return static_cast<int64_t>(first_place(p, s, i)); });
    const int t0 = __ldcg(p.start + b);
    PrUnit u = unit_at(p, place - first_place(p, t0, b), b, t0, __ldcg(p.start + b + 1), rows_of(p.c, b, g_err, 912));
    u.h = static_cast<int>(block % p.c.H);
    return u;
}

// Few units: parts of a unit's tiles each, all of about as many tiles, whichever unit they are of -- which only the device
// can tell.  (16 sequences of 5 tokens over 1 to 16000 rows: with as many parts for each unit 139 us.)
struct PrParts {
    int start[kPrMaxSlots + 1], len[kPrMaxSlots];
    int place[kPrMaxSlots];        // a sequence's first
    PrUnit unit[kPrMaxSlots];      // of a place
    int first[kPrMaxSlots + 1];    // its first part
};
// the last of n numbers that do not fall which is at most x, 0 if there is none
__device__ __forceinline__ int last_upto(const int* v, int n, int x) {
    int lo = 0;
    for (int hi = n; hi - lo > 1;) {
        const int mid = (lo + hi) / 2;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// By one warp: what a block has, its `part` of all parts.  (All else waits for it: 4100 clocks, find_unit's 1900.)
__device__ __forceinline__ PrUnit find_part(const PromptParams& p, PrParts& s, int part) {
    const int lane = threadIdx.x & 31, slots = static_cast<int>(p.slots), batch = p.c.batch;
#pragma unroll 1
    for (int i = lane; i <= batch; i += 32) {
        const int t = __ldcg(p.start + i), n = __ldcg(p.c.lens + min(i, batch - 1));
        s.start[i] = t;
        if (i < batch) {
            s.len[i] = rows_in(p.c, n, g_err, 912);
            s.place[i] = first_place(p, t, i);
        }
    }
    __syncwarp();
    unsigned total = 0, longest = 0, live = 0;
#pragma unroll 1
    for (int i = lane; i < slots; i += 32) {
        const int b = last_upto(s.place, batch, i);
        const PrUnit u = unit_at(p, i - s.place[b], b, s.start[b], s.start[b + 1], s.len[b]);
        s.unit[i] = u;
        total += u.hi;
        longest = max(longest, static_cast<unsigned>(u.hi));
        live += u.ntok > 0;
    }
    total = __reduce_add_sync(0xffffffffu, total);
    longest = __reduce_max_sync(0xffffffffu, longest);
    live = __reduce_add_sync(0xffffffffu, live);
    // A unit of n tiles has 1 + (n - 1) / most parts (one where it sees nothing), so all have p.parts at most: each of
    // `live` units one, and total / most further ones.
    const float most = fmaxf(2.f, fmaxf(__fdividef(total, p.parts - live), longest * (1.f / kPrMaxParts))), inv = __fdividef(1.f, most);
    int at = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < slots; i0 += 32) {
        const int i = i0 + lane;
        const int mine = i >= slots || s.unit[i].ntok == 0 ? 0 : 1 + min(static_cast<int>(max(s.unit[i].hi - 1, 0) * inv), kPrMaxParts - 1);
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += x;
        }
        if (i < slots) s.first[i] = at + upto - mine;
        at += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) s.first[slots] = at;
    __syncwarp();
    if (part >= at) return PrUnit{};
    const int place = last_upto(s.first, slots, part);
    PrUnit u = s.unit[place];
    const int from = part - s.first[place], parts = s.first[place + 1] - s.first[place];
    const float each = __fdividef(u.hi, parts);
    u.lo = static_cast<int>(from * each);
    if (from + 1 < parts) u.hi = static_cast<int>((from + 1) * each);
    return u;
}

// A CTA's form: two halves, one CTA to an SM; or where a unit's tokens are few one half, two CTAs to an SM, whose tiles
// and softmax take turns (8 sequences of 5 tokens over 4099 rows: 32 us, and 40 with two halves of which one is empty, both
// with parts less even than now).
template <int D, int kHalves_>
struct PrForm {
    static constexpr int kHalves = kHalves_, kSoft = 4 * kHalves, kThreads = 32 * (kSoft + 4), kCtas = 3 - kHalves;
    static constexpr int kStages = kHalves == 2 || D == 64 ? 2 : 1;
    // registers of a thread: what the launch gives, then those of a thread per row, and of the others
    static constexpr int kRegs = kHalves == 2 ? 168 : 128, kRegsMore = kHalves == 2 ? 208 : 200, kRegsLess = kHalves == 2 ? 88 : 56;
    static_assert(32 * kSoft * kRegsMore + 128 * kRegsLess <= kThreads * kRegs && kCtas * kThreads * kRegs <= 65536, "");
    static constexpr int kColumns = 256 * kHalves;                   // of the tensor memory: S, then O
    static constexpr int kParts = D / 64;                            // 64 dimensions of 128 rows: 16 KB
    static constexpr int kTileBytes = kParts * 16384;
    static constexpr int kQ = 0, kK = kHalves * kTileBytes, kV = kK + kStages * kTileBytes, kBytes = kV + kStages * kTileBytes;
};
struct PrShared {
    uint64_t q_full, k_full[kPrStages], k_empty[kPrStages], v_full[kPrStages], v_ok[kPrStages], v_empty[kPrStages];
    uint64_t s_full[2], p_full[2], o_full[2];
    PrUnit unit;
    PrWhole whole[3];          // of either half's tokens, and of all
    uint32_t tmem;
    int dead;
    int2 begun;                // tiles whose keys (x) and values (y) were asked for
    int place[2];              // of g_put_by, for either half; -1: none
    int absent[4];             // per tile (mod 4): groups of eight rows whose page is out of range or not looked at
    int wild[kPrStages][2];    // a tile at an edge has values that are not finite (what each of the two warps found)
    uint64_t given_up;         // the products that were under way
    __device__ __forceinline__ bool is_wild(int s) const {
        const volatile int* w = wild[s];
        return (w[0] | w[1]) != 0;
    }
};

// Where sums of whole units are put by: two places for every SM, a CTA of two halves or two CTAs of one.
constexpr int kPrPlaces = 2 * 160;
static __device__ float g_put_by[kPrPlaces * kPrHalf * 128];
static __device__ float2 g_put_by_stat[kPrPlaces * kPrHalf];
static __device__ int g_in_use[kPrPlaces];

// ------------------------------------------------------------------ the roles

// By one thread: a place for each half, or -1 where there is none within the limit, and the unit's results are NaN.
__device__ __noinline__ void pr_take_places(PrShared& sh, int halves) {
    uint32_t sm;
    asm volatile("mov.u32 %0, %%smid;" : "=r"(sm));
    const unsigned long long since = globaltimer();
    for (int x = 0; x < halves; ++x)
        for (int i = 2 * sm; sh.place[x] < 0; ++i) {
            if (atomicCAS(g_in_use + i % kPrPlaces, 0, 1) == 0) sh.place[x] = i % kPrPlaces;
            else if (globaltimer() - since > kWaitLimitNs) {
                return;
            }
        }
    __threadfence();
}
// By one thread, of the warp that loads the rest.
template <int D, class L>
__device__ __forceinline__ void pr_load_queries(const PromptParams& p, const CUtensorMap* mq, PrShared& sh, const PrUnit& u, uint8_t* base) {
    const int halves = u.ntok > p.tq ? 2 : 1;
    mbar_arrive_expect_tx(&sh.q_full, halves * L::kParts * p.tq * p.G * 128);
    for (int x = 0; x < halves; ++x)
        for (int i = 0; i < L::kParts; ++i)
            tma_load_3d(smem_u32(base) + L::kQ + x * L::kTileBytes + i * 16384, mq, i * 64, u.h * p.G, u.tok + x * p.tq, &sh.q_full);
}
// By one warp: the rows behind the last token's heads (G does not divide 128) are zeros.  Nothing is made of their scores, but
// a warp's bases move together, so what lay there before would have a part in how other rows are rounded.
template <int D, class L>
__device__ __forceinline__ void pr_clear_queries(const PromptParams& p, uint8_t* base) {
    const int from = p.tq * p.G, words = (kPrHalf - from) * 8;         // of 16 bytes, of 64 dimensions
    for (int i = threadIdx.x & 31; i < L::kHalves * L::kParts * words; i += 32)
        *reinterpret_cast<uint4*>(base + L::kQ + i / words * 16384 + from * 128 + i % words * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
}
template <int D, class L>
__device__ void pr_load(const PromptParams& p, const CUtensorMap* mk, const CUtensorMap* mv, PrShared& sh,
                        uint8_t* base) {
    const PrUnit u = sh.unit;
    const PrSees both = sees(p, u, 2);
    const int lane = threadIdx.x & 31;
    const int box = min(kPrTile, 1 << p.c.lg), boxes = kPrTile / box, mask = (1 << p.c.lg) - 1;
    const uint32_t at = smem_u32(base);
    const int j = lane % boxes, part = lane / boxes;
    int keys = 0, vals = 0;
    for (int pos = u.lo; pos < u.hi; ++pos) {
        const int n = pos - u.lo, s = n % L::kStages, row = u.tile(pos) * kPrTile;
        const uint32_t parity = (n / L::kStages + 1) & 1;
        int page = -1;
        if (lane < boxes && both.any(row + lane * box, row + lane * box + box - 1)) page = page_of(p.c, u.b, row + lane * box, g_err, 914);
        const uint32_t gone = __ballot_sync(0xffffffffu, page < 0);
        // (a page beyond the pool is read as zeros)
        const int z = __shfl_sync(0xffffffffu, page < 0 ? static_cast<int>(p.c.n_pages) : page, j);
        const int in_page = (row + j * box) & mask;
        const uint32_t to = at + s * L::kTileBytes + part * 16384 + j * box * 128;
        if (!warp_wait_or_give_up(&sh.k_empty[s], parity, &sh.dead)) break;
        if (lane == 0) {
            int absent = 0;
            for (int i = 0; i < 16; ++i) absent |= (gone >> (i * 8 / box) & 1) << i;
            sh.absent[n & 3] = absent;
            mbar_arrive_expect_tx(&sh.k_full[s], L::kTileBytes);
        }
        __syncwarp();
        if (part < L::kParts) tma_load_4d(to + L::kK, mk, part * 64, in_page, u.h, z, &sh.k_full[s]);
        keys = n + 1;
        if (!warp_wait_or_give_up(&sh.v_empty[s], parity, &sh.dead)) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.v_full[s], L::kTileBytes);
        __syncwarp();
        if (part < L::kParts) tma_load_4d(to + L::kV, mv, part * 64, in_page, u.h, z, &sh.v_full[s]);
        vals = n + 1;
    }
    if (lane == 0) sh.begun = make_int2(keys, vals);
}

template <int D, class L>
__device__ void pr_multiply(const PromptParams& p, PrShared& sh, uint8_t* base) {
    const PrUnit u = sh.unit;
    const PrWhole calm = sh.whole[2];
    const uint32_t at = smem_u32(base), tmem = sh.tmem;
    const int halves = u.ntok > p.tq ? 2 : 1, tiles = u.hi - u.lo;
    if (tiles <= 0) return;
    constexpr uint32_t qk = idesc_bf16_f32(kPrHalf, kPrTile), pv = idesc_bf16_f32(kPrHalf, D) | kBIsMN;
    // The whole warp comes this way and one thread of it issues: operands that are the warp's stay in uniform
    // registers (with one thread alone on the path an instruction took 115 clocks to issue, twice its work).
    const bool mine = elect_one();
    const uint64_t q_desc = smem_desc_sw128(at + L::kQ), k_desc = smem_desc_sw128(at + L::kK), v_desc = smem_desc_mn(at + L::kV, 16384);
    auto scores = [&](int x, int n) {
        const uint64_t q = q_desc + x * (L::kTileBytes >> 4), k = k_desc + (n % L::kStages) * (L::kTileBytes >> 4);
        if (!mine) return;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            constexpr int kPart = 16384 >> 4, kStep = 32 >> 4;
            tc_mma_bf16(tmem + x * 128, q + (i / 4) * kPart + (i % 4) * kStep, k + (i / 4) * kPart + (i % 4) * kStep, qk, i > 0);
        }
        tc_commit(&sh.s_full[x]);
    };
    auto values = [&](int x, int n) {
        const uint64_t v = v_desc + (n % L::kStages) * (L::kTileBytes >> 4);
        if (!mine) return;
#pragma unroll
        for (int i = 0; i < kPrTile / 16; ++i)
            tc_mma_bf16_ts(tmem + 128 * L::kHalves + x * 128, tmem + x * 128 + i * 8, v + i * (2048 >> 4), pv, n % kPrHold > 0 || i > 0);
    };
    auto told = [&](uint64_t* bar, uint32_t parity) { return warp_wait_or_give_up(bar, parity, &sh.dead); };
    auto commit = [&](uint64_t* bar) {
        if (mine) tc_commit(bar);
    };
    if (!told(&sh.q_full, 0) || !told(&sh.k_full[0], 0)) return;
    for (int x = 0; x < halves; ++x) scores(x, 0);
    commit(&sh.k_empty[0]);
    for (int n = 0; n < tiles; ++n) {
        const int s = n % L::kStages, next = (n + 1) % L::kStages;
        if (!told(&sh.v_ok[s], (n / L::kStages) & 1)) return;
        const bool wild = !calm.has(u.tile(u.lo + n)) && sh.is_wild(s);
        for (int x = 0; x < halves; ++x) {
            if (!told(&sh.p_full[x], n & 1)) return;
            tc_fence_after();
            if (!wild) values(x, n);       // otherwise the row's threads have done it
            if (x == halves - 1) commit(&sh.v_empty[s]);
            if (n + 1 < tiles) {
                if (x == 0 && !told(&sh.k_full[next], ((n + 1) / L::kStages) & 1)) return;
                scores(x, n + 1);
                if (x == halves - 1) commit(&sh.k_empty[next]);
            } else {
                commit(&sh.o_full[x]);
            }
        }
    }
}

template <int D, class L>
__device__ void pr_look(const PromptParams& p, PrShared& sh, uint8_t* base) {
    const PrUnit u = sh.unit;
    const PrSees both = sees(p, u, 2);
    const PrWhole calm = sh.whole[2];
    const int t = threadIdx.x - 32 * (L::kSoft + 2), warp = t >> 5;   // of 64
    for (int n = 0; n < u.hi - u.lo; ++n) {
        const int s = n % L::kStages, tile = u.tile(u.lo + n);
        if (!warp_wait_or_give_up(&sh.v_full[s], (n / L::kStages) & 1, &sh.dead)) return;
        if (!calm.has(tile)) {
            uint32_t some = 0;
            uint8_t* v = base + L::kV + s * L::kTileBytes;
            for (int part = 0; part < L::kParts; ++part)
#pragma unroll 4
                for (int r = t >> 3; r < kPrTile; r += 8) {
                    uint4* w = reinterpret_cast<uint4*>(v + part * 16384 + r * 128 + (t & 7) * 16);
                    const int row = tile * kPrTile + r;
                    if (!both.any(row, row)) {
                        *w = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    const uint4 x = *w;
                    // an exponent of ones carries into the bit above it
                    some |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                            ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
                }
            const bool found = __any_sync(0xffffffffu, some & 0x80008000u);
            if ((t & 31) == 0) sh.wild[s][warp] = found;
            fence_proxy_async_smem();
        }
        __syncwarp();
        if ((t & 31) == 0) mbar_arrive(&sh.v_ok[s]);
    }
}

// O of this thread's row += P.V on the CUDA cores, element by element that the row sees: for a tile at an edge with
// values that are not finite.
template <int D>
__device__ __noinline__ void pr_by_hand(uint32_t o_tmem, uint32_t p_tmem, const uint8_t* v, bool first) {
    for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t raw[32];
        float o[32];
        if (!first) tmem_get32(o_tmem + d0, raw);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = first ? 0.f : __uint_as_float(raw[i]);
        for (int j = 0; j < kPrTile; ++j) {
            const uint32_t two = tmem_get1(p_tmem + j / 2);
            const float w = j & 1 ? bf16hi(two) : bf16lo(two);
            const uint8_t* row = v + (d0 / 64) * 16384 + j * 128;
            if (w != 0.f) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float x[8];
                    load8(reinterpret_cast<const __nv_bfloat16*>(row + (((d0 / 8 + c) & 7) ^ (j & 7)) * 16), x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[8 * c + i] = fmaf(w, x[i], o[8 * c + i]);
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) raw[i] = __float_as_uint(o[i]);
        tmem_put32(o_tmem + d0, raw);
    }
    tmem_put_wait();
}

// The tensor cores cut a sum off at every 16 rows it takes in, so what it loses grows with the rows.  Every kPrHold tiles O and the
// sum of probabilities of this thread's row are therefore put by, with the base that they were formed with, and begin again at
// zero.  (Equal values in 16M rows: off by 16 % without.)  A part of a unit has its place in the workspace for that, and a whole
// unit takes one of g_put_by while it runs: there are as many as CTAs of either form can be on the device.
// The last time they go back to O instead.  Returns the sum of probabilities.
enum class PrHold { kFirst, kNext, kLast };
template <int D>
__device__ __noinline__ float pr_hold(uint32_t o_tmem, float* place, float2* stat, float m, float l, PrHold time) {
    const float2 was = time == PrHold::kFirst ? make_float2(m, 0.f) : *stat;
    const float w = was.y == 0.f ? 0.f : exp2_fast(was.x - m);
    for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t raw[32];
        tmem_get32(o_tmem + d0, raw);
        if (w != 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 y = reinterpret_cast<const float4*>(place + d0)[i];
                raw[4 * i] = __float_as_uint(fmaf(y.x, w, __uint_as_float(raw[4 * i])));
                raw[4 * i + 1] = __float_as_uint(fmaf(y.y, w, __uint_as_float(raw[4 * i + 1])));
                raw[4 * i + 2] = __float_as_uint(fmaf(y.z, w, __uint_as_float(raw[4 * i + 2])));
                raw[4 * i + 3] = __float_as_uint(fmaf(y.w, w, __uint_as_float(raw[4 * i + 3])));
            }
        }
        __syncwarp();
        if (time == PrHold::kLast) {
            tmem_put32(o_tmem + d0, raw);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                reinterpret_cast<uint4*>(place + d0)[i] = make_uint4(raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]);
        }
    }
    tmem_put_wait();
    l = fmaf(was.y, w, l);
    *stat = make_float2(m, l);
    return l;
}

// O of this thread's row *= w
template <int D>
__device__ __forceinline__ void pr_rescale(uint32_t o_tmem, float w) {
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t o[32];
        tmem_get32(o_tmem + d0, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * w);
        tmem_put32(o_tmem + d0, o);
    }
}

// the lowest k bits
__device__ __forceinline__ uint32_t lowest(int k) { return k <= 0 ? 0u : 0xFFFFFFFFu >> (32 - min(k, 32)); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int D, class L, bool kParts>
__device__ void pr_softmax(const PromptParams& p, PrShared& sh, uint8_t* base) {
    const PrUnit& u = sh.unit;
    const int half = threadIdx.x >> 7, r = threadIdx.x & 127;
    const int lo = u.lo, tiles = u.hi - lo;
    const int token = half * p.tq + min(r / p.G, p.tq - 1);             // (rows beyond the last token repeat its)
    if (half * p.tq >= u.ntok) return;
    const int row = u.row0 + min(token, u.ntok - 1);
    const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;      // 32 lanes of the tensor memory
    const uint32_t s_at = sh.tmem + lanes + half * 128, o_at = s_at + 128 * L::kHalves;
    const float scale = p.scale_log2;
    const bool falls = scale < 0.f;
    const float none = falls ? CUDART_INF_F : -CUDART_INF_F;             // the product that scores -infinity
    float m = -CUDART_INF_F, l = 0.f;
    bool good = true;
    // this row's place where sums are put by
    auto put_by = [&](PrHold time) {
        const int64_t at = kParts ? static_cast<int64_t>(blockIdx.y * p.c.H + blockIdx.x) * (L::kHalves * kPrHalf) + threadIdx.x
                                  : static_cast<int64_t>(sh.place[half]) * kPrHalf + r;
        return pr_hold<D>(o_at, (kParts ? p.part : g_put_by) + at * D, (kParts ? p.part_stat : g_put_by_stat) + at, m, l, time);
    };
    for (int n = 0; n < tiles; ++n) {
        const int tile = u.tile(lo + n);
        good = warp_wait_or_give_up(&sh.s_full[half], n & 1, &sh.dead);
        if (!good) break;
        tc_fence_after();
        if (n > 0 && n % kPrHold == 0) {
            if (!kParts && sh.place[half] < 0) {
                *const_cast<volatile int*>(&sh.dead) = 1;
                good = false;
                break;
            }
            put_by(n == kPrHold ? PrHold::kFirst : PrHold::kNext);
            l = 0.f;
        }
        float x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ask32(s_at + 32 * c, x[c]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_have32(x[c]);
        const int absent = *const_cast<volatile int*>(&sh.absent[n & 3]);
        if (absent || !sh.whole[half].has(tile)) {
            // per 32 rows of the tile, those that this thread's token sees
            const int first = tile * kPrTile, window = p.c.window;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int upto = row - first - 32 * c;
                uint32_t in = lowest(upto + 1);
                if (window) in &= ~lowest(upto + 1 - window) | lowest(p.c.sink - first - 32 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (absent >> (4 * c + e) & 1) in &= ~(0xFFu << (8 * e));
                if (__all_sync(0xffffffffu, in == 0xFFFFFFFFu)) continue;
#pragma unroll
                for (int i = 0; i < 32; ++i) x[c][i] = in >> i & 1 ? x[c][i] : none;
            }
        }
        // eight maxima side by side: one after the other each would wait for the last
        float top[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) top[i] = falls ? fminf(x[0][2 * i], x[0][2 * i + 1]) : fmaxf(x[0][2 * i], x[0][2 * i + 1]);
        if (falls) {
#pragma unroll
            for (int i = 16; i < 128; i += 2) top[i / 2 & 7] = fminf(top[i / 2 & 7], fminf(x[i / 32][i % 32], x[i / 32][i % 32 + 1]));
            top[0] = fminf(fminf(fminf(top[0], top[1]), fminf(top[2], top[3])), fminf(fminf(top[4], top[5]), fminf(top[6], top[7]))) * scale;
        } else {
#pragma unroll
            for (int i = 16; i < 128; i += 2) top[i / 2 & 7] = max3(top[i / 2 & 7], x[i / 32][i % 32], x[i / 32][i % 32 + 1]);
            top[0] = max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], top[5]), fmaxf(top[6], top[7])) * scale;
        }
        if (__any_sync(0xffffffffu, top[0] > m + kPrSlack)) {
            const float now = fmaxf(m, top[0]);
            const float w = m == -CUDART_INF_F ? 0.f : exp2_fast(m - now);
            m = now;
            l *= w;
            if (n > 0) pr_rescale<D>(o_at, w);
        }
        const float minus = m == -CUDART_INF_F ? 0.f : -(m + p.down_bits);
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 scale2 = make_float2(scale, scale), minus2 = make_float2(minus, minus);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float2 e = fma2(make_float2(x[c][i], x[c][i + 1]), scale2, minus2);
                x[c][i] = e.x;
                x[c][i + 1] = e.y;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) x[c][i] = exp2_fast(x[c][i]);
            uint32_t two[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                two[i] = pack_bf16x2(x[c][2 * i], x[c][2 * i + 1]);
                sum[i & 3] = add2(sum[i & 3], make_float2(x[c][2 * i], x[c][2 * i + 1]));
            }
            tmem_put16(s_at + 16 * c, two);
        }
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
        tmem_put_wait();
        if (!sh.whole[2].has(tile)) {
            const int s = n % L::kStages;
            good = warp_wait_or_give_up(&sh.v_ok[s], (n / L::kStages) & 1, &sh.dead);
            if (!good) break;
            if (sh.is_wild(s)) pr_by_hand<D>(o_at, s_at, base + L::kV + s * L::kTileBytes, n % kPrHold == 0);
        }
        tc_fence_before();
        __syncwarp();
        if ((r & 31) == 0) mbar_arrive(&sh.p_full[half]);
    }
    if (good && tiles > 0) {
        good = warp_wait_or_give_up(&sh.o_full[half], 0, &sh.dead);
        tc_fence_after();
    }
    if (good && tiles > kPrHold) l = put_by(PrHold::kLast);
    const bool live = r < p.tq * p.G && token < u.ntok;
    const int g = r % p.G;
    const int64_t head = static_cast<int64_t>(u.h) * p.G + g, tok = u.tok + token;
    const float base2 = m == -CUDART_INF_F ? m : m + p.down_bits;
    // Sums and results go through the place of the warp's 32 queries, which no product reads any more, and from there out by
    // whole rows: a thread's row each would be 32 lines to a store (4 prompts of 4096: 479 us; 468).
    constexpr int kWords = D / 8, kPer = 32 / kWords;          // words of 16 bytes of a row there; rows to a store
    const int lane = r & 31, word = lane % kWords;
    const uint32_t lives = __ballot_sync(0xffffffffu, live);
    uint8_t* stage = base + L::kQ + half * L::kTileBytes + (r & ~31) * D * 2;
    auto put = [&](int row, int w) { return stage + row * D * 2 + (w ^ (row & 7)) * 16; };
    if constexpr (kParts) {
        const int64_t rec = static_cast<int64_t>(blockIdx.y * p.c.H + blockIdx.x) * L::kHalves * kPrHalf + (threadIdx.x & ~31);
        if (live) p.part_stat[rec + lane] = good ? make_float2(base2, l) : make_float2(0.f, CUDART_NAN_F);
        if (!good || tiles <= 0 || !lives) return;
#pragma unroll 1
        for (int half_row = 0; half_row < D; half_row += D / 2) {
#pragma unroll
            for (int d0 = 0; d0 < D / 2; d0 += 32) {
                uint32_t o[32];
                tmem_get32(o_at + half_row + d0, o);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<uint4*>(put(lane, d0 / 4 + i)) = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < 32; i += kPer) {
                const int row = i + lane / kWords;
                if (lives >> row & 1)
                    *reinterpret_cast<uint4*>(p.part + (rec + row) * D + half_row + 4 * word) = *reinterpret_cast<const uint4*>(put(row, word));
            }
            __syncwarp();
        }
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = tok * p.o_tok + head * p.o_head;
    if (good && tiles > 0) {
#pragma unroll 1
        for (int d0 = 0; d0 < D; d0 += 32) {
            uint32_t o[32];
            tmem_get32(o_at + d0, o);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = l == 0.f ? 0.f : __uint_as_float(o[8 * c + i]) * inv;
                store8(reinterpret_cast<__nv_bfloat16*>(put(lane, d0 / 8 + c)), x);
            }
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 32; i += kPer) {
            const int row = i + lane / kWords;
            const int64_t to = __shfl_sync(0xffffffffu, at, row);
            const uint4 x = *reinterpret_cast<const uint4*>(put(row, word));
            if (lives >> row & 1) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + to + 8 * word) = x;
        }
    } else if (live) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = good ? 0.f : CUDART_NAN_F;
        for (int c = 0; c < D / 8; ++c) store8(static_cast<__nv_bfloat16*>(p.out) + at + 8 * c, x);
    }
    if (live && p.lse) p.lse[tok * p.n_q + head] = !good ? CUDART_NAN_F : l == 0.f ? -CUDART_INF_F : (base2 + log2f(l)) * 0.693147180559945309f;
}

template <int D, int kHalves, bool kParts>
__global__ void __launch_bounds__(PrForm<D, kHalves>::kThreads, PrForm<D, kHalves>::kCtas)
    k_prompt_attn(const __grid_constant__ PromptParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv) {
    using L = PrForm<D, kHalves>;
    extern __shared__ uint8_t s_raw[];
    __shared__ PrShared sh;
    __shared__ std::conditional_t<kParts, PrParts, int> all;
    uint8_t* base = s_raw + ((1024 - (smem_u32(s_raw) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == L::kSoft && lane == 0) {
        sh.dead = 0;
        mbar_init(&sh.q_full, 1);
        for (int s = 0; s < kPrStages; ++s) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.k_empty[s], 1);
            mbar_init(&sh.v_full[s], 1);
            mbar_init(&sh.v_ok[s], 2);
            mbar_init(&sh.v_empty[s], 1);
        }
        mbar_init(&sh.given_up, 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(&sh.s_full[x], 1);
            mbar_init(&sh.p_full[x], 4);
            mbar_init(&sh.o_full[x], 1);
        }
        fence_mbar_init();
        prefetch_tensormap(&mq);
        prefetch_tensormap(&mk);
        prefetch_tensormap(&mv);
    }
    __syncwarp();
    begin_call();
    if (warp == L::kSoft) {
        // rows that kernels before this one wrote, to be read by the copy engine (in all of memory, not shared memory's too:
        // that takes 1000 clocks more)
        asm volatile("fence.proxy.async.global;" ::: "memory");
        PrUnit u;
        if constexpr (kParts) {
            u = find_part(p, all, blockIdx.y);
            u.h = blockIdx.x;
        } else {
            u = find_unit(p, blockIdx.x);
        }
        if (lane == 0) {
            if (u.lo < u.hi) pr_load_queries<D, L>(p, &mq, sh, u, base);
            sh.place[0] = sh.place[1] = -1;
            if (!kParts && u.hi - u.lo > kPrHold) pr_take_places(sh, u.ntok > p.tq ? 2 : 1);
            sh.unit = u;
            for (int x = 0; x < 3; ++x) sh.whole[x] = whole(sees(p, u, x));
        }
    } else if (warp == L::kSoft + 1) {
        if (p.tq * p.G < kPrHalf) pr_clear_queries<D, L>(p, base);
        tmem_alloc(&sh.tmem, L::kColumns);
        tmem_relinquish();
        tc_fence_before();
    } else if (warp == L::kSoft + 2) {
        const int64_t block = blockIdx.y * static_cast<int64_t>(gridDim.x) + blockIdx.x, blocks = static_cast<int64_t>(gridDim.x) * gridDim.y;
        for (int64_t b = block * 32 + lane; b < p.c.batch; b += blocks * 32)
            check_sequence(p.c, p.start, p.tokens, static_cast<int>(b), g_err, 915);
    }
    __syncthreads();
    tc_fence_after();
    // the merge's note of all places' parts
    if constexpr (kParts) {
        if (blockIdx.x + blockIdx.y == 0 && warp == L::kSoft + 2)
            for (int i = lane; i < static_cast<int>(p.slots); i += 32)
                p.note[i] = make_int4(all.first[i], all.first[i + 1] - all.first[i], all.unit[i].tok, all.unit[i].ntok);
    }
    if (sh.unit.ntok == 0) {
        if (warp == L::kSoft + 1) tmem_dealloc(sh.tmem, L::kColumns);
        return;
    }
    if (warp < L::kSoft) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kRegsMore));
        pr_softmax<D, L, kParts>(p, sh, base);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kRegsLess));
        if (warp == L::kSoft) pr_load<D, L>(p, &mk, &mv, sh, base);
        else if (warp == L::kSoft + 1) pr_multiply<D, L>(p, sh, base);
        else pr_look<D, L>(p, sh, base);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (sh.dead) {
        // A wait ran out, of whichever warp: no copy and no product may be under way when the CTA ends.
        const unsigned long long since = globaltimer();
        if (threadIdx.x == 0) set_err(g_err, DEV_ERR_TIMEOUT, 911);
        if (warp == L::kSoft && lane == 0) {
            wait_out(&sh.q_full, 0, since);
            for (int n = max(0, sh.begun.x - L::kStages); n < sh.begun.x; ++n) wait_out(&sh.k_full[n % L::kStages], (n / L::kStages) & 1, since);
            for (int n = max(0, sh.begun.y - L::kStages); n < sh.begun.y; ++n) wait_out(&sh.v_full[n % L::kStages], (n / L::kStages) & 1, since);
        } else if (warp == L::kSoft + 1) {
            if (elect_one()) tc_commit(&sh.given_up);
            wait_out(&sh.given_up, 0, since);
        }
        __syncwarp();
    }
    if (!kParts && threadIdx.x < 2 && sh.place[threadIdx.x] >= 0) {
        __threadfence();
        atomicExch(g_in_use + sh.place[threadIdx.x], 0);
    }
    if (warp == L::kSoft + 1) {
        tc_fence_after();
        tmem_dealloc(sh.tmem, L::kColumns);
    }
}

// Joins the parts of the units' rows in their order: a warp per row, a lane per part for the weights, then per
// dimensions.  (37 parts of 20 rows for 8 heads 8 us, most of it the way there; a part at a time 22; a thread per row
// and four dimensions 11.)
template <int D>
__global__ void __launch_bounds__(256) k_prompt_merge(const __grid_constant__ PromptParams p) {
    constexpr int kEach = D / 32;
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x % p.c.H, lane = threadIdx.x & 31;
    const int4 note = __ldcg(p.note + blockIdx.x / p.c.H);
    const int first = note.x, parts = note.y, tok0 = note.z, rows = note.w * p.G;
    for (int i = blockIdx.y * 8 + (threadIdx.x >> 5); i < rows; i += 8 * gridDim.y) {
        const int token = i / p.G, g = i - token * p.G, half = token / p.tq, r = (token - half * p.tq) * p.G + g;
        const int64_t block = p.halves * kPrHalf, step = p.c.H * block, rec = first * step + h * block + half * kPrHalf + r;
        static_assert(kPrMaxParts == 64, "");
        float2 st[2];
        float m = -CUDART_INF_F, l = 0.f, w[2], x[kEach] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int s = 32 * k + lane;
            st[k] = s < parts ? __ldcg(p.part_stat + rec + s * step) : make_float2(-CUDART_INF_F, 0.f);
            m = fmaxf(m, st[k].x);
        }
        m = warp_max(m);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            // (a sum of zero: this part sees nothing; NaN is the row's, or that of a wait that ran out)
            w[k] = st[k].y == 0.f ? 0.f : st[k].y != st[k].y ? CUDART_NAN_F : exp2_fast(st[k].x - m);
            if (w[k] != 0.f) l = fmaf(st[k].y, w[k], l);
        }
        l = warp_sum(l);
        // eight parts' loads under way at a time
        for (int s0 = 0; s0 < parts; s0 += 8) {
            alignas(16) float o[8][kEach];
            float weight[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int s = s0 + k;
                weight[k] = __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31);
                const float* src = p.part + (rec + min(s, parts - 1) * step) * D + kEach * lane;
                if constexpr (kEach == 4) *reinterpret_cast<float4*>(o[k]) = __ldcg(reinterpret_cast<const float4*>(src));
                else *reinterpret_cast<float2*>(o[k]) = __ldcg(reinterpret_cast<const float2*>(src));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (weight[k] != 0.f) x[e] = fmaf(o[k][e], weight[k], x[e]);      // (otherwise nothing may have been written)
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t head = static_cast<int64_t>(h) * p.G + g, tok = tok0 + token;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + tok * p.o_tok + head * p.o_head + kEach * lane;
        const uint32_t lower = pack_bf16x2(x[0] * inv, x[1] * inv);
        if constexpr (kEach == 4) *reinterpret_cast<uint2*>(out) = make_uint2(lower, pack_bf16x2(x[2] * inv, x[3] * inv));
        else *reinterpret_cast<uint32_t*>(out) = lower;
        if (lane == 0 && p.lse) p.lse[tok * p.n_q + head] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.693147180559945309f;
    }
}

// ------------------------------------------------------------------ launches

PromptPlan prompt_plan(int tokens, int batch, int G, int H, int64_t tiles, int nsm) {
    // one half where the sequences have no more tokens than that takes, on average (they are on the device)
    const int tq = kPrHalf / G, halves = tokens <= static_cast<int64_t>(batch) * tq ? 1 : 2;
    PromptPlan plan{halves, 0, tokens / (halves * tq) + static_cast<int64_t>(batch)};
    // parts of the units' tiles, two tiles at least: as many as fill the SMs once, where they can be two for each place
    const int64_t room = (3 - halves) * nsm / H;
    if (tiles > 2 && room >= 2 * plan.slots)
        plan.parts = static_cast<int>(std::min<int64_t>({room, plan.slots * ((tiles + 1) / 2), plan.slots * kPrMaxParts}));
    return plan;
}

template <int D, int kHalves, bool kParts>
static int launch_prompt(const PromptParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
    using L = PrForm<D, kHalves>;
    constexpr int smem = L::kBytes + 1024;
    auto kernel = k_prompt_attn<D, kHalves, kParts>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
    const unsigned units = static_cast<unsigned>(p.slots * p.c.H);
    if (launch_first(kernel, kParts ? dim3(p.c.H, p.parts) : dim3(units), L::kThreads, smem, 1, 100, s, p, mq, mk, mv) != cudaSuccess) return -1;
    // (a block of the merge takes eight rows at a time)
    const unsigned rows = std::min(p.tokens, p.unit_tokens) * p.G;
    if (kParts && launch_first(k_prompt_merge<D>, dim3(units, (rows + 7) / 8), 256, 0, 1, 100, s, p) != cudaSuccess) return -1;
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
}
template <int D>
static int launch_prompt_form(const PromptParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
    if (p.parts) return p.halves == 1 ? launch_prompt<D, 1, true>(p, mq, mk, mv, s) : launch_prompt<D, 2, true>(p, mq, mk, mv, s);
    return p.halves == 1 ? launch_prompt<D, 1, false>(p, mq, mk, mv, s) : launch_prompt<D, 2, false>(p, mq, mk, mv, s);
}
int launch_prompt_attn(int d, const PromptParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
    return d == 64 ? launch_prompt_form<64>(p, mq, mk, mv, s) : launch_prompt_form<128>(p, mq, mk, mv, s);
}

cudaError_t prompt_err(int** e) { return cudaGetSymbolAddress(reinterpret_cast<void**>(e), g_err); }

}  // namespace skv
