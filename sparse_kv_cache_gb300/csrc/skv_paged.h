// Internal types of the paged-cache calls: kernel parameters and launchers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "shadowkv.h"

namespace skv {

// A paged cache as the kernels see it (strides in elements).
struct PagedView {
    void* k; void* v;
    int64_t k_page, k_head, k_row, v_page, v_head, v_row;
    const int32_t* table; int64_t table_seq;
    const int32_t* lens;
    int64_t n_pages;
    int batch, H;
    int lg;        // log2(page_size)
    int cap;       // max_pages * page_size: rows a sequence can have
    int window, sink, s16;      // attention over a part of the rows: last, first, those in whole tiles of 16
};

struct NormRopeParams {
    PagedView c;
    int tokens, nq, rd;
    int groups;               // lane groups per token (set by the launcher)
    float eps;
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, qo_tok, qo_head, ko_tok, ko_head;
    const void *q, *k, *v, *qw, *kw;
    void *qo, *ko;
    const int32_t *positions, *seq, *index;
    int32_t* row_position; float* row_weight; int64_t row_pitch;
    uint64_t turn[64];        // rope_base^(-2i/rd) / (2 pi) in units of 2^-64 turns
};
int launch_norm_rope(int dtype, int d, const NormRopeParams& p, int nsm, cudaStream_t s);

// A unit whose shares CTA i of the attention completes: they lie in the records of CTAs
// from .. i (slot: which of the first one's two); from < 0: there is none.
struct Joint { int from, b, h, slot; };

struct PagedAttnParams {
    PagedView c;
    int G, n_q;
    float scale_log2;         // scale * log2(e)
    float down;               // values are weighed by this much of a probability (set by the launcher)
    int64_t q_seq, q_head, o_seq, o_head;
    const void* q; void* out; float* lse;
    float* rec;               // [ncta][2][G][d]: a CTA's shares of its first and last unit, unnormalised
    float2* rec_stat;         // [ncta][2][G]: their bases and sums
    Joint* joint;             // [ncta]
    // weights: raw products q.k of every row [U][cap][Gp], and (base, 1 / sum) per head [U][G]
    float* z; float2* stat; int Gp;
    const float* weight; float* weight_out; int64_t row_pitch;
    int span;                 // rows that a sequence can show at most
    const float *ks, *vs; int lgb;      // e4m3: scales [n_pages][H][page_size >> lgb]
};
struct alignas(64) PagedCodesParams : PagedAttnParams {
    CUtensorMap mk, mv;       // the pools, d by 16 rows (8 where a page has no more) to a box
};
constexpr int kPaWarps = 4;                  // warps of a CTA of the attention
int paged_attn_ctas(int dtype, int d, int nsm);     // CTAs that fill nsm SMs
int launch_paged_attn(int dtype, int d, const PagedAttnParams& p, int ncta, cudaStream_t s);
int launch_paged_span(int dtype, int d, const PagedAttnParams& p, int ncta, cudaStream_t s);
int launch_paged_codes(int d, const PagedCodesParams& p, int ncta, cudaStream_t s);

struct QuantParams {
    PagedView c;
    int lgb, tokens;          // log2(rows of a block)
    int64_t slots;            // places for blocks: quantise_slots()
    int64_t k_tok, k_head, v_tok, v_head;
    const void *k, *v;
    float *k_scale, *v_scale;
    const int32_t* start;
};
int64_t quantise_slots(int tokens, int batch, int lgb);
int launch_quantise(int dtype, int d, const QuantParams& p, cudaStream_t s);

struct DequantParams {
    PagedView c;
    int lgb, tokens;
    int64_t k_tok, k_head, v_tok, v_head;
    void *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *start, *first;
};
int launch_dequantise(int dtype, int d, const DequantParams& p, cudaStream_t s);

struct PromptParams {
    PagedView c;              // window 0: none
    int G, n_q, tokens;
    int tq;                   // tokens of 128 query rows: 128 / G
    int halves;               // of a unit, of 128 query rows each
    int unit_tokens;          // halves * tq
    int parts;                // of units' tiles, for each KV head at most; 0: units are not taken in parts
    int64_t slots;            // places for units of halves * tq tokens of a sequence
    float scale_log2, down_bits;
    int64_t o_tok, o_head;
    const int32_t* start;
    void* out; float* lse;
    float* part;              // [parts][H][halves * 128][d]: parts of sums, unnormalised
    float2* part_stat;        // [parts][H][halves * 128]: their bases and sums of probabilities
    int4* note;               // [slots]: first part, parts, first token, tokens
};
struct PromptPlan { int halves, parts; int64_t slots; };
PromptPlan prompt_plan(int tokens, int batch, int G, int H, int64_t tiles, int nsm);      // tiles that a unit can see
int launch_prompt_attn(int d, const PromptParams& p, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s);

struct EvictParams {
    PagedView c;
    int d, es, es_v;
    int budget, recent, sink;
    const float* weight; const int32_t* position;
    float* weight_out; int32_t* position_out; int64_t row_pitch;
    int32_t* lens_out;
    int32_t* to; int32_t* of; int list_cap;   // [U][list_cap] rows given up / rows that move there
    int32_t* count;           // [U]: entries of the lists
    int32_t* new_len;         // [batch]: lengths that are updated in place
};
int launch_evict(const EvictParams& p, int nsm, cudaStream_t s);

// The error words of the kernel files on the current device.
cudaError_t norm_rope_err(int** p);
cudaError_t paged_attn_err(int** p);
cudaError_t evict_err(int** p);
cudaError_t paged_span_err(int** p);
cudaError_t quantise_err(int** p);
cudaError_t prompt_err(int** p);

#ifdef __CUDACC__
// A kernel of a call's beginning: a programmatic dependent of whatever is before it in the stream,
// so that its CTAs are in place when that ends (it waits for that before it touches memory), as one
// grid or as clusters of `ranks` CTAs.  carve: percent of an SM's memory that is shared memory, 0 for the
// driver's choice.  While CTAs of the kernel before are on an SM its split stays as that one had it; so kernels
// that follow each other ask for the same one, or the later one finds room for fewer CTAs than it needs and
// runs in two waves (the attention after its merge kernel, 300 units of 1000 rows with e5m2 values: 36 us
// against 28).
constexpr int kCarve = 58;        // room for three CTAs of the attention
constexpr int kSmShared = 228 << 10;      // all that can be shared memory
template <typename... KArgs, typename... Args>
inline cudaError_t launch_first(void (*k)(KArgs...), dim3 grid, int block, size_t smem, int ranks, int carve, cudaStream_t s,
                                Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[3];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (carve) {
        attr[cfg.numAttrs].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
        attr[cfg.numAttrs++].val.sharedMemCarveout = carve;
    }
    if (ranks > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = ranks;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, k, static_cast<Args&&>(args)...);
}
// 2^x, 0 for results below 2^-126
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A wait for a barrier's phase that ends after about a second, or once *dead is set; false then, and *dead is.  One
// statement: with a way out for some threads of a warp alone the compiler keeps what is the warp's in registers of
// each thread behind it (a prompt of 32K tokens: 6.5 ms against 6.3).  The answer is the thread's: each
// looks at the phase and at the clock for itself, so at the limit one may see the phase end and another give up.
__device__ __forceinline__ bool wait_or_give_up(uint64_t* bar, uint32_t parity, int* dead) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 now, end;\n\t.reg .b32 given_up;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "mov.u64 end, %%globaltimer;\n\tadd.u64 end, end, %4;\n\t"
        "AGAIN:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "ld.volatile.shared::cta.u32 given_up, [%3];\n\tsetp.ne.u32 q, given_up, 0;\n\t@q bra DONE;\n\t"
        "mov.u64 now, %%globaltimer;\n\tsetp.lt.u64 q, now, end;\n\t@q bra AGAIN;\n\t"
        "st.volatile.shared::cta.u32 [%3], 1;\n\t"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(smem_u32(dead)), "n"(kWaitLimitNs)
        : "memory");
    return ok != 0;
}
// The same with the warp's answer, by votes, where what comes next takes all of its threads: other votes, tensor memory, what
// lets the barrier's next phase begin.  (Within the statement: a prompt of 32K tokens as without, 1.5 % longer with a vote
// behind it.)
__device__ __forceinline__ bool warp_wait_or_give_up(uint64_t* bar, uint32_t parity, int* dead) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 now, end;\n\t.reg .b32 given_up;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tvote.sync.all.pred q, p, 0xffffffff;\n\t@q bra DONE;\n\t"
        "mov.u64 end, %%globaltimer;\n\tadd.u64 end, end, %4;\n\t"
        "AGAIN:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tvote.sync.all.pred q, p, 0xffffffff;\n\t@q bra DONE;\n\t"
        "ld.volatile.shared::cta.u32 given_up, [%3];\n\tsetp.ne.u32 p, given_up, 0;\n\t"
        "mov.u64 now, %%globaltimer;\n\tsetp.ge.or.u64 p, now, end, p;\n\tvote.sync.any.pred p, p, 0xffffffff;\n\t@!p bra AGAIN;\n\t"
        "st.volatile.shared::cta.u32 [%3], 1;\n\t"
        "DONE:\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(smem_u32(dead)), "n"(kWaitLimitNs)
        : "memory");
    return ok != 0;
}
// Waits for copies or products that nobody has use for any more, before a CTA ends that gave up: for a barrier's phase, and until
// kWaitLimitNs after `since` at most, whatever the number of barriers.
__device__ __forceinline__ void wait_out(uint64_t* bar, uint32_t parity, unsigned long long since) {
    while (!mbar_try_wait(bar, parity) && globaltimer() - since < kWaitLimitNs) {}
}
// A box of a tensor of three or four dimensions to shared memory, counted on `bar`
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}
// Its first lines: the kernels after it may be brought in once it knows that those before it are done.
// So a kernel is on the device while those before it write, and reads what they wrote by coherent loads only:
// the non-coherent ones are for what nothing writes as long as their kernel runs.
__device__ __forceinline__ void begin_call() {
    pdl_wait();
    pdl_trigger();
}

// a length brought into [0, cap], and that of sequence b
__device__ __forceinline__ int rows_in(const PagedView& c, int n, int* err, int where) {
    if (n < 0 || n > c.cap) {
        set_err(err, DEV_ERR_BOUNDS, where);
        n = n < 0 ? 0 : c.cap;
    }
    return n;
}
__device__ __forceinline__ int rows_of(const PagedView& c, int b, int* err, int where) {
    return rows_in(c, __ldcg(c.lens + b), err, where);
}
// The last sequence b whose key(start[b], b) is at most x, by the whole warp: 0 if there is none (keys do not
// fall; where they do, whatever comes out is a sequence).
template <class Key>
__device__ __forceinline__ int find_sequence(const int32_t* start, int batch, int64_t x, Key key) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, i = lo + lane * step;
        const bool in = i < hi && (lane == 0 || key(__ldcg(start + i), i) <= x);
        lo += (31 - __clz(__ballot_sync(0xffffffffu, in))) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}
// Sets the error word where sequence b's tokens are no part of the call's or its length is out of range.  Once for every
// sequence of a call: the searches above pass over some where starts fall.
__device__ __forceinline__ void check_sequence(const PagedView& c, const int32_t* start, int tokens, int b, int* err, int where) {
    const int t0 = __ldcg(start + b), t1 = __ldcg(start + b + 1);
    rows_of(c, b, err, where);
    if (t0 < 0 || t1 < t0 || t1 > tokens) set_err(err, DEV_ERR_BOUNDS, where);
}
// page of row i of sequence b, or -1 (and the error word) if its id is out of range
__device__ __forceinline__ int page_of(const PagedView& c, int b, int i, int* err, int where) {
    const int id = c.table[b * c.table_seq + (i >> c.lg)];
    if (id < 0 || id >= c.n_pages) {
        set_err(err, DEV_ERR_BOUNDS, where);
        return -1;
    }
    return id;
}
#endif

}  // namespace skv
