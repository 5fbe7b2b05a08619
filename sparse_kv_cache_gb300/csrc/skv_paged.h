// Internal types of the paged-cache calls: kernel parameters and launchers.
#pragma once

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
};
constexpr int kPaWarps = 4;                  // warps of a CTA of the attention
int paged_attn_ctas(int dtype, int d, int nsm);     // CTAs that fill nsm SMs
int launch_paged_attn(int dtype, int d, const PagedAttnParams& p, int ncta, cudaStream_t s);

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

// The error words of the three kernel files on the current device.
cudaError_t norm_rope_err(int** p);
cudaError_t paged_attn_err(int** p);
cudaError_t evict_err(int** p);

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
