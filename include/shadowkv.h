/*
 * shadowkv.h — C ABI of the ShadowKV decode-step sparse attention library
 * (libshadowkv.so, sm_103a / GB300).
 *
 * The method: "ShadowKV: KV Cache in Shadows for High-Throughput Long-Context
 * LLM Inference".  The calls map one to one onto the two algorithms of the
 * Chinese digest of that paper (section A2): Algorithm 1 (pre-filling) is
 * shadowkv_prefill_index, Algorithm 2 (decoding) is shadowkv_decode_step.
 * The analytical models (equivalent bandwidth, memory savings, compression
 * ratio) are those of the English summary, section 3.4 and the appendix A.2
 * memory-savings formula.
 *
 * Conventions for every call:
 *  - All tensors are dense row-major in the storage dtype of the config
 *    (float32 or bfloat16), 16-byte aligned.  "dev" marks device memory of the
 *    current CUDA device; "host" marks page-locked host memory.
 *  - Nothing throws across this ABI.  Every int-returning call returns
 *    SKV_OK (0) or one of the negative SKV_ERR_* codes below.
 *  - Calls that take streams enqueue work and return; they do not
 *    synchronise unless stated.  A handle must not be used from two host
 *    threads at once.
 *  - Kernels that index with chunk ids, slots or positions range-check them;
 *    a failed check sets a device error word and skips the access.  The word
 *    is read (with a synchronisation) by shadowkv_stats, which then returns
 *    SKV_ERR_DEVICE_BOUNDS or SKV_ERR_TIMEOUT.
 */
#ifndef SHADOWKV_H
#define SHADOWKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Error codes. */
#define SKV_OK                 0
#define SKV_ERR_INVALID       -1  /* bad config, null or misaligned pointer, bad handle */
#define SKV_ERR_OOM           -2  /* device allocation failed (all partial state freed) */
#define SKV_ERR_NOT_PINNED    -3  /* v_place = host but V is not page-locked host memory */
#define SKV_ERR_CUDA          -4  /* a CUDA runtime/driver call failed */
#define SKV_ERR_DEVICE_BOUNDS -5  /* a kernel met an out-of-range index (access skipped) */
#define SKV_ERR_TIMEOUT       -6  /* a kernel's bounded wait ran out (work abandoned) */
#define SKV_ERR_STEP_LIMIT    -7  /* more decode steps than max_new_tokens */
#define SKV_ERR_UNSUPPORTED   -8  /* valid for the method, not built for this device/shape */

/* A CUDA stream (cudaStream_t) without pulling in the CUDA headers. */
typedef struct CUstream_st* skv_stream;

/*
 * SKV_FP8: the configuration the summary page's precision study runs with
 * float8 e5m2 (section 5, "Precision sensitivity"): the landmarks the library
 * builds and the values V (handed in as e5m2 bytes) are stored in e5m2; A, B,
 * q, k_new, v_new, the keys and out stay bf16.  Scores stay bf16-exact (the
 * query is split into three e5m2 terms for the 8-bit tensor-core product).
 */
/* SKV_E4M3: a paged cache of e4m3 codes with block scales (skv_block_scales); for the paged calls that name it */
typedef enum { SKV_F32 = 0, SKV_BF16 = 1, SKV_FP8 = 2, SKV_E4M3 = 3 } skv_dtype;
typedef enum { SKV_V_HBM = 0, SKV_V_HOST = 1 } skv_vplace;

/*
 * How the keys of generated tokens are kept.
 * SKV_NEWKEYS_EXACT: each decode step's k_new (post-RoPE) joins the exact local
 *   set as it is.
 * SKV_NEWKEYS_LOWRANK: ShadowKV+ (summary page, "The ShadowKV+ extension for
 *   generated tokens"; digest section A7 on newly generated tokens).  k_new is
 *   the PRE-RoPE key; the library keeps its rank-r state a = k'.Psi, where k'
 *   [H*d] is the token's key over the H heads of its batch element and
 *   Psi = B^T (B_b read as [r][H*d]), stored like A, and attends with the key
 *   rebuilt from the stored state, RoPE_{S+t}(a . B[b][h]) -- the same
 *   reconstruction as for context keys, made once when the token arrives and
 *   kept in the local rows as rebuilt context keys are kept in cache slots.
 *   For a true projection B_b's rows should be orthonormal (B = Psi^T from the
 *   SVD); the library does not check.
 */
typedef enum { SKV_NEWKEYS_EXACT = 0, SKV_NEWKEYS_LOWRANK = 1 } skv_newkeys;

/*
 * Sizes of one layer.  Notation of the pages: b batch, H KV heads, G = n_q/H
 * query heads per KV head, d head dim, r rank, C chunk, K selected chunks,
 * O outlier chunks, W local-window tokens, S context length.
 * Requirements: d = 128, C = 8, G in {1, 2, 4, 8}, n_q = G*H, S % C == 0,
 * W % C == 0, n_c = S/C - O - W/C >= K >= 1, O >= 0, 8 <= r <= 256 and
 * r % 8 == 0, max_new_tokens >= 1.
 */
typedef struct {
    int32_t batch;          /* b */
    int32_t n_kv_heads;     /* H */
    int32_t n_q_heads;      /* H*G */
    int32_t head_dim;       /* d */
    int32_t rank;           /* r, A is shared by the H heads of one batch element */
    int32_t chunk;          /* C */
    int32_t n_select;       /* K chunks selected per KV head and step */
    int32_t n_outlier;      /* O static outlier chunks per KV head */
    int32_t local_window;   /* W prefill tokens kept exact (plus every decode token) */
    int32_t max_new_tokens; /* decode steps the handle accepts */
    int64_t seq_len;        /* S */
    double  rope_base;      /* theta_i = rope_base^(-2i/d), half-split pairs (i, i+d/2) */
    int32_t dtype;          /* skv_dtype: storage of A, B, V, q, keys, landmarks, out (SKV_FP8: see above) */
    int32_t v_place;        /* skv_vplace of V */
    int32_t new_keys;       /* skv_newkeys */
} skv_config;

typedef struct skv_layer skv_layer;   /* opaque; one per layer */

/* Host-only check of a config against the requirements above.  No CUDA call. */
int shadowkv_validate_config(const skv_config* cfg);

/*
 * Algorithm 1 (pre-filling) for one layer: rebuilds K~ = RoPE(A.B) for every
 * context token, takes chunk means as landmarks, picks per (b, h) the O
 * chunks outside the local window with the lowest minimum cosine between a
 * token key and its chunk mean (lower chunk id first on ties), removes them
 * from the landmarks, and gathers the outlier chunks' K~/V and the local
 * window's K~/V to the GPU.
 *
 *   A  dev  [b][S][r]      low-rank token coordinates (borrowed)
 *   B  dev  [b][H][r][d]   per-head bases (borrowed)
 *   V  dev or host [b][H][S][d]  values (borrowed).  With v_place = SKV_V_HOST
 *      the GPU reads them in place over the host link: V must be page-locked
 *      (cudaHostAlloc / cudaHostRegister) or, on a device that reads pageable
 *      memory through the host's page tables (Grace + NVLink-C2C), any system
 *      memory.  Otherwise SKV_ERR_NOT_PINNED.  shadowkv_host_alloc provides
 *      suitable page-locked memory.
 *
 * A, B and V must stay valid until shadowkv_destroy: decode steps read A/B
 * rows and V rows of the chunks they miss.  The library owns everything else.
 * Runs on `stream` and synchronises it before returning.  On error *out is
 * NULL and nothing is leaked.
 */
int shadowkv_prefill_index(const skv_config* cfg, const void* A, const void* B, const void* V,
                           skv_stream stream, skv_layer** out);

/*
 * Algorithm 1 as the digest states it (section A2): its inputs are the exact
 * keys K and K_RoPE, and the landmarks, the min-cosine outlier test, the
 * outlier keys and the local window's keys are built from K_RoPE = RoPE(K),
 * while A and B (the SVD of K, computed by the caller) serve only the sparse
 * reconstruction at decode time.
 *
 *   K  dev [b][H][S][d]  exact pre-RoPE keys, storage dtype (bf16; fp32 for
 *      SKV_F32; bf16 for SKV_FP8), 16-byte aligned.  Read during this call
 *      only: the library keeps no reference to it.
 * Everything else as shadowkv_prefill_index; K = NULL is that call.
 */
int shadowkv_prefill_index_keys(const skv_config* cfg, const void* A, const void* B, const void* K,
                                const void* V, skv_stream stream, skv_layer** out);

/*
 * Algorithm 2 (decoding), one step of one layer:
 *   1. appends (k_new, v_new) to the exact local set;
 *   2. P = q.L^T for the G query heads of every KV head (q-head j belongs to
 *      KV head j / G); S2 = max over the group of softmax(P / sqrt(d)) over the
 *      n_c selectable chunks; I = ArgTopK(S2, K), lower chunk id first on ties;
 *   3. index scan against the previous step's I: hit chunks keep their cache
 *      slot, missed chunks take the freed slots;
 *   4. rebuilds the missed chunks' keys RoPE(A[rows].B[b][h]) into their slots
 *      (main stream) while their values are gathered from V (side stream); with
 *      values in HBM and bf16 or e5m2 storage nothing is gathered: attention
 *      reads every cache slot's values in V, and runs on `main` right after the
 *      rebuild;
 *   5. out = softmax(q.K^T / sqrt(d)).V over the O*C outlier tokens, the K*C
 *      cached tokens and the W + t + 1 local tokens (t = 0-based step).
 *
 *   q      dev [b][H*G][d]  post-RoPE queries at position S + t
 *   k_new  dev [b][H][d]    post-RoPE key of the new token (SKV_NEWKEYS_LOWRANK:
 *                           its pre-RoPE key; step 4 then stores a = k'.Psi and
 *                           the new token's key rebuilt from it)
 *   v_new  dev [b][H][d]
 *   out    dev [b][H*G][d]  written
 *   sel_out dev int32 [b][H][K] or NULL: I as original chunk ids, ascending
 *   main, side: streams; side may be NULL or equal to main (then all work runs
 *   on main).  The library orders the two with its own events; the step is
 *   complete when `main` reaches the end of the enqueued work.
 */
int shadowkv_decode_step(skv_layer* layer, const void* q, const void* k_new, const void* v_new,
                         void* out, int32_t* sel_out, skv_stream main, skv_stream side);

/*
 * Micro-batch pipelining.  A caller that splits its batch into independent
 * handles per layer (micro-batches on their own streams) can let one
 * micro-batch's value fetch overlap another's landmark scoring: the fetch
 * moves data over the host link, the scoring reads HBM.  `event` (a
 * cudaEvent_t the caller owns, or NULL to stop) is recorded on the main stream
 * of every later decode step of this layer right after its selection, when
 * the step's miss list is final; the caller makes the next micro-batch's
 * stream wait for it before that micro-batch's decode step.  The library
 * keeps no other reference to the event.
 */
int shadowkv_set_select_event(skv_layer* layer, void* event);

/* Phases timed when profiling is on (CUDA events on the launching stream). */
#define SKV_PH_SCORE   0
#define SKV_PH_SELECT  1
#define SKV_PH_REBUILD 2
#define SKV_PH_FETCH   3
#define SKV_PH_ATTN    4
#define SKV_NPHASE     5

typedef struct {
    int64_t steps;              /* decode steps taken */
    int64_t units;              /* b*H */
    int64_t n_select;           /* K */
    int64_t hits, misses;       /* summed over steps and units */
    double  alpha_last;         /* hit rate of the last step */
    double  alpha_mean;         /* mean hit rate over steps t >= 1 (0 if none) */
    double  hbm_bytes;          /* algorithmic HBM bytes, summed over steps */
    double  link_bytes;         /* algorithmic host-link bytes (v_place = host) */
    double  scratch_bytes;      /* implementation scratch traffic (logits, partials) */
    double  phase_ms[SKV_NPHASE];        /* summed event time per phase (profiling) */
    int64_t phase_launches[SKV_NPHASE];  /* launches timed per phase */
    int32_t device_error;       /* 0, SKV_ERR_DEVICE_BOUNDS or SKV_ERR_TIMEOUT */
    int64_t kernel_launches;    /* kernels the decode steps launched since the last reset */
} skv_stats;

/*
 * Synchronises the layer's streams, reads the device counters and the error
 * word, and fills *out.  Returns the device error (if any) after filling *out.
 */
int shadowkv_stats(skv_layer* layer, skv_stats* out);
int shadowkv_reset_stats(skv_layer* layer);

/* Per-phase CUDA-event timing on (1) or off (0, the default). */
int shadowkv_set_profiling(skv_layer* layer, int enable);

/*
 * Inspection: copies one internal buffer (device to device, on `stream`) into
 * caller memory `dst` of at least shadowkv_export_size(layer, field) bytes.
 */
#define SKV_F_LANDMARKS     0   /* [b*H][n_c][d] dtype, compacted (outliers removed) */
#define SKV_F_CHUNK_IDS     1   /* [b*H][n_c] int32: original chunk id of each landmark */
#define SKV_F_OUTLIER_IDS   2   /* [b*H][O] int32, ascending */
#define SKV_F_MIN_COS       3   /* [b*H][S/C - W/C] float32 */
#define SKV_F_K_OUTLIER     4   /* [b*H][O*C][d] dtype */
#define SKV_F_V_OUTLIER     5   /* [b*H][O*C][d] dtype */
#define SKV_F_K_LOCAL       6   /* [b*H][W + max_new_tokens][d] dtype */
#define SKV_F_V_LOCAL       7   /* [b*H][W + max_new_tokens][d] dtype */
#define SKV_F_K_CACHE       8   /* [b*H][K][C][d] dtype, by slot */
#define SKV_F_V_CACHE       9   /* [b*H][K][C][d] dtype, by slot (values in HBM, bf16 or e5m2: the
                                   rows attention reads in V for each slot, gathered by the export;
                                   dst must be device memory) */
#define SKV_F_SELECTION    10   /* [b*H][K] int32: current I, ascending chunk ids */
#define SKV_F_SLOT_OF_SEL  11   /* [b*H][K] int32: cache slot of each entry of I */
#define SKV_F_MISS_COUNT   12   /* [b*H] int32: misses of the last step */
#define SKV_F_HITS_PER_STEP 13  /* [max_new_tokens] int32: hits summed over units */
#define SKV_F_A_NEW        14   /* [b][max_new_tokens][r] (A's storage: bf16, fp32 for SKV_F32):
                                   rank-r states of generated tokens (SKV_NEWKEYS_LOWRANK;
                                   size 0 otherwise) */
#define SKV_NFIELD         14
int64_t shadowkv_export_size(const skv_layer* layer, int field);
int shadowkv_export(skv_layer* layer, int field, void* dst, size_t bytes, skv_stream stream);

/*
 * Analytical models of the pages, host only:
 *   eq_bandwidth_gbs = 2 S B_GPU / (S/C + 2(K+O)C + (1-alpha) K C B_GPU / B_link)
 *   memory_savings   = 2SM / (SM/C + 2(K+O)C + Sr + rM), literal, M = H d (the
 *                      key width of one token across the KV heads, in elements)
 *   compression      = S d' / (r (S + d')), d' = H d (A is shared by the heads)
 * plus the algorithmic bytes of one decode step of one layer at hit rate alpha
 * and step t, and the predicted step time of that layer
 *   t_pred = hbm_bytes / B_GPU + link_bytes / B_link.
 */
typedef struct {
    double eq_bandwidth_gbs;
    double memory_savings;
    double compression_ratio;
    double hbm_bytes_per_step;
    double link_bytes_per_step;
    double t_pred_us;
} skv_model;
int shadowkv_model(const skv_config* cfg, double alpha, int64_t t, double b_gpu_gbs,
                   double b_link_gbs, skv_model* out);

/*
 * Host memory for values read in place by the GPU (v_place = SKV_V_HOST).
 * Not from the pages: it serves the value offload of the summary page's
 * section 3.4 ("What gets offloaded to the CPU").  Returns page-locked host
 * memory mapped into the GPU's address space (cudaHostAlloc, portable).
 * Allocate the values of every layer in one call and hand out slices: the
 * GPU's translations of one large allocation cover far more memory than
 * those of many small ones, which keeps the random 2 KB chunk reads of the
 * value fetch near link speed (measured for 32 x 2 GiB of values: about
 * 130 GB/s from one allocation against 44 GB/s from one per layer).
 * shadowkv_host_free releases it.  SKV_ERR_INVALID for bytes == 0 or
 * out == NULL, SKV_ERR_OOM if the memory cannot be allocated and locked.
 */
int shadowkv_host_alloc(size_t bytes, void** out);

/*
 * The same with a choice of host memory kind:
 *   SKV_HOST_PINNED  page-locked memory (cudaHostAlloc); what shadowkv_host_alloc returns.
 *   SKV_HOST_HUGE    pageable memory in the host's transparent huge pages (512 MiB on a
 *                    kernel with 64 KiB base pages), which the GPU reads through the host's
 *                    own page tables (Grace with NVLink-C2C; SKV_ERR_UNSUPPORTED elsewhere).
 *                    The mapping is aligned to the huge-page size and advised for huge pages;
 *                    the CUDA driver is told that its preferred location is the host, so it
 *                    does not migrate the pages on the GPU's access counts.  Pages come into
 *                    being when first written (fill it before the first
 *                    shadowkv_prefill_index that reads it).  While its pages are whole, one
 *                    translation covers 512 MiB and the value fetch's scattered 2 KB reads
 *                    run at about 170 GB/s against 125 GB/s from page-locked memory (32 x
 *                    2 GiB of values; link copy peak about 210 GB/s).  But the host kernel
 *                    splits some of them -- measured: a few of 128 pages of a 64 GiB arena on
 *                    most runs, 40-86 on the first run on a freshly booted host -- and a split
 *                    page is read with a translation per 64 KiB; see shadowkv_host_repair.
 *                    SKV_HOST_PINNED is the steady choice.
 * SKV_ERR_INVALID for bytes == 0, out == NULL or an unknown kind; SKV_ERR_OOM if the memory
 * cannot be had.  shadowkv_host_free releases either kind.
 */
#define SKV_HOST_PINNED 0
#define SKV_HOST_HUGE   1
int shadowkv_host_alloc_kind(size_t bytes, int kind, void** out);

/*
 * Puts split huge pages of [p, p + bytes) -- inside one SKV_HOST_HUGE allocation -- back
 * together (madvise MADV_COLLAPSE, Linux 6.1+; a page that is whole costs nothing).  Measured
 * on a 64 GiB arena: about ten of its 128 pages split while the layers were pre-filled, and a
 * split page costs the fetch a translation per 64 KiB instead of per 512 MiB.
 * shadowkv_prefill_index repairs the layer's own values before it returns.  From the first
 * decode step that reads such memory until the last SKV_HOST_HUGE allocation is freed, a
 * library thread watches the host's split count (/proc/vmstat thp_split_pmd, every 5 ms) and
 * repairs every such allocation when it moves, resting 50 ms after each repair.  A caller may
 * also repair a range itself, e.g. after its warm-up.  Synchronous.
 * SKV_ERR_INVALID if the range is not inside such an allocation, SKV_ERR_UNSUPPORTED if the
 * host kernel lacks the call, SKV_ERR_OOM if no huge page could be had.
 */
int shadowkv_host_repair(void* p, size_t bytes);
void shadowkv_host_free(void* p);

/*
 * Sparse attention that allocates nothing.  The pages have no counterpart to
 * this call; it exists for callers that cannot allocate device memory while
 * they run -- a server that hands all of HBM to one pool at start-up, code
 * that runs under an allocator lock, or a hot path where an allocation (which
 * may synchronise the device) is forbidden.
 *
 * It computes what step 5 of shadowkv_decode_step computes -- for each unit u
 * (a batch element's KV head) and each of its G query heads,
 * out = softmax(q.K^T / sqrt(d)).V over the unit's outlier rows, then its
 * cache rows, then its first n_local_tokens local rows -- but with its own
 * kernel (k_attn_bulk: 128-token splits staged by bulk copies, merged by the
 * last CTA of each unit), not the decode step's persistent tensor-core kernel.
 * All bf16, d = 128, rows of a region contiguous per unit:
 *   q         dev [units*group][128]                    (post-RoPE)
 *   k/v_outlier dev [units][n_outlier_tokens][128]      (may be NULL if 0 rows)
 *   k/v_cache dev [units][n_cache_tokens][128]          (may be NULL if 0 rows)
 *   k/v_local dev [units][local_capacity][128]
 *   out       dev [units*group][128]                    written
 * The caller owns every buffer; each must be device memory (a host pointer is
 * refused with SKV_ERR_INVALID before anything runs).
 *
 * Scratch: the partial results of the splits, one merge ticket per unit and an
 * error word live in a fixed 16 MiB array compiled into the library, which
 * every GPU that loads the library holds until the process exits.  Refused
 * with SKV_ERR_INVALID: more than 16384 units; partials above
 * 16 MiB - 64.25 KiB (units * ceil(rows / 128) * group * 528 bytes); or a unit
 * whose merge state does not fit in one CTA's shared memory (64 KiB +
 * 8 * ceil(rows / 128) * group bytes above the device's per-block limit, e.g.
 * about 333K rows at group 8).  fp32 data: SKV_ERR_UNSUPPORTED.
 *
 * No cudaMalloc, cudaFree or other allocating call is made.  With CUDA's lazy
 * module loading, though, the array itself comes into being when this part of
 * the library is first used on a device -- by the first call here, or by the
 * first decode step, whose attention kernels live in the same module.  A
 * caller that gives all free HBM to a pool should therefore make a set-up call
 * first: args->units == 0 launches nothing and only loads the array, resolves
 * its device address for the current device and sets the kernel's
 * shared-memory limit.  The first call on a device (set-up or not) does that
 * set-up, with that device current; make it before any stream capture.  The
 * address is resolved again if the device's context changes (after
 * cudaDeviceReset).
 *
 * Every call shares the one array and clears the merge tickets itself
 * (asynchronously, on `stream`); calls that overlap on the GPU -- on different
 * streams, or from different threads -- race on it, so serialise them.
 *
 * Errors inside the kernel (a bounded wait for the staged rows that ran out,
 * after about one second) are not seen by the call, which has returned
 * already: the affected units' outputs are written as NaN, and the error is
 * kept in the array's error word until shadowkv_sparse_attention_noalloc_status
 * reads it.
 */
typedef struct {
    int32_t units;              /* b*H; 0: set-up only (see above) */
    int32_t group;              /* G in {1, 2, 4, 8} */
    int32_t dtype;              /* skv_dtype; only SKV_BF16 */
    int32_t n_outlier_tokens;   /* rows per unit in k/v_outlier */
    int32_t n_cache_tokens;     /* rows per unit in k/v_cache */
    int32_t n_local_tokens;     /* rows per unit used from k/v_local, >= 1 */
    int32_t local_capacity;     /* rows per unit allocated in k/v_local */
    const void* q;
    const void* k_outlier;
    const void* v_outlier;
    const void* k_cache;
    const void* v_cache;
    const void* k_local;
    const void* v_local;
    void* out;
} skv_attention_args;
int shadowkv_sparse_attention_noalloc(const skv_attention_args* args, skv_stream stream);

/*
 * Status of the no-allocation calls made so far on the current device:
 * synchronises `stream`, reads the error word of the fixed array and clears it.
 * Returns SKV_OK, SKV_ERR_TIMEOUT (a kernel's wait ran out; those units' outputs
 * are NaN), or SKV_ERR_CUDA.  Allocates nothing.  The pages have no counterpart.
 */
int shadowkv_sparse_attention_noalloc_status(skv_stream stream);

/*
 * Measurement aid, not from the pages: the rate of the decode step's value
 * fetch on its own.  Reads n_chunks distinct random chunks of chunk_bytes
 * (1024, 2048 or 4096: one chunk of C = 8 rows of e5m2, bf16 or fp32 values)
 * spread over [src, src + bytes) -- host memory the GPU reads in place, or
 * device memory -- into device scratch with the fetch kernel, in address
 * order as the decode step reads its miss lists, on `stream`, reps + 1 times
 * (the first untimed).  fresh = 0 reads the same chunks every time (the GPU's
 * translations of them are warm after the first); fresh = 1 draws new chunks
 * for every repetition, as successive layers' fetches do.  *gbs_out = chunk
 * bytes per second of the fastest timed repetition (CUDA events).  Allocates
 * and frees its own device scratch and synchronises `stream`.
 * SKV_ERR_INVALID for bad sizes or a null or misaligned src.
 */
int shadowkv_fetch_probe(const void* src, size_t bytes, int64_t n_chunks, int chunk_bytes, uint64_t seed,
                         int reps, int fresh, skv_stream stream, double* gbs_out);

/*
 * Paged caches: the dense path beside the sparse one.  The pages have no
 * counterpart to these calls; they serve what surrounds a decode step --
 * the projections' outputs that have to be normed and rotated before
 * shadowkv_decode_step takes them, layers that attend over their whole cache,
 * and caches that are held to a budget by giving rows up instead of by
 * offloading them.
 *
 * A paged cache is the caller's memory.  Keys and values live in two pools of
 * n_pages pages of page_size rows (one row: one token's key or value of one KV
 * head); sequence b owns the pages table[b][0 .. max_pages), and row i of it is
 * row i % page_size of page table[b][i / page_size].  Only the pages of its
 * first lens[b] rows are read.  Strides are in elements and free (page-major,
 * head-major or token-major pools), the head dimension is contiguous.
 *   dtype      SKV_BF16, SKV_F32, or SKV_FP8 (bf16 keys, e5m2 values); SKV_E4M3 where a call says so
 *   head_dim   64 or 128;  page_size a power of two from 8 to 1024
 *   strides    multiples of 16 bytes; pools 16-byte aligned device memory of the
 *              current device; rows of pools and outputs that are written do not overlap
 * A negative length counts as 0 and one above max_pages * page_size as that;
 * a page id outside [0, n_pages) is not followed (its rows count as absent).
 * Both set an error word of the device, which shadowkv_paged_status reads.
 *
 * Calls enqueue their work on `stream`, allocate nothing, keep nothing for the
 * next call, and give the same bits for the same inputs.  They can be captured
 * into graphs.  Calls that overlap on the GPU need workspaces of their own (so
 * do two graphs that may replay at once, and the calls of host threads that
 * enqueue on one stream side by side); calls that only read a cache may
 * overlap on it.
 */
typedef struct {
    int32_t dtype;              /* skv_dtype of the cache, of q, k, v and of the outputs (SKV_FP8: those are bf16) */
    int32_t n_kv_heads;         /* H */
    int32_t head_dim;           /* d */
    int32_t page_size;
    int32_t batch;              /* sequences; 0: nothing is done */
    int32_t max_pages;          /* entries per sequence in table, >= 1 */
    int64_t n_pages;            /* pages of the pools */
    int64_t k_page, k_head, k_row;   /* strides of the key pool, elements */
    int64_t v_page, v_head, v_row;   /* strides of the value pool, elements */
    int64_t table_seq;          /* entries between sequences of table, >= max_pages */
    void* k;                    /* dev */
    void* v;                    /* dev */
    const int32_t* table;       /* dev [batch][max_pages] */
    const int32_t* lens;        /* dev [batch] (not used by shadowkv_qk_norm_rope) */
} skv_paged_cache;

/*
 * Norm, rotation and append of the queries and keys of `tokens` tokens in one
 * pass.  For every head x of q and k
 *   y = x / sqrt(mean(x^2) + eps) * w     (w NULL: y = x)
 *   (y_i, y_{i+rd/2}) -> (y_i cos a - y_{i+rd/2} sin a, y_{i+rd/2} cos a + y_i sin a),
 *   a = position * rope_base^(-2i/rd),  i < rd/2
 * in fp32 (the angle's turns in 64-bit fixed point), rounded once.  With
 * rd = head_dim these are the keys and queries shadowkv_decode_step takes;
 * dimensions from rd on pass through.  The squares add up in fp32 too: a normed
 * head has elements below 10^18.
 *
 * With cache.k set, k and v also become row index[t] of sequence seq[t] of the
 * cache (v is rounded to e5m2 for SKV_FP8, saturating), and where given
 * row_position[b][h][row] = position and row_weight[b][h][row] = 0.  lens is
 * the caller's to advance.  No two tokens of a call may name the same row, nor
 * two sequences share the page of a row that is written.
 *
 * A token with a negative position is padding: nothing of it is written.  One
 * with a negative seq is not appended.  An index or seq beyond the cache, or a
 * bad page, sets the error word and skips the append.
 * q_out may be q and k_out may be k (same strides); other overlaps are not
 * allowed.  tokens == 0 does nothing.
 */
typedef struct {
    skv_paged_cache cache;      /* dtype, n_kv_heads, head_dim always; the rest with cache.k */
    int32_t tokens;
    int32_t n_q_heads;          /* any number >= 0, not tied to n_kv_heads */
    int32_t rotary_dim;         /* rd: a multiple of 16, 16 .. head_dim; 0: head_dim */
    float eps;                  /* > 0 where a weight is given */
    double rope_base;           /* > 1 */
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;   /* strides, elements */
    int64_t q_out_tok, q_out_head, k_out_tok, k_out_head;
    const void* q;              /* dev [tokens][n_q_heads][d] */
    const void* k;              /* dev [tokens][n_kv_heads][d] */
    const void* v;              /* dev [tokens][n_kv_heads][d]; with a cache only */
    const void* q_weight;       /* dev [d], dtype of q, or NULL: q is not normed */
    const void* k_weight;       /* dev [d], or NULL: k is not normed */
    void* q_out;                /* dev [tokens][n_q_heads][d] */
    void* k_out;                /* dev [tokens][n_kv_heads][d], or NULL with a cache */
    const int32_t* positions;   /* dev [tokens] */
    const int32_t* seq;         /* dev [tokens]; with a cache */
    const int32_t* index;       /* dev [tokens]; with a cache */
    int32_t* row_position;      /* dev [batch][n_kv_heads][row_pitch], or NULL */
    float* row_weight;          /* dev, the same shape, or NULL */
    int64_t row_pitch;          /* >= max_pages * page_size */
} skv_qk_norm_rope_args;
int shadowkv_qk_norm_rope(const skv_qk_norm_rope_args* args, skv_stream stream);

/*
 * Attention of one new token per sequence over its whole paged cache:
 *   out = softmax(scale q.K^T).V,  lse = ln sum exp(scale q.k_j)
 * for the G = n_q_heads / n_kv_heads query heads of every KV head (q-head j
 * belongs to KV head j / G; G from 1 to 8).  A sequence of no rows gives out = 0 and
 * lse = -inf; what lies behind a sequence's last row, in its last page or in
 * its table, is not read.  The token's own key has to be in the cache (and
 * counted in lens) if it is to attend to itself.  Nothing that is written
 * overlaps anything else.
 *
 * Lengths are on the device, so the host goes by the table's width: it picks the
 * kernels for sequences that fill it, and the workspace of a call with weights
 * has 4 bytes per row of that width and query head (an odd number of heads per
 * KV head counts as one more).  A table no wider than the longest sequence is
 * the fastest: one sequence of 1013 rows takes 6.4 us, and 13 in a table for
 * 128K rows.
 *
 * With weight_out set, the weight every row received is added to the running
 * sums that shadowkv_paged_evict goes by:
 *   weight_out[b][h][j] = weight[b][h][j] + sum over the G heads of p_j
 * for j < lens[b]; rows behind are left as they are.  weight_out may be weight.
 * Only these calls add weight, one token a sequence at a time: the rows of a
 * prompt, which shadowkv_qk_norm_rope sets to 0, have none before the first
 * step after it.
 *
 * Accumulation, softmax statistics and sums are fp32.  bf16 values are
 * multiplied by probabilities in two bf16 terms (16 bits), e5m2 ones by
 * probabilities in fp16.  Values may be as large as their type's largest; the
 * products of those below 2^-118 times the table's rows lose bits.  An infinite
 * value gives that infinity, one of each sign or a NaN gives NaN.  A row 2^-75
 * below the heaviest (e5m2: 2^-32) may weigh nothing, and an infinity there give
 * NaN.  Rows that score -infinity count as absent.
 */
typedef struct {
    skv_paged_cache cache;
    int32_t n_q_heads;
    float scale;                /* 0: 1 / sqrt(head_dim) */
    int64_t q_seq, q_head, out_seq, out_head;   /* strides, elements */
    const void* q;              /* dev [batch][n_q_heads][d] */
    void* out;                  /* dev [batch][n_q_heads][d]; q and out 16-byte aligned, strides of whole 16 bytes */
    float* lse;                 /* dev [batch][n_q_heads], or NULL */
    const float* weight;        /* dev [batch][n_kv_heads][row_pitch]; with weight_out */
    float* weight_out;          /* dev, the same shape, or NULL */
    int64_t row_pitch;          /* >= max_pages * page_size */
    void* workspace;            /* dev, 16-byte aligned */
    int64_t workspace_bytes;    /* >= shadowkv_paged_attention_workspace(args) */
} skv_paged_attention_args;
int64_t shadowkv_paged_attention_workspace(const skv_paged_attention_args* args);   /* bytes, or SKV_ERR_*; goes by the sizes alone, no CUDA call */
int shadowkv_paged_attention(const skv_paged_attention_args* args, skv_stream stream);

/*
 * Brings every (sequence, KV head) of more than `budget` rows down to budget
 * rows.  Kept are the rows whose position is above last - recent (last: the
 * largest position of the sequence's rows of that head) or below sink, and of
 * the rest those with the largest weight; a lower row before a higher one among equal
 * weights (a NaN weighs more than any number).  The kept rows with row >= budget then move, key, value, position and
 * weight, into the rows below budget that were given up: the i-th such row, in
 * ascending order, into the i-th given-up one.  Rows so lose their order, which attention does
 * not depend on; row_position records where each belongs.  Afterwards
 * lens_out[b] = min(lens[b], budget) and the pages behind are free.  Straight
 * after a prompt all weights are equal and the lowest rows stay, so a caller
 * that gives up rows of a prompt has weights of its own for them.  A table much
 * wider than lens costs here too (64 units one row over a budget of 2080: 12 us,
 * and 24 in tables for 128K rows).
 *
 * position_out, weight_out and lens_out may be position, weight and lens (in
 * place) or buffers of their own, which then hold the rows below lens_out[b]
 * (rows behind are left as they are).  The key and value pools are changed in
 * place; the rows at budget and behind stay as they were.  A sequence that
 * gives up rows must not share its pages.  A bad page sets the error word; a
 * row that would move out of or into one does not, and its place keeps the key,
 * value, weight and position of the row that was given up there.
 */
typedef struct {
    skv_paged_cache cache;
    int32_t budget;             /* >= 1 */
    int32_t recent, sink;       /* >= 0, recent + sink <= budget */
    const float* weight;        /* dev [batch][n_kv_heads][row_pitch]; this and the next three 16-byte aligned */
    const int32_t* position;    /* dev, the same shape; >= 0 */
    float* weight_out;
    int32_t* position_out;
    int64_t row_pitch;          /* >= max_pages * page_size, a multiple of 4 */
    int32_t* lens_out;          /* dev [batch] */
    void* workspace;            /* dev, 16-byte aligned */
    int64_t workspace_bytes;    /* >= shadowkv_paged_evict_workspace(args) */
} skv_paged_evict_args;
int64_t shadowkv_paged_evict_workspace(const skv_paged_evict_args* args);   /* bytes, or SKV_ERR_* */
int shadowkv_paged_evict(const skv_paged_evict_args* args, skv_stream stream);

/*
 * The same for one new token per sequence over a part of its rows, and over caches of 8-bit codes.
 *
 * With window > 0 the token sees its sequence's last `window` rows and its first `sink` ones: row j < lens[b] with
 * j >= lens[b] - window or j < sink, by the place in the cache (a cache that has lost rows in an eviction has no
 * such order).  window 0: all rows, whatever sink is.  Pages without a row that is seen are not looked
 * at, nor are their ids: a server may give the pages between back.  What is in a row that is not seen has no part
 * in the result, whatever it is.
 *
 * A cache of dtype SKV_E4M3 holds codes of four significant bits, keys and values alike, and their scales beside
 * the pools: a value is code * scale[page][head][row % page_size / block].  q and out are bf16.  The
 * scales are powers of two as shadowkv_paged_quantise writes them; any positive ones do here.  Strides of the pools are
 * above zero where there is more than one to step through, and below 2^40 bytes; rows are read by tiles of 16, also
 * those of a tile that are not seen or lie behind the last one.  A code of NaN in a row that is seen gives NaN.
 * Scores are formed from fp16 queries, a power of two per head apart (what is below 2^-39 of a head's largest
 * element is lost), probabilities take their value's scale and are rounded to fp16: a row whose probability times
 * scale is 2^-32 below the unit's heaviest may weigh nothing.  Everything else is as above.  Where a kernel's bounded
 * wait ran out (shadowkv_paged_status: SKV_ERR_TIMEOUT) results are NaN.
 *
 * attn.weight and attn.weight_out go with whole caches of the other types (window 0), where this call is
 * shadowkv_paged_attention; anywhere else they are refused.
 */
typedef struct {
    float* k;                   /* dev [n_pages][n_kv_heads][page_size / block] */
    float* v;                   /* dev, the same shape */
    int32_t block;              /* rows of a scale: a power of two from 8 to 128, at most page_size */
    int32_t reserved;           /* 0 */
} skv_block_scales;
typedef struct {
    skv_paged_attention_args attn;
    skv_block_scales scales;    /* with SKV_E4M3; otherwise zeros */
    int32_t window;             /* >= 0 */
    int32_t sink;               /* >= 0 */
} skv_paged_attention_ext_args;
int64_t shadowkv_paged_attention_ext_workspace(const skv_paged_attention_ext_args* args);   /* bytes, or SKV_ERR_* */
int shadowkv_paged_attention_ext(const skv_paged_attention_ext_args* args, skv_stream stream);

/*
 * Writes new rows of a cache of dtype SKV_E4M3.  Tokens start[b] .. start[b+1] of k and v (bf16 or fp32) become rows
 * lens[b] on of sequence b; lens is the caller's to advance.  For every block (scales.block rows of a page, from the
 * page's first) and head, of keys and of values:
 *   scale = 2^e, the smallest e >= -100 with |x| <= 448 * 2^e for the finite x among the block's new rows
 * and, where the block holds rows of the sequence already, the larger of that and the scale it has;
 * held codes are then rounded to the new one (between powers of two, as this call leaves them, only what falls below
 * 2^-9 of it is lost).
 *   code = x / scale, to the nearest, ties to even; NaN for a NaN and for an infinity
 * start does not fall, start[0] >= 0, start[batch] <= tokens; a sequence for which it does, or whose rows
 * would pass its table, sets the error word, and what is out of range is not written.  Where start falls, rows of other
 * sequences may be left out too.  A bad page sets it too and
 * its rows are left out.  A sequence that is written to does not share its last page, and no block of the
 * call's is another's: no page is in two tables' places that are written.
 */
typedef struct {
    skv_paged_cache cache;      /* dtype SKV_E4M3; lens: rows held before the call */
    skv_block_scales scales;
    int32_t tokens;             /* 0: nothing is done */
    int32_t dtype;              /* SKV_BF16 or SKV_F32: of k and v */
    int64_t k_tok, k_head, v_tok, v_head;   /* strides, elements, of whole 16 bytes */
    const void* k;              /* dev [tokens][n_kv_heads][d], 16-byte aligned */
    const void* v;
    const int32_t* start;       /* dev [batch + 1] */
} skv_paged_quantise_args;
int shadowkv_paged_quantise(const skv_paged_quantise_args* args, skv_stream stream);

/*
 * Reads rows of a cache of dtype SKV_E4M3 back: tokens start[b] .. start[b+1] of k and v (bf16 or fp32) become
 * rows first[b] on of sequence b, code * scale in fp32, rounded once.  Rows from lens[b] on and tokens of no
 * sequence are left as they are, and so are the rows of a bad page, which sets the error word, and the
 * tokens of a sequence whose start or first is out of range, which does too (where start falls, other sequences' may be left
 * out with them).  k and v do not overlap.
 */
typedef struct {
    skv_paged_cache cache;      /* dtype SKV_E4M3 */
    skv_block_scales scales;
    int32_t tokens;             /* 0: nothing is done */
    int32_t dtype;              /* SKV_BF16 or SKV_F32: of k and v */
    int64_t k_tok, k_head, v_tok, v_head;   /* strides, elements, of whole 16 bytes; rows do not overlap */
    void* k;                    /* dev [tokens][n_kv_heads][d], 16-byte aligned, written */
    void* v;
    const int32_t* start;       /* dev [batch + 1], does not fall */
    const int32_t* first;       /* dev [batch], >= 0 */
} skv_paged_dequantise_args;
int shadowkv_paged_dequantise(const skv_paged_dequantise_args* args, skv_stream stream);

/*
 * Attention of many new tokens per sequence: prompts, chunks of prompts, drafted tokens.  Tokens start[b] ..
 * start[b+1] of q are the last rows of sequence b, whose keys and values are in the cache already and counted in
 * lens[b]; token start[b+1] - 1 is row lens[b] - 1.  Token of row r sees row j <= r where window is 0, and
 * otherwise where j > r - window or j < sink besides.  out and lse as for one token; a token that sees nothing (there
 * are more tokens than rows, or its pages are bad) has out = 0 and lse = -inf.  out overlaps nothing else.
 *
 * dtype SKV_BF16 (others: SKV_ERR_UNSUPPORTED; a cache of codes is read back by shadowkv_paged_dequantise into rows
 * that make pages).  Strides of q and of the pools are above zero where there is more than one
 * to step through, and below 2^40 bytes.  Whole pages are read, also behind a sequence's last row; what is in
 * a row that a token does not see has no part in its result, whatever it is.  Pages of which no row is
 * seen are not looked at.  start does not fall, start[0] >= 0, start[batch] <= tokens: the tokens of a sequence
 * for which it does are left out and set the error word, and with them others may be.  Tokens of no sequence are left as they are.
 *
 * Scores, sums and softmax statistics are fp32; probabilities are rounded to bf16 (2^-8 at most), and what is
 * 2^-88 below a row's heaviest may weigh nothing (an infinite value there gives NaN or is passed over).  Sums of values
 * are cut off at every 16 rows, by 2^-22 of what is there, for 131072 rows at most: then they are put by, in the workspace or in a
 * fixed array of the library's (21 MB, a place for each CTA while it runs).  Keys that score -infinity count as absent.  Where a kernel's bounded wait ran
 * out (shadowkv_paged_status: SKV_ERR_TIMEOUT) results are NaN.
 */
typedef struct {
    skv_paged_cache cache;      /* dtype SKV_BF16; lens: with the new tokens' rows */
    int32_t n_q_heads;
    float scale;                /* 0: 1 / sqrt(head_dim) */
    int32_t window, sink;       /* >= 0 */
    int32_t tokens;             /* 0: nothing is done */
    int32_t reserved;           /* 0 */
    int64_t q_tok, q_head, out_tok, out_head;   /* strides, elements, of whole 16 bytes */
    const void* q;              /* dev [tokens][n_q_heads][d], 16-byte aligned */
    void* out;                  /* dev [tokens][n_q_heads][d], 16-byte aligned */
    float* lse;                 /* dev [tokens][n_q_heads], or NULL */
    const int32_t* start;       /* dev [batch + 1] */
    void* workspace;            /* dev, 16-byte aligned; may be NULL where no bytes are asked for */
    int64_t workspace_bytes;    /* >= shadowkv_paged_prompt_attention_workspace(args) */
} skv_paged_prompt_args;
int64_t shadowkv_paged_prompt_attention_workspace(const skv_paged_prompt_args* args);   /* bytes, or SKV_ERR_*; no CUDA call */
int shadowkv_paged_prompt_attention(const skv_paged_prompt_args* args, skv_stream stream);

/*
 * Status of the paged calls on the current device, of all streams: waits for
 * `stream`, then takes the error words and clears them in one step.  A call that
 * still runs on another stream is in it as far as it has come; what it sets
 * later is in the next status.  Returns SKV_OK, SKV_ERR_DEVICE_BOUNDS (a length,
 * index or page id was out of range; its access was skipped), SKV_ERR_TIMEOUT (a bounded wait inside a
 * kernel ran out), or SKV_ERR_CUDA.
 * Not for use during stream capture.
 */
int shadowkv_paged_status(skv_stream stream);

void shadowkv_destroy(skv_layer* layer);   /* frees everything the handle owns; NULL ok */
const char* shadowkv_strerror(int code);
int shadowkv_version(void);                 /* major*10000 + minor*100 + patch */

#ifdef __cplusplus
}
#endif
#endif /* SHADOWKV_H */
