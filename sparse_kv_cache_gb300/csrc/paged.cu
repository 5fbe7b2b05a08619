// Host side of the paged-cache calls (include/shadowkv.h): argument checks, workspace layout,
// launches and the error words.
#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <mutex>

#include "skv_common.cuh"
#include "skv_internal.h"
#include "skv_paged.h"

using namespace skv;

namespace {

struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;
};

// rows of a sequence above this are refused: row arithmetic in the kernels is 32-bit
constexpr int64_t kMaxRows = int64_t(1) << 30;
// units (KV heads of sequences): with it, sizes in bytes stay below 2^60
constexpr int64_t kMaxUnits = int64_t(1) << 24;
// SMs that the attention's records have room for (a GB300 has 152)
constexpr int kMaxSms = 160;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// device memory of the current device
bool on_device(const void* p, int dev) {
    cudaPointerAttributes a;
    if (!p || cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return (a.type == cudaMemoryTypeDevice && a.device == dev) || a.type == cudaMemoryTypeManaged;
}

int wide_bytes(int dtype) { return dtype == SKV_F32 ? 4 : 2; }         // q and outputs
int key_bytes(int dtype) { return dtype == SKV_E4M3 ? 1 : wide_bytes(dtype); }
int value_bytes(int dtype) { return dtype == SKV_F32 ? 4 : dtype == SKV_BF16 ? 2 : 1; }

// the types that a call takes: those of all calls, one more, or that one alone
enum Types { kPlain, kAll, kCodes };
bool good_type(const skv_paged_cache& c, Types types = kPlain) {
    const bool plain = c.dtype == SKV_F32 || c.dtype == SKV_BF16 || c.dtype == SKV_FP8, codes = c.dtype == SKV_E4M3;
    return ((plain && types != kCodes) || (codes && types != kPlain)) && c.n_kv_heads >= 1 && c.n_kv_heads <= (1 << 16) &&
           (c.head_dim == 64 || c.head_dim == 128);
}

// a stride of whole 16-byte words
bool good_stride(int64_t s, int bytes) { return s >= 0 && s * bytes % 16 == 0; }
// Rows of d elements that are written must not overlap: every dimension that is stepped through (n steps
// of s) moves past all that the shorter steps reach.
struct Dim { int64_t n, s; };
template <int N>
bool apart(Dim (&x)[N], int64_t d) {
    std::sort(x, x + N, [](const Dim& a, const Dim& b) { return a.s < b.s; });
    int64_t reach = d;       // elements from the first row's first to the last one's last
    for (const Dim& e : x) {
        if (e.n <= 1) continue;
        if (e.s < reach || e.s > (INT64_MAX - reach) / e.n) return false;
        reach += (e.n - 1) * e.s;
    }
    return true;
}
bool apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t d) {
    Dim x[] = {{n0, s0}, {n1, s1}};
    return apart(x, d);
}

// what the host can tell without the device
int check_cache(const skv_paged_cache& c, bool written, Types types = kPlain) {
    if (!good_type(c, types)) return SKV_ERR_INVALID;
    if (c.page_size < 8 || c.page_size > 1024 || (c.page_size & (c.page_size - 1))) return SKV_ERR_INVALID;
    if (c.max_pages < 1 || c.n_pages < 1 || c.n_pages > INT32_MAX || c.table_seq < c.max_pages) return SKV_ERR_INVALID;
    if (static_cast<int64_t>(c.max_pages) * c.page_size > kMaxRows) return SKV_ERR_INVALID;
    if (static_cast<int64_t>(c.batch) * c.n_kv_heads > kMaxUnits) return SKV_ERR_INVALID;
    const int es = key_bytes(c.dtype), ev = value_bytes(c.dtype);
    for (int64_t s : {c.k_page, c.k_head, c.k_row})
        if (!good_stride(s, es)) return SKV_ERR_INVALID;
    for (int64_t s : {c.v_page, c.v_head, c.v_row})
        if (!good_stride(s, ev)) return SKV_ERR_INVALID;
    if (written) {
        Dim k[] = {{c.n_pages, c.k_page}, {c.n_kv_heads, c.k_head}, {c.page_size, c.k_row}};
        Dim v[] = {{c.n_pages, c.v_page}, {c.n_kv_heads, c.v_head}, {c.page_size, c.v_row}};
        if (!apart(k, c.head_dim) || !apart(v, c.head_dim)) return SKV_ERR_INVALID;
    }
    if (!c.k || !c.v || !c.table || !aligned16(c.k) || !aligned16(c.v)) return SKV_ERR_INVALID;
    return SKV_OK;
}

// every one of the pointers, where set, begins at an element of four bytes
int check_words(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 3) return SKV_ERR_INVALID;
    return SKV_OK;
}

// every one of the pointers that is set has to be device memory of the current device
int check_memory(std::initializer_list<const void*> ptrs, int dev) {
    for (const void* p : ptrs)
        if (p && !on_device(p, dev)) return SKV_ERR_INVALID;
    return SKV_OK;
}

// scales of a cache that check_cache has seen
int check_scales(const skv_paged_cache& c, const skv_block_scales& s) {
    if (s.block < 8 || s.block > 128 || s.block > c.page_size || (s.block & (s.block - 1)) || s.reserved) return SKV_ERR_INVALID;
    if (!s.k || !s.v) return SKV_ERR_INVALID;
    return check_words({s.k, s.v});
}
int log2_of(int x) {
    int lg = 0;
    while ((1 << lg) < x) ++lg;
    return lg;
}

PagedView view(const skv_paged_cache& c) {
    PagedView v{};
    v.k = c.k; v.v = c.v;
    v.k_page = c.k_page; v.k_head = c.k_head; v.k_row = c.k_row;
    v.v_page = c.v_page; v.v_head = c.v_head; v.v_row = c.v_row;
    v.table = c.table; v.table_seq = c.table_seq;
    v.lens = c.lens;
    v.n_pages = c.n_pages;
    v.batch = c.batch; v.H = c.n_kv_heads;
    v.lg = log2_of(c.page_size);
    v.cap = c.max_pages * c.page_size;
    return v;
}

struct Device { int id, nsm; };
int device(Device* d) {
    int major = 0;
    if (cudaGetDevice(&d->id) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d->id) != cudaSuccess ||
        cudaDeviceGetAttribute(&d->nsm, cudaDevAttrMultiProcessorCount, d->id) != cudaSuccess) {
        cudaGetLastError();
        return SKV_ERR_CUDA;
    }
    return major < 10 ? SKV_ERR_UNSUPPORTED : SKV_OK;
}

int done(int rc) {
    if (rc == 0) return SKV_OK;
    cudaGetLastError();
    return SKV_ERR_CUDA;
}

int64_t round16(int64_t n) { return (n + 15) & ~int64_t(15); }

// ------------------------------------------------------------------ tensor maps

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn find_encode() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    return reinterpret_cast<EncodeFn>(f);
}
// Map of a tensor [..][d] of bf16 or bytes (sizes and strides in elements, innermost first without d), for boxes of
// `width` elements of d, swizzled by their width of 128 or 64 bytes.  Steps of zero (a dimension that is expanded) and of 2^40
// bytes and more have no map.
int tensor_map(CUtensorMap* m, const void* base, int bytes, int d, uint32_t width, std::initializer_list<Dim> dims,
               std::initializer_list<uint32_t> box) {
    static const EncodeFn encode = find_encode();
    if (!encode) return SKV_ERR_CUDA;
    cuuint64_t size[4] = {static_cast<cuuint64_t>(d)}, step[3];
    cuuint32_t boxes[4] = {width}, ones[4] = {1, 1, 1, 1};
    int n = 1;
    for (const Dim& x : dims) {
        size[n] = x.n;
        step[n - 1] = static_cast<cuuint64_t>(x.n > 1 ? x.s : d) * bytes;     // (a step that is never taken has to be some step)
        if (step[n - 1] == 0 || step[n - 1] >= cuuint64_t(1) << 40) return SKV_ERR_INVALID;
        ++n;
    }
    std::copy(box.begin(), box.end(), boxes + 1);
    return encode(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, n, const_cast<void*>(base), size,
                  step, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  width * bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? SKV_OK
               : SKV_ERR_INVALID;
}

// SHADOWKV_FAULT=wait:q, wait:k or wait:v (tests): copies of that tensor's tiles are half as high as the kernels count on, so that
// their waits for them run out.
bool falls_short(char tensor) {
    const char* e = std::getenv("SHADOWKV_FAULT");
    return e && std::strncmp(e, "wait:", 5) == 0 && e[5] == tensor;
}

// ------------------------------------------------------------------ attention

struct AttnSpace { int Gp; int64_t joint, rec, rec_stat, stat, z, bytes; };

// host-only part of the checks, and the workspace's layout
int attn_space(const skv_paged_attention_args* a, AttnSpace* w, Types types = kPlain) {
    const skv_paged_cache& c = a->cache;
    if (!good_type(c, types) || c.batch < 0 || a->n_q_heads < 1 || a->n_q_heads % c.n_kv_heads) return SKV_ERR_INVALID;
    const int G = a->n_q_heads / c.n_kv_heads;
    if (G > 8 || !std::isfinite(a->scale)) return SKV_ERR_INVALID;
    if (c.max_pages < 1 || c.page_size < 1 || static_cast<int64_t>(c.max_pages) * c.page_size > kMaxRows)
        return SKV_ERR_INVALID;
    const int64_t U = static_cast<int64_t>(c.batch) * c.n_kv_heads, cap = static_cast<int64_t>(c.max_pages) * c.page_size;
    if (U > kMaxUnits) return SKV_ERR_INVALID;
    w->Gp = (G + 1) & ~1;
    const int64_t ctas = paged_attn_ctas(c.dtype, c.head_dim, kMaxSms);
    w->joint = 0;
    w->rec = ctas * static_cast<int64_t>(sizeof(Joint));
    w->rec_stat = w->rec + ctas * 2 * G * c.head_dim * 4;
    w->stat = w->rec_stat + round16(ctas * 2 * G * 8);
    w->z = w->stat;
    w->bytes = w->stat;
    if (a->weight_out) {
        w->z = w->stat + round16(U * G * 8);
        w->bytes = w->z + U * cap * w->Gp * 4;
    }
    return SKV_OK;
}

// ------------------------------------------------------------------ eviction

struct EvictSpace { int64_t to, of, count, len, bytes; int list_cap; };

int evict_space(const skv_paged_evict_args* a, EvictSpace* w) {
    const skv_paged_cache& c = a->cache;
    if (!good_type(c) || c.batch < 0 || a->budget < 1 || a->recent < 0 || a->sink < 0 ||
        static_cast<int64_t>(a->recent) + a->sink > a->budget)
        return SKV_ERR_INVALID;
    if (c.max_pages < 1 || c.page_size < 1 || static_cast<int64_t>(c.max_pages) * c.page_size > kMaxRows)
        return SKV_ERR_INVALID;
    const int64_t U = static_cast<int64_t>(c.batch) * c.n_kv_heads, cap = static_cast<int64_t>(c.max_pages) * c.page_size;
    if (U > kMaxUnits) return SKV_ERR_INVALID;
    // rows that can move: no more than the budget, no more than lie behind it
    const int64_t behind = cap > a->budget ? cap - a->budget : 0;
    w->list_cap = static_cast<int>(behind < a->budget ? behind : a->budget);
    if (w->list_cap < 1) w->list_cap = 1;
    w->to = 0;
    w->of = round16(U * w->list_cap * 4);
    w->count = w->of + round16(U * w->list_cap * 4);
    w->len = w->count + round16(U * 4);
    w->bytes = w->len + round16(static_cast<int64_t>(c.batch) * 4);
    return SKV_OK;
}

// ------------------------------------------------------------------ attention of prompts

struct PromptSpace { int64_t tiles, stat, note, bytes; };

int prompt_space(const skv_paged_prompt_args* a, PromptSpace* w) {
    const skv_paged_cache& c = a->cache;
    if (!good_type(c, kAll) || c.batch < 0 || a->tokens < 0 || a->reserved || a->n_q_heads < 1 || a->n_q_heads % c.n_kv_heads)
        return SKV_ERR_INVALID;
    const int G = a->n_q_heads / c.n_kv_heads;
    if (G > 8 || !std::isfinite(a->scale) || a->window < 0 || a->sink < 0) return SKV_ERR_INVALID;
    if (c.max_pages < 1 || c.page_size < 1 || static_cast<int64_t>(c.max_pages) * c.page_size > kMaxRows) return SKV_ERR_INVALID;
    if (static_cast<int64_t>(c.batch) * c.n_kv_heads > kMaxUnits) return SKV_ERR_INVALID;
    if (c.dtype != SKV_BF16) return SKV_ERR_UNSUPPORTED;
    // tiles of 128 rows that a unit of 256 / G tokens can see
    const int64_t all = (static_cast<int64_t>(c.max_pages) * c.page_size + 127) / 128;
    w->tiles = a->window ? std::min<int64_t>(all, (static_cast<int64_t>(a->sink) + 127) / 128 + (static_cast<int64_t>(a->window) + 256) / 128 + 2) : all;
    const PromptPlan plan = prompt_plan(a->tokens, c.batch, G, c.n_kv_heads, w->tiles, kMaxSms);
    const int64_t rows = static_cast<int64_t>(plan.parts) * c.n_kv_heads * plan.halves * 128;
    w->stat = rows * c.head_dim * 4;
    w->note = w->stat + rows * 8;
    w->bytes = w->note + (plan.parts ? plan.slots * 16 : 0);
    return SKV_OK;
}

// ------------------------------------------------------------------ status

// The error words are shared by all streams: reading and clearing is one step, so that nothing another
// stream's kernel sets in between is lost.
__device__ int g_taken;
std::mutex g_taking;       // g_taken is one call's at a time
struct ErrorWords { int* at[6]; };
__global__ void k_take_status(ErrorWords words) {
    int taken = 0;
    for (int* word : words.at) {
        const int x = atomicExch(word, 0);
        if (!taken) taken = x;
    }
    g_taken = taken;
}

// what attention takes of the rows: all of them, or the last `window` and the first `sink`
struct Part { const skv_block_scales* scales; int window, sink; };

int attend(const skv_paged_attention_args* a, const Part* part, const char* name, skv_stream stream);

}  // namespace

extern "C" {

int shadowkv_qk_norm_rope(const skv_qk_norm_rope_args* a, skv_stream stream) {
    if (!a) return SKV_ERR_INVALID;
    const skv_paged_cache& c = a->cache;
    if (!good_type(c) || a->tokens < 0 || a->n_q_heads < 0 || a->n_q_heads > (1 << 16)) return SKV_ERR_INVALID;
    const int rd = a->rotary_dim ? a->rotary_dim : c.head_dim;
    if (rd < 16 || rd > c.head_dim || rd % 16) return SKV_ERR_INVALID;
    if (!(a->rope_base > 1.0) || !std::isfinite(a->rope_base)) return SKV_ERR_INVALID;
    if ((a->q_weight || a->k_weight) && !(a->eps > 0.f && std::isfinite(a->eps))) return SKV_ERR_INVALID;
    if (a->tokens == 0) return SKV_OK;
    const int es = key_bytes(c.dtype);
    const bool cache = c.k != nullptr;
    if (cache) {
        if (c.batch < 1) return SKV_ERR_INVALID;
        if (int rc = check_cache(c, true)) return rc;
        if (!a->seq || !a->index || !a->v) return SKV_ERR_INVALID;
        if ((a->row_position || a->row_weight) && a->row_pitch < static_cast<int64_t>(c.max_pages) * c.page_size)
            return SKV_ERR_INVALID;
    } else if (!a->k_out || a->row_position || a->row_weight) {
        return SKV_ERR_INVALID;
    }
    if (!a->positions) return SKV_ERR_INVALID;
    struct { const void* p; int64_t tok, head; bool need; bool written; int heads; } t[] = {
        {a->q, a->q_tok, a->q_head, a->n_q_heads > 0, false, a->n_q_heads},
        {a->k, a->k_tok, a->k_head, true, false, c.n_kv_heads},
        {a->v, a->v_tok, a->v_head, cache, false, c.n_kv_heads},
        {a->q_out, a->q_out_tok, a->q_out_head, a->n_q_heads > 0, true, a->n_q_heads},
        {a->k_out, a->k_out_tok, a->k_out_head, a->k_out != nullptr, true, c.n_kv_heads},
        {a->q_weight, 0, 0, a->q_weight != nullptr, false, 1},
        {a->k_weight, 0, 0, a->k_weight != nullptr, false, 1}};
    for (const auto& x : t) {
        if (!x.need) continue;
        if (!x.p || !aligned16(x.p) || !good_stride(x.tok, es) || !good_stride(x.head, es)) return SKV_ERR_INVALID;
        if (x.written && !apart(a->tokens, x.tok, x.heads, x.head, c.head_dim)) return SKV_ERR_INVALID;
    }
    if (int rc = check_words({a->positions})) return rc;
    if (cache)
        if (int rc = check_words({c.table, a->seq, a->index, a->row_position, a->row_weight})) return rc;
    Device dev;
    if (int rc = device(&dev)) return rc;
    if (int rc = check_memory({a->positions, a->k, a->n_q_heads ? a->q : nullptr, a->n_q_heads ? a->q_out : nullptr, a->k_out,
                               a->q_weight, a->k_weight},
                              dev.id))
        return rc;
    if (cache)
        if (int rc = check_memory({c.k, c.v, c.table, a->seq, a->index, a->v, a->row_position, a->row_weight}, dev.id))
            return rc;
    Range range("shadowkv_qk_norm_rope");
    NormRopeParams p{};
    p.c.H = c.n_kv_heads;
    if (cache) p.c = view(c);
    p.tokens = a->tokens; p.nq = a->n_q_heads; p.rd = rd; p.eps = a->eps;
    p.q_tok = a->q_tok; p.q_head = a->q_head; p.k_tok = a->k_tok; p.k_head = a->k_head;
    p.v_tok = a->v_tok; p.v_head = a->v_head;
    p.qo_tok = a->q_out_tok; p.qo_head = a->q_out_head; p.ko_tok = a->k_out_tok; p.ko_head = a->k_out_head;
    p.q = a->q; p.k = a->k; p.v = a->v; p.qw = a->q_weight; p.kw = a->k_weight; p.qo = a->q_out; p.ko = a->k_out;
    p.positions = a->positions; p.seq = a->seq; p.index = a->index;
    p.row_position = a->row_position; p.row_weight = a->row_weight; p.row_pitch = a->row_pitch;
    // rope_base^(-2i/rd) from the powers of i's bits: six calls of pow, not 64, and off by at most a few
    // units of 2^-53 (64 calls were 1.5 us of the host's 4.4)
    double power[64] = {1.0};
    for (int bit = 1; bit < rd / 2; bit *= 2) {
        const double f = std::pow(a->rope_base, -2.0 * bit / rd);
        for (int i = bit; i < 2 * bit && i < rd / 2; ++i) power[i] = power[i - bit] * f;
    }
    for (int i = 0; i < rd / 2; ++i)
        p.turn[i] = static_cast<uint64_t>(power[i] * (18446744073709551616.0 / 6.283185307179586476925));
    return done(launch_norm_rope(c.dtype, c.head_dim, p, dev.nsm, stream));
}

int64_t shadowkv_paged_attention_workspace(const skv_paged_attention_args* a) {
    if (!a) return SKV_ERR_INVALID;
    AttnSpace w;
    const int rc = attn_space(a, &w);
    return rc ? rc : w.bytes;
}

int shadowkv_paged_attention(const skv_paged_attention_args* a, skv_stream stream) {
    return a ? attend(a, nullptr, "shadowkv_paged_attention", stream) : SKV_ERR_INVALID;
}

}  // extern "C"

namespace {
int attend(const skv_paged_attention_args* a, const Part* part, const char* name, skv_stream stream) {
    const skv_paged_cache& c = a->cache;
    const Types types = part ? kAll : kPlain;
    AttnSpace w;
    if (int rc = attn_space(a, &w, types)) return rc;
    if (c.batch == 0) return SKV_OK;
    if (int rc = check_cache(c, false, types)) return rc;
    const bool codes = c.dtype == SKV_E4M3;
    if (codes)
        if (int rc = check_scales(c, *part->scales)) return rc;
    const int es = wide_bytes(c.dtype), G = a->n_q_heads / c.n_kv_heads;
    if (!c.lens || !a->q || !a->out || !a->workspace || !aligned16(a->q) || !aligned16(a->workspace)) return SKV_ERR_INVALID;
    if (!good_stride(a->q_seq, es) || !good_stride(a->q_head, es)) return SKV_ERR_INVALID;
    if (!aligned16(a->out) || !good_stride(a->out_seq, es) || !good_stride(a->out_head, es)) return SKV_ERR_INVALID;
    if (!apart(c.batch, a->out_seq, a->n_q_heads, a->out_head, c.head_dim)) return SKV_ERR_INVALID;
    if (a->workspace_bytes < w.bytes) return SKV_ERR_INVALID;
    if ((a->weight != nullptr) != (a->weight_out != nullptr)) return SKV_ERR_INVALID;
    if (a->weight && a->row_pitch < static_cast<int64_t>(c.max_pages) * c.page_size) return SKV_ERR_INVALID;
    if (int rc = check_words({c.table, c.lens, a->lse, a->weight, a->weight_out})) return rc;
    Device dev;
    if (int rc = device(&dev)) return rc;
    if (int rc = check_memory({c.k, c.v, c.table, c.lens, a->q, a->out, a->lse, a->weight, a->weight_out, a->workspace}, dev.id))
        return rc;
    if (codes)
        if (int rc = check_memory({part->scales->k, part->scales->v}, dev.id)) return rc;
    Range range(name);
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    PagedCodesParams p{};
    if (codes) {
        const uint32_t d = c.head_dim, box = std::min(c.page_size, 16);
        if (int rc = tensor_map(&p.mk, c.k, 1, d, d, {{c.page_size, c.k_row}, {c.n_kv_heads, c.k_head}, {c.n_pages, c.k_page}},
                                {falls_short('k') ? box / 2 : box, 1, 1}))
            return rc;
        if (int rc = tensor_map(&p.mv, c.v, 1, d, d, {{c.page_size, c.v_row}, {c.n_kv_heads, c.v_head}, {c.n_pages, c.v_page}},
                                {falls_short('v') ? box / 2 : box, 1, 1}))
            return rc;
    }
    p.c = view(c);
    p.span = p.c.cap;
    if (part) {
        // a window of more rows than there can be shows them all
        p.c.window = part->window ? std::min<int64_t>(part->window, kMaxRows) : static_cast<int>(kMaxRows);
        p.c.sink = part->window ? std::min<int64_t>(part->sink, kMaxRows) : 0;
        p.c.s16 = (p.c.sink + 15) & ~15;
        p.span = static_cast<int>(std::min<int64_t>(p.c.cap, static_cast<int64_t>(p.c.window) + 15 + p.c.s16));
        if (codes) {
            p.ks = part->scales->k;
            p.vs = part->scales->v;
            p.lgb = log2_of(part->scales->block);
        }
    }
    p.G = G; p.n_q = a->n_q_heads;
    p.scale_log2 = static_cast<float>((a->scale != 0.f ? static_cast<double>(a->scale) : 1.0 / std::sqrt(double(c.head_dim))) *
                                      1.4426950408889634074);
    p.q_seq = a->q_seq; p.q_head = a->q_head; p.o_seq = a->out_seq; p.o_head = a->out_head;
    p.q = a->q; p.out = a->out; p.lse = a->lse;
    p.joint = reinterpret_cast<Joint*>(ws + w.joint);
    p.rec = reinterpret_cast<float*>(ws + w.rec);
    p.rec_stat = reinterpret_cast<float2*>(ws + w.rec_stat);
    if (a->weight_out) {
        p.stat = reinterpret_cast<float2*>(ws + w.stat);
        p.z = reinterpret_cast<float*>(ws + w.z);
        p.Gp = w.Gp;
        p.weight = a->weight; p.weight_out = a->weight_out; p.row_pitch = a->row_pitch;
    }
    const int ctas = paged_attn_ctas(c.dtype, c.head_dim, dev.nsm < kMaxSms ? dev.nsm : kMaxSms);
    if (codes) return done(launch_paged_codes(c.head_dim, p, ctas, stream));
    return done((part ? launch_paged_span : launch_paged_attn)(c.dtype, c.head_dim, p, ctas, stream));
}
}  // namespace

extern "C" {

int64_t shadowkv_paged_attention_ext_workspace(const skv_paged_attention_ext_args* a) {
    if (!a || a->window < 0 || a->sink < 0) return SKV_ERR_INVALID;
    if (a->attn.weight_out && (a->window || a->attn.cache.dtype == SKV_E4M3)) return SKV_ERR_INVALID;
    AttnSpace w;
    const int rc = attn_space(&a->attn, &w, kAll);
    return rc ? rc : w.bytes;
}

int shadowkv_paged_attention_ext(const skv_paged_attention_ext_args* a, skv_stream stream) {
    if (!a || a->window < 0 || a->sink < 0) return SKV_ERR_INVALID;
    const bool codes = a->attn.cache.dtype == SKV_E4M3;
    if (!codes && (a->scales.k || a->scales.v || a->scales.block || a->scales.reserved)) return SKV_ERR_INVALID;
    if (!codes && !a->window) return shadowkv_paged_attention(&a->attn, stream);
    if (a->attn.weight || a->attn.weight_out) return SKV_ERR_INVALID;
    const Part part{&a->scales, a->window, a->sink};
    return attend(&a->attn, &part, "shadowkv_paged_attention_ext", stream);
}

int shadowkv_paged_quantise(const skv_paged_quantise_args* a, skv_stream stream) {
    if (!a) return SKV_ERR_INVALID;
    const skv_paged_cache& c = a->cache;
    if (!good_type(c, kCodes) || c.batch < 0 || a->tokens < 0 || (a->dtype != SKV_BF16 && a->dtype != SKV_F32)) return SKV_ERR_INVALID;
    if (c.batch == 0 || a->tokens == 0) return SKV_OK;
    if (int rc = check_cache(c, true, kCodes)) return rc;
    if (int rc = check_scales(c, a->scales)) return rc;
    const int es = wide_bytes(a->dtype);
    if (!a->k || !a->v || !a->start || !c.lens || !aligned16(a->k) || !aligned16(a->v)) return SKV_ERR_INVALID;
    for (int64_t s : {a->k_tok, a->k_head, a->v_tok, a->v_head})
        if (!good_stride(s, es)) return SKV_ERR_INVALID;
    if (int rc = check_words({c.table, c.lens, a->start})) return rc;
    Device dev;
    if (int rc = device(&dev)) return rc;
    if (int rc = check_memory({c.k, c.v, c.table, c.lens, a->scales.k, a->scales.v, a->k, a->v, a->start}, dev.id)) return rc;
    Range range("shadowkv_paged_quantise");
    QuantParams p{};
    p.c = view(c);
    p.lgb = log2_of(a->scales.block);
    p.tokens = a->tokens;
    p.slots = quantise_slots(a->tokens, c.batch, p.lgb);
    if (p.slots * 2 * c.n_kv_heads > INT32_MAX) return SKV_ERR_INVALID;
    p.k_tok = a->k_tok; p.k_head = a->k_head; p.v_tok = a->v_tok; p.v_head = a->v_head;
    p.k = a->k; p.v = a->v; p.k_scale = a->scales.k; p.v_scale = a->scales.v; p.start = a->start;
    return done(launch_quantise(a->dtype, c.head_dim, p, stream));
}

int shadowkv_paged_dequantise(const skv_paged_dequantise_args* a, skv_stream stream) {
    if (!a) return SKV_ERR_INVALID;
    const skv_paged_cache& c = a->cache;
    if (!good_type(c, kCodes) || c.batch < 0 || a->tokens < 0 || (a->dtype != SKV_BF16 && a->dtype != SKV_F32)) return SKV_ERR_INVALID;
    if (c.batch == 0 || a->tokens == 0) return SKV_OK;
    if (int rc = check_cache(c, false, kCodes)) return rc;
    if (int rc = check_scales(c, a->scales)) return rc;
    const int es = wide_bytes(a->dtype);
    if (!a->k || !a->v || !a->start || !a->first || !c.lens || !aligned16(a->k) || !aligned16(a->v)) return SKV_ERR_INVALID;
    for (int64_t s : {a->k_tok, a->k_head, a->v_tok, a->v_head})
        if (!good_stride(s, es)) return SKV_ERR_INVALID;
    if (!apart(a->tokens, a->k_tok, c.n_kv_heads, a->k_head, c.head_dim) ||
        !apart(a->tokens, a->v_tok, c.n_kv_heads, a->v_head, c.head_dim))
        return SKV_ERR_INVALID;
    if (int rc = check_words({c.table, c.lens, a->start, a->first})) return rc;
    Device dev;
    if (int rc = device(&dev)) return rc;
    if (int rc = check_memory({c.k, c.v, c.table, c.lens, a->scales.k, a->scales.v, a->k, a->v, a->start, a->first}, dev.id))
        return rc;
    Range range("shadowkv_paged_dequantise");
    DequantParams p{};
    p.c = view(c);
    p.lgb = log2_of(a->scales.block);
    p.tokens = a->tokens;
    p.k_tok = a->k_tok; p.k_head = a->k_head; p.v_tok = a->v_tok; p.v_head = a->v_head;
    p.k = a->k; p.v = a->v; p.k_scale = a->scales.k; p.v_scale = a->scales.v; p.start = a->start; p.first = a->first;
    return done(launch_dequantise(a->dtype, c.head_dim, p, stream));
}

int64_t shadowkv_paged_prompt_attention_workspace(const skv_paged_prompt_args* a) {
    if (!a) return SKV_ERR_INVALID;
    PromptSpace w;
    const int rc = prompt_space(a, &w);
    return rc ? rc : w.bytes;
}

int shadowkv_paged_prompt_attention(const skv_paged_prompt_args* a, skv_stream stream) {
    if (!a) return SKV_ERR_INVALID;
    const skv_paged_cache& c = a->cache;
    PromptSpace w;
    if (int rc = prompt_space(a, &w)) return rc;
    if (c.batch == 0 || a->tokens == 0) return SKV_OK;
    if (int rc = check_cache(c, false)) return rc;
    if (!c.lens || !a->q || !a->out || !a->start || !aligned16(a->q) || !aligned16(a->out)) return SKV_ERR_INVALID;
    for (int64_t s : {a->q_tok, a->q_head, a->out_tok, a->out_head})
        if (!good_stride(s, 2)) return SKV_ERR_INVALID;
    if (!apart(a->tokens, a->out_tok, a->n_q_heads, a->out_head, c.head_dim)) return SKV_ERR_INVALID;
    if (a->workspace_bytes < w.bytes || (w.bytes && (!a->workspace || !aligned16(a->workspace)))) return SKV_ERR_INVALID;
    if (int rc = check_words({c.table, c.lens, a->lse, a->start})) return rc;
    Device dev;
    if (int rc = device(&dev)) return rc;
    if (int rc = check_memory({c.k, c.v, c.table, c.lens, a->q, a->out, a->lse, a->start, w.bytes ? a->workspace : nullptr}, dev.id))
        return rc;
    const uint32_t G = a->n_q_heads / c.n_kv_heads, tq = 128 / G, box = std::min(c.page_size, 128);
    CUtensorMap mq, mk, mv;
    if (int rc = tensor_map(&mq, a->q, 2, c.head_dim, 64, {{a->n_q_heads, a->q_head}, {a->tokens, a->q_tok}}, {G, falls_short('q') ? tq / 2 : tq}))
        return rc;
    if (int rc = tensor_map(&mk, c.k, 2, c.head_dim, 64, {{c.page_size, c.k_row}, {c.n_kv_heads, c.k_head}, {c.n_pages, c.k_page}},
                            {falls_short('k') ? box / 2 : box, 1, 1}))
        return rc;
    if (int rc = tensor_map(&mv, c.v, 2, c.head_dim, 64, {{c.page_size, c.v_row}, {c.n_kv_heads, c.v_head}, {c.n_pages, c.v_page}},
                            {falls_short('v') ? box / 2 : box, 1, 1}))
        return rc;
    Range range("shadowkv_paged_prompt_attention");
    PromptParams p{};
    p.c = view(c);
    p.c.window = static_cast<int>(std::min<int64_t>(a->window, kMaxRows));
    p.c.sink = static_cast<int>(std::min<int64_t>(a->sink, kMaxRows));
    p.G = G; p.n_q = a->n_q_heads; p.tokens = a->tokens; p.tq = tq;
    const PromptPlan plan = prompt_plan(a->tokens, c.batch, G, c.n_kv_heads, w.tiles, dev.nsm < kMaxSms ? dev.nsm : kMaxSms);
    if (plan.slots * c.n_kv_heads > INT32_MAX) return SKV_ERR_INVALID;
    p.halves = plan.halves; p.unit_tokens = plan.halves * tq; p.parts = plan.parts; p.slots = plan.slots;
    p.scale_log2 = static_cast<float>((a->scale != 0.f ? static_cast<double>(a->scale) : 1.0 / std::sqrt(double(c.head_dim))) *
                                      1.4426950408889634074);
    p.down_bits = static_cast<float>(8 + log2_of(p.c.cap));
    p.o_tok = a->out_tok; p.o_head = a->out_head;
    p.start = a->start; p.out = a->out; p.lse = a->lse;
    p.part = static_cast<float*>(a->workspace);
    p.part_stat = reinterpret_cast<float2*>(static_cast<uint8_t*>(a->workspace) + w.stat);
    p.note = reinterpret_cast<int4*>(static_cast<uint8_t*>(a->workspace) + w.note);
    return done(launch_prompt_attn(c.head_dim, p, mq, mk, mv, stream));
}

int64_t shadowkv_paged_evict_workspace(const skv_paged_evict_args* a) {
    if (!a) return SKV_ERR_INVALID;
    EvictSpace w;
    const int rc = evict_space(a, &w);
    return rc ? rc : w.bytes;
}

int shadowkv_paged_evict(const skv_paged_evict_args* a, skv_stream stream) {
    if (!a) return SKV_ERR_INVALID;
    const skv_paged_cache& c = a->cache;
    EvictSpace w;
    if (int rc = evict_space(a, &w)) return rc;
    if (c.batch == 0) return SKV_OK;
    if (int rc = check_cache(c, true)) return rc;
    if (!c.lens || !a->weight || !a->position || !a->weight_out || !a->position_out || !a->lens_out || !a->workspace)
        return SKV_ERR_INVALID;
    if (a->row_pitch < static_cast<int64_t>(c.max_pages) * c.page_size || a->row_pitch % 4) return SKV_ERR_INVALID;
    for (const void* q : {static_cast<const void*>(a->weight), static_cast<const void*>(a->position),
                          static_cast<const void*>(a->weight_out), static_cast<const void*>(a->position_out)})
        if (!aligned16(q)) return SKV_ERR_INVALID;
    if (!aligned16(a->workspace) || a->workspace_bytes < w.bytes) return SKV_ERR_INVALID;
    if (int rc = check_words({c.table, c.lens, a->lens_out})) return rc;
    Device dev;
    if (int rc = device(&dev)) return rc;
    if (int rc = check_memory({c.k, c.v, c.table, c.lens, a->weight, a->position, a->weight_out, a->position_out, a->lens_out,
                               a->workspace},
                              dev.id))
        return rc;
    Range range("shadowkv_paged_evict");
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    EvictParams p{};
    p.c = view(c);
    p.d = c.head_dim; p.es = key_bytes(c.dtype); p.es_v = value_bytes(c.dtype);
    p.budget = a->budget; p.recent = a->recent; p.sink = a->sink;
    p.weight = a->weight; p.position = a->position;
    p.weight_out = a->weight_out; p.position_out = a->position_out; p.row_pitch = a->row_pitch;
    p.lens_out = a->lens_out;
    p.to = reinterpret_cast<int32_t*>(ws + w.to);
    p.of = reinterpret_cast<int32_t*>(ws + w.of);
    p.list_cap = w.list_cap;
    p.count = reinterpret_cast<int32_t*>(ws + w.count);
    p.new_len = reinterpret_cast<int32_t*>(ws + w.len);
    return done(launch_evict(p, dev.nsm, stream));
}

int shadowkv_paged_status(skv_stream stream) {
    std::lock_guard<std::mutex> mine(g_taking);
    ErrorWords words;
    int taken = 0;
    if (cudaStreamSynchronize(stream) != cudaSuccess || norm_rope_err(&words.at[0]) != cudaSuccess ||
        paged_attn_err(&words.at[1]) != cudaSuccess || evict_err(&words.at[2]) != cudaSuccess ||
        paged_span_err(&words.at[3]) != cudaSuccess || quantise_err(&words.at[4]) != cudaSuccess ||
        prompt_err(&words.at[5]) != cudaSuccess) {
        cudaGetLastError();
        return SKV_ERR_CUDA;
    }
    k_take_status<<<1, 1, 0, stream>>>(words);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&taken, g_taken, sizeof(taken), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess) {
        cudaGetLastError();
        return SKV_ERR_CUDA;
    }
    return taken == DEV_ERR_TIMEOUT ? SKV_ERR_TIMEOUT : taken ? SKV_ERR_DEVICE_BOUNDS : SKV_OK;
}

}  // extern "C"
