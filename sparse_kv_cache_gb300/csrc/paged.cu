// Host side of the paged-cache calls (include/shadowkv.h): argument checks, workspace layout,
// launches and the error words.
#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>
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

int key_bytes(int dtype) { return dtype == SKV_F32 ? 4 : 2; }
int value_bytes(int dtype) { return dtype == SKV_F32 ? 4 : dtype == SKV_FP8 ? 1 : 2; }

bool good_type(const skv_paged_cache& c) {
    return (c.dtype == SKV_F32 || c.dtype == SKV_BF16 || c.dtype == SKV_FP8) && c.n_kv_heads >= 1 &&
           c.n_kv_heads <= (1 << 16) && (c.head_dim == 64 || c.head_dim == 128);
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
int check_cache(const skv_paged_cache& c, bool written) {
    if (!good_type(c)) return SKV_ERR_INVALID;
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

PagedView view(const skv_paged_cache& c) {
    PagedView v{};
    v.k = c.k; v.v = c.v;
    v.k_page = c.k_page; v.k_head = c.k_head; v.k_row = c.k_row;
    v.v_page = c.v_page; v.v_head = c.v_head; v.v_row = c.v_row;
    v.table = c.table; v.table_seq = c.table_seq;
    v.lens = c.lens;
    v.n_pages = c.n_pages;
    v.batch = c.batch; v.H = c.n_kv_heads;
    while ((1 << v.lg) < c.page_size) ++v.lg;
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

// ------------------------------------------------------------------ attention

struct AttnSpace { int Gp; int64_t joint, rec, rec_stat, stat, z, bytes; };

// host-only part of the checks, and the workspace's layout
int attn_space(const skv_paged_attention_args* a, AttnSpace* w) {
    const skv_paged_cache& c = a->cache;
    if (!good_type(c) || c.batch < 0 || a->n_q_heads < 1 || a->n_q_heads % c.n_kv_heads) return SKV_ERR_INVALID;
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

// ------------------------------------------------------------------ status

// The error words are shared by all streams: reading and clearing is one step, so that nothing another
// stream's kernel sets in between is lost.
__device__ int g_taken;
std::mutex g_taking;       // g_taken is one call's at a time
__global__ void k_take_status(int* a, int* b, int* c) {
    const int x = atomicExch(a, 0), y = atomicExch(b, 0), z = atomicExch(c, 0);
    g_taken = x ? x : y ? y : z;
}

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
    if (!a) return SKV_ERR_INVALID;
    const skv_paged_cache& c = a->cache;
    AttnSpace w;
    if (int rc = attn_space(a, &w)) return rc;
    if (c.batch == 0) return SKV_OK;
    if (int rc = check_cache(c, false)) return rc;
    const int es = key_bytes(c.dtype), G = a->n_q_heads / c.n_kv_heads;
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
    Range range("shadowkv_paged_attention");
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    PagedAttnParams p{};
    p.c = view(c);
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
    return done(launch_paged_attn(c.dtype, c.head_dim, p,
                                  paged_attn_ctas(c.dtype, c.head_dim, dev.nsm < kMaxSms ? dev.nsm : kMaxSms), stream));
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
    int *norm = nullptr, *attn = nullptr, *evict = nullptr, taken = 0;
    if (cudaStreamSynchronize(stream) != cudaSuccess || norm_rope_err(&norm) != cudaSuccess ||
        paged_attn_err(&attn) != cudaSuccess || evict_err(&evict) != cudaSuccess) {
        cudaGetLastError();
        return SKV_ERR_CUDA;
    }
    k_take_status<<<1, 1, 0, stream>>>(norm, attn, evict);
    if (cudaGetLastError() != cudaSuccess ||
        cudaMemcpyFromSymbolAsync(&taken, g_taken, sizeof(taken), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess) {
        cudaGetLastError();
        return SKV_ERR_CUDA;
    }
    return taken ? SKV_ERR_DEVICE_BOUNDS : SKV_OK;
}

}  // extern "C"
