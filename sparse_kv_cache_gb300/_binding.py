"""ctypes binding of libshadowkv.so (argument marshalling only).

Every step of the decode path runs in the library's CUDA kernels; this module
only turns torch tensors into pointers and streams into handles, and checks
return codes.  There is no fallback: if the library is missing, loading fails.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libshadowkv.so")

SKV_F32, SKV_BF16, SKV_FP8 = 0, 1, 2
DTYPE_CODES = {"f32": SKV_F32, "bf16": SKV_BF16, "fp8": SKV_FP8}
SKV_V_HBM, SKV_V_HOST = 0, 1
HOST_KINDS = {"pinned": 0, "huge": 1}   # SKV_HOST_PINNED, SKV_HOST_HUGE
PHASES = ("score", "select", "rebuild", "fetch", "attn")
FIELDS = {
    "landmarks": 0, "chunk_ids": 1, "outlier_ids": 2, "min_cos": 3, "k_outlier": 4, "v_outlier": 5,
    "k_local": 6, "v_local": 7, "k_cache": 8, "v_cache": 9, "selection": 10, "slot_of_sel": 11,
    "miss_count": 12, "hits_per_step": 13, "a_new": 14,
}
NEW_KEYS = {"exact": 0, "lowrank": 1}
ERRORS = {0: "OK", -1: "INVALID", -2: "OOM", -3: "NOT_PINNED", -4: "CUDA", -5: "DEVICE_BOUNDS",
          -6: "TIMEOUT", -7: "STEP_LIMIT", -8: "UNSUPPORTED"}
EXPORTED = ("shadowkv_validate_config", "shadowkv_prefill_index", "shadowkv_prefill_index_keys",
            "shadowkv_decode_step",
            "shadowkv_stats", "shadowkv_reset_stats", "shadowkv_set_profiling",
            "shadowkv_set_select_event", "shadowkv_export_size", "shadowkv_export", "shadowkv_model", "shadowkv_destroy",
            "shadowkv_strerror", "shadowkv_version", "shadowkv_host_alloc", "shadowkv_host_alloc_kind",
            "shadowkv_host_repair", "shadowkv_host_free",
            "shadowkv_sparse_attention_noalloc", "shadowkv_sparse_attention_noalloc_status",
            "shadowkv_fetch_probe",
            "shadowkv_qk_norm_rope", "shadowkv_paged_attention", "shadowkv_paged_attention_workspace",
            "shadowkv_paged_evict", "shadowkv_paged_evict_workspace", "shadowkv_paged_status")

# C layouts of the paged calls' argument structs (native sizes and alignment, as the header declares
# them).  They are packed in one go: a decode step calls these once per layer, where filling a
# ctypes.Structure field by field would take longer than the kernels.
_CACHE = "6i q 6q q 4P"                                  # skv_paged_cache
_NORM_ROPE = struct.Struct(_CACHE + " 3i f d 10q 7P 3P 2P q")
_PAGED_ATTN = struct.Struct(_CACHE + " i f 4q 5P q P q")
_EVICT = struct.Struct(_CACHE + " 3i 4P q 2P q")


class SkvConfig(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rank", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("n_select", ctypes.c_int32), ("n_outlier", ctypes.c_int32),
                ("local_window", ctypes.c_int32), ("max_new_tokens", ctypes.c_int32),
                ("seq_len", ctypes.c_int64), ("rope_base", ctypes.c_double),
                ("dtype", ctypes.c_int32), ("v_place", ctypes.c_int32),
                ("new_keys", ctypes.c_int32)]


class SkvStats(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int64), ("units", ctypes.c_int64), ("n_select", ctypes.c_int64),
                ("hits", ctypes.c_int64), ("misses", ctypes.c_int64),
                ("alpha_last", ctypes.c_double), ("alpha_mean", ctypes.c_double),
                ("hbm_bytes", ctypes.c_double), ("link_bytes", ctypes.c_double),
                ("scratch_bytes", ctypes.c_double),
                ("phase_ms", ctypes.c_double * 5), ("phase_launches", ctypes.c_int64 * 5),
                ("device_error", ctypes.c_int32), ("kernel_launches", ctypes.c_int64)]


class SkvAttentionArgs(ctypes.Structure):
    _fields_ = [("units", ctypes.c_int32), ("group", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("n_outlier_tokens", ctypes.c_int32), ("n_cache_tokens", ctypes.c_int32),
                ("n_local_tokens", ctypes.c_int32), ("local_capacity", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("k_outlier", ctypes.c_void_p), ("v_outlier", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("k_local", ctypes.c_void_p),
                ("v_local", ctypes.c_void_p), ("out", ctypes.c_void_p)]


class SkvModel(ctypes.Structure):
    _fields_ = [("eq_bandwidth_gbs", ctypes.c_double), ("memory_savings", ctypes.c_double),
                ("compression_ratio", ctypes.c_double), ("hbm_bytes_per_step", ctypes.c_double),
                ("link_bytes_per_step", ctypes.c_double), ("t_pred_us", ctypes.c_double)]


class ShadowKVError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {ERRORS.get(code, code)} ({strerror(code)})")


_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libshadowkv.so (built in-tree by ``sparse_kv_cache_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with sparse_kv_cache_gb300.build.build()")
    lib = ctypes.CDLL(p)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    lib.shadowkv_validate_config.argtypes = [ctypes.POINTER(SkvConfig)]
    lib.shadowkv_prefill_index.argtypes = [ctypes.POINTER(SkvConfig), vp, vp, vp, vp, ctypes.POINTER(vp)]
    lib.shadowkv_prefill_index_keys.argtypes = [ctypes.POINTER(SkvConfig), vp, vp, vp, vp, vp, ctypes.POINTER(vp)]
    lib.shadowkv_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp]
    lib.shadowkv_stats.argtypes = [vp, ctypes.POINTER(SkvStats)]
    lib.shadowkv_reset_stats.argtypes = [vp]
    lib.shadowkv_set_profiling.argtypes = [vp, i32]
    lib.shadowkv_set_select_event.argtypes = [vp, vp]
    lib.shadowkv_export_size.argtypes = [vp, i32]
    lib.shadowkv_export_size.restype = i64
    lib.shadowkv_export.argtypes = [vp, i32, vp, sz, vp]
    lib.shadowkv_model.argtypes = [ctypes.POINTER(SkvConfig), ctypes.c_double, i64, ctypes.c_double,
                                   ctypes.c_double, ctypes.POINTER(SkvModel)]
    lib.shadowkv_destroy.argtypes = [vp]
    lib.shadowkv_destroy.restype = None
    lib.shadowkv_strerror.argtypes = [i32]
    lib.shadowkv_strerror.restype = ctypes.c_char_p
    lib.shadowkv_version.argtypes = []
    lib.shadowkv_host_alloc.argtypes = [sz, ctypes.POINTER(vp)]
    lib.shadowkv_host_alloc.restype = i32
    lib.shadowkv_host_alloc_kind.argtypes = [sz, i32, ctypes.POINTER(vp)]
    lib.shadowkv_host_alloc_kind.restype = i32
    lib.shadowkv_host_repair.argtypes = [vp, sz]
    lib.shadowkv_host_repair.restype = i32
    lib.shadowkv_host_free.argtypes = [vp]
    lib.shadowkv_host_free.restype = None
    lib.shadowkv_sparse_attention_noalloc.argtypes = [ctypes.POINTER(SkvAttentionArgs), vp]
    lib.shadowkv_sparse_attention_noalloc.restype = i32
    lib.shadowkv_sparse_attention_noalloc_status.argtypes = [vp]
    lib.shadowkv_fetch_probe.argtypes = [vp, sz, i64, i32, ctypes.c_uint64, i32, i32, vp,
                                         ctypes.POINTER(ctypes.c_double)]
    lib.shadowkv_fetch_probe.restype = i32
    lib.shadowkv_sparse_attention_noalloc_status.restype = i32
    for name in ("shadowkv_qk_norm_rope", "shadowkv_paged_attention", "shadowkv_paged_evict"):
        getattr(lib, name).argtypes = [ctypes.c_char_p, vp]
        getattr(lib, name).restype = i32
    for name in ("shadowkv_paged_attention_workspace", "shadowkv_paged_evict_workspace"):
        getattr(lib, name).argtypes = [ctypes.c_char_p]
        getattr(lib, name).restype = i64
    lib.shadowkv_paged_status.argtypes = [vp]
    lib.shadowkv_paged_status.restype = i32
    for name in ("shadowkv_validate_config", "shadowkv_prefill_index", "shadowkv_decode_step",
                 "shadowkv_stats", "shadowkv_reset_stats", "shadowkv_set_profiling",
                 "shadowkv_set_select_event", "shadowkv_export", "shadowkv_model", "shadowkv_version"):
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return load().shadowkv_strerror(code).decode()


def _check(code: int, where: str):
    if code != 0:
        raise ShadowKVError(code, where)


def make_config(w=None, **kw) -> SkvConfig:
    """Config from a ``workload.Workload`` (or keyword fields)."""
    f = {}
    if w is not None:
        f = dict(batch=w.batch, n_kv_heads=w.n_kv_heads, n_q_heads=w.n_q_heads,
                 head_dim=w.head_dim, rank=w.rank, chunk=w.chunk, n_select=w.n_select,
                 n_outlier=w.n_outlier, local_window=w.local_window, max_new_tokens=w.steps,
                 seq_len=w.seq_len, rope_base=w.rope_base,
                 dtype=DTYPE_CODES[w.dtype],
                 v_place=SKV_V_HOST if w.v_place == "host" else SKV_V_HBM,
                 new_keys=NEW_KEYS[w.new_keys])
    f.update(kw)
    return SkvConfig(**f)


def validate_config(cfg: SkvConfig) -> int:
    return load().shadowkv_validate_config(ctypes.byref(cfg))


def model(cfg: SkvConfig, alpha: float, t: int, b_gpu_gbs: float, b_link_gbs: float) -> dict:
    out = SkvModel()
    _check(load().shadowkv_model(ctypes.byref(cfg), alpha, t, b_gpu_gbs, b_link_gbs, ctypes.byref(out)),
           "shadowkv_model")
    return {k: getattr(out, k) for k, _ in SkvModel._fields_}


def sparse_attention_noalloc(q, k_outlier, v_outlier, k_cache, v_cache, k_local, v_local, out,
                             units: int, group: int, n_outlier_tokens: int, n_cache_tokens: int,
                             n_local_tokens: int, local_capacity: int, stream=None) -> int:
    """shadowkv_sparse_attention_noalloc (bf16 tensors); returns the status code."""
    a = SkvAttentionArgs(units=units, group=group, dtype=SKV_BF16, n_outlier_tokens=n_outlier_tokens,
                         n_cache_tokens=n_cache_tokens, n_local_tokens=n_local_tokens,
                         local_capacity=local_capacity, q=_ptr(q), k_outlier=_ptr(k_outlier),
                         v_outlier=_ptr(v_outlier), k_cache=_ptr(k_cache), v_cache=_ptr(v_cache),
                         k_local=_ptr(k_local), v_local=_ptr(v_local), out=_ptr(out))
    return load().shadowkv_sparse_attention_noalloc(ctypes.byref(a), _stream(stream))


def sparse_attention_noalloc_setup(stream=None) -> int:
    """shadowkv_sparse_attention_noalloc with units = 0: the per-device set-up only."""
    a = SkvAttentionArgs(units=0, group=1, dtype=SKV_BF16)
    return load().shadowkv_sparse_attention_noalloc(ctypes.byref(a), _stream(stream))


def sparse_attention_noalloc_status(stream=None) -> int:
    """shadowkv_sparse_attention_noalloc_status: the kept kernel status, cleared on read."""
    return load().shadowkv_sparse_attention_noalloc_status(_stream(stream))


def fetch_probe(src_ptr: int, nbytes: int, n_chunks: int, chunk_bytes: int = 2048, seed: int = 1,
                reps: int = 3, fresh: bool = False, stream=None) -> float:
    """shadowkv_fetch_probe: GB/s of the fetch kernel on random chunks of [src, src + nbytes)
    (fresh: new chunks for every repetition)."""
    g = ctypes.c_double()
    _check(load().shadowkv_fetch_probe(src_ptr, nbytes, n_chunks, chunk_bytes, seed, reps, 1 if fresh else 0,
                                       _stream(stream), ctypes.byref(g)), "shadowkv_fetch_probe")
    return g.value


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


# ---------------------------------------------------------------- paged caches
#
# A decode step makes these calls once per layer, so their host time counts.  What a call's tensors
# look like -- shapes, strides, types, never addresses -- decides all of its checks and most of its
# argument struct; both are worked out once per form and kept, and a call fills in the pointers.

def _refuse(where: str, why: str):
    raise ShadowKVError(-1, f"{where}: {why}")


def _form(t):
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _steps(t, n: int):
    """The first n strides, 0 where a dimension is never stepped through."""
    return tuple(0 if size == 1 else step for size, step in zip(t[0][:n], t[1]))


def _pool_fields(where: str, k, v, table, lens, batch: int):
    """The fields of skv_paged_cache before its pointers, from the forms of the tensors: pools
    [n_pages][H][page_size][d] with any strides over a contiguous head dimension, table int32
    [batch][max_pages], lens int32 [batch]."""
    kd, vd = str(k[2]), str(v[2])
    code = {("torch.bfloat16", "torch.bfloat16"): SKV_BF16, ("torch.float32", "torch.float32"): SKV_F32,
            ("torch.bfloat16", "torch.float8_e5m2"): SKV_FP8}.get((kd, vd))
    if code is None:
        _refuse(where, f"no cache of {kd} keys and {vd} values")
    if len(k[0]) != 4 or k[0] != v[0] or k[1][3] != 1 or v[1][3] != 1:
        _refuse(where, "the pools are [n_pages][n_kv_heads][page_size][head_dim], alike, head_dim contiguous")
    if len(table[0]) != 2 or table[0][0] != batch or table[1][1] != 1 or str(table[2]) != "torch.int32":
        _refuse(where, "table is int32 [batch][max_pages]")
    if lens is not None:
        _vector(where, "lens", lens, batch)
    pages, heads, size, d = k[0]
    return (code, heads, d, size, batch, table[0][1], pages, *_steps(k, 3), *_steps(v, 3),
            table[1][0] if batch > 1 else table[0][1])


def _rows(where: str, name: str, t, dtype: str, batch: int, heads: int, need: int) -> int:
    """Row pitch of a per-row array [batch][n_kv_heads][>= need]."""
    if (len(t[0]) != 3 or t[0][:2] != (batch, heads) or t[0][2] < need or str(t[2]) != dtype
            or t[1] != (heads * t[0][2], t[0][2], 1)):
        _refuse(where, f"{name} is {dtype} [batch][n_kv_heads][max_pages * page_size or more], contiguous")
    return t[0][2]


def _heads(where: str, name: str, t, dtype, shape):
    """Strides over (token or sequence, head) of a [..][heads][d] tensor, head dimension contiguous."""
    if t is None or t[0] != shape or t[1][2] != 1 or t[2] != dtype:
        _refuse(where, f"{name} is {dtype} {list(shape)}, head_dim contiguous")
    return _steps(t, 2)


def _vector(where: str, name: str, t, n: int, dtype: str = "torch.int32"):
    if t is None or t[0] != (n,) or (n > 1 and t[1] != (1,)) or str(t[2]) != dtype:
        _refuse(where, f"{name} is {dtype} [{n}], contiguous")


def _raw_stream(device, stream) -> int:
    """The handle of a call's stream: the given one, or torch's current one."""
    if stream is not None:
        return _stream(stream)
    if device.type != "cuda":
        return 0
    import torch
    try:
        return torch._C._cuda_getCurrentRawStream(device.index)
    except AttributeError:   # a build without the short way
        return torch.cuda.current_stream().cuda_stream


_KEPT_BYTES = 8 << 20


class _Space:
    """A workspace, at the address `at`.  Its lock is held while a call is put into the stream, or the
    kernels of two host threads' calls could come there alternately, with one workspace for both."""
    __slots__ = ("lock", "mem", "at", "size")

    def __init__(self):
        self.lock, self.mem, self.at, self.size = threading.RLock(), None, 0, 0

    def grow(self, nbytes: int, device):
        import torch
        self.mem = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.at, self.size = self.mem.data_ptr(), nbytes


_kept_spaces: dict = {}      # (device, stream) -> _Space of that stream's calls


def _space(nbytes: int, device, stream, raw: int) -> _Space:
    """Workspace of one call, its lock taken: the caller releases it.  Calls on torch's current stream
    run one after the other and share one per stream; a captured call, one on a stream that was
    handed in, and one that needs much have their own from torch's allocator, on the call's stream --
    so neither streams nor graphs that run side by side ever share one."""
    import torch
    if stream is None and device.type == "cuda" and nbytes <= _KEPT_BYTES and not torch.cuda.is_current_stream_capturing():
        space = _kept_spaces.get((device.index, raw))
        if space is None:
            space = _kept_spaces.setdefault((device.index, raw), _Space())
        space.lock.acquire()
        try:
            if space.size < nbytes:
                space.grow(nbytes, device)
        except BaseException:
            space.lock.release()
            raise
        return space
    space = _Space()
    if stream is None or device.type != "cuda":
        space.grow(nbytes, device)
    else:
        with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(raw, device)):
            space.grow(nbytes, device)
    space.lock.acquire()
    return space


@functools.lru_cache(maxsize=1024)
def _norm_rope_plan(q, k, positions, q_out, k_out, q_weight, k_weight, v, k_cache, v_cache, table, seq, index, position,
                    weight, rotary_dim, eps, rope_base):
    w = "qk_norm_rope"
    if len(q[0]) != 3 or len(k[0]) != 3 or str(q[2]) not in ("torch.bfloat16", "torch.float32"):
        _refuse(w, "q is bf16 or fp32 [tokens][n_q_heads][d], k [tokens][n_kv_heads][d]")
    (n, nq, d), nk, dt = q[0], k[0][1], q[2]
    qs, ks = _heads(w, "q", q, dt, (n, nq, d)), _heads(w, "k", k, dt, (n, nk, d))
    qo = _heads(w, "q_out", q_out, dt, (n, nq, d))
    ko = _heads(w, "k_out", k_out, dt, (n, nk, d)) if k_out is not None else (0, 0)
    for name, x in (("q_weight", q_weight), ("k_weight", k_weight)):
        if x is not None:
            _vector(w, name, x, d, str(dt))
    _vector(w, "positions", positions, n)
    vs, pitch = (0, 0), 0
    if k_cache is not None:
        if v is None or v_cache is None or table is None:
            _refuse(w, "an append takes v, k_cache, v_cache, table, seq and index")
        if len(k_cache[0]) != 4 or k_cache[2] != dt or k_cache[0][1] != nk or k_cache[0][3] != d:
            _refuse(w, f"k_cache is {dt} [n_pages][{nk}][page_size][{d}]")
        batch = table[0][0]
        cache = _pool_fields(w, k_cache, v_cache, table, None, batch)
        vs = _heads(w, "v", v, dt, (n, nk, d))
        _vector(w, "seq", seq, n)
        _vector(w, "index", index, n)
        need = table[0][1] * k_cache[0][2]
        if position is not None:
            pitch = _rows(w, "position", position, "torch.int32", batch, nk, need)
        if weight is not None:
            wp = _rows(w, "weight", weight, "torch.float32", batch, nk, need)
            if position is not None and wp != pitch:
                _refuse(w, "position and weight have rows of different lengths")
            pitch = wp
    else:
        if any(x is not None for x in (position, weight, v_cache, table, seq, index)):
            _refuse(w, "v_cache, table, seq, index, position and weight go with k_cache")
        cache = (SKV_F32 if str(dt) == "torch.float32" else SKV_BF16, nk, d) + (0,) * 11
    return cache, (n, nq, rotary_dim, eps, rope_base, *qs, *ks, *vs, *qo, *ko), pitch


def qk_norm_rope(q, k, positions, q_out, k_out=None, *, q_weight=None, k_weight=None, eps: float = 1e-6,
                 rope_base: float = 500000.0, rotary_dim: int = 0, v=None, k_cache=None, v_cache=None, table=None,
                 seq=None, index=None, position=None, weight=None, stream=None):
    """shadowkv_qk_norm_rope: norm (where a weight is given) and rotation of q [T][n_q][d] and
    k [T][H][d] at int32 positions [T] into q_out and k_out; with k_cache, v_cache and table also
    the append of k and v as row index[t] of sequence seq[t], with row_position and row_weight in
    position and weight [batch][H][rows] where given.  Returns (q_out, k_out)."""
    cache, fixed, pitch = _norm_rope_plan(
        _form(q), _form(k), _form(positions), _form(q_out), _form(k_out), _form(q_weight), _form(k_weight),
        _form(v) if k_cache is not None else None, _form(k_cache), _form(v_cache), _form(table), _form(seq), _form(index),
        _form(position), _form(weight), rotary_dim, eps, rope_base)
    if k_cache is None:
        pools, more = (0, 0, 0, 0), (0, 0, 0)
    else:
        pools = (k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), 0)
        more = (v.data_ptr(), seq.data_ptr(), index.data_ptr())
    packed = _NORM_ROPE.pack(
        *cache, *pools, *fixed, q.data_ptr(), k.data_ptr(), more[0], _ptr(q_weight) or 0, _ptr(k_weight) or 0,
        q_out.data_ptr(), _ptr(k_out) or 0, positions.data_ptr(), more[1], more[2], _ptr(position) or 0, _ptr(weight) or 0,
        pitch)
    _check(load().shadowkv_qk_norm_rope(packed, _raw_stream(q.device, stream)), "shadowkv_qk_norm_rope")
    return q_out, k_out


@functools.lru_cache(maxsize=1024)
def _paged_attention_plan(q, k_cache, v_cache, table, lens, out, lse, weight, weight_out, scale):
    w = "paged_attention"
    if len(q[0]) != 3:
        _refuse(w, "q is [batch][n_q_heads][d]")
    batch, nq, d = q[0]
    cache = _pool_fields(w, k_cache, v_cache, table, lens, batch)
    if q[2] != k_cache[2] or cache[2] != d:
        _refuse(w, f"q is {k_cache[2]} [batch][n_q_heads][{cache[2]}]")
    qs, os_ = _heads(w, "q", q, q[2], (batch, nq, d)), _heads(w, "out", out, q[2], (batch, nq, d))
    if lse is not None and (lse[0] != (batch, nq) or lse[1] != (nq, 1) or str(lse[2]) != "torch.float32"):
        _refuse(w, "lse is fp32 [batch][n_q_heads], contiguous")
    pitch = 0
    if weight is not None:
        need = cache[5] * cache[3]
        pitch = _rows(w, "weight", weight, "torch.float32", batch, cache[1], need)
        if _rows(w, "weight_out", weight_out, "torch.float32", batch, cache[1], need) != pitch:
            _refuse(w, "weight and weight_out have rows of different lengths")
    elif weight_out is not None:
        _refuse(w, "weight_out goes with weight")
    # the workspace's size goes by these fields alone
    size = _PAGED_ATTN.pack(*cache[:6], *(0,) * 12, nq, scale, *(0,) * 8, 0 if weight is None else 1, 0, 0, 0)
    nbytes = load().shadowkv_paged_attention_workspace(size)
    if nbytes < 0:
        _check(int(nbytes), "shadowkv_paged_attention_workspace")
    return cache, (nq, scale, *qs, *os_), pitch, nbytes


def paged_attention(q, k_cache, v_cache, table, lens, out, lse=None, weight=None, weight_out=None,
                    scale: float = 0.0, stream=None):
    """shadowkv_paged_attention: attention of q [batch][n_q][d] over each sequence's first lens[b]
    rows of the paged cache into out (and its log-sum-exp into lse [batch][n_q], fp32).  With
    weight [batch][H][rows] the weight that each row received is added to it, in place or into
    weight_out.  scale 0: 1/sqrt(d).  Returns out."""
    if weight is not None and weight_out is None:
        weight_out = weight
    cache, fixed, pitch, nbytes = _paged_attention_plan(
        _form(q), _form(k_cache), _form(v_cache), _form(table), _form(lens), _form(out), _form(lse), _form(weight),
        _form(weight_out), scale)
    device = q.device
    raw = _raw_stream(device, stream)
    space = _space(nbytes, device, stream, raw)
    try:
        packed = _PAGED_ATTN.pack(
            *cache, k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lens.data_ptr(), *fixed, q.data_ptr(),
            out.data_ptr(), _ptr(lse) or 0, _ptr(weight) or 0, _ptr(weight_out) or 0, pitch, space.at, nbytes)
        _check(load().shadowkv_paged_attention(packed, raw), "shadowkv_paged_attention")
    finally:
        space.lock.release()
    return out


@functools.lru_cache(maxsize=1024)
def _paged_evict_plan(k_cache, v_cache, table, lens, weight, position, lens_out, weight_out, position_out, budget, recent,
                      sink):
    w = "paged_evict"
    batch = table[0][0] if len(table[0]) == 2 else -1
    cache = _pool_fields(w, k_cache, v_cache, table, lens, batch)
    need = cache[5] * cache[3]
    pitch = _rows(w, "weight", weight, "torch.float32", batch, cache[1], need)
    for name, t, dt in (("position", position, "torch.int32"), ("weight_out", weight_out, "torch.float32"),
                        ("position_out", position_out, "torch.int32")):
        if _rows(w, name, t, dt, batch, cache[1], need) != pitch:
            _refuse(w, f"weight and {name} have rows of different lengths")
    _vector(w, "lens_out", lens_out, batch)
    size = _EVICT.pack(*cache[:6], *(0,) * 12, budget, recent, sink, *(0,) * 8)
    nbytes = load().shadowkv_paged_evict_workspace(size)
    if nbytes < 0:
        _check(int(nbytes), "shadowkv_paged_evict_workspace")
    return cache, (budget, recent, sink), pitch, nbytes


def paged_evict(k_cache, v_cache, table, lens, weight, position, budget: int, recent: int = 0, sink: int = 0,
                lens_out=None, weight_out=None, position_out=None, stream=None):
    """shadowkv_paged_evict: brings every (sequence, KV head) down to budget rows by the weights
    [batch][H][rows] and int32 positions of its rows.  weight, position and lens are updated in
    place, or into weight_out, position_out and lens_out.  Returns lens_out."""
    lens_out = lens if lens_out is None else lens_out
    weight_out = weight if weight_out is None else weight_out
    position_out = position if position_out is None else position_out
    cache, fixed, pitch, nbytes = _paged_evict_plan(
        _form(k_cache), _form(v_cache), _form(table), _form(lens), _form(weight), _form(position), _form(lens_out),
        _form(weight_out), _form(position_out), budget, recent, sink)
    device = weight.device
    raw = _raw_stream(device, stream)
    space = _space(nbytes, device, stream, raw)
    try:
        packed = _EVICT.pack(
            *cache, k_cache.data_ptr(), v_cache.data_ptr(), table.data_ptr(), lens.data_ptr(), *fixed, weight.data_ptr(),
            position.data_ptr(), weight_out.data_ptr(), position_out.data_ptr(), pitch, lens_out.data_ptr(), space.at, nbytes)
        _check(load().shadowkv_paged_evict(packed, raw), "shadowkv_paged_evict")
    finally:
        space.lock.release()
    return lens_out


def paged_status(stream=None) -> int:
    """shadowkv_paged_status: waits for the stream, then the kept status of the paged calls' kernels of
    all streams as far as they have come, cleared on read."""
    return load().shadowkv_paged_status(_stream(stream))


class HostBuffer:
    """Host memory for values from shadowkv_host_alloc_kind, viewed as a CPU tensor:
    kind "pinned" (page-locked) or "huge" (transparent huge pages read through the
    host's page tables)."""

    def __init__(self, shape, dtype, kind: str = "pinned"):
        import numpy as np
        import torch
        self.shape, self.dtype, self.kind = tuple(shape), dtype, kind
        elem = torch.empty((), dtype=dtype).element_size()
        self.nbytes = int(np.prod(self.shape)) * elem
        p = ctypes.c_void_p()
        _check(load().shadowkv_host_alloc_kind(self.nbytes, HOST_KINDS[kind], ctypes.byref(p)),
               "shadowkv_host_alloc_kind")
        self._p = p
        raw = (ctypes.c_uint8 * self.nbytes).from_address(p.value)
        self.tensor = torch.frombuffer(raw, dtype=torch.uint8).view(dtype).view(self.shape)

    def data_ptr(self) -> int:
        return self._p.value

    def fill_from(self, src, offset_elems: int = 0):
        """Copy a tensor (any device) into the buffer starting at element offset_elems."""
        flat = self.tensor.view(-1)
        s = src.contiguous().view(-1)
        flat[offset_elems:offset_elems + s.numel()].copy_(s)

    def repair(self) -> int:
        """shadowkv_host_repair over the whole buffer (huge-page kind); returns the status."""
        return load().shadowkv_host_repair(self._p, self.nbytes)

    def slice(self, offset_elems: int, shape):
        """A view of part of the buffer (data_ptr() gives its address)."""
        import numpy as np
        n = int(np.prod(shape))
        return self.tensor.view(-1)[offset_elems:offset_elems + n].view(*shape)

    def free(self):
        if getattr(self, "_p", None) and self._p.value:
            self.tensor = None
            load().shadowkv_host_free(self._p)
            self._p = ctypes.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class Layer:
    """One layer's ShadowKV state (the handle of shadowkv_prefill_index)."""

    def __init__(self, cfg: SkvConfig, A, B, V, stream=None, K=None):
        """K: optional exact pre-RoPE keys [b][H][S][d] (pre-filling from exact keys)."""
        lib = load()
        self.cfg = cfg
        self._keep = (A, B, V)   # the library borrows these
        h = ctypes.c_void_p()
        if K is None:
            _check(lib.shadowkv_prefill_index(ctypes.byref(cfg), _ptr(A), _ptr(B), _ptr(V), _stream(stream),
                                              ctypes.byref(h)), "shadowkv_prefill_index")
        else:
            _check(lib.shadowkv_prefill_index_keys(ctypes.byref(cfg), _ptr(A), _ptr(B), _ptr(K), _ptr(V),
                                                   _stream(stream), ctypes.byref(h)),
                   "shadowkv_prefill_index_keys")
        self._h = h

    @property
    def handle(self) -> int:
        return self._h.value

    def decode_step(self, q, k_new, v_new, out, sel_out=None, main=None, side=None):
        _check(load().shadowkv_decode_step(self._h, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out),
                                           _ptr(sel_out), _stream(main),
                                           None if side is None else _stream(side)),
               "shadowkv_decode_step")

    def decode_step_raw(self, q, k_new, v_new, out, sel_out, main, side) -> int:
        """Same call with integer pointers/handles; returns the status code."""
        return load().shadowkv_decode_step(self._h, q, k_new, v_new, out, sel_out, main, side)

    def stats(self, check: bool = True) -> dict:
        s = SkvStats()
        rc = load().shadowkv_stats(self._h, ctypes.byref(s))
        if check:
            _check(rc, "shadowkv_stats")
        d = {k: getattr(s, k) for k, _ in SkvStats._fields_ if k not in ("phase_ms", "phase_launches")}
        d["phase_ms"] = dict(zip(PHASES, list(s.phase_ms)))
        d["phase_launches"] = dict(zip(PHASES, list(s.phase_launches)))
        d["status"] = rc
        return d

    def reset_stats(self):
        _check(load().shadowkv_reset_stats(self._h), "shadowkv_reset_stats")

    def set_profiling(self, on: bool):
        _check(load().shadowkv_set_profiling(self._h, 1 if on else 0), "shadowkv_set_profiling")

    def set_select_event(self, event):
        """Record ``event`` (a torch.cuda.Event, or None to stop) after each step's selection."""
        if event is not None and not event.cuda_event:
            import torch
            event.record(torch.cuda.current_stream())   # torch creates its events on first record
        _check(load().shadowkv_set_select_event(self._h, None if event is None else event.cuda_event),
               "shadowkv_set_select_event")

    def export_size(self, field: str) -> int:
        return load().shadowkv_export_size(self._h, FIELDS[field])

    def export(self, field: str, dst, stream=None):
        _check(load().shadowkv_export(self._h, FIELDS[field], _ptr(dst),
                                      dst.numel() * dst.element_size(), _stream(stream)),
               f"shadowkv_export({field})")

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            load().shadowkv_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
