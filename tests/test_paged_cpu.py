"""The paged-cache calls without a GPU: argument layouts, refusals that the host decides, and pins
of the float64 forms that the GPU tests compare with."""
import math
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def skv():
    import sparse_kv_cache_gb300 as pkg
    from sparse_kv_cache_gb300 import _binding, build
    if not os.path.exists(_binding.LIB_PATH):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("nvcc not available to build the library")
        build.build()
    return pkg


def test_packed_arguments_match_the_header(tmp_path):
    from sparse_kv_cache_gb300 import _binding as b
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc missing")
    src = tmp_path / "sizes.c"
    src.write_text('#include "shadowkv.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(){printf("'
                   + "%zu " * 9 + '\\n", sizeof(skv_paged_cache), offsetof(skv_paged_cache, table_seq), '
                   'sizeof(skv_qk_norm_rope_args), offsetof(skv_qk_norm_rope_args, q), '
                   'offsetof(skv_qk_norm_rope_args, row_pitch), sizeof(skv_paged_attention_args), '
                   'offsetof(skv_paged_attention_args, workspace), sizeof(skv_paged_evict_args), '
                   'offsetof(skv_paged_evict_args, lens_out));return 0;}\n')
    exe = tmp_path / "sizes"
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    import struct
    size = struct.calcsize
    assert got == [size(b._CACHE), size("6i q 6q"), b._NORM_ROPE.size, size(b._CACHE + " 3i f d 10q"),
                   b._NORM_ROPE.size - 8, b._PAGED_ATTN.size, b._PAGED_ATTN.size - 16, b._EVICT.size,
                   size(b._CACHE + " 3i 4P q")]


# ------------------------------------------------------------------ refusals on the host

def cache(batch=2, heads=2, d=128, ps=16, pages=8, width=4, kind=torch.bfloat16, val=None):
    k = torch.zeros((pages, heads, ps, d), dtype=kind)
    v = torch.zeros((pages, heads, ps, d), dtype=kind).to(val or kind)
    return dict(k_cache=k, v_cache=v, table=torch.zeros((batch, width), dtype=torch.int32),
                lens=torch.zeros(batch, dtype=torch.int32))


def off(t):
    """A copy of t that begins one element behind a 16-byte boundary."""
    return torch.zeros(t.numel() + 8, dtype=t.dtype)[1:t.numel() + 1].view(t.shape)


def refused(skv, call):
    with pytest.raises(skv.ShadowKVError) as e:
        call()
    assert e.value.code == -1


@pytest.mark.parametrize("change", [
    dict(d=96), dict(ps=4), dict(ps=24), dict(ps=2048), dict(kind=torch.float16), dict(val=torch.float8_e4m3fn),
    dict(kind=torch.float32, val=torch.bfloat16)])
def test_caches_of_other_forms_are_refused(skv, change):
    c = cache(**change)
    q = torch.zeros((2, 4, c["k_cache"].shape[3]), dtype=c["k_cache"].dtype)
    refused(skv, lambda: skv.paged_attention(q, **c, out=torch.empty_like(q), stream=0))
    rows = torch.zeros((2, 2, c["table"].shape[1] * c["k_cache"].shape[2]))
    refused(skv, lambda: skv.paged_evict(**c, weight=rows, position=rows.int(), budget=8, stream=0))


@pytest.mark.parametrize("heads", [3, 18, 32])
def test_attention_refuses_head_counts(skv, heads):
    c, q = cache(), torch.zeros((2, heads, 128), dtype=torch.bfloat16)     # 1.5, 9 and 16 heads per KV head
    refused(skv, lambda: skv.paged_attention(q, **c, out=torch.empty_like(q), stream=0))


def test_attention_refuses_tensors_of_other_shapes(skv):
    c, q = cache(), torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    out = torch.empty_like(q)
    go = lambda **kw: skv.paged_attention(**{**dict(q=q, out=out, stream=0), **c, **kw})  # noqa: E731
    for bad in (dict(q=q[:1]), dict(q=q.float()), dict(out=out[:, :2]), dict(out=out.float()), dict(q=q[..., :64]),
                dict(lens=c["lens"].long()), dict(table=c["table"].long()), dict(table=c["table"][:1]),
                dict(table=c["table"][:1].expand(2, -1)), dict(table=c["table"].t().contiguous().t()),
                dict(lse=torch.zeros(2, 4, dtype=torch.float64)), dict(lse=torch.zeros(2, 2)),
                dict(weight=torch.zeros(2, 2, 63)), dict(weight=torch.zeros(2, 2, 64, dtype=torch.float64)),
                dict(weight_out=torch.zeros(2, 2, 64)),
                dict(weight=torch.zeros(2, 2, 64), weight_out=torch.zeros(2, 2, 80)),
                dict(out=out[:1].expand(2, -1, -1)),                                   # one row for two results
                dict(q=torch.zeros((2, 4, 256), dtype=torch.bfloat16)[..., ::2]),
                dict(q=torch.zeros(2 * 4 * 129, dtype=torch.bfloat16).as_strided((2, 4, 128), (516, 129, 1))),
                dict(q=off(q)), dict(out=off(q)),                                      # 2 bytes off a 16-byte boundary
                dict(scale=math.inf), dict(scale=math.nan)):
        refused(skv, lambda: go(**bad))


def test_norm_refuses(skv):
    x = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t)  # noqa: E731
    q, k, pos = x(3, 4, 128), x(3, 2, 128), torch.zeros(3, dtype=torch.int32)
    c = cache()
    c.pop("lens")
    at = dict(c, v=k, seq=pos, index=pos)
    go = lambda **kw: skv.qk_norm_rope(**{**dict(q=q, k=k, positions=pos, q_out=q, k_out=k, stream=0), **kw})  # noqa: E731
    rows = torch.zeros(2, 2, 64)
    for bad in (dict(q=q.half(), q_out=q.half()), dict(q_out=q[:2]), dict(k_out=None), dict(k=k.float()),
                dict(positions=pos.long()), dict(positions=pos[:2]), dict(q_weight=x(64)), dict(k_weight=x(128, t=torch.float32)),
                dict(q_weight=x(128), eps=0.0), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=-16),
                dict(rope_base=1.0), dict(rope_base=math.inf), dict(position=rows.int()), dict(weight=rows),
                dict(at, index=None), dict(at, v=None), dict(at, table=None), dict(at, seq=pos[:1]),
                dict(at, weight=rows[..., :60]), dict(at, weight=rows, position=torch.zeros(2, 2, 80).int()),
                dict(q=off(q)), dict(k_out=off(k)), dict(k_weight=off(x(128))),
                dict(at, k_cache=c["k_cache"][:, :1]), dict(at, k_cache=c["k_cache"].float()),
                dict(at, k_cache=c["k_cache"][:1].expand(8, -1, -1, -1)),              # pages that are one
                dict(q_out=q[:1].expand(3, -1, -1))):
        refused(skv, lambda: go(**bad))


def test_evict_refuses(skv):
    c = cache()
    rows = torch.zeros(2, 2, 64)
    go = lambda **kw: skv.paged_evict(**{**c, **dict(weight=rows, position=rows.int(), budget=8, stream=0), **kw})  # noqa: E731
    for bad in (dict(budget=0), dict(budget=-1), dict(recent=-1), dict(sink=-1), dict(recent=5, sink=4),
                dict(weight=rows.double()), dict(position=rows), dict(weight=rows[:, :1]), dict(position=rows[..., :63].int()),
                dict(weight=torch.zeros(2, 2, 66), position=torch.zeros(2, 2, 66).int()),     # rows 8 bytes off
                dict(weight=off(rows)), dict(weight_out=off(rows)), dict(position_out=off(rows.int())),
                dict(weight_out=torch.zeros(2, 2, 65)), dict(lens_out=torch.zeros(3, dtype=torch.int32)),
                dict(lens_out=torch.zeros(2)), dict(table=c["table"][0]),
                dict(k_cache=c["k_cache"][:, :1].expand(-1, 2, -1, -1))):
        refused(skv, lambda: go(**bad))


def test_c_entries_refuse_null_and_host_only_mistakes(skv):
    from sparse_kv_cache_gb300 import _binding as b
    lib = skv.load()
    for name in ("shadowkv_qk_norm_rope", "shadowkv_paged_attention", "shadowkv_paged_evict"):
        assert getattr(lib, name)(None, None) == -1
    for name in ("shadowkv_paged_attention_workspace", "shadowkv_paged_evict_workspace"):
        assert getattr(lib, name)(None) == -1
    # null pools, then rows beyond what 32-bit row numbers hold
    for pages, k in ((4, 0), (1 << 27, 1 << 20)):
        packed = b._PAGED_ATTN.pack(1, 2, 128, 16, 1, pages, 8, 4096, 2048, 128, 4096, 2048, 128, pages, k, k, 64, 64,
                                    4, 0.0, 512, 128, 512, 128, 64, 64, 0, 0, 0, 0, 64, 1 << 30)
        assert lib.shadowkv_paged_attention(packed, None) == -1
        packed = b._EVICT.pack(1, 2, 128, 16, 1, pages, 8, 4096, 2048, 128, 4096, 2048, 128, pages, k, k, 64, 64,
                               8, 0, 0, 64, 64, 64, 64, 1 << 31, 64, 64, 1 << 40)
        assert lib.shadowkv_paged_evict(packed, None) == -1


@pytest.mark.parametrize("size,stride,good", [
    ((8, 2, 16), (4096, 2048, 128), True), ((8, 2, 16), (4096, 128, 256), True), ((8, 2, 16), (2048, 16384, 128), True),
    ((8, 2, 16), (8192, 2048, 128), True),       # with room between pages
    ((8, 1, 16), (2048, 0, 128), True),          # one head: its stride is not stepped through
    ((8, 2, 16), (2048, 2048, 128), False),      # a page's second head is the next page's first
    ((8, 2, 16), (4096, 1920, 128), False),      # heads share a row
    ((8, 2, 16), (4096, 128, 128), False), ((8, 2, 16), (4088, 2048, 128), False), ((8, 2, 16), (4096, 2048, 120), False),
    ((8, 2, 16), (1 << 60, 2048, 128), False)])  # beyond what 64 bits hold
def test_written_pools_whose_rows_overlap_are_refused(skv, size, stride, good):
    from sparse_kv_cache_gb300 import _binding as b
    (pages, heads, ps), host = size, torch.zeros(64)
    at = host.data_ptr() + 15 & ~15
    dev = skv.load().shadowkv_paged_status(None) == 0
    for k, v in ((stride, (4096, 2048, 128)), ((4096, 2048, 128), stride)):
        packed = b._EVICT.pack(1, heads, 128, ps, 1, 4, pages, *k, *v, 4, at, at, at, at, 8, 0, 0, at, at, at, at, 64, at, at,
                               1 << 40)
        # good ones get as far as the look at the device (or at the memory, which is the host's)
        assert skv.load().shadowkv_paged_evict(packed, None) == (-1 if dev or not good else -4)


def test_outputs_whose_rows_overlap_are_refused(skv):
    x = torch.zeros(1 << 12, dtype=torch.bfloat16)
    k, pos = torch.zeros((3, 2, 128), dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for strides in ((256, 128, 1), (128, 256, 1), (128, 128, 1)):     # four heads of three tokens
        q_out = x.as_strided((3, 4, 128), strides)
        refused(skv, lambda: skv.qk_norm_rope(torch.zeros((3, 4, 128), dtype=x.dtype), k, pos, q_out, k.clone(), stream=0))
        c = cache(batch=3)
        refused(skv, lambda: skv.paged_attention(torch.zeros((3, 4, 128), dtype=x.dtype), **c, out=q_out, stream=0))


def test_workspaces_of_too_many_units_are_refused(skv):
    from sparse_kv_cache_gb300 import _binding as b
    c = (1, 1 << 16, 128, 1024, (1 << 31) - 1, 1 << 20, *(0,) * 12)
    assert skv.load().shadowkv_paged_attention_workspace(b._PAGED_ATTN.pack(*c, 1 << 16, 0.0, *(0,) * 8, 64, 0, 0, 0)) == -1
    assert skv.load().shadowkv_paged_evict_workspace(b._EVICT.pack(*c, 8, *(0,) * 10)) == -1
    c = (1, 1 << 16, 128, 1024, 1 << 8, 1 << 20, *(0,) * 12)          # the most that there may be
    assert skv.load().shadowkv_paged_attention_workspace(
        b._PAGED_ATTN.pack(*c, 1 << 19, 0.0, *(0,) * 8, 64, 0, 0, 0)) > 1 << 59
    assert skv.load().shadowkv_paged_evict_workspace(b._EVICT.pack(*c, 1 << 29, *(0,) * 10)) > 1 << 56


def test_host_threads_do_not_share_a_workspace_in_the_middle_of_a_call(skv, monkeypatch):
    """Threads that call on one stream: while one is enqueueing, the workspace is its own."""
    import threading
    import time
    from sparse_kv_cache_gb300 import _binding as b
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw))
    monkeypatch.setattr(b, "_kept_spaces", {})
    busy, clashes, done = set(), [], []

    def work(raw):
        for n in (100, 5000, 200):
            space = b._space(n, torch.device("cuda", 0), None, raw)
            if space.at in busy or space.size < n:
                clashes.append((raw, n))
            busy.add(space.at)
            time.sleep(0.002)
            busy.discard(space.at)
            done.append(raw)
            space.lock.release()

    threads = [threading.Thread(target=work, args=(raw,)) for raw in (0, 0, 0, 7)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not clashes and len(done) == 12


def test_empty_calls_do_nothing(skv):
    q = torch.zeros((0, 4, 128), dtype=torch.bfloat16)
    k = torch.zeros((0, 2, 128), dtype=torch.bfloat16)
    skv.qk_norm_rope(q, k, torch.zeros(0, dtype=torch.int32), q, k, stream=0)
    from sparse_kv_cache_gb300 import _binding as b
    c = (1, 2, 128, 16, 0, 4, 8, 4096, 2048, 128, 4096, 2048, 128, 4, 0, 0, 0, 0)
    assert skv.load().shadowkv_paged_attention(b._PAGED_ATTN.pack(*c, 4, 0.0, *(0,) * 12), None) == 0
    assert skv.load().shadowkv_paged_evict(b._EVICT.pack(*c, 8, 0, 0, *(0,) * 8), None) == 0


def test_host_pools_are_refused_or_need_a_device(skv):
    """Well-formed calls on CPU tensors: refused as host memory, or no device to run on."""
    c, q = cache(), torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    from sparse_kv_cache_gb300 import _binding as b
    pools = [c[n] for n in ("k_cache", "v_cache", "table", "lens")]
    packed = b._PAGED_ATTN.pack(*b._pool_fields("t", *(b._form(t) for t in pools), 2), *(t.data_ptr() for t in pools), 4,
                                0.0, 512, 128, 512, 128, q.data_ptr(), q.data_ptr(), 0, 0, 0, 0, q.data_ptr(), 1 << 40)
    assert skv.load().shadowkv_paged_attention(packed, None) in (-1, -4)


# ------------------------------------------------------------------ the float64 forms

def test_norm_rope_pins():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal(64), rng.standard_normal(64)
    y = ref.norm_rope(x, 0, w, 1e-6, 10000.0, 64)                    # position 0: the norm alone
    assert np.allclose(y, x * w / math.sqrt((x ** 2).sum() / 64 + 1e-6))
    y = ref.norm_rope(x, 12345, None, 1.0, 10000.0, 32)              # a rotation keeps every pair's length
    assert np.allclose(np.hypot(y[:16], y[16:32]), np.hypot(x[:16], x[16:32])) and np.array_equal(y[32:], x[32:])
    # scores of rotated heads depend on the distance alone
    a, b = rng.standard_normal(64), rng.standard_normal(64)
    dot = lambda i, j: ref.norm_rope(a, i, None, 1, 1e4, 64) @ ref.norm_rope(b, j, None, 1, 1e4, 64)  # noqa: E731
    assert abs(dot(907, 900) - dot(7, 0)) < 1e-9
    # the first pair turns by its position in radians
    e = np.zeros(64)
    e[0] = 1
    assert np.allclose(ref.norm_rope(e, 2, None, 1, 1e4, 64)[[0, 32]], [math.cos(2), math.sin(2)])


def test_attend_pins():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    out, lse, p = ref.attend(q, k, v, 0.3)
    want = torch.nn.functional.scaled_dot_product_attention(*(torch.from_numpy(x)[None] for x in (q, k, v)), scale=0.3)
    assert np.allclose(out, want[0].numpy()) and np.allclose(p.sum(1), 1)
    assert np.allclose(lse, np.log(np.exp(0.3 * q @ k.T).sum(1)))
    out, lse, _ = ref.attend(q, k[:0], v[:0], 0.3)
    assert not out.any() and np.all(lse == -np.inf)


def test_evict_pins():
    w = np.array([5.0, 0.0, 3.0, 0.0, 4.0, 0.0, 1.0, 0.0])
    pos = np.arange(8)
    assert list(np.flatnonzero(ref.kept_rows(w, pos, 3, 0, 0))) == [0, 2, 4]
    assert list(np.flatnonzero(ref.kept_rows(w, pos, 3, 2, 0))) == [0, 6, 7]         # the last two positions
    assert list(np.flatnonzero(ref.kept_rows(w, pos, 3, 0, 2))) == [0, 1, 4]         # the first two
    assert list(np.flatnonzero(ref.kept_rows(w, pos, 6, 0, 0))) == [0, 1, 2, 3, 4, 6]  # ties: lower rows
    assert list(np.flatnonzero(ref.kept_rows(w, pos[::-1], 3, 1, 0))) == [0, 2, 4]   # recent by position, not by row
    assert ref.kept_rows(w, pos, 8, 0, 0).all()
    w[5] = np.nan
    assert list(np.flatnonzero(ref.kept_rows(w, pos, 2, 0, 0))) == [0, 5]
    assert ref.moves(np.array([1, 0, 0, 1, 1, 0], bool), 3) == [(1, 3), (2, 4)]
