"""The calls over 8-bit paged caches and windows without a GPU: argument layouts, refusals that the host decides, pins of
the float64 forms."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged_ref as ref
from tests.test_paged_cpu import cache, off, refused, skv  # noqa: F401 (skv is a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn


def codes(batch=2, heads=2, d=128, ps=16, block=8, pages=8, width=4):
    c = cache(batch, heads, d, ps, pages, width, torch.bfloat16)
    c["k_cache"], c["v_cache"] = c["k_cache"].to(E4M3), c["v_cache"].to(E4M3)
    return dict(c, k_scale=torch.ones(pages, heads, ps // block), v_scale=torch.ones(pages, heads, ps // block))


def test_packed_arguments_of_the_further_calls_match_the_header(tmp_path):
    from sparse_kv_cache_gb300 import _binding as b
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc missing")
    pairs = [("skv_paged_attention_ext_args", b._PAGED_ATTN_EXT.size), ("skv_paged_quantise_args", b._QUANTISE.size),
             ("skv_paged_dequantise_args", b._DEQUANTISE.size)]
    import struct
    size = struct.calcsize
    places = [("skv_paged_attention_ext_args", "scales", b._PAGED_ATTN.size), ("skv_paged_attention_ext_args", "sink", b._PAGED_ATTN_EXT.size - 4),
              ("skv_paged_quantise_args", "tokens", size(b._CACHE + b._SCALES)), ("skv_paged_quantise_args", "start", b._QUANTISE.size - 8),
              ("skv_paged_dequantise_args", "k", size(b._CACHE + b._SCALES + "2i 4q"))]
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text('#include "shadowkv.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(){'
                   + "".join(f'printf("%zu ", sizeof({n}));' for n, _ in pairs)
                   + "".join(f'printf("%zu ", offsetof({n}, {f}));' for n, f, _ in places) + "return 0;}\n")
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    assert got == [n for _, n in pairs] + [n for _, _, n in places]


def test_attention_over_codes_refuses(skv):  # noqa: F811
    c, q = codes(), torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    go = lambda **kw: skv.paged_attention(**{**dict(q=q, out=torch.empty_like(q), stream=0), **c, **kw})  # noqa: E731
    rows = torch.zeros(2, 2, 64)
    for bad in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=c["k_scale"].double()), dict(v_scale=c["v_scale"][:4]),
                dict(k_scale=torch.ones(8, 2, 3), v_scale=torch.ones(8, 2, 3)),      # blocks that are no power of two
                dict(k_scale=torch.ones(8, 2, 4), v_scale=torch.ones(8, 2, 4)),      # of four rows
                dict(k_scale=torch.ones(8, 2, 0), v_scale=torch.ones(8, 2, 0)),
                dict(k_scale=torch.ones(8, 2, 4)[..., ::2]), dict(k_scale=torch.ones(2, 8, 2).transpose(0, 1)),
                dict(k_scale=torch.ones(8, 1, 2).expand(8, 2, 2), v_scale=torch.ones(8, 1, 2).expand(8, 2, 2)),
                dict(k_cache=c["k_cache"].to(torch.bfloat16)), dict(v_cache=c["v_cache"].float().to(torch.float8_e5m2)),
                dict(q=q.float(), out=q.float()), dict(weight=rows), dict(weight=rows, window=3)):
        refused(skv, lambda: go(**bad))
    # scales go with codes alone, and codes with no other call
    refused(skv, lambda: skv.paged_attention(q, **cache(), out=torch.empty_like(q), k_scale=c["k_scale"], v_scale=c["v_scale"], stream=0))
    plain = {n: c[n] for n in ("k_cache", "v_cache", "table", "lens")}
    refused(skv, lambda: skv.paged_evict(**plain, weight=rows, position=rows.int(), budget=8, stream=0))
    k = torch.zeros((2, 2, 128), dtype=torch.bfloat16)
    refused(skv, lambda: skv.qk_norm_rope(k, k, c["lens"], k, v=k, k_cache=c["k_cache"], v_cache=c["v_cache"], table=c["table"],
                                          seq=c["lens"], index=c["lens"], stream=0))


def test_a_block_is_no_longer_than_128_rows(skv):  # noqa: F811
    c, q = codes(ps=256, block=256), torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    refused(skv, lambda: skv.paged_attention(q, **c, out=torch.empty_like(q), stream=0))


@pytest.mark.parametrize("bad", [dict(window=-1), dict(sink=-1), dict(window=1.5), dict(window=1 << 31), dict(sink=1 << 31),
                                 dict(window=4, weight=torch.zeros(2, 2, 64))])
def test_windows_are_refused(skv, bad):  # noqa: F811
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    refused(skv, lambda: skv.paged_attention(q, **cache(), out=torch.empty_like(q), stream=0, **bad))


@pytest.mark.parametrize("call", ["paged_quantise", "paged_dequantise"])
def test_writing_and_reading_back_refuse(skv, call):  # noqa: F811
    c, k = codes(), torch.zeros((5, 2, 128), dtype=torch.bfloat16)
    start, first = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    names = ("k", "v") if call == "paged_quantise" else ("k_out", "v_out")

    def go(k=k, v=k.clone(), **kw):
        a = {**c, "start": start, "stream": 0, names[0]: k, names[1]: v, **kw}
        if call == "paged_dequantise":
            a.setdefault("first", first)
        getattr(skv, call)(**a)
    bad = [dict(k=k.half(), v=k.half()), dict(v=k.float()), dict(v=k[:4]), dict(k=k[:, :1], v=k[:, :1]), dict(k=k[..., :64], v=k[..., :64]),
           dict(start=start[:2]), dict(start=start.long()), dict(start=start.repeat(2)[::2]), dict(k=off(k)),
           dict(k=torch.zeros(5 * 2 * 136 + 1, dtype=k.dtype).as_strided((5, 2, 128), (260, 129, 1))),
           dict(k_scale=torch.ones(8, 2, 16), v_scale=torch.ones(8, 2, 16)), dict(v_scale=torch.ones(8, 2, 1)),
           dict(k_cache=c["k_cache"].to(torch.bfloat16), v_cache=c["v_cache"].to(torch.bfloat16)), dict(table=c["table"].long()),
           dict(table=c["table"][0]), dict(lens=c["lens"][:1])]
    if call == "paged_quantise":
        bad.append(dict(k_cache=c["k_cache"][:1].expand(8, -1, -1, -1)))             # pages that are one
    else:
        bad += [dict(first=first[:1]), dict(first=None), dict(k=k[:1].expand(5, -1, -1))]      # one row for five tokens
    for x in bad:
        refused(skv, lambda: go(**x))


def test_c_entries_of_the_further_calls_refuse(skv):  # noqa: F811
    from sparse_kv_cache_gb300 import _binding as b
    lib, host = skv.load(), torch.zeros(64)
    at = (host.data_ptr() + 15) & ~15
    for name in ("shadowkv_paged_attention_ext", "shadowkv_paged_quantise", "shadowkv_paged_dequantise"):
        assert getattr(lib, name)(None, None) == -1
    assert lib.shadowkv_paged_attention_ext_workspace(None) == -1
    pools = (3, 2, 128, 16, 1, 4, 8, 4096, 2048, 128, 4096, 2048, 128, 4, at, at, at, at)
    dev = lib.shadowkv_paged_status(None) == 0
    good = -1 if dev else -4          # as far as the look at the device, or at the memory, which is the host's

    def attend(scales=(at, at, 8, 0), window=0, sink=0, weight=0, kind=3, pools=pools):
        return lib.shadowkv_paged_attention_ext(b._PAGED_ATTN_EXT.pack(
            kind, *pools[1:], 4, 0.0, 512, 128, 512, 128, at, at, 0, weight, weight, 64, at, 1 << 40, *scales, window, sink), None)
    assert attend() == good and attend(window=5, sink=2) == good and attend((0, 0, 0, 0), kind=1, window=3) == good
    for x in (dict(scales=(0, at, 8, 0)), dict(scales=(at, at + 2, 8, 0)), dict(scales=(at, at, 8, 1)), dict(scales=(at, at, 32, 0)),
              dict(scales=(at, at, 4, 0)), dict(scales=(at, at, 12, 0)), dict(window=-1), dict(sink=-1), dict(weight=at),
              dict(kind=1, window=3), dict(kind=4), dict(scales=(0, 0, 0, 0), kind=1, window=3, weight=at)):
        assert attend(**x) == -1, x
    for name, pack in (("shadowkv_paged_quantise", b._QUANTISE), ("shadowkv_paged_dequantise", b._DEQUANTISE)):
        extra = (at,) if pack is b._DEQUANTISE else ()

        def call(scales=(at, at, 8, 0), tokens=3, kind=1, steps=(256, 128, 256, 128), k=at, start=at, cache=pools):
            return getattr(lib, name)(pack.pack(*cache, *scales, tokens, kind, *steps, k, at, start, *extra), None)
        assert call() == good and call(tokens=0) == 0
        for x in (dict(tokens=-1), dict(kind=2), dict(kind=3), dict(k=0), dict(k=at + 8), dict(start=0), dict(start=at + 2),
                  dict(steps=(256, 124, 256, 128)), dict(scales=(at, 0, 8, 0)), dict(scales=(at, at, 32, 0)),
                  dict(cache=(1, *pools[1:])), dict(cache=(*pools[:14], at + 8, *pools[15:])), dict(cache=(*pools[:17], 0))):
            assert call(**x) == -1, x


def test_calls_of_no_tokens_and_no_sequences_do_nothing(skv):  # noqa: F811
    for batch, tokens in ((2, 0), (0, 0), (0, 5)):
        c = codes(batch=batch)
        k, start, first = torch.zeros((tokens, 2, 128), dtype=torch.bfloat16), torch.zeros(batch + 1, dtype=torch.int32), torch.zeros(batch, dtype=torch.int32)
        skv.paged_quantise(k, k, *(c[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "lens")), start, stream=0)
        skv.paged_dequantise(*(c[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "table", "lens")), first, start, k, k.clone(), stream=0)
        q = torch.zeros((tokens, 4, 128), dtype=torch.bfloat16)
        p = cache(batch=batch)
        skv.paged_prompt_attention(q, p["k_cache"], p["v_cache"], p["table"], p["lens"], start, torch.empty_like(q), stream=0)
    c, q = codes(batch=0), torch.zeros((0, 4, 128), dtype=torch.bfloat16)
    skv.paged_attention(q, **c, out=torch.empty_like(q), window=3, sink=1, stream=0)


# ------------------------------------------------------------------ the float64 forms

def test_e4m3_pins():
    x = np.concatenate([np.random.default_rng(0).standard_normal(5000) * np.exp2(np.random.default_rng(1).integers(-14, 8, 5000)),
                        [448.0, -448.0, 0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11, 17.0, 19.0, 464.0 - 17]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    assert np.array_equal(ref.e4m3(x.astype(np.float64)), torch.from_numpy(x).to(E4M3).float().double().numpy())


def test_block_scale_pins():
    one = lambda x: ref.block_scale(np.array([x, -0.5 * x]))  # noqa: E731
    assert one(448.0) == 1.0 and one(448.1) == 2.0 and one(224.0) == 0.5 and one(1.75) == 2.0 ** -8 and one(1.76) == 2.0 ** -7
    assert one(0.0) == 2.0 ** -100 and ref.block_scale(np.array([np.inf, np.nan, 3.0])) == one(3.0)
    got, size = ref.append_block(np.array([[448.0, 3.0]]), 1.0, np.array([[500.0, 0.0]]))
    assert size == 2.0 and np.array_equal(got, [[224.0, 1.5], [256.0, 0.0]])         # 250 lies nearer to 256 than to 240
    got, size = ref.append_block(np.array([[448.0, 3.0]]), 4.0, np.array([[500.0, np.inf]]))
    assert size == 4.0 and np.array_equal(got, [[448.0, 3.0], [128.0, np.nan]], equal_nan=True)


def test_seen_rows_pins():
    assert list(ref.seen_rows(9, 3, 2)) == [0, 1, 7, 8, 9] and list(ref.seen_rows(2, 3, 2)) == [0, 1, 2]
    assert list(ref.seen_rows(3, 0, 0)) == [0, 1, 2, 3] and list(ref.seen_rows(3, 1, 0)) == [3] and len(ref.seen_rows(-1, 2, 2)) == 0


def test_sources_of_the_further_kernels_read_coherently():
    from tests.test_paged_source import code_of
    import re
    for name in ("paged_attn.cuh", "k_paged_span.cu", "k_quantise.cu"):
        assert not re.findall(r"\.nc\b|__ldg\b|__restrict__", code_of(name)), name


# ------------------------------------------------------------------ prompts

def test_packed_arguments_of_prompts_match_the_header(tmp_path):
    from sparse_kv_cache_gb300 import _binding as b
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc missing")
    src, exe = tmp_path / "sizes.c", tmp_path / "sizes"
    src.write_text('#include "shadowkv.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(){printf("%zu %zu %zu", '
                   'sizeof(skv_paged_prompt_args), offsetof(skv_paged_prompt_args, q_tok), offsetof(skv_paged_prompt_args, workspace));return 0;}\n')
    subprocess.run([gcc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    import struct
    assert got == [b._PROMPT.size, struct.calcsize(b._CACHE + " i f 4i"), b._PROMPT.size - 16]


def test_prompt_attention_refuses(skv):  # noqa: F811
    c, q = cache(), torch.zeros((5, 4, 128), dtype=torch.bfloat16)
    start = torch.zeros(3, dtype=torch.int32)
    go = lambda **kw: skv.paged_prompt_attention(**{**dict(q=q, out=torch.empty_like(q), start=start, stream=0), **c, **kw})  # noqa: E731
    odd = torch.zeros((5, 3, 128), dtype=torch.bfloat16)
    many = torch.zeros((5, 18, 128), dtype=torch.bfloat16)
    for bad in (dict(q=q[:4]), dict(q=q.float()), dict(q=q[0]), dict(out=q[:, :2]), dict(out=q.float()), dict(q=odd, out=odd.clone()),
                dict(q=many, out=many.clone()), dict(start=start[:2]), dict(start=start.long()), dict(start=None), dict(lens=c["lens"][:1]),
                dict(table=c["table"].long()), dict(table=c["table"][0]), dict(lse=torch.zeros(5, 2)), dict(window=-1), dict(sink=-1),
                dict(window=2.5), dict(scale=float("nan")), dict(q=off(q)), dict(out=off(q)), dict(out=q[:1].expand(5, -1, -1)),
                dict(k_cache=c["k_cache"].to(E4M3), v_cache=c["v_cache"].to(E4M3)), dict(k_cache=c["k_cache"][:, :, :, :64])):
        refused(skv, lambda: go(**bad))


def test_prompt_entry_and_workspace(skv):  # noqa: F811
    from sparse_kv_cache_gb300 import _binding as b
    lib, host = skv.load(), torch.zeros(64)
    at = (host.data_ptr() + 15) & ~15
    pools = (1, 2, 128, 16, 1, 4, 8, 4096, 2048, 128, 4096, 2048, 128, 4, at, at, at, at)
    dev = lib.shadowkv_paged_status(None) == 0
    assert lib.shadowkv_paged_prompt_attention(None, None) == -1 and lib.shadowkv_paged_prompt_attention_workspace(None) == -1

    def args(pools=pools, heads=4, scale=0.0, window=0, sink=0, tokens=9, reserved=0, steps=(512, 128, 512, 128), q=at, out=at, start=at,
             space=at, nbytes=1 << 40):
        return b._PROMPT.pack(*pools, heads, scale, window, sink, tokens, reserved, *steps, q, out, 0, start, space, nbytes)
    call = lambda **kw: lib.shadowkv_paged_prompt_attention(args(**kw), None)  # noqa: E731
    long = (1, 2, 128, 1024, 1, 4, *pools[6:])
    good = -1 if dev else -4          # as far as the look at the device, or at the memory, which is the host's
    assert call() == good and call(nbytes=0, space=0) == good and call(pools=long) == good
    assert call(tokens=0) == 0 and call(pools=(*pools[:4], 0, *pools[5:])) == 0
    for x in (dict(heads=3), dict(heads=18), dict(heads=0), dict(window=-1), dict(sink=-1), dict(tokens=-1), dict(reserved=1), dict(q=0),
              dict(q=at + 8), dict(out=at + 8), dict(start=0), dict(start=at + 2), dict(steps=(512, 124, 512, 128)),
              dict(steps=(512, 128, 512, 120)), dict(steps=(512, 128, 128, 128)), dict(scale=float("inf")), dict(pools=long, nbytes=0),
              dict(pools=long, space=0), dict(pools=long, space=at + 8), dict(pools=(*pools[:17], 0)), dict(pools=(*pools[:3], 24, *pools[4:]))):
        assert call(**x) == -1, x
    for kind in (0, 2, 3):
        assert call(pools=(kind, *pools[1:])) == -8
    # parts take room, one unit per SM and more takes none; the most that there may be does not overflow
    size = lambda **kw: lib.shadowkv_paged_prompt_attention_workspace(args(**kw))  # noqa: E731
    wide = (1, 2, 128, 1024, 1, 1 << 20, *pools[6:])
    assert size() == 0 and 0 < size(pools=wide) <= 160 * 256 * (128 * 4 + 8) and size(pools=wide, tokens=100000) == 0
    assert size(pools=(1, 1 << 16, 128, 16, 1 << 8, 4, *pools[6:]), heads=1 << 16, tokens=(1 << 31) - 1) == 0
    assert size(pools=wide, window=(1 << 31) - 1, sink=(1 << 31) - 1) == size(pools=wide)


def test_sources_of_prompts_read_coherently():
    from tests.test_paged_source import code_of
    import re
    assert not re.findall(r"\.nc\b|__ldg\b|__restrict__", code_of("k_prompt_attn.cu"))
