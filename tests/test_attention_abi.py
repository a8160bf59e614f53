"""Refusals of the attention side's entry points: every check runs on the host
before any HIP call, so wrong calls are shown here without a GPU."""

import ctypes
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

import moe_layer_05_amd as mm
from moe_layer_05_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUP, WS = 0, 1, 2, 3, 4
P = 4096                       # a stand-in for an aligned device pointer; never read


@pytest.fixture(scope="module")
def L():
    return binding.lib()


def norm_rope(L, **kw):
    a = dict(q=P, qs=256, k=P, ks=128, pos=P, cs=P, max_pos=10, T=3, qw=P, kw=P, qo=P, qos=256, ko=P,
             kos=128, NHq=2, NHk=1, D=128, R=128, inter=0, f32=0, eps=1e-6)
    a.update(kw)
    return L.moe_qk_norm_rope(binding.pack_norm_rope(*a.values()), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), SHAPE), (dict(NHq=0), SHAPE), (dict(NHk=-1), SHAPE), (dict(R=0), SHAPE),
    (dict(R=144), SHAPE), (dict(R=33), SHAPE), (dict(max_pos=0), SHAPE), (dict(D=0), SHAPE),
    (dict(D=132), UNSUP), (dict(D=520, R=64, qs=2080, ks=2080, qos=2080, kos=2080), UNSUP),
    (dict(R=24), UNSUP), (dict(R=12, inter=1), UNSUP), (dict(eps=-1.0), UNSUP),
    (dict(eps=float("nan")), UNSUP), (dict(eps=float("inf")), UNSUP), (dict(qs=248), UNSUP),
    (dict(qs=260), UNSUP), (dict(ks=120), UNSUP), (dict(qos=255), UNSUP), (dict(kos=64), UNSUP),
    (dict(T=1 << 31), UNSUP), (dict(q=0), NULL), (dict(k=0), NULL), (dict(pos=0), NULL),
    (dict(cs=0), NULL), (dict(qo=0), NULL), (dict(ko=0), NULL), (dict(q=P + 8), UNSUP),
    (dict(qw=P + 2), UNSUP), (dict(ko=P + 4), UNSUP), (dict(T=0), OK),
    (dict(T=0, NHk=0, k=0, ko=0, kw=0, ks=0, kos=0), OK),
])
def test_norm_rope(L, kw, want):
    assert norm_rope(L, **kw) == want


def cache(pages=P, n=4, size=16, heads=2, D=128):
    return ctypes.byref(binding.Cache4(pages, n, size, heads, D))


CACHES = [(dict(n=0), SHAPE), (dict(size=0), SHAPE), (dict(heads=0), SHAPE), (dict(D=-64), SHAPE),
          (dict(size=24), UNSUP), (dict(size=8192), UNSUP), (dict(D=96), UNSUP), (dict(D=512), UNSUP),
          (dict(n=1 << 31), UNSUP), (dict(heads=70000), UNSUP)]


def places(fn, c, **kw):
    a = dict(k=P, ks=256, v=P, vs=256, table=P, ts=5, start=P, cu=P, T=9, B=2, pages=5, tail=0)
    a.update(kw)
    return fn(c, binding.pack_tokens(*a.values()), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(pages=-1), SHAPE), (dict(ts=4), SHAPE),
    (dict(cu=0), SHAPE), (dict(T=1 << 31), UNSUP), (dict(ks=128), UNSUP), (dict(vs=260), UNSUP),
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(table=0), NULL), (dict(start=0), NULL),
    (dict(k=P + 2), UNSUP), (dict(v=P + 8), UNSUP), (dict(T=0), OK), (dict(T=0, B=0, cu=0), OK),
])
def test_cache_write_and_read(L, kw, want):
    assert places(L.moe_cache4_write, cache(), **kw) == want
    assert places(L.moe_cache4_read, cache(), **kw) == want


@pytest.mark.parametrize("c,want", CACHES + [(dict(pages=None), NULL), (dict(pages=P + 8), UNSUP)])
def test_cache_shapes(L, c, want):
    assert places(L.moe_cache4_write, cache(**c)) == want
    assert places(L.moe_cache4_read, cache(**c)) == want
    if "D" not in c and "heads" not in c:
        assert attend(L, cache(**c)) == want


def test_cache_null(L):
    assert places(L.moe_cache4_write, None) == NULL
    assert attend(L, None) == NULL
    assert L.moe_cache4_attend_workspace_bytes(None, 1, 2, 1) == 0


def attend(L, c, **kw):
    a = dict(q=P, qs=512, table=P, ts=5, lens=P, out=P, os=512, lse=0, ws=P, wsb=1 << 40, B=2, pages=5,
             NHq=4, scale=0.1)
    a.update(kw)
    return L.moe_cache4_attend(c, binding.pack_attend(*a.values()), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(NHq=0), SHAPE), (dict(NHq=3), SHAPE), (dict(pages=-1), SHAPE),
    (dict(ts=4), SHAPE), (dict(B=70000), UNSUP), (dict(pages=(1 << 24) + 1, ts=1 << 30), UNSUP),
    (dict(scale=0.0), UNSUP), (dict(scale=-1.0), UNSUP), (dict(scale=float("nan")), UNSUP),
    (dict(scale=float("inf")), UNSUP), (dict(qs=384), UNSUP), (dict(os=516), UNSUP),
    (dict(q=0), NULL), (dict(lens=0), NULL), (dict(out=0), NULL), (dict(table=0), NULL),
    (dict(q=P + 4), UNSUP), (dict(out=P + 8), UNSUP), (dict(B=0), OK),
    (dict(pages=1000, ts=1000, ws=0), WS), (dict(pages=1000, ts=1000, wsb=16), WS),
    (dict(pages=1000, ts=1000, ws=P + 8), UNSUP),
])
def test_attend(L, kw, want):
    assert attend(L, cache(), **kw) == want


def test_attend_workspace(L):
    need = L.moe_cache4_attend_workspace_bytes
    assert need(cache(), 0, 4, 1000) == 0 and need(cache(), 2, 3, 1000) == 0
    assert need(cache(), 2, 4, 1) == 0                     # one split: nothing to join
    assert need(cache(), 1, 4, 1000) > 0
    a, b = need(cache(), 1, 4, 1000), need(cache(), 1, 8, 1000)
    assert b == 2 * a


def prompt(L, **kw):
    a = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, cq=P, ck=P, out=P, os=512, lse=0, ws=0, wsb=0, Tq=9,
             Tk=9, B=2, NHq=4, NKV=2, D=128, causal=1, tail=0, scale=0.1)
    a.update(kw)
    return L.moe_prompt_attention(binding.pack_prompt(*a.values()), None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), SHAPE), (dict(Tq=-1), SHAPE), (dict(Tk=-1), SHAPE), (dict(NHq=3), SHAPE),
    (dict(NKV=0), SHAPE), (dict(D=0), SHAPE), (dict(D=80), UNSUP), (dict(scale=0.0), UNSUP),
    (dict(scale=float("nan")), UNSUP), (dict(Tq=(1 << 31) - 1), UNSUP), (dict(Tk=1 << 31), UNSUP),
    (dict(Tq=1 << 30, NHq=128, qs=16384, os=16384), UNSUP), (dict(qs=384), UNSUP),
    (dict(ks=250), UNSUP), (dict(vs=128), UNSUP), (dict(os=513), UNSUP), (dict(tail=4), UNSUP),
    (dict(ks=(1 << 24) + 8), UNSUP), (dict(vs=1 << 30), UNSUP),
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(cq=0), NULL),
    (dict(ck=0), NULL), (dict(out=0), NULL), (dict(q=P + 8), UNSUP), (dict(v=P + 2), UNSUP),
    (dict(Tq=0), OK), (dict(B=0), OK), (dict(Tk=4096), WS), (dict(Tk=4096, ws=P, wsb=64), WS),
    (dict(Tk=4096, ws=P + 8, wsb=1 << 40), UNSUP),
])
def test_prompt(L, kw, want):
    assert prompt(L, **kw) == want


def test_prompt_workspace(L):
    need = L.moe_prompt_attention_workspace_bytes
    assert need(2, 9, 9, 4, 2, 128) == 0                   # few keys: one split
    assert need(1, 8192, 8192, 32, 4, 128) == 0            # enough query tiles
    assert need(2, 9, 4096, 4, 2, 128) > 0
    assert need(2, 9, 4096, 3, 2, 128) == 0 and need(-1, 9, 4096, 4, 2, 128) == 0


def test_launches_of_more_than_32_bits(L):
    """The largest calls that a launch's 32-bit count of threads holds pass the
    shape checks (and are refused for their null pointer), one more is
    refused."""
    big = dict(NHk=0, k=0, ko=0, kw=0, ks=0, kos=0)
    assert norm_rope(L, T=(1 << 26) - 5, q=0, **big) == NULL
    assert norm_rope(L, T=(1 << 26) - 4, **big) == UNSUP
    most = 16 * (0xFFFFFFFF // 256 - 8)                    # 256 threads for 16 tokens of a head
    for fn in (L.moe_cache4_write, L.moe_cache4_read):
        assert places(fn, cache(heads=1), T=most, k=0, ks=128, vs=128) == NULL
        assert places(fn, cache(heads=1), T=most + 1, ks=128, vs=128) == UNSUP
        assert places(fn, cache(heads=4), T=most, k=0, ks=512, vs=512) == NULL
        assert places(fn, cache(heads=4), T=most + 1, ks=512, vs=512) == UNSUP
    room = (1 << 23) - 9                                   # workgroups of 512 threads
    assert prompt(L, B=room // 2 - 8, q=0) == NULL
    assert prompt(L, B=room // 2 - 7) == UNSUP


def test_binding_refuses_host_tensors():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        mm.qk_norm_rope(x, x, torch.zeros(3, dtype=torch.int64), torch.zeros(4, 64), 64)
    with pytest.raises(TypeError):
        mm.prompt_attention(x, x, x, i32)
    with pytest.raises(TypeError):
        mm.KVCache4.of(torch.zeros(2, 2, 1, 17 * 64, dtype=torch.uint8))
    with pytest.raises(mm.MoEError):
        mm.KVCache4(4, 24, 2, 128)
    with pytest.raises(mm.MoEError):
        mm.KVCache4(0, 16, 2, 128)


def test_null_arguments(L):
    assert L.moe_qk_norm_rope(None, None) == NULL
    assert L.moe_cache4_write(cache(), None, None) == NULL and L.moe_cache4_read(cache(), None, None) == NULL
    assert L.moe_cache4_attend(cache(), None, None) == NULL and L.moe_prompt_attention(None, None) == NULL


def test_struct_layouts_match_c():
    """The packed bytes have the sizes and the offsets of the C structures."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    fields = {
        "moe_cache4": "pages num_pages page_size NKV D",
        "moe_qk_norm_rope_args": "q q_token_stride k k_token_stride positions cos_sin max_pos T q_weight k_weight "
                                 "q_out q_out_token_stride k_out k_out_token_stride NHq NHk D R interleaved "
                                 "weights_f32 eps",
        "moe_cache4_tokens": "k k_token_stride v v_token_stride block_table table_stride start cu_seqlens T B "
                             "max_pages zero_tail",
        "moe_cache4_attend_args": "q q_token_stride block_table table_stride lens out out_token_stride lse workspace "
                                  "workspace_bytes B max_pages NHq scale",
        "moe_prompt_attention_args": "q q_token_stride k k_token_stride v v_token_stride cu_seqlens_q cu_seqlens_k "
                                     "out out_token_stride lse workspace workspace_bytes Tq Tk B NHq NKV D causal "
                                     "zero_tail scale",
    }
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\nint main(void) {\n'
    for t, names in fields.items():
        prog += f'  printf("%zu", sizeof({t}));\n'
        prog += "".join(f'  printf(" %zu", offsetof({t}, {n}));\n' for n in names.split())
        prog += '  printf("\\n");\n'
    prog += "  return 0;\n}\n"
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write(prog)
        r = subprocess.run([gcc, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", f"-I{ROOT}/include", src, "-o",
                            exe], capture_output=True, text=True)
        if r.returncode:
            pytest.skip("cannot compile against hip_runtime_api.h: " + r.stderr[:200])
        rows = [[int(v) for v in line.split()] for line in subprocess.check_output([exe], text=True).splitlines()]
    F = binding.Cache4
    assert rows[0] == [ctypes.sizeof(F)] + [getattr(F, n).offset for n, _ in F._fields_]
    packs = (binding.pack_norm_rope, binding.pack_tokens, binding.pack_attend, binding.pack_prompt)
    for (t, names), row, pack in zip(list(fields.items())[1:], rows[1:], packs):
        n = len(names.split())
        zero = pack(*([0] * n))
        assert len(zero) == row[0], t
        for i in range(n):                       # field i alone is not zero from its offset on
            one = pack(*[1 if j == i else 0 for j in range(n)])
            at = [k for k in range(len(one)) if one[k]]
            assert row[1 + i] <= at[0] < row[1 + i] + 4, (t, names.split()[i])
