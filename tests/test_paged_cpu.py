"""Host side of the paged cache and the filtered sampler: struct layouts,
argument refusals before any launch, RoPE frequencies."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import block_attention_b200 as ba
from block_attention_b200 import build as ba_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"orthrus_filter_args": ba.FilterArgs, "orthrus_rope_scaling": ba.RopeScaling,
           "orthrus_rope_args": ba.RopeArgs, "orthrus_append_args": ba.AppendArgs,
           "orthrus_paged_attn_args": ba.PagedAttnArgs}


@pytest.fixture(scope="module")
def L():
    ba_build.build()
    return ba.lib()


def test_struct_layouts_match_c(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'printf("{name} {f[0]} %zu\\n", offsetof({name}, {f[0]}));'
                  for f in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "orthrus_paged.h"\n'
                   'int main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines():
        name, field, off = line.split()
        cls = STRUCTS[name]
        got = ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset
        assert got == int(off), line


def freqs(rot, theta, kind=0, factor=1.0, ctx=0.0, low=0.0, high=0.0, mscale=0.0):
    f = (ctypes.c_double * max(rot // 2, 1))()
    m = ctypes.c_double()
    s = ba.RopeScaling(kind, factor, ctx, low, high, mscale)
    rc = ba.lib().orthrus_rope_freqs(rot, theta, ctypes.byref(s), f, ctypes.byref(m))
    return rc, np.array(f[:]), m.value


def test_rope_freqs_values(L):
    i = np.arange(32)
    base = 1e6 ** (-2 * i / 64)
    rc, f, m = freqs(64, 1e6)
    assert rc == 0 and m == 1.0
    np.testing.assert_allclose(f, base, rtol=1e-14)
    np.testing.assert_allclose(freqs(64, 1e6, 1, 4.0)[1], base / 4, rtol=1e-14)
    # NTK: the slowest frequency is divided by the factor, the fastest kept
    f = freqs(64, 1e6, 2, 4.0)[1]
    np.testing.assert_allclose(f[0], 1.0, rtol=1e-14)
    np.testing.assert_allclose(f[-1], base[-1] / 4, rtol=1e-12)
    # bands: few turns over the trained length divided, many kept, in between mixed
    f = freqs(64, 1e6, 3, 8.0, 8192.0, 1.0, 4.0)[1]
    turns = 8192 * base / (2 * np.pi)
    np.testing.assert_allclose(f[turns >= 4], base[turns >= 4], rtol=1e-14)
    np.testing.assert_allclose(f[turns <= 1], base[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    t = (turns[mid] - 1) / 3
    np.testing.assert_allclose(f[mid], base[mid] * ((1 - t) / 8 + t), rtol=1e-12)
    # YaRN: the ramp over indexes and the factor on the values
    rc, f, m = freqs(64, 1e6, 4, 8.0, 16384.0, 1.0, 32.0)
    assert m == pytest.approx(0.1 * math.log(8) + 1, rel=1e-15)
    dim = lambda n: 64 * math.log(16384 / (2 * math.pi * n)) / (2 * math.log(1e6))
    lo, hi = math.floor(dim(32)), math.ceil(dim(1))
    t = np.clip((i - lo) / (hi - lo), 0, 1)
    np.testing.assert_allclose(f, base * ((1 - t) + t / 8), rtol=1e-12)
    assert freqs(64, 1e6, 4, 8.0, 16384.0, 1.0, 32.0, 1.5)[2] == 1.5


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=3), dict(theta=1.0), dict(theta=math.nan), dict(kind=5), dict(kind=-1),
    dict(kind=1, factor=0.5), dict(kind=1, factor=math.inf), dict(kind=2, factor=2.0, rot=2),
    dict(kind=3, factor=2.0, ctx=0.0, low=1.0, high=4.0),
    dict(kind=3, factor=2.0, ctx=100.0, low=4.0, high=1.0),
    dict(kind=4, factor=2.0, ctx=100.0, low=0.0, high=1.0),
    dict(kind=4, factor=2.0, ctx=100.0, low=1.0, high=2.0, mscale=-1.0)])
def test_rope_freqs_refusals(L, kw):
    args = dict(rot=64, theta=1e6)
    args.update(kw)
    assert freqs(**args)[0] == -1


def filled(cls, **kw):
    a = cls()
    for name, t in cls._fields_:
        if t is ctypes.c_void_p:
            setattr(a, name, 4096)  # an aligned address that is never dereferenced
    for k, v in kw.items():
        setattr(a, k, v)
    return a


ROPE = dict(dtype=0, layout=0, rows=4, H=2, D=64, rot=64, mscale=1.0, x_row_stride=128,
            x_head_stride=64, out_row_stride=128, out_head_stride=64, out=8192)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -1), (dict(layout=2), -1), (dict(rows=-1), -1), (dict(H=0), -1),
    (dict(rot=63), -1), (dict(rot=66), -1), (dict(rot=-2), -1), (dict(D=1026, rot=2), -2),
    (dict(mscale=math.inf), -1), (dict(inv_freq=None), -1), (dict(inv_freq=4100), -1),
    (dict(x=None), -1), (dict(out=None), -1), (dict(positions=None), -1), (dict(x=4098), -1),
    (dict(x_row_stride=-1), -1), (dict(inverse=2), -1),
    (dict(out=4096, out_row_stride=256), -1), (dict(rows=0), 0)])
def test_rope_refusals(L, kw, code):
    a = filled(ba.RopeArgs, **{**ROPE, **kw})
    assert L.orthrus_rope(ctypes.byref(a), None) == code


APPEND = dict(dtype=1, layers=1, B=2, blk=4, rows=8, Hq=2, Hkv=1, D=64, page_size=16, pages=4,
              max_pages=3, rot=64, layout=0, mscale=1.0, row_starts=None, workspace_bytes=256)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -1), (dict(layers=0), -1), (dict(layers=2), -1), (dict(B=-1), -1),
    (dict(rows=9), -1), (dict(Hq=0), -1), (dict(q=None), -1), (dict(Hkv=0), -1),
    (dict(page_size=0), -1), (dict(pages=0), -1), (dict(max_pages=0), -1), (dict(layout=5), -1),
    (dict(mscale=math.nan), -1), (dict(k=None), -1), (dict(v_pages=None), -1), (dict(k=4097), -1),
    (dict(q_out=None), -1), (dict(page_table=None), -1), (dict(ctx_lens=None), -1),
    (dict(k_row_stride=-8), -1), (dict(row_starts=4096), -1),  # n_rows goes with blocks
    (dict(advance=1, workspace=None), -3), (dict(advance=1, workspace_bytes=255), -3),
    (dict(advance=2), -1), (dict(D=2048, rot=64), -2), (dict(B=0, rows=0), 0),
    (dict(blk=0, rows=0), 0)])
def test_append_refusals(L, kw, code):
    a = filled(ba.AppendArgs, **{**APPEND, **kw})
    assert L.orthrus_paged_append(ctypes.byref(a), None) == code


def test_append_refuses_overlapping_layers(L):
    a = filled(ba.AppendArgs, **{**APPEND, "layers": 2, "q": None, "Hq": 0,
                                 "pages_layer_stride": 4 * 16 * 64 - 1})
    assert L.orthrus_paged_append(ctypes.byref(a), None) == -1


ATTN = dict(dtype=1, mask_mode=0, B=2, Hq=4, Hkv=2, D=64, blk=8, page_size=16, pages=10,
            max_pages=8, max_ctx=128, shared_prefix=0, scale=0.125, workspace_bytes=1 << 40)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("kw,code", [
    (dict(mask_mode=2), -1), (dict(B=-1), -1), (dict(Hq=5), -1), (dict(Hkv=0), -1),
    (dict(blk=0), -1), (dict(blk=33), -2), (dict(Hq=64, blk=5), -2), (dict(D=96), -2),
    (dict(page_size=24), -2), (dict(page_size=8, max_ctx=64), -2), (dict(page_size=512), -2),
    (dict(pages=0), -1), (dict(max_pages=0), -1), (dict(max_ctx=129), -4), (dict(max_ctx=-1), -1),
    (dict(shared_prefix=129), -1), (dict(shared_prefix=-1), -1), (dict(scale=0.0), -1),
    (dict(scale=math.nan), -1), (dict(k_blk=None), -1), (dict(v_blk=None), -1), (dict(q=None), -1),
    (dict(q=4104), -1), (dict(k_blk=4104), -1), (dict(v_pages=None), -1), (dict(out=None), -1),
    (dict(page_table=None), -1), (dict(ctx_lens=None), -1), (dict(B=1 << 20), -2),
    (dict(pages=1 << 28), -2), (dict(B=0), 0)])
def test_paged_attention_refusals(L, dtype, kw, code):
    a = filled(ba.PagedAttnArgs, **{**ATTN, "dtype": dtype, **kw})
    assert L.orthrus_paged_attn(ctypes.byref(a), None) == code


@pytest.mark.parametrize("dtype,ctx,code", [(1, 64 * 16380, -3), (1, 64 * 16381, -2),
                                            (0, 64 * 16381, -2)])
def test_paged_attention_schedule_limit(L, dtype, ctx, code):
    """4096 sequences and 2 kv-heads: 16380 pieces of 64 keys each fit, more do not
    (those that fit are turned away for the workspace, which bf16 always needs)."""
    a = filled(ba.PagedAttnArgs, **{**ATTN, "B": 4096, "max_pages": 1 << 16, "workspace": None,
                                    "dtype": dtype, "max_ctx": ctx})
    assert L.orthrus_paged_attn(ctypes.byref(a), None) == code


@pytest.mark.parametrize("dtype", [0, 1])
def test_paged_attention_workspace(L, dtype):
    a = filled(ba.PagedAttnArgs, **{**ATTN, "dtype": dtype, "max_pages": 500, "max_ctx": 8000})
    need = L.orthrus_paged_attn_workspace(ctypes.byref(a))
    assert need > 0
    a.workspace_bytes = need - 1
    assert L.orthrus_paged_attn(ctypes.byref(a), None) == -3
    a.workspace_bytes, a.workspace = need, 4096 + 128
    assert L.orthrus_paged_attn(ctypes.byref(a), None) == -3
    a.workspace = None
    assert L.orthrus_paged_attn(ctypes.byref(a), None) == -3
    a.dtype = 2
    assert L.orthrus_paged_attn(ctypes.byref(a), None) == -1
    assert L.orthrus_paged_attn_workspace(ctypes.byref(a)) == 0
    b = filled(ba.PagedAttnArgs, **{**ATTN, "dtype": dtype, "shared_prefix": 100})
    assert L.orthrus_paged_attn_workspace(ctypes.byref(b)) >= 0


FILTER = dict(dtype=0, rows=3, vocab=100, row_stride=100)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=4), -1), (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(row_stride=99), -1),
    (dict(rows=65536), -2), (dict(vocab=(1 << 24) + 1, row_stride=1 << 25), -2),
    (dict(logits=None), -1), (dict(logits=4098), -1), (dict(u=None), -1), (dict(idx=None), -1),
    (dict(rows=0), 0)])
def test_filter_refusals(L, kw, code):
    a = filled(ba.FilterArgs, **{**FILTER, **kw})
    assert L.orthrus_vocab_sample_filtered(ctypes.byref(a), None) == code


def test_binding_refuses_cpu_tensors_and_unknown_scalings():
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        ba.rope(x, torch.zeros(2, dtype=torch.int32), None)
    with pytest.raises(ValueError):
        ba.paged_append(x, x, x, x, x, x)
    with pytest.raises(ValueError):
        ba.paged_block_attn(x, None, None, x, x, x, x, 0)
    with pytest.raises(ValueError):
        ba.vocab_sample_filtered(x[0], x[0])
    with pytest.raises(ValueError):
        ba.rope_freqs(64, 1e6, scaling="cubic", device="cpu")
    with pytest.raises(ba.OrthrusError):
        ba.rope_freqs(63, 1e6, device="cpu")
