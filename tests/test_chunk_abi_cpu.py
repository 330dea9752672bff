"""Refusals of the prompt-chunk entry points, on the CPU: arguments are checked
before anything is launched, so none of the fake pointers is ever used."""
import ctypes

import pytest
import torch

from head_latent_attention_02_b200 import build as B
from head_latent_attention_02_b200 import mla

FAKE = 0x1000
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    B.build()
    return mla.lib()


def _dims(**kw):
    d = dict(H=128, d_c=512, d_r=64, d_n=128, d_v=128, d_model=7168, page_size=64,
             dtype=mla.MLA_BF16, scale=1 / 192 ** 0.5, rope_base=10000.0)
    d.update(kw)
    return mla.Dims(**d)


def _ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


def _rope(L, dims=None, **kw):
    a = dict(dims=ctypes.byref(dims or _dims()), n=4, heads=8, x=FAKE, xt=8 * 64, xh=64, pos=FAKE,
             axes=3, sections=_ints(8, 12, 12), inverse=0, out=FAKE, ot=8 * 64, oh=64, stream=None)
    a.update(kw)
    return L.mla_rope_axes(*a.values())


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(heads=0), dict(axes=0), dict(sections=None), dict(inverse=2), dict(x=None),
    dict(pos=None), dict(out=None), dict(x=FAKE + 1), dict(pos=FAKE + 2),
    dict(sections=_ints(8, 12, 11)), dict(sections=_ints(40, -4, -4)), dict(sections=_ints(8, 30, 2)),
    dict(xt=-1), dict(xh=-64),
    dict(oh=32),            # out's heads overlap
    dict(ot=64),            # out's tokens overlap its heads
    dict(ot=0),
])
def test_rope_refuses(L, kw):
    assert _rope(L, **kw) == INVALID


def test_null_dims(L):
    assert L.mla_rope_axes(None, 4, 8, FAKE, 512, 64, FAKE, 1, _ints(32), 0, FAKE, 512, 64, None) == INVALID
    assert L.mla_append_tokens(None, 1, 4, FAKE, 576, FAKE, FAKE, FAKE, 1, _ints(32), None, 0.0, 0, 0, None,
                               None, FAKE, 4, FAKE, 2, None) == INVALID
    assert L.mla_chunk_attn(None, 1, 4, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, 2, FAKE, 1, _ints(0), 1,
                            64, FAKE, None, FAKE, 0, None) == INVALID


def test_rope_limits_and_empty_call(L):
    assert _rope(L, axes=5, sections=_ints(8, 8, 8, 4, 4)) == UNSUPPORTED
    assert _rope(L, dims=_dims(d_r=256), sections=_ints(128, 0, 0)) == UNSUPPORTED
    assert _rope(L, dims=_dims(d_r=63)) == INVALID
    assert _rope(L, dims=_dims(dtype=3)) == INVALID
    assert _rope(L, dims=_dims(rope_base=0.0)) == INVALID
    assert _rope(L, n=0, x=None, pos=None, out=None) == OK


def _append(L, dims=None, **kw):
    a = dict(dims=ctypes.byref(dims or _dims()), B=2, n=4, kv=FAKE, stride=576, ts=FAKE, row0=FAKE,
             pos=FAKE, axes=1, sections=_ints(32), norm=None, eps=0.0, bc=0, br=0, sc=None, sr=None,
             cache=FAKE, n_pages=4, bt=FAKE, max_pages=2, stream=None)
    a.update(kw)
    return L.mla_append_tokens(*a.values())


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(n=-1), dict(stride=575), dict(kv=None), dict(ts=None), dict(row0=None),
    dict(pos=None), dict(axes=0), dict(sections=_ints(31)), dict(norm=FAKE, eps=-1.0),
    dict(norm=FAKE, eps=float("nan")), dict(cache=None), dict(cache=FAKE + 1), dict(kv=FAKE + 1),
    dict(n_pages=0), dict(bt=None), dict(max_pages=0), dict(sc=FAKE), dict(sr=FAKE),
    dict(bc=4, br=4), dict(bc=4, br=4, sc=FAKE), dict(bc=4, br=4, sc=FAKE, sr=FAKE, cache=FAKE + 2),
])
def test_append_refuses(L, kw):
    assert _append(L, **kw) == INVALID


def test_append_limits_and_empty_call(L):
    low = dict(sc=FAKE, sr=FAKE)
    assert _append(L, bc=3, br=4, **low) == UNSUPPORTED
    assert _append(L, bc=4, br=2, **low) == UNSUPPORTED
    assert _append(L, bc=0, br=4, **low) == UNSUPPORTED
    assert _append(L, dims=_dims(d_c=500), stride=564, bc=2, br=4, **low) == UNSUPPORTED
    assert _append(L, dims=_dims(page_size=32)) == UNSUPPORTED
    assert _append(L, dims=_dims(d_r=192), stride=704, sections=_ints(96)) == UNSUPPORTED
    assert _append(L, n=0, kv=None, ts=None, row0=None, pos=None, cache=None, bt=None) == OK
    assert _append(L, B=0, kv=None, ts=None, row0=None, pos=None, cache=None, bt=None) == OK


def _chunk(L, dims=None, **kw):
    a = dict(dims=ctypes.byref(dims or _dims()), B=2, n=4, q=FAKE, ts=FAKE, q_pos=FAKE, uk=FAKE, uv=FAKE,
             cache=FAKE, n_pages=4, bt=FAKE, max_pages=2, segs=FAKE, max_segs=1, delta=_ints(0), n_ver=1,
             max_rows=256, v=FAKE, lse=None, ws=FAKE, ws_bytes=0, stream=None)
    a.update(kw)
    return L.mla_chunk_attn(*a.values())


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(n=-1), dict(q=None), dict(ts=None), dict(q_pos=None), dict(uk=None), dict(uv=None),
    dict(cache=None), dict(bt=None), dict(segs=None), dict(delta=None), dict(n_ver=0), dict(v=None),
    dict(n_pages=0), dict(max_pages=0), dict(max_segs=0), dict(max_rows=-1), dict(q=FAKE + 8),
    dict(cache=FAKE + 16), dict(v=FAKE + 8), dict(uk=FAKE + 2), dict(uv=FAKE + 2), dict(lse=FAKE + 2),
])
def test_chunk_refuses(L, kw):
    assert _chunk(L, **kw) == INVALID


def test_chunk_limits_and_empty_call(L):
    assert _chunk(L, dims=_dims(scale=0.0)) == INVALID
    assert _chunk(L, dims=_dims(scale=-0.1)) == INVALID
    assert _chunk(L, dims=_dims(scale=float("inf"))) == INVALID
    assert _chunk(L, dims=_dims(d_r=0)) == INVALID
    assert _chunk(L, dims=_dims(page_size=128)) == UNSUPPORTED
    assert _chunk(L, n_ver=9) == UNSUPPORTED
    assert _chunk(L, n_pages=1 << 25) == UNSUPPORTED
    assert _chunk(L, max_pages=1 << 26) == UNSUPPORTED
    assert _chunk(L, max_rows=1 << 31) == UNSUPPORTED
    # generic widths whose query and latent do not fit in shared memory
    assert _chunk(L, dims=_dims(dtype=mla.MLA_F32, d_c=16384)) == UNSUPPORTED
    # a chunk (expanded route): too small a workspace is refused before any launch
    assert _chunk(L, n=4096, max_rows=8192, ws_bytes=4096) == WORKSPACE
    assert _chunk(L, n=4096, max_rows=8192, ws=None) == WORKSPACE
    assert _chunk(L, n=0, q=None, ts=None, q_pos=None, v=None, ws=None) == OK
    assert _chunk(L, B=0, q=None, ts=None, q_pos=None, v=None, ws=None) == OK


def test_sizes_whose_products_overflow(L):
    assert _chunk(L, n_pages=1 << 58) == UNSUPPORTED
    assert _chunk(L, n_pages=(1 << 63) - 1) == UNSUPPORTED
    assert _append(L, dims=_dims(d_c=2 ** 31 - 8)) == INVALID      # rows longer than their stride
    assert _append(L, dims=_dims(d_c=1 << 30), stride=1 << 31, bc=4, br=4, sc=FAKE, sr=FAKE) == UNSUPPORTED
    assert _chunk(L, dims=_dims(H=65536)) == UNSUPPORTED
    f32 = dict(dtype=mla.MLA_F32, d_c=32)
    assert _chunk(L, dims=_dims(**f32, d_r=1 << 30), n_ver=4, delta=_ints(0, 0, 0, 0)) == UNSUPPORTED


def test_chunk_workspace_size(L):
    size = lambda d, B, n, rows, n_ver=1, mp=64, ms=1: L.mla_chunk_workspace_size(
        ctypes.byref(d), B, n, n_ver, mp, ms, rows)
    d = _dims()
    # expanded: keys and values of every row and head, at most about 1 GiB of them at a time
    need = size(d, 1, 2048, 4096)
    assert 4096 * 128 * 512 < need < 1.1 * 4352 * 128 * 512 + 2 ** 21
    assert size(d, 1, 2048, 1 << 20) < 3 * 2 ** 30
    assert size(_dims(dtype=mla.MLA_F32, d_c=32, d_r=16, H=8), 3, 75, 400) == 256
    assert size(d, 0, 4, 64) == 0 and size(d, 1, 0, 64) == 0 and size(d, 1, 4, -1) == 0
    assert size(d, 1, 4, 64, n_ver=9) == 0 and size(d, 1, 4, 64, mp=0) == 0
    assert size(_dims(scale=0.0), 1, 4, 64) == 0
    assert L.mla_chunk_workspace_size(None, 1, 4, 1, 1, 1, 64) == 0


def _linear(L, **kw):
    a = dict(dtype=mla.MLA_BF16, M=4, N=8, K=16, x=FAKE, xs=16, w=FAKE, ws_=16, bias=None, act=0,
             res=None, rs=0, out=FAKE, os=8, ws=None, ws_bytes=0, stream=None)
    a.update(kw)
    return L.mla_linear(*a.values())


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(M=-1), dict(N=-1), dict(K=0), dict(act=3), dict(act=-1), dict(xs=15), dict(ws_=15),
    dict(os=7), dict(res=FAKE, rs=7), dict(x=None), dict(w=None), dict(out=None), dict(x=FAKE + 1),
    dict(w=FAKE + 1), dict(out=FAKE + 1), dict(bias=FAKE + 2), dict(res=FAKE + 1, rs=8),
])
def test_linear_refuses(L, kw):
    assert _linear(L, **kw) == INVALID


def test_linear_empty_call_and_sizes(L):
    assert _linear(L, M=0, x=None, w=None, out=None) == OK
    assert _linear(L, N=0, x=None, w=None, out=None) == OK
    assert L.mla_linear_workspace_size(mla.MLA_F32, 4, 4, 4) == 0
    assert L.mla_linear_workspace_size(mla.MLA_BF16, 0, 4, 4) == 0
    # CUDA-core rows beyond the launch grid
    assert _linear(L, dtype=mla.MLA_F32, M=(1 << 22) + 1) == UNSUPPORTED


def test_binding_refuses_tensors_of_another_kind(monkeypatch):
    """Types, sizes, strides and devices are checked before the call."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)     # CPU tensors answer -1
    monkeypatch.setattr(mla, "_raw_stream", lambda dev: 0)
    d = _dims(H=2)
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros(4, 2, 64, dtype=bf)
    pos = torch.zeros(1, 4, dtype=i32)
    bad = [dict(x=x.float()), dict(x=torch.zeros(4, 2, 32, dtype=bf)), dict(pos=pos.long()),
           dict(pos=torch.zeros(2, 4, dtype=i32)), dict(out=torch.zeros(4, 3, 64, dtype=bf)),
           dict(x=torch.zeros(4, 64, 2, dtype=bf).transpose(1, 2)), dict(pos=torch.zeros(1, 8, dtype=i32)[:, ::2])]
    for kw in bad:
        a = dict(x=x, pos=pos, out=x.clone())
        a.update(kw)
        with pytest.raises(ValueError):
            mla.rope_axes(d, a["x"], a["pos"], [32], a["out"])
    w = torch.zeros(8, 16, dtype=bf)
    with pytest.raises(ValueError):
        mla.linear(torch.zeros(4, 16), w, torch.zeros(4, 8))
    with pytest.raises(ValueError):
        mla.linear(torch.zeros(4, 16, dtype=bf), w, torch.zeros(4, 8, dtype=bf), act="tanh")
    with pytest.raises(ValueError):
        mla.linear(torch.zeros(4, 16, dtype=torch.float16), w.half(), torch.zeros(4, 8).half())
    with pytest.raises(ValueError):
        mla.linear(torch.zeros(16, 4, dtype=bf).T, w, torch.zeros(4, 8, dtype=bf))
    with pytest.raises(ValueError):
        mla.linear(torch.zeros(4, 16, dtype=bf), w, torch.zeros(4, 8, dtype=bf), bias=torch.zeros(8, dtype=bf))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current CUDA device"):
        mla.linear(torch.zeros(4, 16, dtype=bf), w, torch.zeros(4, 8, dtype=bf))
