"""Host side of the generation path: argument checks of its entry points (no GPU: they fail before
any CUDA call), of the binding, and the rotation frequencies."""
import ctypes
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import attn, build

A = 0x10000  # fake, never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.lib()


class CacheStruct(ctypes.Structure):  # attn_kv_cache in the header
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


def cache(**kw):
    a = dict(k=A, v=A, k_scale=None, v_scale=None, page_stride=2 * 64 * 128, num_pages=9, page_size=64,
             dtype=0)
    a.update(kw)
    return CacheStruct(*a.values())


def paged(lib, c=None, **kw):
    a = dict(q=A, cache=ctypes.byref(cache() if c is None else c), table=A, lens=A, o=A, lse=A, B=2,
             H=8, H_kv=2, d=128, max_pages=4, scale=0.1, ws=A, nb=1 << 30)
    a.update(kw)
    return lib.attn_fwd_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -3), (dict(H=-1), -3), (dict(max_pages=-1), -3), (dict(d=96), -2),
    (dict(H_kv=3), -3), (dict(H_kv=0), -3), (dict(q=None), -1), (dict(cache=None), -1),
    (dict(table=None), -1), (dict(lens=None), -1), (dict(o=None), -1), (dict(lse=None), -1),
    (dict(q=A + 8), -4), (dict(o=A + 2), -4), (dict(lse=A + 2), -4), (dict(lens=A + 1), -4),
    (dict(scale=0.0), -7), (dict(scale=float("nan")), -7), (dict(scale=float("inf")), -7),
    (dict(max_pages=1 << 26), -3), (dict(ws=None), -8), (dict(ws=A + 16), -8), (dict(nb=100), -8),
    (dict(B=0), 0), (dict(H=0), 0), (dict(B=0, q=None, cache=None), 0),
])
def test_paged_checks(lib, kw, code):
    assert paged(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=8), -9), (dict(page_size=48), -9), (dict(page_size=512), -9), (dict(dtype=2), -9),
    (dict(num_pages=0), -3), (dict(page_stride=100), -3), (dict(page_stride=2 * 64 * 128 + 4), -3),
    (dict(page_stride=1 << 40), -3), (dict(k=None), -1), (dict(v=A + 8), -4),
    (dict(dtype=1), -1), (dict(dtype=1, k_scale=A, v_scale=A + 4), -4),
    (dict(dtype=1, k_scale=A, v_scale=A, page_stride=2 * 64 * 128 + 8), -3),
])
def test_cache_checks(lib, kw, code):
    assert paged(lib, cache(**kw)) == code
    assert rope(lib, cache=ctypes.byref(cache(**kw)), slots=A) == code


def test_paged_workspace(lib):
    f = lib.attn_fwd_paged_workspace_bytes
    def need(rows, d):  # partial outputs, maxima and sums, each up to 256 bytes
        return sum(-(-n // 256) * 256 for n in (2 * 608 * rows * d * 4, 2 * 608 * rows * 8))

    assert f(2, 8, 2, 128) == need(4, 128)
    assert f(1, 40, 1, 64) == need(20, 64)  # two groups of 20 rows
    assert f(1000, 8, 2, 128) == f(1, 8, 2, 128)
    assert f(2, 8, 3, 128) == f(2, 8, 2, 96) == f(0, 8, 2, 64) == 0


def rope(lib, **kw):
    a = dict(qkv=A, ld=12 * 128, wq=A, wk=A, eps=1e-6, f=A, rot=128, inter=0, rs=1.0, pos=A, q=A, k=A,
             v=A, cache=None, slots=None, B=2, N=5, H=8, H_kv=2, d=128)
    a.update(kw)
    return lib.attn_qkv_rope(*a.values(), None)


def rope_bwd(lib, **kw):
    a = dict(dq=A, dk=A, dv=A, qkv=A, ld=12 * 128, wq=A, wk=A, eps=1e-6, f=A, rot=128, inter=0, rs=1.0,
             pos=A, dqkv=A, ldo=12 * 128, dwq=A, dwk=A, B=2, N=5, H=8, H_kv=2, d=128, ws=A, nb=1 << 30)
    a.update(kw)
    return lib.attn_qkv_rope_bwd(*a.values(), None)


COMMON = [
    (dict(B=-1), -3), (dict(N=-1), -3), (dict(d=80), -2), (dict(rot=8), -3), (dict(rot=144), -3),
    (dict(rot=-16), -3), (dict(H_kv=3), -3), (dict(H_kv=0), -3), (dict(ld=11 * 128), -3),
    (dict(ld=12 * 128 + 4), -3), (dict(qkv=None), -1), (dict(f=None), -1), (dict(pos=None), -1),
    (dict(qkv=A + 8), -4), (dict(wq=A + 2), -4), (dict(f=A + 4), -4), (dict(pos=A + 2), -4),
    (dict(eps=-1.0), -7), (dict(eps=float("nan")), -7), (dict(rs=float("inf")), -7),
    (dict(B=1 << 20, N=1 << 20), -3), (dict(ld=1 << 62), -3),
    (dict(B=0), 0), (dict(N=0), 0), (dict(H=0), 0),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(cache=ctypes.byref(cache())), -1),
    (dict(q=A + 8), -4), (dict(v=A + 2), -4), (dict(q=None, k=None, v=None), 0),
    (dict(cache=ctypes.byref(cache()), slots=A + 4), -4),
])
def test_rope_checks(lib, kw, code):
    assert rope(lib, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(dq=None), -1), (dict(dk=None), -1), (dict(dqkv=None), -1), (dict(dwq=None), -1),
    (dict(dv=A + 8), -4), (dict(dqkv=A + 4), -4), (dict(dwk=A + 2), -4), (dict(ldo=128), -3),
    (dict(ldo=12 * 128 + 2), -3), (dict(ws=None), -8), (dict(ws=A + 16), -8), (dict(nb=10), -8),
])
def test_rope_bwd_checks(lib, kw, code):
    assert rope_bwd(lib, **kw) == code


def test_rope_bwd_workspace(lib):
    f = lib.attn_qkv_rope_bwd_workspace_bytes
    assert f(2, 5, 8, 2, 128) == 304 * 2 * 128 * 4 and f(1, 1, 1, 1, 64) == 304 * 2 * 64 * 4
    assert f(1, 1, 1, 1, 96) == f(0, 1, 1, 1, 64) == f(1, 1, 0, 1, 64) == 0


def slots(lib, **kw):
    a = dict(lens=A, cu=A, table=A, free=A, head=A, slots=A, pos=A, lens_out=A + 64, head_out=A + 64, B=3,
             T=7, max_pages=4, n_free=9, page=16)
    a.update(kw)
    return lib.attn_kv_slots(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -3), (dict(T=-1), -3), (dict(max_pages=-1), -3), (dict(n_free=-1), -3),
    (dict(page=0), -3), (dict(page=65537), -3), (dict(B=16385), -3), (dict(B=0), -3),
    (dict(B=0, T=0), 0), (dict(lens=None), -1), (dict(cu=None), -1), (dict(table=None), -1),
    (dict(free=None), -1), (dict(head=None), -1), (dict(slots=None), -1), (dict(pos=None), -1),
    (dict(lens_out=None), -1), (dict(head_out=None), -1), (dict(slots=A + 4), -4),
    (dict(cu=A + 2), -4), (dict(table=A + 1), -4), (dict(lens_out=A), -9), (dict(head_out=A), -9),
])
def test_slots_checks(lib, kw, code):
    assert slots(lib, **kw) == code


def test_binding_refuses(lib):
    c = attn.kv_cache(2, 2, 16, 64, device="cpu")
    x = torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_fwd_paged(x, c, i, i[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        attn.qkv_rope(torch.zeros(3, 12 * 64, dtype=torch.bfloat16), 8, 2)
    with pytest.raises(ValueError, match="CUDA"):
        attn.qkv_rope_bwd(x, x[:, :2], x[:, :2], torch.zeros(2, 1, 12 * 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        attn.kv_slots(i[:, 0], i[:, 0], 0, i, i[:, 0], i[:1, 0], 16)
    with pytest.raises(TypeError):
        attn.kv_slots([0], i[:, 0], 0, i, i[:, 0], i[:1, 0], 16)
    with pytest.raises(ValueError, match="32 bits"):
        attn.kv_slots(i[:, 0], i[:, 0], 1 << 40, i, i[:, 0], i[:1, 0], 16)


def test_cache_layouts(lib):
    def layout(c, H_kv=2, d=64):
        return attn._native().cache_layout(*c, H_kv, d)

    c = attn.kv_cache(5, 2, 16, 64, device="cpu")
    assert layout(c) == (2 * 16 * 64, 5, 16, 0)
    both = torch.zeros(5, 2, 2, 16, 64, dtype=torch.bfloat16)  # K and V page by page
    assert layout(attn.KVCache(both[:, 0], both[:, 1])) == (2 * 2 * 16 * 64, 5, 16, 0)
    one = torch.zeros(3, 16, 1, 64, dtype=torch.bfloat16).transpose(1, 2)  # one head: its stride is free
    assert layout(attn.KVCache(one, one), 1) == (16 * 64, 3, 16, 0)
    e = attn.kv_cache(5, 2, 16, 64, torch.float8_e4m3fn, "cpu")
    assert layout(e) == (2 * 16 * 64, 5, 16, 1)
    assert layout(attn.KVCache(e.k.view(torch.uint8), e.v.view(torch.uint8), e.k_scale, e.v_scale))[3] == 1
    for bad in (attn.KVCache(c.k.transpose(1, 2), c.v.transpose(1, 2)), attn.KVCache(c.k, c.v[:4]),
                attn.KVCache(e.k, e.v), attn.KVCache(e.k, e.v, e.k_scale, e.v_scale[:4]),
                attn.KVCache(c.k.float(), c.v.float()), attn.KVCache(c.k, both[:, 1]),
                attn.KVCache(both[:, 0, :, ::2], both[:, 1, :, ::2])):
        with pytest.raises(ValueError):
            layout(bad)
    with pytest.raises(ValueError):
        layout(c, H_kv=1)


def test_inv_freq():
    f = attn.rope_inv_freq(8, base=100.0, device="cpu").numpy()
    assert np.allclose(f, [1, 100 ** -0.25, 0.1, 100 ** -0.75], rtol=1e-15) and f.dtype == np.float64
    assert np.allclose(attn.rope_inv_freq(8, base=100.0, factor=4, device="cpu"), f / 4)
    # by wavelength: over 128 positions the pairs turn 20.4, 6.4, 2.04 and 0.64 times
    g = attn.rope_inv_freq(8, base=100.0, factor=4, original_len=128, low=1.0, high=4.0,
                           device="cpu").numpy()
    keep = (128 * 0.1 / (2 * math.pi) - 1) / 3
    assert np.allclose(g, [f[0], f[1], f[2] * (keep + (1 - keep) / 4), f[3] / 4])
    assert attn.rope_inv_freq(0, device="cpu").numel() == 0
