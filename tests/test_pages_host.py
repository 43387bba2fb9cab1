"""Host side of work over a paged cache beyond one new token a request: argument checks of its entry points (no GPU: they
fail before any CUDA call), workspace sizes, the binding's own checks, and the work split against counting."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

from io_aware_attention_attn_gb300 import attn, build
from test_generation_host import A, CacheStruct, cache

INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.lib()


def call(lib, name, a, kw):
    assert not set(kw) - set(a)
    a.update(kw)
    c = a["cache"]
    if isinstance(c, CacheStruct):
        a["cache"] = ctypes.byref(c)
    return getattr(lib, name)(*a.values(), None)


def varlen(lib, **kw):
    return call(lib, "attn_fwd_paged_varlen", dict(
        q=A, cache=cache(), table=A, lens=A, cu=A, o=A, lse=A, B=2, T=9, H=8, H_kv=2, d=128, max_pages=4, causal=1, scale=0.1,
        ws=A, nb=1 << 40), kw)


def shared(lib, **kw):
    return call(lib, "attn_fwd_paged_shared", dict(
        q=A, cache=cache(), ptable=A, plens=A, cu=A, table=A, lens=A, o=A, lse=A, groups=2, B=9, H=8, H_kv=2, d=128,
        max_prefix=7, max_pages=4, scale=0.1, ws=A, nb=1 << 40), kw)


def strides(*v):
    return (ctypes.c_int64 * 3)(*v)


def write(lib, **kw):
    return call(lib, "attn_kv_write", dict(
        k=A, ks=strides(5 * 2 * 128, 5 * 128, 128), v=A, vs=strides(5 * 2 * 128, 5 * 128, 128), cache=cache(), slots=A, B=3,
        N=5, H_kv=2, d=128), kw)


def read(lib, **kw):
    return call(lib, "attn_kv_read", dict(
        cache=cache(), table=A, cu=A, first=A, k=A, v=A, B=2, T=9, H_kv=2, d=128, max_pages=4), kw)


ATTEND = [
    (dict(B=-1), -3), (dict(H=-1), -3), (dict(H_kv=-1), -3), (dict(max_pages=-1), -3), (dict(d=96), -2), (dict(d=0), -2),
    (dict(H_kv=3), -3), (dict(H_kv=0), -3), (dict(H_kv=16), -3), (dict(q=None), -1), (dict(cache=None), -1),
    (dict(table=None), -1), (dict(lens=None), -1), (dict(cu=None), -1), (dict(o=None), -1), (dict(lse=None), -1),
    (dict(q=A + 8), -4), (dict(o=A + 2), -4), (dict(lse=A + 2), -4), (dict(lens=A + 1), -4), (dict(cu=A + 2), -4),
    (dict(table=A + 3), -4), (dict(scale=0.0), -7), (dict(scale=-1.0), -7), (dict(scale=float("nan")), -7),
    (dict(scale=float("inf")), -7), (dict(max_pages=1 << 26), -3), (dict(max_pages=INT_MAX), -3),
    (dict(ws=None), -8), (dict(ws=A + 16), -8), (dict(nb=1000), -8), (dict(B=0), -3), (dict(H=0), 0),
    (dict(H=0, q=None, cache=None, ws=None), 0),
]


@pytest.mark.parametrize("kw,code", ATTEND + [
    (dict(T=-1), -3), (dict(T=0), 0), (dict(B=0, T=0), 0), (dict(T=INT_MAX), -3), (dict(T=1 << 28, H=16), -3),
    (dict(T=1 << 24, H_kv=8, max_pages=1 << 14), -3),
])
def test_varlen_checks(lib, kw, code):
    assert varlen(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [(k, c) for k, c in ATTEND if "B" not in k] + [
    (dict(B=-1), -3), (dict(groups=-1), -3), (dict(groups=0), -3), (dict(groups=0, B=0), 0), (dict(B=0), 0),
    (dict(max_prefix=-1), -3), (dict(ptable=None), -1), (dict(plens=None), -1), (dict(ptable=A + 2), -4),
    (dict(plens=A + 2), -4), (dict(max_prefix=1 << 26), -3), (dict(B=INT_MAX), -3),
])
def test_shared_checks(lib, kw, code):
    assert shared(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -3), (dict(N=-1), -3), (dict(H_kv=-1), -3), (dict(d=32), -2), (dict(k=None), -1), (dict(ks=None), -1),
    (dict(v=None), -1), (dict(vs=None), -1), (dict(cache=None), -1), (dict(slots=None), -1), (dict(k=A + 8), -4),
    (dict(v=A + 4), -4), (dict(slots=A + 4), -4), (dict(B=1 << 16, N=1 << 16), -3),
    (dict(ks=strides(1284, 640, 128)), -3), (dict(vs=strides(1280, 644, 128)), -3), (dict(vs=strides(1280, 640, 129)), -3),
    (dict(ks=strides(-1280, 640, 128)), -3), (dict(ks=strides(1 << 62, 640, 128)), -3),
    (dict(ks=strides(1 << 60, 1 << 61, 128)), -3), (dict(B=0), 0), (dict(N=0), 0), (dict(H_kv=0), 0),
    (dict(B=0, k=None, cache=None), 0),
])
def test_write_checks(lib, kw, code):
    assert write(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -3), (dict(T=-1), -3), (dict(H_kv=-1), -3), (dict(max_pages=-1), -3), (dict(B=0), -3), (dict(d=127), -2),
    (dict(cache=None), -1), (dict(table=None), -1), (dict(cu=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(k=A + 8), -4), (dict(v=A + 8), -4), (dict(table=A + 2), -4), (dict(cu=A + 1), -4), (dict(first=A + 2), -4),
    (dict(T=INT_MAX), -3), (dict(T=0), 0), (dict(H_kv=0), 0), (dict(B=0, T=0, cu=None), 0),
])
def test_read_checks(lib, kw, code):
    assert read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(page_size=8), -9), (dict(page_size=48), -9), (dict(page_size=512), -9), (dict(dtype=2), -9),
    (dict(num_pages=0), -3), (dict(page_stride=100), -3), (dict(page_stride=1 << 40), -3), (dict(k=None), -1),
    (dict(v=A + 8), -4), (dict(dtype=1), -1), (dict(dtype=1, k_scale=A, v_scale=A + 4), -4),
])
def test_cache_checks(lib, kw, code):
    for f in (varlen, shared, write, read):
        assert f(lib, cache=cache(**kw)) == code


# ------------------------------------------------------------------------------ workspaces
def up(n):
    return -(-n // 256) * 256


def few(rows, d):  # 608 CTAs with two parts each: O, maximum and sum; a record of 28 bytes each; a head
    return up(2 * 608 * rows * d * 4) + up(2 * 608 * rows * 8) + up(608 * 28) + 256


def many(group, T, d):  # 76 pairs of CTAs, up to four rounds, two parts each; a record of 24 bytes
    groups = -(-group // 128)
    rows = -(-group // groups)
    tokens = 128 // rows
    part = T * rows if T <= tokens else 256
    shares = 76 * (1 if T <= 2 * tokens else 4)
    return up(2 * shares * part * d * 4) + up(2 * shares * part * 8) + up(shares * 24) + 256


def need(group, T, d):
    rows = group * T
    return max(few(8 if rows <= 8 else 16 if rows <= 16 else 32, d), many(group, T, d))


def test_workspaces(lib):
    f = lib.attn_fwd_paged_varlen_workspace_bytes
    for T, H, H_kv, d in ((1, 1, 1, 64), (5, 8, 2, 128), (2048, 32, 8, 128), (33, 20, 4, 64), (3, 130, 1, 64)):
        assert f(T, H, H_kv, d) == need(H // H_kv, T, d), (T, H, H_kv, d)
        g = lib.attn_fwd_paged_shared_workspace_bytes
        one = lib.attn_fwd_paged_workspace_bytes(T, H, H_kv, d)
        assert g(T, H, H_kv, d) == one + up(2 * T * H * d * 4) + up(2 * T * H * 4) + need(H // H_kv, T, d)
    assert f(0, 8, 2, 128) == f(4, 8, 3, 128) == f(4, 8, 0, 128) == f(4, 8, 2, 96) == f(-1, 8, 2, 64) == 0
    assert g(0, 8, 2, 128) == g(4, 8, 3, 128) == g(4, 0, 1, 128) == g(4, 8, 2, 32) == 0
    assert attn.paged_varlen_workspace_bytes(5, 8, 2, 128) == need(4, 5, 128)
    assert attn.paged_shared_workspace_bytes(5, 8, 2, 128) == g(5, 8, 2, 128)
    # a byte less than that is refused, with the check before any CUDA call
    for T in (1, 9, 40, 5000):
        assert varlen(lib, T=T, nb=need(4, T, 128) - 1) == -8
        assert shared(lib, B=T, nb=g(T, 8, 2, 128) - 1) == -8


def test_binding_refuses(lib):
    c = attn.kv_cache(2, 2, 16, 64, device="cpu")
    q = torch.zeros(8, 3, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_fwd_paged_varlen(q, c, i, i[0], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        attn.attn_fwd_paged_shared(q, c, i, i[0], torch.zeros(2, dtype=torch.int32), i, i[0])
    with pytest.raises(ValueError, match="CUDA"):
        attn.kv_write(q[:2], q[:2], c, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        attn.kv_read(c, i, torch.zeros(2, dtype=torch.int32), 3)
    with pytest.raises(TypeError):
        attn.attn_fwd_paged_varlen([0], c, i, i[0], i[0])
    with pytest.raises((AttributeError, TypeError)):
        attn.kv_write(q[:2], None, c, torch.zeros(3, dtype=torch.int64))
    big = torch.empty(64 << 20, dtype=torch.uint8)
    for ws in (big[::2], big[:1].expand(64 << 20), torch.empty(64 << 20, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            attn.attn_fwd_paged_varlen(q, c, i, i[0], torch.zeros(2, dtype=torch.int32), workspace=ws)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            attn.attn_fwd_paged_shared(q, c, i, i[0], torch.zeros(2, dtype=torch.int32), i, i[0], workspace=ws)


# -------------------------------------------------------------------------------- work split
PROGRAM = r"""
#include <cstdio>
#include "attn_chunk_split.h"
using namespace attn;
// per request: new tokens, rows, tokens of a row tile, causal, cost; then totals, pairs, kilobytes, rounds
int main() {
  int n, L, tokens, causal, cost;
  while (std::scanf("%d %d %d %d %d", &n, &L, &tokens, &causal, &cost) == 5 && tokens > 0) {
    const ChunkReq r{n, L};
    const ChunkShape c{tokens, causal, cost};
    std::printf("%d %d", row_tiles(r, c), unit_row_places(r, c));
    for (int t = 0; t < row_tiles(r, c) && t < 400; ++t) std::printf(" %d %d", key_tiles(r, c, t), places_before(r, c, t));
    std::printf("\n");
  }
  unsigned total;
  int pairs, kb, most;
  while (std::scanf("%u %d %d %d", &total, &pairs, &kb, &most) == 4) {
    const int rounds = chunk_rounds(total, pairs, kb * 1024.f, most);
    std::printf("%d %d\n", rounds, chunk_shares(total, pairs, rounds));
  }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    cxx = os.environ.get("CXX", "g++")
    if shutil.which(cxx) is None:
        pytest.skip("needs a host compiler")
    at = tmp_path_factory.mktemp("pages")
    (at / "split.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-Wno-unused-result", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-I", build.CSRC, str(at / "split.cpp"), "-o", str(at / "split")], check=True)
    return str(at / "split")


def requests():
    r = random.Random(3)
    yield from [(1, 0, 1, 1, 2), (1, 1, 256, 1, 2), (256, 128, 256, 1, 2), (257, 129, 256, 0, 0), (1, INT_MAX - 1024, 1, 1, 2),
                (100000, 100000, 256, 1, 2), (5000, 10, 254, 1, 2), (10000, 0, 2, 1, 2), (1 << 18, 1 << 18, 2, 1, 2)]
    for _ in range(600):
        n = r.choice([r.randint(1, 20), r.randint(1, 3000)])
        yield n, r.choice([r.randint(0, 300), r.randint(0, 9000), n]), r.randint(1, 256), r.choice([1, 1, 0]), r.choice([0, 1, 2])


def lines(program, text):
    out = subprocess.run([program], input=text, capture_output=True, text=True, check=True).stdout
    return [[int(x) for x in s.split()] for s in out.splitlines()]


def test_places_are_those_counted(program):
    todo = list(requests())
    got = lines(program, "".join("%d %d %d %d %d\n" % x for x in todo))
    assert len(got) == len(todo)
    for (n, L, tokens, causal, cost), line in zip(todo, got):
        want, places, tiles = [], 0, -(-n // tokens)
        for t in range(tiles):
            seen = L - n + min((t + 1) * tokens, n) if causal else L  # what the tile's last token sees
            k = max(1, -(-seen // 128))
            want += [k, places] if t < 400 else []
            places += k + cost
        assert line == [tiles, places, *want], (n, L, tokens, causal, cost)


def test_shares_and_rounds(program):
    r = random.Random(4)
    todo = [(r.choice([r.randint(1, 600), r.randint(1, 1 << 17), r.randint(1, INT_MAX)]), r.randint(1, 76),
             r.randint(0, 1 << 20), r.choice([1, 4])) for _ in range(300)]
    got = lines(program, "0 0 0 0 0\n" + "".join("%d %d %d %d\n" % x for x in todo))
    for (total, pairs, kb, most), (rounds, shares) in zip(todo, got):
        assert rounds in (1, 2, 4) and rounds <= most and 1 <= shares <= pairs * rounds
        assert shares == min(max(1, total // 4), pairs * rounds)
        if rounds > 1:                                    # shares stay long, and there was more than the rounds before hold
            assert total // (pairs * rounds) >= 256 and kb * 1024 > rounds // 2 * (96 << 20)
