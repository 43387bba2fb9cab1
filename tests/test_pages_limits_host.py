"""Host side of work over a paged cache at the ends of what it takes: sizes that are refused and sizes that are not (no GPU:
a call with a workspace of no bytes fails after the check of sizes and before any CUDA call)."""
import pytest

from test_generation_host import cache
from test_pages_host import INT_MAX, lib, read, shared, varlen  # noqa: F401


@pytest.mark.parametrize("B", [INT_MAX, INT_MAX - 1023])
def test_more_requests_than_a_block_can_step_over(lib, B):
    # loops over requests go on by up to 640 after the last one
    assert varlen(lib, B=B, nb=0) == -3
    assert shared(lib, groups=B, nb=0) == -3
    assert shared(lib, groups=B - 9, nb=0) == -3       # prefixes and the own rows of requests are counted on together
    assert read(lib, B=B) == -3
    assert varlen(lib, B=INT_MAX - 1024, nb=0) == -8
    assert shared(lib, groups=INT_MAX - 1024 - 9, nb=0) == -8


@pytest.mark.parametrize("kw", [
    # one request, 2 to 6 % of the places that the kernel that takes it numbers; the other kernel's, which is not launched, not
    dict(B=1, T=32768, H=32, H_kv=8, max_pages=1 << 14), dict(B=1, T=65536, H=32, H_kv=8, max_pages=1 << 13),
    dict(B=1, T=16384, H=64, H_kv=8, max_pages=1 << 14),
    # 64 rows a request, of which the kernel for few rows counts 32 to a unit; then 64 and one, of which only the other can
    # number the places, and takes all
    dict(B=4096, T=65536, H=32, H_kv=8, max_pages=1 << 13), dict(B=65536, T=1 << 20, H=32, H_kv=8, max_pages=1 << 11),
    dict(B=1 << 17, T=1 << 17, H=8, H_kv=8, max_pages=1 << 11),
])
def test_sizes_within_the_limit_are_taken(lib, kw):
    tiles = kw["max_pages"] * 64 // 128 + 1
    tokens = 256 // (kw["H"] // kw["H_kv"])
    assert (kw["T"] // tokens + min(kw["B"], kw["T"])) * (tiles + 2) * kw["H_kv"] < 2 ** 31
    for pages, code in ((1, -8), (64, -3)):
        assert varlen(lib, nb=0, **{**kw, "max_pages": kw["max_pages"] * pages}, cache=cache(page_stride=8 * 64 * 128)) == code


@pytest.mark.parametrize("kw", [
    dict(groups=1, B=32768, H=32, H_kv=8, max_prefix=1 << 14, max_pages=1), dict(groups=64, B=65536, H=32, H_kv=8,
                                                                                max_prefix=1 << 13, max_pages=1)])
def test_shared_sizes_within_the_limit_are_taken(lib, kw):
    for pages, code in ((1, -8), (64, -3)):
        assert shared(lib, nb=0, **{**kw, "max_prefix": kw["max_prefix"] * pages}, cache=cache(page_stride=8 * 64 * 128)) == code
