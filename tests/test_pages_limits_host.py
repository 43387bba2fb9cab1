"""Host side of work over a paged cache at the ends of what it takes: sizes that are refused and sizes that are not (no GPU:
a call with a workspace of no bytes fails after the check of sizes and before any CUDA call)."""
import pytest

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
