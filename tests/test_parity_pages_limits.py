"""Work over a paged cache at the limits of what its entry points promise: more requests than a block looks at in one
step, prefix sums that are not sums, values that are not finite, scales at the ends of their range, groups without requests.

Tolerances as in test_parity_pages.py unless a test derives its own."""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import attn
from test_parity_generation import _gpu, i32, normal, paged_inputs  # noqa: F401
from test_parity_pages import check_varlen, sums

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_short_requests_of_many_rows(kind):
    # the first shares end after a tile or two, while other warps may still look for where theirs begin
    B, d = 520, 64
    new = [17 + i % 5 for i in range(B)]
    lens = [n + i % 3 for i, n in enumerate(new)]
    _, cache, table, n, vals = paged_inputs(3, lens, 4, 1, d, 16, kind)
    q, cu = normal(4, 4, sum(new), d), sums(new)
    first = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    for _ in range(50):
        assert same(first, attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu)))
    tokens = set(range(0, cu[-1], 53)) | {cu[-1] - 1}
    check_varlen(*first, q, vals, table, lens, cu, True, 1 / math.sqrt(d), kind, f"varlen {kind} many short", tokens)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("B", [5, 40, 300])
@pytest.mark.parametrize("T", [12, 60, 2000])
def test_nothing_is_computed_for_sums_that_fall(T, B, kind):
    # each of the requests behind a fall would be as many tokens as there are, together more than the host's check of sizes
    # counts: both kernels leave O and lse alone, with either way of adding the requests up
    _, cache, table, n, _ = paged_inputs(3, [40] * B, 4, 2, 64, 16, kind)
    q = normal(2, 4, T, 64)
    for cu in ([0] + [T if i % 2 else 0 for i in range(B)], [0] * (B - 1) + [T, T - 1], [0] * B + [-1]):
        o = torch.full((4, T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, T), 7.0, device="cuda")
        attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu), out=o, lse=lse)
        assert attn.decode_status(attn.last_device_error())["kind"] == 2
        assert (o == 7).all() and (lse == 7).all()
    cu = [0] * B + [T]
    o, lse = attn.attn_fwd_paged_varlen(q, cache, table, n, i32(*cu))
    assert torch.isfinite(o.float()[:, -40:]).all() and attn.last_device_error() == 0
