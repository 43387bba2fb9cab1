"""GPU parity of attention over an E4M3 cache against the float64 oracle where the scales of a request's
rows differ in size and sign (tolerances as in test_parity_generation.py)."""
import math

import numpy as np
import pytest
import torch

from io_aware_attention_attn_gb300 import attn
from test_parity_generation import _gpu, check_paged, paged_inputs  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = [(64, 4), (64, 16), (64, 32), (128, 4), (128, 16), (128, 32)]  # d, query rows a K/V head


@pytest.mark.parametrize("d,rows", ROWS)
@pytest.mark.parametrize("share", [0.5, 1.0])
def test_negative_scales(d, rows, share):
    lens = [300, 17, 1]
    q, cache, table, n, vals = paged_inputs(40 + rows, lens, 2 * rows, 2, d, 16, "e4m3")
    r = np.random.default_rng(rows)
    signs = [np.where(r.random(t.shape) < share, -1.0, 1.0) for t in (cache.k_scale, cache.v_scale)]
    scales = [t * torch.from_numpy(s).float().cuda() for t, s in zip(cache[2:], signs)]
    vals = [v * s[..., None] for v, s in zip(vals, signs)]
    o, lse = attn.attn_fwd_paged(q, attn.KVCache(cache.k, cache.v, *scales), table, n)
    check_paged(o, lse, q, vals, table, lens, 1 / math.sqrt(d), "e4m3", f"paged negative scales d{d} {rows}")
