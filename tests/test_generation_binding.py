"""Refusals of the generation path's binding that the entry points' own checks cannot make: they see an
address and a size."""
import pytest
import torch

from io_aware_attention_attn_gb300 import attn, build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def calls(device):
    x = torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device=device)
    k = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16, device=device)
    w = torch.ones(64, dtype=torch.bfloat16, device=device)
    i = torch.zeros(2, 1, dtype=torch.int32, device=device)
    rows = torch.zeros(2, 1, 12 * 64, dtype=torch.bfloat16, device=device)
    cache = attn.kv_cache(2, 2, 16, 64, device=device)
    return {"attn_fwd_paged": lambda ws: attn.attn_fwd_paged(x, cache, i, i[:, 0], workspace=ws),
            "qkv_rope_bwd": lambda ws: attn.qkv_rope_bwd(x, k, k, rows, wq=w, wk=w, workspace=ws)}


BIG = 64 << 20  # more than either call needs


def refused(call, device, other):
    byte = torch.zeros(1, dtype=torch.uint8, device=device)
    for ws in (torch.empty(BIG, dtype=torch.uint8, device=other),           # not where the inputs are
               byte.expand(BIG),                                            # one byte of memory
               torch.empty(BIG, dtype=torch.uint8, device=device)[::2]):                    # strided
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(ws)


@pytest.mark.parametrize("name", ["attn_fwd_paged", "qkv_rope_bwd"])
def test_workspace_of_another_device_or_layout(name):
    refused(calls("cpu")[name], "cpu", "meta")
    with pytest.raises(ValueError, match="CUDA"):
        calls("cpu")[name](torch.empty(BIG, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["attn_fwd_paged", "qkv_rope_bwd"])
def test_workspace_of_another_device_or_layout_on_the_gpu(name):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    call = calls("cuda")[name]
    refused(call, "cuda", "cpu")
    with pytest.raises(attn.AttnError, match="ATTN_ERR_WORKSPACE"):
        call(torch.empty(4096, dtype=torch.uint8, device="cuda"))
    for ws in (None, torch.empty(BIG, dtype=torch.uint8, device="cuda"), torch.empty(BIG // 4, device="cuda")):
        call(ws)
    torch.cuda.synchronize()
    assert attn.last_device_error() == 0
