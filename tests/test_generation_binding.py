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


@pytest.mark.gpu
def test_lengths_do_not_hold_a_prompts_slots():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()

    def i32(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    table = torch.full((2, 80), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(200, dtype=torch.int32, device="cuda")
    lens, head = i32(0, 0), i32(0)
    for cu in ((0, 1000, 1001), (0, 1, 2), (0, 0, 1), (0, 0, 0), (0, 2, 3)):
        old, T = lens.tolist(), cu[-1]
        slots, pos, _, lens, head = attn.kv_slots(lens, i32(*cu), T, table, free, head, 16)
        assert lens.tolist() == [old[0] + cu[1], old[1] + cu[2] - cu[1]]
        assert int(head) == sum(-(-n // 16) for n in lens.tolist())
        want = [n + i for n, a, b in zip(old, cu, cu[1:]) for i in range(b - a)]
        assert pos.tolist() == want and slots.shape == (T,)
        for t in (lens, head):
            assert t.untyped_storage().nbytes() <= 4 * 3 + 12 * 2
        assert slots.data_ptr() % 8 == pos.data_ptr() % 4 == lens.data_ptr() % 4 == 0
