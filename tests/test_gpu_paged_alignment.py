"""Paged batches on buffers that keep the 16 bytes of include/msa_paged.h and no more: every
one of them starts at an odd multiple of 16."""
import pytest
import torch

import top_kv_routing_b200 as msa
from paged_ref import D, Batch

pytestmark = pytest.mark.gpu


def _odd16(t):
    """A copy of t that starts 16 bytes behind a multiple of 32."""
    n = 16 // t.element_size()
    room = torch.empty(t.numel() + 2 * n, dtype=t.dtype, device=t.device)
    at = n if room.data_ptr() % 32 == 0 else 0
    out = room[at:at + t.numel()].view(t.shape)
    assert out.data_ptr() % 32 == 16
    return out.copy_(t)


def _shift(x):
    for name in ("q", "k", "v", "pages", "mem", "out"):
        if getattr(x, name) is not None:
            setattr(x, name, _odd16(getattr(x, name)))
    n = msa.msa_shared_attend_workspace_size(x.T, x.B, x.NG, x.L, x.HQ, x.H)
    x.ws = _odd16(torch.zeros(n, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("launches,case", [
    # row form, block form (short and long units, values that are taken out), memory form (groups of
    # at most and of more than a row tile)
    (1, dict(new=[1, 2, 20], past=[50, 600, 70], H=2, G=4, groups=[0, 2, 3], mem=[300, 17])),
    (1, dict(new=[40, 33, 1], past=[150, 0, 90], L=8, H=16, G=4, page=32, groups=[0, 2], mem=[[140] * 8])),
    (1, dict(new=[129, 64], past=[5, 300], L=8, H=16, G=1, page=64)),
    (2, dict(new=[1] * 20, past=[9] * 20, L=8, H=16, G=4, groups=[0, 10, 20], mem=[[700] * 8, [3] * 8])),
    (2, dict(new=[1] * 70, past=[5] * 70, L=8, H=16, G=8, groups=[0, 69], mem=[[400] * 8])),
])
def test_attend(launches, case):
    x = Batch(seed=41, **case)
    _shift(x)
    assert x.call_attend(msa) == launches
    x.check()
    assert x.err.item() == 0


def test_values_that_are_not_finite():
    x = Batch([40, 33], [150, 7], L=8, H=16, G=4, page=32, groups=[0, 2], mem=[[140] * 8], seed=42)
    _shift(x)
    assert x.call_attend(msa) == 1
    first = x.out.clone()
    page, slot = x.ids[0][189 // 32], 189 % 32
    x.pages[:, page, 1, :, slot, 3] = float("inf")
    x.call_attend(msa)
    rest = torch.ones(x.T, dtype=torch.bool, device="cuda")
    rest[39] = False
    assert torch.equal(first[:, rest].view(torch.int16), x.out[:, rest].view(torch.int16))
    assert (x.out[:, 39, :, 3] == float("inf")).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append(dtype):
    x = Batch([3, 1, 40], [14, 0, 63], L=2, H=2, G=4, page=32, dtype=dtype, seed=43)
    before, q_rot = x.pages.clone(), torch.empty_like(x.out)
    x.call_append(msa, q_rot=q_rot)
    want, want_pages = q_rot, x.pages
    x.pages = before
    _shift(x)
    q_rot = _odd16(torch.zeros((2, x.T, x.HQ, D), dtype=torch.bfloat16, device="cuda"))
    x.call_append(msa, q_rot=q_rot)
    assert torch.equal(q_rot.view(torch.int16), want.view(torch.int16))
    assert torch.equal(x.pages.view(torch.int16), want_pages.view(torch.int16))
    assert x.err.item() == 0
