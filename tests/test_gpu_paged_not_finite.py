"""Infinite values that a row does see: a weight above zero times an infinity, in every form of
msa_shared_attend and for both sizes of the row kernel's units."""
import pytest
import torch

import top_kv_routing_b200 as msa
from paged_ref import Batch
from test_gpu_paged_forms import forms

pytestmark = pytest.mark.gpu

CASES = {
    "rows of eight": (dict(new=[1, 1, 1], past=[40, 700, 3], H=2, G=4, groups=[0, 2], mem=[90]), ["rows"]),
    "rows of eight, one head": (dict(new=[2, 2, 2], past=[40, 700, 3], H=2, G=1, groups=[0, 2], mem=[90]), ["rows"]),
    "rows of sixteen": (dict(new=[5, 5, 5], past=[40, 700, 3], H=2, G=4, groups=[0, 2], mem=[90]), ["rows"]),
    "memory and rows of eight": (dict(new=[1] * 40, past=[30] * 40, L=8, H=16, G=4, groups=[0, 20, 39],
                                      mem=[[200] * 8, [300] * 8]), ["memory", "rows"]),
    "memory and rows of sixteen": (dict(new=[3] * 40, past=[30] * 40, L=8, H=16, G=4, groups=[0, 20, 39],
                                        mem=[[400] * 8, [350] * 8]), ["memory", "rows"]),
    "blocks": (dict(new=[40, 33], past=[150, 7], L=8, H=16, G=4, groups=[0, 2], mem=[[140] * 8]), ["blocks"]),
}


@pytest.mark.parametrize("where", ["memory", "first page row", "last page row"])
@pytest.mark.parametrize("name", CASES)
def test_infinite_values(name, where):
    case, kernels = CASES[name]
    x = Batch(seed=71, **case)
    assert [f[0] for f in forms(x)] == kernels
    x.out.fill_(7.0)
    x.call_attend(msa)
    x.check()
    plain = x.out.clone()
    b, g = 0, 0
    last = x.new[b] - 1  # the token that sees the value in any case
    if where == "memory":
        v = x.mem[g, :, 1, :, 17]
        hit = list(range(x.off[x.groups[g + 1]].item()))
    else:
        row = 0 if where == "first page row" else x.past[b] + last
        v = x.pages[:, x.ids[b][row // x.page], 1, :, row % x.page]
        hit = [i for i in range(x.new[b]) if x.past[b] + i >= row]
    v[..., 3], v[..., 64] = float("inf"), float("-inf")
    x.call_attend(msa)
    mine = torch.zeros(x.T, dtype=torch.bool, device="cuda")
    mine[hit] = True
    assert (x.out[:, mine, :, 3] == float("inf")).all() and (x.out[:, mine, :, 64] == float("-inf")).all()
    x.out[:, mine, :, 3], x.out[:, mine, :, 64] = plain[:, mine, :, 3], plain[:, mine, :, 64]
    assert torch.equal(x.out.view(torch.int16), plain.view(torch.int16))
