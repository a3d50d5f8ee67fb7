"""The paged path as it is served: each question's documents gathered once (msa_gather_kv), the
questions appended and attended, then several answers a question token by token, in buffers with
room to grow, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

import top_kv_routing_b200 as msa
from paged_ref import D, Batch
from test_gpu_paged_forms import forms

pytestmark = pytest.mark.gpu


def _room(x, pages, table, ids, max_pages):
    """x over a pool and a page table that are larger than its own."""
    x.pages, x.n_pages, x.table, x.max_pages = pages, pages.shape[1], table, max_pages
    x.ids = [ids[b][:-(-(n + p) // x.page)] for b, (n, p) in enumerate(zip(x.new, x.past))]
    return x


@pytest.mark.parametrize("L,H,G,page,answers,step", [
    (2, 2, 4, 16, 2, ["rows"]),           # small batches, row form
    (4, 16, 4, 32, 14, ["memory", "rows"]),  # many answers, memory once for all of a question
    (3, 4, 8, 64, 3, ["rows"]),
])
def test_gather_append_attend(L, H, G, page, answers, step):
    gen = np.random.default_rng(91)
    n_docs, k, NQ = 12, 4, 3
    blocks = gen.integers(1, 30, n_docs)
    offs = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int64)
    C = int(offs[-1])
    host = torch.randn((L, C, 2, H, D), dtype=torch.float32).to(torch.bfloat16).pin_memory()
    ids = np.stack([[gen.choice(n_docs, k, replace=False) for _ in range(L)] for _ in range(NQ)]).astype(np.int32)
    M = int(k * blocks.max()) + 100  # (room for longer documents)
    mem = torch.full((NQ, L, 2, H, M, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    mem_len = torch.zeros((NQ, L), dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    msa.msa_gather_kv(host, C, torch.from_numpy(offs).cuda(), None, n_docs, torch.from_numpy(ids).cuda(), NQ, L, k, H, D,
                      M, mem, mem_len, err)
    B, question = NQ * answers, [17, 40, 26]
    groups = [answers * g for g in range(NQ + 1)]
    # every answer holds its question's tokens in pages of its own; room for 500 rows each
    max_pages = -(-500 // page)
    need = -(-60 // page)
    order = gen.permutation(B * need + 5).tolist()
    own = [order[b * need:(b + 1) * need] for b in range(B)]
    pages = torch.full((L, len(order), 2, H, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, max_pages), 0x7FFFFFF0, dtype=torch.int32, device="cuda")
    table[:, :need] = torch.tensor(own, dtype=torch.int32, device="cuda")

    def batch(new, past, seed):
        x = Batch(new, past, L=L, H=H, G=G, page=page, groups=groups, mem=[[1] * L] * NQ, M=M, pad=1, seed=seed)
        x.mem, x.mem_len = mem, mem_len
        return _room(x, pages, table, own, max_pages)

    def run(x):
        q_rot = torch.full_like(x.out, 7.0)
        x.call_append(msa, pos=k, q_rot=q_rot)
        assert (q_rot[:, -1] == 7.0).all()
        x.q = q_rot
        x.call_attend(msa)
        x.check()
        assert x.err.item() == 0

    new = [question[b // answers] for b in range(B)]
    run(batch(new, [0] * B, 92))
    assert err.item() == 0
    for g in range(NQ):  # (what was gathered, and with it what `check` compared with)
        for l in range(L):
            want = torch.cat([host[l, offs[d]:offs[d + 1]] for d in ids[g, l]]).permute(1, 2, 0, 3)
            n = want.shape[2]
            assert mem_len[g, l].item() == n
            assert torch.equal(mem[g, l, :, :, :n].cpu().view(torch.int16), want.contiguous().view(torch.int16))
    past = new
    for i in range(4):
        x = batch([1] * B, past, 93 + i)
        run(x)
        past = [p + 1 for p in past]
    assert [f[0] for f in forms(x)] == step
    run(batch([b % 4 for b in range(B)], past, 99))  # drafts of all lengths, none among them
