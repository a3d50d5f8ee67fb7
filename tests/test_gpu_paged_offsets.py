"""Paged batches with unusable offsets: the sequences and groups that have them are skipped, all
others get what include/msa_paged.h defines, in every form of the kernels."""
import pytest
import torch

import top_kv_routing_b200 as msa
from paged_ref import Batch, rope
from test_gpu_paged_forms import forms

pytestmark = pytest.mark.gpu


def _check_only(x, good):
    """Outputs of the sequences in `good` as defined, those of all others untouched."""
    want, tol = x.attend(only=good)
    own = torch.zeros(x.T, dtype=torch.bool, device="cuda")
    for b in good:
        at = slice(x.off[b].item(), x.off[b].item() + x.new[b])
        own[at] = True
        assert ((x.out[:, at].double() - want[:, at]).abs() <= tol[:, at]).all(), b
    assert (x.out[:, ~own] == 7.0).all()


# batches of 40 sequences in three groups, one for each form: few rows a group; memory once for all
# rows, groups of at most and of more than a row tile; long blocks
FORMS = {
    "rows": dict(new=[1] * 40, past=[30 + b for b in range(40)], L=1, H=1, G=1, mem=[20, 30, 10]),
    "memory": dict(new=[1] * 40, past=[30 + b for b in range(40)], L=8, H=16, G=4, mem=[200, 300, 50]),
    "memory, two row tiles": dict(new=[1] * 40, past=[30 + b for b in range(40)], L=8, H=16, G=8, mem=[200, 300, 50]),
    "memory, drafts": dict(new=[3] * 40, past=[30 + b for b in range(40)], L=8, H=16, G=4, mem=[400, 300, 350]),
    "blocks": dict(new=[20] * 40, past=[3 + b for b in range(40)], L=2, H=16, G=4, mem=[100, 130, 50]),
}
GROUPS = [0, 12, 25, 40]


def _batch(form):
    case = FORMS[form]
    mem = [[m - l for l in range(case["L"])] for m in case["mem"]]
    x = Batch(**{**case, "mem": mem}, groups=GROUPS, seed=61)
    assert [f[0] for f in forms(x)] == {"rows": ["rows"], "blocks": ["blocks"]}.get(form, ["memory", "rows"])
    x.out.fill_(7.0)
    return x


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("at,value", [(12, 100000), (12, -3), (25, 0), (18, 100000), (18, 0), (0, -1), (40, 100000),
                                      (39, -7)])
def test_attend_one_bad_token_offset(form, at, value):
    # an offset at a border between groups, inside a group, the first and the last one
    x = _batch(form)
    x.off[at] = value
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_BAD_OFFSETS
    if value == 0:
        # sequence `at` is [0, ...): it shares its tokens with the ones before it, which are then undefined
        want, tol = x.attend(only=range(at + 1, 40))
        assert ((x.out.double() - want).abs() <= tol)[tol >= 0].all() and (tol >= 0).any()
        return
    _check_only(x, [b for b in range(40) if b not in (at - 1, at)])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("at,value,lost", [(0, -1, [0]), (1, 99, [0, 1]), (1, -5, [0, 1]), (2, 2000, [1, 2]), (3, 41, [2])])
def test_attend_one_bad_group_offset(form, at, value, lost):
    # the groups on both sides of it have no memory, the third keeps its own
    x = _batch(form)
    x.goff[at] = value
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_BAD_OFFSETS
    group_of = x.group_of
    x.group_of = lambda b: None if group_of(b) in lost else group_of(b)
    want, tol = x.attend()
    assert ((x.out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("form", ["memory", "memory, two row tiles", "memory, drafts", "blocks"])
def test_attend_device_conditions(form):
    x = _batch(form)
    good = x.table.clone()
    x.mem_len[1, 0] += 200                      # clamped
    x.table[3, 0] = x.n_pages                   # rows 0..15 of sequence 3 are not seen
    x.call_attend(msa)
    x.mem_len[1, 0] = min(x.mem_len[1, 0].item(), x.M)
    assert x.err.item() == msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_CAPACITY
    x.mem.nan_to_num_(0.25)
    x.call_attend(msa)
    rest = [b for b in range(40) if b != 3]
    want, tol = x.attend(only=rest)
    assert ((x.out.double() - want).abs() <= tol)[tol >= 0].all()
    assert not x.out[:, x.off[3]:x.off[4]].isnan().any()
    x.table.copy_(good)
    x.err.zero_()
    x.seq_len[5] = x.max_pages * x.page + 3     # clamped to the table's rows
    x.pages.nan_to_num_(0.25)
    spare = [i for i in range(x.n_pages) if all(i not in r for r in x.ids)]
    x.ids[5] = (x.ids[5] + spare * x.max_pages)[:x.max_pages]
    x.table[5] = torch.tensor(x.ids[5], dtype=torch.int32)
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_LOCAL_FULL
    want, tol = x.attend()
    assert ((x.out.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("B", [4, 33, 100, 1024])
@pytest.mark.parametrize("value", [-5, 0, 100000])
def test_append_stores_the_tokens_of_usable_sequences(B, value):
    # one bad offset in turn at every place that a search of the offsets may look at
    for at in sorted({1, 2, B // 2, B - 2, B - 1} | set(range(0, B, max(1, -(-B // 32) * 5)))):
        if at == 0 and value == 0:
            continue
        x = Batch([1] * B, [b % 15 for b in range(B)], H=1, G=1, page=16, pad=2, seed=62)
        before, q_rot = x.pages.clone(), torch.full_like(x.out, 7.0)
        x.off[at] = value
        if at == 1 and value == 0:  # (sequence 0 without tokens, sequence 1 with two: nothing is wrong)
            continue
        x.call_append(msa, q_rot=q_rot)
        assert x.err.item() & msa.MSA_DEVERR_BAD_OFFSETS
        skip = {at - 1, at}
        good = torch.tensor([b for b in range(B) if b not in skip and (value != 0 or b > at)], dtype=torch.long)
        row = torch.tensor([b % 15 for b in range(B)])[good]
        ids = torch.tensor([x.ids[b][0] for b in good.tolist()], dtype=torch.long)
        want = rope(x.q[0, good].cpu(), 16 + row)
        assert ((q_rot[0, good].cpu().double() - want).abs() <= want.abs() * 2 ** -8 + 2 ** -15).all(), (at, value)
        assert torch.equal(x.pages[0, ids, 1, 0, row].cpu(), x.v[0, good, 0].cpu()), (at, value)
        if value != 0:
            left = [b for b in range(B) if b in skip]
            assert (q_rot[0, left] == 7.0).all() and (q_rot[0, -2:] == 7.0).all()
            own = torch.zeros(x.n_pages, dtype=torch.bool)
            own[ids] = True
            a, b = x.pages[0, ~own].nan_to_num(9.0), before[0, ~own].nan_to_num(9.0)
            assert torch.equal(a, b), (at, value)


@pytest.mark.parametrize("form", FORMS)
def test_batches_without_tokens(form):
    # every sequence empty (all tokens padding): nothing is written, and the workspace stays ready
    x = _batch(form)
    off = x.off.clone()
    pages, q_rot = x.pages.clone(), torch.full_like(x.out, 7.0)
    for value in (0, 7, x.T):
        x.off.fill_(value)
        x.call_append(msa, q_rot=q_rot)
        x.call_attend(msa)
    assert (x.out == 7.0).all() and (q_rot == 7.0).all() and x.err.item() == 0
    assert torch.equal(x.pages.view(torch.int16), pages.view(torch.int16))
    x.off.copy_(off)
    x.call_attend(msa)
    x.check()


@pytest.mark.parametrize("form", FORMS)
def test_any_offsets_leave_the_workspace_ready(form):
    # offsets of all kinds, many unusable, sequences that share tokens and groups that share
    # sequences: no row past the tokens is written, and the next usable call is as ever
    x = _batch(form)
    x.call_attend(msa)
    first, off, goff = x.out.clone(), x.off.clone(), x.goff.clone()
    room = torch.full((x.out.numel() + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(63)
    for i in range(12):
        bad = torch.randint(-3, x.T + 4, (41,), generator=gen, dtype=torch.int32)
        if i % 3 == 0:  # mostly usable ones, some exchanged
            bad = torch.where(torch.rand(41, generator=gen) < 0.2, bad, off.cpu())
        if i % 3 == 1:  # every second sequence has all tokens
            bad = torch.tensor([0, x.T] * 20 + [0], dtype=torch.int32)
        x.off.copy_(bad)
        x.goff.copy_(torch.randint(-2, 43, (4,), generator=gen, dtype=torch.int32) if i % 2 else goff)
        x.out = room[:x.out.numel()].view(x.out.shape)
        x.call_attend(msa)
        torch.cuda.synchronize()
        assert (room[x.out.numel():] == 7.0).all()
        assert x.err.item() & ~(msa.MSA_DEVERR_BAD_OFFSETS) == 0
        x.off.copy_(off)
        x.goff.copy_(goff)
        x.call_attend(msa)
        assert torch.equal(first.view(torch.int16), x.out.view(torch.int16))
