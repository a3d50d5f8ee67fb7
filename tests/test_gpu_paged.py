"""Paged batches on the GPU (include/msa_paged.h) against their definition in 64 bits.

Tolerances are derived in paged_ref.py.  Slots and rows that no key occupies hold NaN in
every case, and unused page-table entries an id outside the pool."""
import pytest
import torch

import top_kv_routing_b200 as msa
from paged_ref import D, Batch, rope

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------------------- append

def _check_append(x, q_rot, before, pos_offset, pos, theta=1e6):
    """Stored rows and rotated queries: half a bf16 step of the exact rotation, plus the fp32
    rotation's own error (angles within 2^-22 of a half turn as sine and cosine, two products
    and a sum: at most 2^-20 of |lo| + |hi|)."""
    want = before.clone().double()
    for b, (new, past) in enumerate(zip(x.new, x.past)):
        if new == 0:
            continue
        t0 = x.off[b].item()
        row = torch.arange(past, past + new, device=x.q.device)
        at = (pos + int(pos_offset[b]) if pos_offset is not None else pos) + row
        rq = rope(x.q[:, t0:t0 + new], at, theta)
        mag = lambda z: z.double().abs().amax(-1, keepdim=True) * 2  # noqa: E731
        got = q_rot[:, t0:t0 + new].double()
        assert ((got - rq).abs() <= rq.abs() * 2 ** -8 + mag(x.q[:, t0:t0 + new]) * 2 ** -20).all()
        rk = rope(x.k[:, t0:t0 + new], at, theta)
        ids = torch.tensor(x.ids[b], device=x.q.device)[row // x.page]
        gk = x.pages[:, ids, 0, :, row % x.page].double().transpose(0, 1)
        assert ((gk - rk).abs() <= rk.abs() * 2 ** -8 + mag(x.k[:, t0:t0 + new]) * 2 ** -20).all()
        gv = x.pages[:, ids, 1, :, row % x.page].transpose(0, 1)
        assert torch.equal(gv, x.v[:, t0:t0 + new].to(torch.bfloat16))
        want[:, ids, 0, :, row % x.page] = gk.transpose(0, 1)
        want[:, ids, 1, :, row % x.page] = gv.double().transpose(0, 1)
    got = x.pages.double()  # every other slot is as it was (NaN or an earlier row)
    assert torch.equal(got.nan_to_num(123.0), want.nan_to_num(123.0))


@pytest.mark.parametrize("new,past,L,H,G,page,pad,lead", [
    ([1], [0], 1, 1, 1, 16, 0, 0),
    ([1], [383], 18, 8, 4, 64, 0, 0),
    ([1] * 33, list(range(33)), 2, 2, 8, 16, 0, 0),
    ([1, 0, 17, 64, 3, 0], [5, 9, 0, 15, 63, 0], 2, 4, 2, 32, 5, 3),
    ([130, 1, 257], [7, 200, 0], 1, 16, 1, 128, 2, 0),
    ([5] * 70, [250] * 70, 1, 2, 4, 256, 0, 1),
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append(new, past, L, H, G, page, pad, lead, dtype):
    x = Batch(new, past, L=L, H=H, G=G, page=page, pad=pad, lead=lead, dtype=dtype, seed=1)
    off = torch.arange(x.B, dtype=torch.int32, device="cuda") * 37
    before, q_rot = x.pages.clone(), torch.full_like(x.out, 7.0)
    assert x.call_append(msa, off, 16, q_rot=q_rot) == 1
    _check_append(x, q_rot, before, off, 16)
    own = torch.zeros(x.T, dtype=torch.bool)
    own[lead:lead + sum(new)] = True
    assert (q_rot[:, ~own.cuda()] == 7.0).all()
    assert x.err.item() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_from_a_fused_projection_at_far_positions(dtype):
    x = Batch([3, 40, 1], [100, 0, 31], L=2, H=2, G=4, page=16, pad=2, seed=2, dtype=dtype)
    w = torch.randn((2, x.T, x.HQ + 2 * x.H, D), device="cuda").to(dtype)
    x.q, x.k, x.v = w[:, :, :x.HQ], w[:, :, x.HQ:x.HQ + x.H], w[:, :, x.HQ + x.H:]
    before, q_rot = x.pages.clone(), torch.full_like(x.out, 7.0)
    stride = w.stride(1)
    x.call_append(msa, None, 2_000_000_000, theta=5e5, q_rot=q_rot, q_stride=stride, k_stride=stride, v_stride=stride)
    _check_append(x, q_rot, before, None, 2_000_000_000, 5e5)


def test_append_without_queries_and_twice():
    x = Batch([4, 9], [2, 0], L=2, H=4, G=2, page=16, seed=3)
    before, q = x.pages.clone(), x.q
    x.q = None
    x.call_append(msa)
    first = x.pages.clone()
    x.call_append(msa)  # lengths are not advanced: the same rows again
    assert torch.equal(first.view(torch.int16), x.pages.view(torch.int16))
    x.q = q
    q_rot = torch.empty_like(x.out)
    x.call_append(msa, q_rot=q_rot)
    assert torch.equal(first.view(torch.int16), x.pages.view(torch.int16))
    _check_append(x, q_rot, before, None, 16)


def test_append_device_conditions():
    x = Batch([4, 4, 4, 4], [14, 0, 3, 2], L=2, H=2, G=2, page=16, seed=4)
    ok = Batch([4, 4, 4, 4], [14, 0, 3, 2], L=2, H=2, G=2, page=16, seed=4)
    q_rot = torch.full_like(x.out, 7.0)
    ok.call_append(msa, q_rot=torch.empty_like(q_rot))
    x.seq_len[0] = x.max_pages * x.page + 2  # the last two of four rows do not fit
    for p in range(2, x.max_pages):  # (its table: real pages throughout)
        x.table[0, p] = x.n_pages - 1
    x.table[1, 0] = x.n_pages                # a page that does not exist
    x.seq_len[2] = 3                         # fewer rows than new tokens
    x.call_append(msa, q_rot=q_rot)
    assert x.err.item() == msa.MSA_DEVERR_LOCAL_FULL | msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_BAD_OFFSETS
    ids3 = x.ids[3][0]  # the last sequence is unaffected
    assert torch.equal(x.pages[:, ids3].view(torch.int16), ok.pages[:, ids3].view(torch.int16))
    x.err.zero_()
    x.off[2] = 9999  # sequences 1 and 2 unusable
    x.call_append(msa, q_rot=q_rot)
    assert x.err.item() & msa.MSA_DEVERR_BAD_OFFSETS


# ----------------------------------------------------------------------------- attend

CASES = {
    "one row": dict(new=[1], past=[0]),
    "one token, nothing before": dict(new=[1], past=[0], H=8, G=4, groups=[0, 1], mem=[0]),
    "one long sequence": dict(new=[1], past=[5000], H=1, G=8, page=64),
    "tile edges": dict(new=[1] * 8, past=[14, 15, 16, 17, 30, 31, 32, 63], groups=[0, 3, 8], mem=[16, 33]),
    "ragged groups": dict(new=[1] * 9, past=[0, 400, 3, 77, 150, 31, 8, 250, 1], L=3, H=2, G=4, page=32,
                          groups=[0, 4, 5, 8], mem=[[100, 0, 257], [1, 2, 3], [700, 64, 65]], pad=3, lead=2),
    "one query head": dict(new=[1] * 5, past=[20, 100, 3, 0, 64], H=4, G=1, groups=[0, 5], mem=[300]),
    "two query heads": dict(new=[1, 0, 2, 0], past=[20, 4, 3, 0], H=3, G=2, groups=[0, 4], mem=[129]),
    "drafts": dict(new=[5] * 7, past=[0, 1, 11, 12, 100, 250, 31], L=2, H=2, G=4, groups=[0, 7], mem=[200]),
    "wide drafts": dict(new=[3] * 6, past=[0, 13, 14, 15, 90, 41], H=2, G=8, groups=[0, 2, 6], mem=[5, 64]),
    "many tokens": dict(new=[70, 1, 33, 0, 129], past=[0, 300, 64, 5, 13], H=2, G=4, page=64, groups=[0, 4],
                        mem=[150], pad=1),
    "many tokens alone": dict(new=[100, 90], past=[0, 31], H=1, G=2, page=128),
    "questions": dict(new=[128, 200, 97], past=[0, 0, 50], H=1, G=4, page=16, groups=[0, 3], mem=[256]),
    "long memory": dict(new=[1] * 40, past=[i * 5 for i in range(40)], H=1, G=4, page=16, groups=[0, 38, 40],
                        mem=[4100, 130]),
    "sixteen key heads": dict(new=[1] * 3, past=[10, 20, 30], H=16, G=2, groups=[0, 3], mem=[70]),
    "peaked": dict(new=[1, 2, 20], past=[50, 60, 70], H=2, G=4, groups=[0, 3], mem=[300], scale=8.0),
}


@pytest.mark.parametrize("name", CASES)
def test_attend(name):
    x = Batch(seed=5, **CASES[name])
    x.call_attend(msa)
    x.check()
    assert x.err.item() == 0
    first = x.out.clone()
    x.call_attend(msa)  # the workspace is ready again, and the order of arrival changes nothing
    assert torch.equal(first.view(torch.int16), x.out.view(torch.int16))


def test_one_workspace_for_calls_of_other_sizes():
    a = Batch([1] * 3, [2000, 7, 900], H=2, G=4, groups=[0, 3], mem=[40], seed=6)
    b = Batch([1], [700], H=1, G=8, page=64, seed=7)
    c = Batch([60, 50], [0, 20], H=2, G=4, groups=[0, 2], mem=[300], seed=8)
    need = max(msa.msa_shared_attend_workspace_size(x.T, x.B, x.NG, x.L, x.HQ, x.H) for x in (a, b, c))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    a.ws = b.ws = c.ws = ws
    for x in (a, b, c, b, a, c):
        x.out.fill_(7.0)
        x.call_attend(msa)
        x.check()


def test_rows_that_see_nothing_are_zero():
    x = Batch([3, 2, 1], [0, 0, 0], H=2, G=4, groups=[1, 2], mem=[20], seed=9)
    x.seq_len[0], x.seq_len[1] = 1, 0  # fewer stored rows than new tokens: the first tokens see none
    x.call_attend(msa)
    x.check()
    assert (x.out[:, :2] == 0).all() and (x.out[:, 2] != 0).any()


@pytest.mark.parametrize("G,new", [(4, 4), (8, 3), (1, 16), (2, 40), (4, 150)])
def test_values_that_are_not_finite_stay_behind_the_causal_limit(G, new):
    x = Batch([new, 2], [21, 3], H=1, G=G, groups=[0, 2], mem=[18], seed=10)
    last = x.ids[0][(21 + new - 1) // 16], (21 + new - 1) % 16
    x.pages[:, last[0], 1, :, last[1]] = float("inf")
    x.pages[:, last[0], 0, :, last[1]] = float("nan")
    x.call_attend(msa)
    got = x.out.clone()
    assert got[:, new - 1].isnan().all()  # the last token sees its own row
    x.pages[:, last[0], :, :, last[1]] = 0.0
    x.call_attend(msa)
    assert torch.equal(got[:, :new - 1].view(torch.int16), x.out[:, :new - 1].view(torch.int16))
    assert torch.equal(got[:, new:].view(torch.int16), x.out[:, new:].view(torch.int16))
    x.check()


def test_attend_device_conditions():
    x = Batch([1, 1, 1, 1], [40, 40, 40, 40], H=2, G=4, groups=[0, 2, 4], mem=[30, 50], seed=11)
    good = x.table.clone()
    x.table[1, 1] = -1                          # rows 16..31 of sequence 1 are not seen
    x.mem_len[1, 0] = 60                        # clamped to 50
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_CAPACITY
    want, tol = x.attend()
    for b in (0, 2, 3):
        assert ((x.out[:, b].double() - want[:, b]).abs() <= tol[:, b]).all()
    loc = x.rows(1, 41)
    keep = torch.tensor([i for i in range(41) if not 16 <= i < 32], device="cuda")
    k = torch.cat([x.mem[0, 0, 0, :, :30].double(), loc[0, 0][:, keep]], 1)
    v = torch.cat([x.mem[0, 0, 1, :, :30].double(), loc[1, 0][:, keep]], 1)
    s = torch.einsum("hgd,hkd->hgk", x.q[0, 1].double().view(2, 4, D), k) * D ** -0.5
    w = torch.einsum("hgk,hkd->hgd", torch.softmax(s, -1), v).reshape(8, D)
    assert ((x.out[0, 1].double() - w).abs() <= tol[0, 1] + 2 ** -7 * w.abs()).all()
    x.table.copy_(good)
    x.mem_len[1, 0] = 50
    x.err.zero_()
    x.off[2] = 4000                             # sequences 1 and 2 unusable: left as they were
    x.out.fill_(7.0)
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_BAD_OFFSETS
    assert (x.out[:, 1:3] == 7.0).all()
    for b in (0, 3):
        assert ((x.out[:, b].double() - want[:, b]).abs() <= tol[:, b]).all()
    x.off[2] = 2
    x.err.zero_()
    x.goff[1] = -5                              # both groups unusable: no memory
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_BAD_OFFSETS
    x.goff[1] = 2
    x.NG, x.err[0] = 0, 0
    x.check()
    x.seq_len[0] = 10_000                       # past the table: clamped to its 64 rows
    x.table[0, 3] = x.ids[0][0]
    x.ids[0] = x.ids[0] + [x.ids[0][0]]
    x.pages.nan_to_num_(0.25)
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_LOCAL_FULL
    x.check()


def test_offsets_past_32_bits():
    # a pool of more than 2^31 elements; the sequence's rows lie in its last pages
    H, page = 8, 64
    n_pages = (2 ** 31) // (2 * H * page * D) + 40
    x = Batch([1, 2], [300, 70], H=H, G=4, page=page, groups=[0, 2], mem=[30], seed=12)
    big = torch.empty((1, n_pages, 2, H, page, D), dtype=torch.bfloat16, device="cuda")
    big[:, -x.n_pages:] = x.pages
    shift = n_pages - x.n_pages
    x.pages, x.n_pages = big, n_pages
    x.ids = [[i + shift for i in r] for r in x.ids]
    x.table += shift * (x.table < 0x7FFFFFF0).int()
    before, q_rot = big[:, shift:].clone(), torch.empty_like(x.out)
    x.call_append(msa, q_rot=q_rot)
    x.q = q_rot
    x.call_attend(msa)
    x.check()
    assert not torch.equal(before.view(torch.int16), big[:, shift:].view(torch.int16))
    assert x.err.item() == 0


def test_append_then_attend_captured_and_replayed_on_its_own_stream():
    x = Batch([1, 1, 1], [30, 0, 200], L=2, H=2, G=4, groups=[0, 3], mem=[100], seed=13)
    q_rot, s = torch.empty_like(x.out), torch.cuda.Stream()
    raw = x.q
    x.call_attend(msa)  # (allocates the workspace)

    def step():
        x.q = raw
        x.call_append(msa, q_rot=q_rot, stream=s)
        x.q = q_rot
        x.call_attend(msa, stream=s)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(3):  # the replays read the lengths of the moment
        x.seq_len += 1
        x.past = [p + 1 for p in x.past]
        for b in range(3):
            need = -(-(x.past[b] + 1) // x.page)
            if need > len(x.ids[b]):  # a spare page
                x.ids[b].append([i for i in range(x.n_pages) if all(i not in r for r in x.ids)][0])
                x.table[b, need - 1] = x.ids[b][-1]
        raw.normal_()
        x.k.normal_()
        graph.replay()
        torch.cuda.synchronize()
        x.check()
    assert x.err.item() == 0


def test_agrees_with_the_single_query_decode_step():
    # one sequence, one group: msa_sparse_decode of the same query, memory and local rows
    L, H, G, M, n = 3, 8, 4, 120, 77
    x = Batch([1], [n], L=L, H=H, G=G, page=32, groups=[0, 1], mem=[[120, 64, 9]], M=M, seed=14)
    loc = x.rows(0, n).to(torch.bfloat16)
    local = [torch.zeros((1, L, H, 128, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for c, src in zip(local, loc):
        c[0, :, :, :n] = src
    out = torch.empty((1, L, H * G, D), dtype=torch.bfloat16, device="cuda")
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = torch.zeros(msa.msa_sparse_decode_workspace_size(1, L, H * G, H), dtype=torch.uint8, device="cuda")
    mem = x.mem.nan_to_num(0.0)
    msa.msa_sparse_decode(x.q[:, 0].contiguous(), x.k[:, 0].contiguous(), x.v[:, 0].contiguous(), 1, L, H * G, H, D,
                          local[0], local[1], ln, 128, mem, x.mem_len, M, 16, 1e6, D ** -0.5, out, ws)
    q_rot = torch.empty_like(x.out)
    x.call_append(msa, q_rot=q_rot)
    x.q = q_rot
    x.call_attend(msa)
    x.check()
    assert torch.equal(x.rows(0, n + 1)[0, :, :, n].to(torch.bfloat16), local[0][0, :, :, n])
    # the two differ by the rounding of the rotated query to bf16 and the two outputs' own
    a, b = x.out[:, 0].double(), out[0].double()
    assert (a - b).norm() / b.norm() <= 2 ** -7


# ----------------------------------------------------------------------------- long blocks, many rows

BLOCKS = {
    # long blocks of new tokens: memory and pages in one walk
    "one short block": dict(new=[16], past=[0], H=1, G=4),
    "edges of a tile pair": dict(new=[31, 32, 33, 63, 64, 65], past=[0, 127, 128, 1, 97, 64], H=2, G=4, page=32),
    "one query head": dict(new=[127, 128, 129, 257], past=[0, 5, 130, 260], H=2, G=1, page=256, groups=[0, 4], mem=[129]),
    "two query heads": dict(new=[64, 200], past=[100, 0], H=1, G=2, page=128, groups=[0, 1, 2], mem=[1, 128]),
    "eight query heads": dict(new=[20, 50, 8], past=[200, 3, 77], H=2, G=8, groups=[0, 2], mem=[255]),
    "empty memory": dict(new=[40, 40], past=[0, 30], H=1, G=4, groups=[0, 1, 2], mem=[0, 17]),
    "layers of other lengths": dict(new=[50, 30], past=[20, 260], L=3, H=1, G=4, groups=[0, 2], mem=[[0, 128, 300]]),
    "some without tokens": dict(new=[0, 90, 0, 1, 70], past=[3, 0, 0, 500, 33], H=1, G=4, groups=[1, 4], mem=[60],
                                pad=5, lead=4),
    "a long past": dict(new=[33], past=[3000], H=1, G=4, page=64, groups=[0, 1], mem=[700]),
    "peaked": dict(new=[60, 45], past=[200, 3], H=1, G=4, groups=[0, 2], mem=[300], scale=8.0),
    "sixteen key heads": dict(new=[40], past=[150], H=16, G=2, groups=[0, 1], mem=[140]),
}

MANY_ROWS = {
    # groups of more than one, two, four row tiles; the memory split over few and many units
    "one tile": dict(new=[1] * 32, past=[i for i in range(32)], H=1, G=4, groups=[0, 32], mem=[401]),
    "a tile and a row": dict(new=[1] * 33, past=[2] * 33, H=1, G=4, groups=[0, 33], mem=[500]),
    "pairs of tiles": dict(new=[1] * 150, past=[i % 40 for i in range(150)], H=2, G=4, groups=[0, 150], mem=[300]),
    "groups of all sizes": dict(new=[1] * 100, past=[i % 23 for i in range(100)], L=2, H=2, G=8,
                                groups=[0, 1, 3, 20, 37, 99], mem=[[5, 700], [64, 0], [0, 128], [256, 255], [33, 1]]),
    "drafts of all lengths": dict(new=[i % 6 for i in range(60)], past=[7 * i % 50 for i in range(60)], H=2, G=4,
                                  groups=[2, 30, 58], mem=[150, 400], pad=2, lead=1),
    "many empty splits": dict(new=[1] * 20, past=[9] * 20, H=1, G=4, groups=[0, 10, 20], mem=[8000, 3]),
}


def _wide(case):
    """The case with key heads and layers enough that the tensor-core kernels are taken."""
    L = 8
    mem = [(m if isinstance(m, list) else [m]) for m in case.get("mem", [])]
    return {**case, "H": 16, "L": L, "mem": [(m * L)[:L] for m in mem] or None}


@pytest.mark.parametrize("name", list(BLOCKS) + list(MANY_ROWS))
def test_attend_blocks_and_many_rows(name):
    x = Batch(seed=21, **_wide({**BLOCKS, **MANY_ROWS}[name]))
    launches = x.call_attend(msa)
    assert launches == (1 if name in BLOCKS else 2)
    x.check()
    assert x.err.item() == 0
    first = x.out.clone()
    x.call_attend(msa)
    assert torch.equal(first.view(torch.int16), x.out.view(torch.int16))


@pytest.mark.parametrize("G,new", [(4, 70), (2, 140), (8, 33)])
def test_values_that_are_not_finite_in_many_blocks(G, new):
    # several units per SM, every one with rows that must not see the last token's values
    B, H = 24, 16
    x = Batch([new] * B, [(37 * b) % 150 for b in range(B)], L=2, H=H, G=G, page=32, groups=[0, B], mem=[130], seed=22)
    last = [(x.ids[b][(p + new - 1) // 32], (p + new - 1) % 32) for b, p in enumerate(x.past)]
    kept = []
    for b, (page, slot) in enumerate(last):
        kept.append(x.pages[:, page, 1, :, slot].clone())
        x.pages[:, page, 1, :, slot, b % D] = float("inf") if b % 3 else float("nan")
    assert x.call_attend(msa) == 1
    got = x.out.clone()
    for b, (page, slot) in enumerate(last):
        x.pages[:, page, 1, :, slot] = kept[b]
    x.out.fill_(7.0)
    x.call_attend(msa)
    x.check()
    ends = x.off[1:].long() - 1
    rest = torch.ones(x.T, dtype=torch.bool, device="cuda")
    rest[ends] = False
    assert torch.equal(got[:, rest].view(torch.int16), x.out[:, rest].view(torch.int16))
    for b in range(B):
        row = got[:, ends[b]]
        at = torch.arange(D, device="cuda") == b % D
        assert (row[..., at].isnan().all() if b % 3 == 0 else (row[..., at] == float("inf")).all())
        assert torch.equal(row[..., ~at].view(torch.int16), x.out[:, ends[b]][..., ~at].view(torch.int16))


def test_block_device_conditions():
    x = Batch([40, 40, 40], [60, 60, 60], L=8, H=16, G=4, page=32, groups=[0, 3], mem=[50], seed=23)
    assert x.call_attend(msa) == 1
    good = x.out.clone()
    x.check()
    x.table[1, 1] = x.n_pages + 3               # rows 32..63 of sequence 1 are not seen
    x.mem_len[0, 0] = 60                        # clamped to 50
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_BAD_PAGE | msa.MSA_DEVERR_CAPACITY
    for b in (0, 2):
        assert torch.equal(x.out[:, 40 * b:40 * b + 40].view(torch.int16), good[:, 40 * b:40 * b + 40].view(torch.int16))
    want, tol = x.attend()
    loc = x.rows(1, 100)
    for i in (0, 17, 39):
        keep = torch.tensor([r for r in range(61 + i) if not 32 <= r < 64], device="cuda")
        k = torch.cat([x.mem[0, 0, 0, :, :50].double(), loc[0, 0][:, keep]], 1)
        v = torch.cat([x.mem[0, 0, 1, :, :50].double(), loc[1, 0][:, keep]], 1)
        s = torch.einsum("hgd,hkd->hgk", x.q[0, 40 + i].double().view(16, 4, D), k) * D ** -0.5
        w = torch.einsum("hgk,hkd->hgd", torch.softmax(s, -1), v).reshape(64, D)
        assert ((x.out[0, 40 + i].double() - w).abs() <= tol[0, 40 + i] + 2 ** -7 * w.abs()).all()
    x.err.zero_()
    x.mem_len[0, 0] = 50
    x.off[2] = 4000                             # sequences 1 and 2 unusable: left as they were
    x.out.fill_(7.0)
    x.call_attend(msa)
    assert x.err.item() == msa.MSA_DEVERR_BAD_OFFSETS
    assert (x.out[:, 40:] == 7.0).all()
    assert torch.equal(x.out[:, :40].view(torch.int16), good[:, :40].view(torch.int16))


def test_blocks_whose_first_rows_see_nothing():
    x = Batch([50, 60], [0, 0], H=1, G=4, seed=24)
    x.seq_len[0], x.seq_len[1] = 20, 0
    x.call_attend(msa)
    x.check()
    assert (x.out[:, :30] == 0).all() and (x.out[:, 30:50] != 0).any() and (x.out[:, 50:] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_q", [True, False])
def test_append_of_many_tokens_and_layers(dtype, with_q):
    # a CTA takes a run of layers of its token: runs that do not divide the layers
    x = Batch([300, 1, 211, 170], [3, 60, 0, 31], L=7, H=2, G=4, page=64, pad=3, seed=25, dtype=dtype)
    before, q_rot = x.pages.clone(), torch.full_like(x.out, 7.0)
    off = torch.tensor([5, 0, 1000, 77], dtype=torch.int32, device="cuda")
    q = x.q
    if not with_q:
        x.call_append(msa, off, 16, q_rot=q_rot)
        once, x.q = x.pages.clone(), None
        x.pages.copy_(before)
        x.call_append(msa, off, 16)
        assert torch.equal(once.view(torch.int16), x.pages.view(torch.int16))
        x.q = q
    else:
        x.call_append(msa, off, 16, q_rot=q_rot)
    _check_append(x, q_rot, before, off, 16)
    assert (q_rot[:, -3:] == 7.0).all() and x.err.item() == 0


def test_calls_follow_the_current_stream():
    # captured from the current stream, without a stream argument: append, block form and memory form
    x = Batch([70, 60], [0, 20], L=8, H=16, G=4, groups=[0, 2], mem=[100], seed=26)
    y = Batch([1] * 40, [30] * 40, L=8, H=16, G=4, groups=[0, 40], mem=[300], seed=27)
    for z in (x, y):
        z.call_attend(msa)
    q_rot = [torch.empty_like(z.out) for z in (x, y)]
    raw = [z.q for z in (x, y)]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        for z, r, w in zip((x, y), q_rot, raw):
            z.q = w
            z.call_append(msa, q_rot=r)
            z.q = r
            z.call_attend(msa)
    for _ in range(2):
        for z, w in zip((x, y), raw):
            w.normal_()
            z.k.normal_()
            z.v.normal_()
            z.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        x.check()
        y.check()


def test_two_streams_with_their_own_workspaces():
    xs = [Batch([1] * 40, [25] * 40, L=4, H=16, G=4, groups=[0, 40], mem=[900], seed=28),
          Batch([50] * 6, [40] * 6, L=4, H=16, G=4, groups=[0, 6], mem=[500], seed=29),
          Batch([1] * 9, [700] * 9, L=2, H=4, G=4, seed=30)]
    assert [x.call_attend(msa) for x in xs] == [2, 1, 1]
    torch.cuda.synchronize()
    alone = [x.out.clone() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for x, s in zip(xs, streams):
            x.call_attend(msa, stream=s)
    torch.cuda.synchronize()
    for x, want in zip(xs, alone):
        assert torch.equal(x.out.view(torch.int16), want.view(torch.int16)) and x.err.item() == 0


@pytest.mark.parametrize("G,new", [(4, 20), (1, 100), (8, 33), (2, 64)])
def test_one_row_tile_over_keys_of_all_lengths(G, new):
    # sequences of one row tile: no key tile, one, two, odd and even numbers of them; one sequence
    # with values that are not finite
    past = [0, 100, 128 - new, 129, 300, 513, 40, 700, 1, 255]
    x = Batch([new] * 10, [max(0, p) for p in past], L=4, H=16, G=G, page=16, groups=[0, 3, 6, 10], mem=[0, 128, 200],
              seed=31)
    x.seq_len[0] = 0  # (its rows see nothing)
    assert x.call_attend(msa) == 1
    x.check()
    first = x.out.clone()
    last = x.ids[5][(513 + new - 1) // 16], (513 + new - 1) % 16
    x.pages[:, last[0], 1, :, last[1], 7] = float("-inf")
    x.call_attend(msa)
    end = 6 * new - 1
    rest = torch.ones(x.T, dtype=torch.bool, device="cuda")
    rest[end] = False
    assert torch.equal(first[:, rest].view(torch.int16), x.out[:, rest].view(torch.int16))
    assert (x.out[:, end, :, 7] == float("-inf")).all()
    assert torch.equal(first[:, end, :, 8:].view(torch.int16), x.out[:, end, :, 8:].view(torch.int16))


def test_few_sequences_over_a_long_memory_are_cut():
    # blocks of new tokens, but too few for the GPU: the memory form, which cuts the memory
    x = Batch([60, 90], [10, 70], H=8, G=4, groups=[0, 1, 2], mem=[9000, 1], seed=32)
    assert x.call_attend(msa) == 2
    x.check()


@pytest.mark.parametrize("B", [511, 513])
def test_blocks_of_many_sequences(B):
    # both sides of the number of sequences that are put in order
    new = [17 + b % 3 for b in range(B)]
    x = Batch(new, [(11 * b) % 29 for b in range(B)], H=1, G=8, groups=[0, 5, B - 1], mem=[3, 20], seed=33)
    x.call_attend(msa)
    pick = [0, 4, 5, 77, B - 2, B - 1]
    want, tol = x.attend(only=pick)
    for b in pick:
        at = slice(x.off[b].item(), x.off[b + 1].item())
        assert ((x.out[:, at].double() - want[:, at]).abs() <= tol[:, at]).all()
    assert not x.out.isnan().any() and x.err.item() == 0
