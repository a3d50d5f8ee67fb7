"""The serving operators of a paged local cache, as workloads: what is timed and compared.

Two operators.  ``append``: the new tokens' keys are rotated (RoPE at each token's position)
and stored with the values in the pages of their sequences, and the queries are rotated.
``attend``: every new token attends its group's shared memory (one gathered selection for
all sequences of the group) followed by its own sequence's pages, causal over the new
tokens.  With ``own`` false ``run`` is plain torch in 32 bits, with ``own`` true it is the
calls a user makes of the package.
"""
import math
import random

import torch

own = False

D = 128          # head size of the package's attention kernels
THETA = 1e6


# ----------------------------------------------------------------------------- the cases

def _append(name, **kw):
    c = {"name": name, "op": "append", "dtype": "bf16", "layers": 18, "hq": 32, "h": 8, "seqs": 1, "new_lo": 1,
         "new_hi": 1, "past_lo": 0, "past_hi": 256, "page": 64, "fused": False, "pad": 0, "pos": 16, "layout": 0}
    c.update(kw)
    return c


def _attend(name, **kw):
    c = {"name": name, "op": "attend", "layers": 18, "hq": 32, "h": 8, "seqs": 1, "groups": 1, "mem_lo": 256,
         "mem_hi": 256, "new_lo": 1, "new_hi": 1, "past_lo": 256, "past_hi": 383, "page": 64, "bare": 0, "pad": 0,
         "layout": 0}
    c.update(kw)
    return c


def listed():
    return [
        # one answer's next token, all 18 memory layers: the smallest call, latency alone
        _append("append one token"),
        # one step of 128 answers sampled at once
        _append("append 128 answers", seqs=128, past_hi=400, layout=1),
        # questions of different lengths arriving together, fp32 activations, small pages, a padded batch
        _append("append ragged questions", dtype="f32", layers=4, seqs=24, new_hi=511, past_hi=40, page=16, pad=7,
                layout=2),
        # long raw documents of one layer out of a fused projection, far positions
        _append("append long texts", layers=2, hq=64, h=8, seqs=5, new_lo=3000, new_hi=8192, past_hi=5000, page=128,
                fused=True, pos=1 << 20, layout=3),
        # one answer's next token over 16 selected documents (256 blocks): the package's own decode step
        _attend("attend one token"),
        # sixteen answers to one question, sharing its documents
        _attend("attend 16 answers", seqs=16, layout=4),
        # sixteen questions, eight answers each, selections of different sizes
        _attend("attend 16 groups", seqs=128, groups=16, mem_lo=100, mem_hi=700, past_lo=30, past_hi=400, layout=5),
        # one layer of a batch that shares a long text, answers of 1 to 600 tokens
        _attend("attend long memory", layers=1, seqs=64, mem_lo=32768, mem_hi=32768, past_lo=0, past_hi=600, page=32,
                layout=6),
        # the same with eight query heads a key head and a large batch: bound by arithmetic
        _attend("attend wide batch", layers=1, hq=64, seqs=256, mem_lo=16384, mem_hi=16384, past_lo=15, past_hi=500,
                layout=7),
        # five drafted tokens checked at once
        _attend("attend drafts", layers=4, seqs=33, mem_lo=1000, mem_hi=1000, new_lo=5, new_hi=5, past_lo=100,
                past_hi=900, page=16, layout=8),
        # the questions themselves: 100 to 256 new tokens each over the shared documents
        _attend("attend questions", seqs=8, mem_lo=256, mem_hi=256, new_lo=100, new_hi=256, past_lo=0, past_hi=0,
                layout=9),
        # a mixed batch: next tokens and chunks of questions, some sequences without a memory, padded
        _attend("attend mixed", layers=2, hq=16, seqs=40, groups=3, mem_lo=0, mem_hi=1500, new_hi=200, past_lo=0,
                past_hi=1800, page=128, bare=4, pad=3, layout=10),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    heads = rng.choice([(32, 8), (32, 8), (64, 8), (16, 8), (8, 8), (32, 4), (16, 16), (4, 2), (16, 2)])
    page = rng.choice([16, 32, 64, 128])
    layout = rng.randrange(1 << 20)
    if rng.random() < 0.35:
        new = _log(rng, 1, 4096)
        c = _append("", dtype=rng.choice(["bf16", "f32"]), layers=_log(rng, 1, 18), hq=heads[0], h=heads[1],
                    seqs=_log(rng, 1, 128), new_lo=rng.choice([1, new]), new_hi=new, past_hi=_log(rng, 1, 4000),
                    page=page, fused=rng.random() < 0.4, pad=rng.choice([0, 0, 1, 13]), pos=_log(rng, 1, 1 << 22),
                    layout=layout)
        most = 1.2e9
    else:
        new = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 9, 400)])
        seqs, mem, past = _log(rng, 1, 256), _log(rng, 1, 32768), _log(rng, 1, 4000)
        c = _attend("", layers=_log(rng, 1, 18), hq=heads[0], h=heads[1], seqs=seqs,
                    groups=rng.choice([1, 1, _log(rng, 1, max(1, seqs // 2))]), mem_lo=rng.choice([0, mem // 2, mem]),
                    mem_hi=mem, new_lo=rng.choice([1, new]), new_hi=new, past_lo=rng.choice([0, past]), past_hi=past,
                    page=page, bare=rng.choice([0, 0, seqs // 3]), pad=rng.choice([0, 0, 5]), layout=layout)
        most = 2.0e9
    c.pop("name")
    while True:  # no more than the largest listed case
        w = work(c)
        if w["bytes"] + w["flops"] / 50 <= most and (c["op"] == "append" or _plain_floats(c) < 2.5e9):
            return c
        for key in ("layers", "seqs", "new_hi", "mem_hi", "past_hi"):
            if c.get(key, 1) > 1 and rng.random() < 0.5:
                c[key] = max(1, c[key] * 2 // 3)
        c["new_lo"] = min(c["new_lo"], c["new_hi"])
        c["past_lo"] = min(c["past_lo"], c["past_hi"])
        if c["op"] == "attend":
            c["mem_lo"] = min(c["mem_lo"], c["mem_hi"])
            c["groups"] = min(c["groups"], c["seqs"])
            c["bare"] = min(c["bare"], c["seqs"] // 3)


def _layout(c):
    """Lengths of a case (from the case alone): new tokens and rows before them per
    sequence, the sequences of each group, each group's memory rows per layer."""
    r = random.Random(c["layout"] * 7919 + 13)
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["seqs"])]
    past = [r.randint(c.get("past_lo", 0), c["past_hi"]) for _ in range(c["seqs"])]
    out = {"new": new, "past": past, "tokens": sum(new) + c["pad"]}
    out["longest"] = max(n + p for n, p in zip(new, past))
    if c["op"] == "attend":
        grouped = c["seqs"] - c["bare"]  # the last `bare` sequences have no memory
        cuts = sorted(r.sample(range(1, grouped), c["groups"] - 1)) if c["groups"] > 1 else []
        out["groups"] = [0] + cuts + [grouped]
        out["mem"] = [[r.randint(c["mem_lo"], c["mem_hi"]) for _ in range(c["layers"])] for _ in range(c["groups"])]
    return out


def _plain_floats(c):
    """Values that the plain form of an attend case holds at once, about."""
    y = _layout(c)
    n, rows = max(y["new"]), max(sum(y["new"][a:b]) for a, b in zip(y["groups"], y["groups"][1:]))
    loc = c["layers"] * c["seqs"] * y["longest"] * (2 * c["h"] * D + 2 * c["hq"] * n)
    mem = c["layers"] * c["groups"] * c["mem_hi"] * (2 * c["h"] * D + 2 * c["hq"] * rows)
    return loc + mem + 4 * c["layers"] * c["seqs"] * n * c["hq"] * D


def work(case):
    c, y = case, _layout(case)
    n_tok = sum(y["new"])
    row = (c["hq"] + 2 * c["h"]) * D
    ints = 4 * (3 * c["seqs"] + sum(-(-(n + p) // c["page"]) for n, p in zip(y["new"], y["past"])))
    if c["op"] == "append":
        each = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["layers"] * n_tok * row * (each + 2) + ints,
                "flops": c["layers"] * n_tok * (c["hq"] + c["h"]) * D * 3}
    kv = 2 * c["h"] * D * 2
    size = c["layers"] * n_tok * c["hq"] * D * 4 + ints  # q in, out back
    size += sum(sum(m) for m in y["mem"]) * kv
    size += c["layers"] * sum(n + p for n, p in zip(y["new"], y["past"])) * kv
    pairs = c["layers"] * sum(n * p + n * (n + 1) // 2 for n, p in zip(y["new"], y["past"]))
    for g, (a, b) in enumerate(zip(y["groups"], y["groups"][1:])):
        pairs += sum(y["new"][a:b]) * sum(y["mem"][g])
    return {"bytes": size, "flops": pairs * c["hq"] * 4 * D}


# ----------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    c, y = case, _layout(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    offs = [0]
    for n in y["new"]:
        offs.append(offs[-1] + n)
    s = dict(c)
    s.update(n_tokens=y["tokens"], n_valid=offs[-1], most_new=max(y["new"]), longest=y["longest"],
             q_offsets=ints(offs), seq_len=ints([n + p for n, p in zip(y["new"], y["past"])]))
    # pages dealt to the sequences in a random order, a few spare ones, unused entries pointing at page 0
    need = [-(-(n + p) // c["page"]) for n, p in zip(y["new"], y["past"])]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, device=dev, generator=gen).to(torch.int32)
    wide = max(max(need), 1)
    table = torch.zeros((c["seqs"], wide), dtype=torch.int32, device=dev)
    at = torch.arange(wide, device=dev)[None] < ints(need)[:, None]
    table[at] = order[:sum(need)]
    s.update(n_pages=n_pages, max_pages=wide, page_table=table)
    L, H, HQ, T = c["layers"], c["h"], c["hq"], y["tokens"]
    s["pages"] = torch.randn((L, n_pages, 2, H, c["page"], D), device=dev, generator=gen, dtype=torch.bfloat16)
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    if c["op"] == "append":
        if c["fused"]:  # one projection's rows: all query heads, then keys, then values
            x = torch.randn((L, T, HQ + 2 * H, D), device=dev, generator=gen, dtype=dt)
            s["q"], s["k"], s["v"] = x[:, :, :HQ], x[:, :, HQ:HQ + H], x[:, :, HQ + H:]
        else:
            s["q"], s["k"], s["v"] = (torch.randn((L, T, n, D), device=dev, generator=gen, dtype=dt)
                                      for n in (HQ, H, H))
        s["q_rot"] = torch.zeros((L, T, HQ, D), device=dev, dtype=torch.bfloat16)
        s["pos_offset"] = torch.randint(0, 1000, (c["seqs"],), device=dev, generator=gen, dtype=torch.int32)
        return s
    s["q"] = 1.5 * torch.randn((L, T, HQ, D), device=dev, generator=gen, dtype=torch.bfloat16)
    s["mem_rows"] = max(1, c["mem_hi"])
    s["mem"] = torch.randn((c["groups"], L, 2, H, s["mem_rows"], D), device=dev, generator=gen, dtype=torch.bfloat16)
    s["mem_len"] = ints(y["mem"])
    s["group_offsets"] = ints(y["groups"])
    s["most_rows"] = max(sum(y["new"][a:b]) for a, b in zip(y["groups"], y["groups"][1:]))
    s["out"] = torch.zeros((L, T, HQ, D), device=dev, dtype=torch.bfloat16)
    return s


# ----------------------------------------------------------------------------- one pass

def run(state):
    s = state
    if s["op"] == "append":
        return _own_append(s) if own else _plain_append(s)
    return _own_attend(s) if own else _plain_attend(s)


def _own_append(s):
    import top_kv_routing_b200 as msa
    msa.msa_paged_append(s["q"], s["k"], s["v"], s["q_offsets"], s["n_tokens"], s["seqs"], s["layers"], s["hq"],
                         s["h"], D, s["pages"], s["n_pages"], s["page"], s["page_table"], s["max_pages"],
                         s["seq_len"], s["pos_offset"], s["pos"], THETA, s["q_rot"], q_stride=s["q"].stride(1),
                         k_stride=s["k"].stride(1), v_stride=s["v"].stride(1))
    return s["q_rot"], s["pages"]


def _own_attend(s):
    import top_kv_routing_b200 as msa
    if "workspace" not in s:
        n = msa.msa_shared_attend_workspace_size(s["n_tokens"], s["seqs"], s["groups"], s["layers"], s["hq"], s["h"])
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=s["q"].device)
    msa.msa_shared_attend(s["q"], s["q_offsets"], s["n_tokens"], s["seqs"], s["layers"], s["hq"], s["h"], D,
                          s["mem"], s["mem_len"], s["mem_rows"], s["group_offsets"], s["groups"], s["pages"],
                          s["n_pages"], s["page"], s["page_table"], s["max_pages"], s["seq_len"], D ** -0.5, s["out"],
                          s["workspace"])
    return s["out"]


def _plain_append(s):
    dev, n = s["q"].device, s["n_valid"]
    off, length = s["q_offsets"].long(), s["seq_len"].long()
    tok = torch.arange(n, device=dev)
    b = torch.searchsorted(off[1:], tok, right=True)
    row = length[b] - (off[b + 1] - tok)
    at = (s["pos"] + s["pos_offset"].long()[b] + row).double()
    freq = THETA ** (-torch.arange(D // 2, device=dev, dtype=torch.float64) / (D // 2))
    angle = at[:, None] * freq
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x):
        lo, hi = x[..., :D // 2].float(), x[..., D // 2:].float()
        return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], dim=-1).to(torch.bfloat16)

    s["q_rot"][:, :n] = turned(s["q"][:, :n])
    page, slot = s["page_table"].long()[b, row // s["page"]], row % s["page"]
    s["pages"][:, page, 0, :, slot] = turned(s["k"][:, :n]).transpose(0, 1)
    s["pages"][:, page, 1, :, slot] = s["v"][:, :n].to(torch.bfloat16).transpose(0, 1)
    return s["q_rot"], s["pages"]


def _part(q, k, v, seen):
    """Running maximum, sum and weighted values of rows q over keys k where `seen`."""
    x = torch.matmul(q, k.transpose(-1, -2)).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-1e30)
    x = torch.exp(x.sub_(top))
    return top, x.sum(-1, keepdim=True), torch.matmul(x, v)


def _plain_attend(s):
    dev, L, H, HQ, B, n = s["q"].device, s["layers"], s["h"], s["hq"], s["seqs"], s["n_valid"]
    G, NG, S, R = HQ // H, s["groups"], s["most_new"], s["most_rows"]
    off, length, goff = s["q_offsets"].long(), s["seq_len"].long(), s["group_offsets"].long()
    q = s["q"][:, :n].float().mul_(D ** -0.5).view(L, n, H, G, D)
    tok = torch.arange(n, device=dev)
    b = torch.searchsorted(off[1:], tok, right=True)  # each token's sequence, and its place there
    i = tok - off[b]
    # the sequences' own pages: rows of one sequence padded to the longest block
    pad = torch.zeros((L, B, S, H, G, D), device=dev)
    pad[:, b, i] = q
    used = -(-s["longest"] // s["page"])
    kv = s["pages"][:, s["page_table"].long()[:, :used]]  # [L, B, used, 2, H, page, D]
    kv = kv.permute(3, 0, 1, 4, 2, 5, 6).reshape(2, L, B, H, used * s["page"], D).float()
    key = torch.arange(used * s["page"], device=dev)
    last = (length - off.diff())[:, None] + torch.arange(S, device=dev)
    seen = (key <= last[..., None])[:, None, :, None].expand(B, 1, S, G, -1).reshape(B, 1, S * G, -1)
    loc = _part(pad.permute(0, 1, 3, 2, 4, 5).reshape(L, B, H, S * G, D), kv[0], kv[1], seen)
    loc = [x.view(L, B, H, S, G, -1).permute(0, 1, 3, 2, 4, 5)[:, b, i] for x in loc]  # [L, n, H, G, .]
    del kv, pad
    # the groups' memory: all rows of a group at once
    g = torch.searchsorted(goff[1:], b, right=True)
    has, g = g < NG, g.clamp_max(NG - 1)
    r = (tok - off[goff[g]]).clamp_max(R - 1)
    pad = torch.zeros((L, NG, R, H, G, D), device=dev)
    pad[:, g[has], r[has]] = q[:, has]
    mem = s["mem"].permute(2, 1, 0, 3, 4, 5).float()  # [2, L, NG, H, M, D]
    seen = (torch.arange(s["mem_rows"], device=dev) < s["mem_len"].long().t()[..., None])[:, :, None, None]
    far = _part(pad.permute(0, 1, 3, 2, 4, 5).reshape(L, NG, H, R * G, D), mem[0], mem[1], seen)
    far = [x.view(L, NG, H, R, G, -1).permute(0, 1, 3, 2, 4, 5)[:, g, r] for x in far]
    top = torch.maximum(loc[0], torch.where(has[:, None, None, None], far[0], -math.inf))
    wl = torch.exp(loc[0] - top)
    wf = torch.where(has[:, None, None, None], torch.exp(far[0] - top), 0.0)
    total = wl * loc[1] + wf * far[1]
    o = (wl * loc[2] + wf * far[2]) / torch.where(total > 0, total, 1.0)
    s["out"][:, :n] = o.reshape(L, n, HQ, D).to(torch.bfloat16)
    return s["out"]


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s, y = prepare(case, seed), _layout(case)
    L, H, HQ, ps = s["layers"], s["h"], s["hq"], s["page"]
    G, at = HQ // H, 0
    if s["op"] == "append":
        q_rot, pages = s["q_rot"].double(), s["pages"].double()
        j = torch.arange(D // 2, dtype=torch.float64, device=s["q"].device)
        freq = torch.exp(-2.0 * j / D * math.log(THETA))
        for b, (new, past) in enumerate(zip(y["new"], y["past"])):
            row = past + torch.arange(new, device=j.device)
            turn = torch.exp(1j * ((s["pos"] + s["pos_offset"][b].item() + row)[:, None] * freq))[:, None]
            pair = lambda x: torch.complex(x[..., :D // 2].double(), x[..., D // 2:].double()) * turn  # noqa: E731,B023
            rot = lambda x: torch.cat([pair(x).real, pair(x).imag], -1)  # noqa: E731,B023
            q_rot[:, at:at + new] = rot(s["q"][:, at:at + new])
            page, slot = s["page_table"][b].long()[row // ps], row % ps
            pages[:, page, 0, :, slot] = rot(s["k"][:, at:at + new]).transpose(0, 1)
            pages[:, page, 1, :, slot] = s["v"][:, at:at + new].double().transpose(0, 1)
            at += new
        return q_rot, pages
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    group = {b: g for g, (lo, hi) in enumerate(zip(y["groups"], y["groups"][1:])) for b in range(lo, hi)}
    kept = (None, None)
    for b, (new, past) in enumerate(zip(y["new"], y["past"])):
        n = new + past
        ids = s["page_table"][b, :-(-n // ps)].long()
        kv = s["pages"][:, ids].double().permute(2, 0, 3, 1, 4, 5).reshape(2, L, H, -1, D)[:, :, :, :n]
        q = s["q"][:, at:at + new].double().view(L, new, H, G, D).permute(0, 2, 3, 1, 4)  # [L, H, G, new, D]
        x = torch.einsum("lhgnd,lhkd->lhgnk", q, kv[0]) / math.sqrt(D)
        row, key = torch.arange(new, device=q.device)[:, None], torch.arange(n, device=q.device)[None]
        x = torch.where(key <= past + row, x, -math.inf)
        if b in group:
            if kept[0] != group[b]:
                kept = (group[b], s["mem"][group[b]].double().permute(1, 0, 2, 3, 4))  # [2, L, H, M, D]
            m = torch.arange(s["mem_rows"], device=q.device) < s["mem_len"][group[b]][:, None]
            z = torch.einsum("lhgnd,lhkd->lhgnk", q, kept[1][0]) / math.sqrt(D)
            z = torch.where(m[:, None, None, None], z, -math.inf)
            w = torch.softmax(torch.cat([z, x], -1), -1)
            o = torch.einsum("lhgnk,lhkd->lhgnd", w[..., :z.shape[-1]], kept[1][1])
            o = o + torch.einsum("lhgnk,lhkd->lhgnd", w[..., z.shape[-1]:], kv[1])
        else:
            o = torch.einsum("lhgnk,lhkd->lhgnd", torch.softmax(x, -1), kv[1])
        out[:, at:at + new] = o.permute(0, 3, 1, 2, 4).reshape(L, new, HQ, D)
        at += new
    return out
