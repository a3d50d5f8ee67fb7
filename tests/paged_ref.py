"""Inputs and 64-bit results of the paged-batch tests (no product code).

``Batch`` lays out a ragged batch: packed tokens, pages dealt in a shuffled order, unused
page slots and memory rows filled with NaN, unused page-table entries with an id that no pool
has.  ``append`` and ``attend`` compute what ``include/msa_paged.h`` defines, sequence by
sequence in fp64.

Tolerances.  An output is a sum of weights times values, rounded to bf16 (half a step: 2^-8 of
the value).  Before that rounding, with A = sum of |weight * value|: the weights may be bf16
operands of the tensor cores (2^-8 of each, and of their sum: 2^-7 A); fp32 accumulation over
n keys adds at most n 2^-22 A for sum and denominator together; a score is an fp32 sum of 128
products, off by at most 128 * 2^-23 times the sum of their magnitudes (times the softmax
scale), which moves a weight by the same fraction, numerator and denominator: twice that.
"""
import math

import torch

D = 128
U = 2.0 ** -8  # half a bf16 step, relative


class Batch:
    def __init__(self, new, past, *, L=1, H=2, G=4, page=16, groups=None, mem=None, M=None, pad=0, lead=0, seed=0,
                 dtype=torch.bfloat16, spare=2, scale=1.0, device="cuda"):
        gen = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
        self.new, self.past, self.L, self.H, self.G, self.page, self.lead = list(new), list(past), L, H, G, page, lead
        self.HQ, self.B, self.T = H * G, len(new), lead + sum(new) + pad
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
        off = [lead]
        for n in new:
            off.append(off[-1] + n)
        self.off, self.seq_len = ints(off), ints([n + p for n, p in zip(new, past)])
        need = [-(-(n + p) // page) for n, p in zip(new, past)]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=gen).tolist()
        self.max_pages = max(need + [1]) + 1
        self.ids, table = [], []
        for k in need:
            mine, order = order[:k], order[k:]
            self.ids.append(mine)
            table.append(mine + [0x7FFFFFF0] * (self.max_pages - k))
        self.table = ints(table)
        pages = torch.full((L, self.n_pages, 2, H, page, D), float("nan"))
        for b, (n, p) in enumerate(zip(new, past)):
            for r0 in range(0, n + p, page):
                rows = min(page, n + p - r0)
                pages[:, self.ids[b][r0 // page], :, :, :rows] = rnd(L, 2, H, rows, D)
        self.pages = pages.to(torch.bfloat16).to(device)
        self.q = (scale * rnd(L, self.T, self.HQ, D)).to(dtype).to(device)
        self.k = rnd(L, self.T, H, D).to(dtype).to(device)
        self.v = rnd(L, self.T, H, D).to(dtype).to(device)
        self.groups = groups if groups is not None else []
        self.NG = max(0, len(self.groups) - 1)
        self.goff = ints(self.groups) if self.NG else None
        self.mem = self.mem_len = None
        self.M = M or 1
        if self.NG:
            mem = [[m] * L if isinstance(m, int) else list(m) for m in mem]
            self.M = M or max(1, max(max(r) for r in mem))
            kv = torch.full((self.NG, L, 2, H, self.M, D), float("nan"))
            for g in range(self.NG):
                for l in range(L):
                    m = min(mem[g][l], self.M)
                    kv[g, l, :, :, :m] = rnd(2, H, m, D)
            self.mem, self.mem_len = kv.to(torch.bfloat16).to(device), ints(mem)
        self.out = torch.full((L, self.T, self.HQ, D), 7.0, dtype=torch.bfloat16, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.ws = None

    # ------------------------------------------------------------------ the calls
    def call_append(self, msa, pos_offset=None, pos=16, theta=1e6, q_rot=None, stream=None, **kw):
        return msa.msa_paged_append(self.q, self.k, self.v, self.off, self.T, self.B, self.L, self.HQ, self.H, D,
                                    self.pages, self.n_pages, self.page, self.table, self.max_pages, self.seq_len,
                                    pos_offset, pos, theta, q_rot, dev_err=self.err, stream=stream, **kw)

    def call_attend(self, msa, stream=None, scale=D ** -0.5):
        if self.ws is None:
            n = msa.msa_shared_attend_workspace_size(self.T, self.B, self.NG, self.L, self.HQ, self.H)
            self.ws = torch.zeros(n, dtype=torch.uint8, device=self.q.device)
        return msa.msa_shared_attend(self.q, self.off, self.T, self.B, self.L, self.HQ, self.H, D, self.mem,
                                     self.mem_len, self.M, self.goff, self.NG, self.pages, self.n_pages, self.page,
                                     self.table, self.max_pages, self.seq_len, scale, self.out, self.ws,
                                     dev_err=self.err, stream=stream)

    # ------------------------------------------------------------------ in 64 bits
    def rows(self, b, n):
        """The first n page rows of sequence b: [2, L, H, n, D] in fp64."""
        if n == 0:
            return torch.zeros((2, self.L, self.H, 0, D), dtype=torch.float64, device=self.pages.device)
        ids = torch.tensor(self.ids[b][:-(-n // self.page)], device=self.pages.device)
        kv = self.pages[:, ids].double()  # [L, P, 2, H, page, D]
        return kv.permute(2, 0, 3, 1, 4, 5).reshape(2, self.L, self.H, -1, D)[:, :, :, :n]

    def group_of(self, b):
        for g in range(self.NG):
            if self.groups[g] <= b < self.groups[g + 1]:
                return g
        return None

    def attend(self, scale=D ** -0.5, only=None):
        """(expected output, tolerance), both [L, T, HQ, D] fp64; tolerance < 0 where the output
        is to be left as it was (and for sequences not in `only`)."""
        L, H, G = self.L, self.H, self.G
        want = torch.zeros((L, self.T, self.HQ, D), dtype=torch.float64, device=self.q.device)
        tol = torch.full_like(want, -1.0)
        for b, (new, past) in enumerate(zip(self.new, self.past)):
            if only is not None and b not in only:
                continue
            t0 = self.off[b].item()
            ln = self.seq_len[b].item()
            cut = ln - new
            kept = max(0, min(ln, self.max_pages * self.page))
            loc = self.rows(b, kept)
            g = self.group_of(b)
            for i in range(new):
                n_loc = max(0, min(cut + i + 1, kept))
                for l in range(L):
                    k, v = loc[0, l, :, :n_loc], loc[1, l, :, :n_loc]
                    if g is not None:
                        m = max(0, min(int(self.mem_len[g, l]), self.M))
                        k = torch.cat([self.mem[g, l, 0, :, :m].double(), k], 1)
                        v = torch.cat([self.mem[g, l, 1, :, :m].double(), v], 1)
                    q = self.q[l, t0 + i].double().view(H, G, D)
                    if k.shape[1] == 0:
                        want[l, t0 + i] = 0.0
                        tol[l, t0 + i] = 0.0
                        continue
                    s = torch.einsum("hgd,hkd->hgk", q, k) * scale
                    mag = torch.einsum("hgd,hkd->hgk", q.abs(), k.abs()).amax(-1, keepdim=True) * scale
                    w = torch.softmax(s, -1)
                    o = torch.einsum("hgk,hkd->hgd", w, v)
                    a = torch.einsum("hgk,hkd->hgd", w, v.abs())
                    want[l, t0 + i] = o.reshape(self.HQ, D)
                    slack = a * (2 * U + k.shape[1] * 2.0 ** -22 + 2 * 128 * 2.0 ** -23 * mag)
                    tol[l, t0 + i] = (U * (o.abs() + slack) + slack).reshape(self.HQ, D)
        return want, tol

    def check(self, scale=D ** -0.5):
        want, tol = self.attend(scale)
        own = tol >= 0
        got = self.out.double()
        assert torch.all(got[~own] == 7.0), "rows of no sequence were written"
        bad = own & ~((got - want).abs() <= tol)
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist())
        # two independent roundings of at most half a step each (weights, output): each has an
        # rms of at most 2^-8 / sqrt(3) of the output's norm, together below 2^-8
        if own.any() and want[own].norm() > 0:
            rel = ((got - want)[own].norm() / want[own].norm()).item()
            assert rel <= U, rel


def rope(x, pos, theta=1e6):
    """fp64 rotate-half of x [..., heads, D] at positions pos [...]."""
    j = torch.arange(D // 2, dtype=torch.float64, device=x.device)
    ang = pos.double()[..., None] * torch.exp(-2.0 * j / D * math.log(theta))
    c, s = torch.cos(ang)[..., None, :], torch.sin(ang)[..., None, :]
    lo, hi = x[..., :D // 2].double(), x[..., D // 2:].double()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)
