"""The paged memory, the attention over it, eviction and 4-bit weights restated in 64 bits (torch on the CPU), for the
tests, with the tolerances that the kernels' number formats give."""
from __future__ import annotations

import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}     # half a step, relative


class Pages:
    """A paged memory on the CPU in 64 bits, filled at random: sequence b holds lens[b] positions, of which the next is
    first[b]; its pages lie anywhere in the pool."""

    def __init__(self, B, H, D, lens, page_len, dtype, room=0, first=None, seed=0, spare=2, order=False):
        g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.D, self.page_len, self.dtype = B, H, D, page_len, dtype
        most = max(max(lens) + room, 1)
        per = (most + page_len - 1) // page_len
        n = B * per + spare
        self.k, self.v = (torch.randn(n, H, page_len, D, generator=g).to(dtype) for _ in range(2))
        self.table = torch.randperm(n, generator=g)[: B * per].view(B, per).int()
        self.length = torch.tensor(lens, dtype=torch.int32)
        first = list(lens) if first is None else first
        self.next_pos = torch.tensor(first, dtype=torch.int32)
        self.pos = torch.zeros(n, page_len, dtype=torch.int32)
        self.weight = torch.rand(n, page_len, generator=g)
        for b in range(B):
            p = torch.randperm(first[b], generator=g)[: lens[b]]
            p = p.sort().values if order else p
            for s in range(lens[b]):
                self.pos[self.at(b, s)] = int(p[s])

    def at(self, b, s):
        return int(self.table[b, s // self.page_len]), s % self.page_len

    def index(self, b, n):
        s = torch.arange(n)
        return self.table[b, s // self.page_len].long(), s % self.page_len

    def push(self, k, v, counts=None):
        for b in range(self.B):
            for t in range(k.shape[1] if counts is None else int(counts[b])):
                p, row = self.at(b, int(self.length[b]))
                self.k[p, :, row], self.v[p, :, row] = k[b, t], v[b, t]
                self.pos[p, row], self.weight[p, row] = self.next_pos[b], 0.0
                self.length[b] += 1
                self.next_pos[b] += 1

    def evict(self, keep, recent):
        for b in range(self.B):
            n = int(self.length[b])
            if n <= keep:
                continue
            p, row = self.index(b, n)
            pos, w = self.pos[p, row].tolist(), self.weight[p, row].tolist()
            may = [s for s in range(n) if pos[s] < int(self.next_pos[b]) - recent]
            may.sort(key=lambda s: (math.inf, 1, pos[s]) if math.isnan(w[s]) else (w[s], 0, pos[s]))
            gone = set(may[: n - keep])
            holes = [s for s in range(keep) if s in gone]
            movers = [s for s in range(keep, n) if s not in gone]
            assert len(holes) == len(movers)
            for to, fr in zip(holes, movers):
                a, c = self.at(b, to), self.at(b, fr)
                for t in (self.k, self.v):
                    t[a[0], :, a[1]] = t[c[0], :, c[1]]
                self.pos[a], self.weight[a] = self.pos[c].clone(), self.weight[c].clone()
            self.length[b] = keep

    def to_gpu(self, txl):
        """The same memory on the device (rows padded, what a row holds past D is NaN)."""
        unit = 16 // self.k.element_size()
        ld = (self.D + unit - 1) // unit * unit

        def pool(x):
            store = torch.full((*x.shape[:3], ld), math.nan, dtype=self.dtype, device="cuda")
            store[..., : self.D] = x.cuda()
            return store[..., : self.D]

        return txl.PagedMemory(pool(self.k), pool(self.v), self.pos.cuda(), self.weight.cuda(), self.table.cuda(),
                               self.length.cuda(), self.next_pos.cuda())


def attend(mem: Pages, q, u, vb, r, C, counts=None, scale=None):
    """Outputs [B, T, H, D] (NaN where a row is left alone), what each slot receives [n_pages, page_len], and bounds on
    the kernels' errors of both."""
    B, T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    C = min(C, r.shape[0] - 1)
    out = torch.full(q.shape, math.nan, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    got = torch.zeros(mem.weight.shape, dtype=torch.float64)
    got_tol = torch.zeros_like(got)
    f32 = mem.dtype == torch.float32
    r = r[..., :D].double()
    for b in range(B):
        n = T if counts is None else int(counts[b])
        L = int(mem.length[b])
        if n == 0:
            continue
        p, row = mem.index(b, L)
        k, v = mem.k[p, :, row].double(), mem.v[p, :, row].double()             # [L, H, D]
        pos = mem.pos[p, row].long()
        for i in range(n):
            at = int(mem.next_pos[b]) - n + i
            seen = pos <= at
            out[b, i] = 0.0
            if not bool(seen.any()):
                continue
            ks, vs = k[seen], v[seen]
            rs = r[(at - pos[seen]).clamp(max=C)]                               # [S, H, D]
            qu, qv = q[b, i].double() + u.double(), q[b, i].double() + vb.double()
            s = scale * ((qu * ks).sum(-1) + (qv * rs).sum(-1))                 # [S, H]
            w = torch.softmax(s, 0)
            out[b, i] = (w[..., None] * vs).sum(0)
            # a score's error: fp32 products and sums of 2 D terms, and in bf16 the operand's 2^-17 that two bf16 leave
            size = scale * ((qu.abs() * ks.abs()).sum(-1) + (qv.abs() * rs.abs()).sum(-1)).max(0).values     # [H]
            ds = size * ((2 * D + 8) * 2.0 ** -24 if f32 else 2.0 ** -16 + (2 * D + 8) * 2.0 ** -24)
            # a weight's: e^(2 ds) - 1, the exponential's own 2^-22 of scores up to `size`, sums of its share of L keys
            dw = 2 * ds + (size + 2) * 2.0 ** -22 + L * 2.0 ** -24 + (0 if f32 else 2.0 ** -16)              # [H]
            tol[b, i] = HALF[mem.dtype] * out[b, i].abs() + dw[:, None] * (w[..., None] * vs.abs()).sum(0) * 2
            sl = torch.nonzero(seen).flatten()
            got.index_put_((p[sl], row[sl]), w.sum(1), accumulate=True)
            got_tol.index_put_((p[sl], row[sl]), (w * (dw + H * n * 2.0 ** -23)).sum(1), accumulate=True)
    return out, tol, got, got_tol


def bf16_toward(x: torch.Tensor, up: bool) -> torch.Tensor:
    """fp64 x to the neighbouring bf16 toward +inf (up) or -inf, by comparing the candidates."""
    y = x.float().bfloat16()                                    # either neighbour of x
    for _ in range(2):
        wrong = (y.double() < x) if up else (y.double() > x)
        bits = y.view(torch.int16).int()
        away = torch.where(y == 0, torch.full_like(bits, 1 if up else -32767),
                           torch.where((y > 0) == up, bits + 1, bits - 1))
        y = torch.where(wrong, away.short().view(torch.bfloat16), y)
    return y


def q4(W: torch.Tensor, group: int):
    """codes [k, n], step and lo [groups, n] (fp64) of bf16 W, and what they stand for [k, n]."""
    k, n = W.shape
    code, held = torch.zeros(k, n, dtype=torch.float64), torch.zeros(k, n, dtype=torch.float64)
    steps, los = [], []
    for a in range(0, k, group):
        x = W[a:a + group].double()
        bad = ~torch.isfinite(x).all(0)
        x = torch.where(bad, torch.zeros_like(x), x)
        lo = x.min(0).values
        step = bf16_toward((x.max(0).values - lo) / 15, True).double()
        c = torch.where(step > 0, torch.round((x - lo) / torch.where(step > 0, step, torch.ones_like(step))), torch.zeros_like(x))
        assert int(c.min()) >= 0 and int(c.max()) <= 15
        bad |= ~torch.isfinite(step)
        code[a:a + group] = torch.where(bad, torch.zeros_like(c), c)
        held[a:a + group] = torch.where(bad, torch.full_like(c, math.nan), lo + step * c)
        steps.append(step)
        los.append(lo)
    return code, torch.stack(steps), torch.stack(los), held
