"""The quantised memory and the attention over it restated in 64 bits (numpy), for the tests.

quantise64 follows the definition in include/txl.h: per group of 32 channels lo = bf16 floor of the
minimum, step = bf16 ceiling of (max - lo) / n, code = nearest integer to (x - lo) / step, ties to
even.  quantise_exact does the same in rational arithmetic, for values whose differences 64 bits do
not hold."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

GROUP = 32


def bf16_grid(x: np.ndarray, up: bool) -> np.ndarray:
    """Float64 x to the neighbouring bf16 value toward +inf (up) or -inf; bf16 keeps 8 bits above
    2^-126 and multiples of 2^-133 below."""
    with np.errstate(all="ignore"):
        e = np.floor(np.log2(np.where(x == 0, 1.0, np.abs(x))))
        e = np.where(np.exp2(e) > np.abs(x), e - 1, e)          # log2 may round up across a power of two
        e = np.where(np.exp2(e + 1) <= np.abs(x), e + 1, e)
        unit = np.exp2(np.maximum(e, -126) - 7)
        y = (np.ceil(x / unit) if up else np.floor(x / unit)) * unit
    return np.where(np.isfinite(x), y, np.nan)


def quantise64(x: np.ndarray, bits: int):
    """x [..., D] float64 -> codes [..., G*32] (uint8), step and lo [..., G] (float64)."""
    n, D = 2 ** bits - 1, x.shape[-1]
    G = (D + GROUP - 1) // GROUP
    code = np.zeros(x.shape[:-1] + (G * GROUP,), np.uint8)
    step, lo = np.zeros(x.shape[:-1] + (G,)), np.zeros(x.shape[:-1] + (G,))
    for g in range(G):
        y = x[..., g * GROUP:min(D, (g + 1) * GROUP)]
        bad = ~np.isfinite(y).all(-1)
        z = np.where(bad[..., None], 0.0, y)
        a = bf16_grid(z.min(-1), up=False)
        s = bf16_grid((z.max(-1) - a) / n, up=True)
        big = float(np.finfo(np.float32).max)
        bad |= (np.abs(a) > 3.4e38) | (z.max(-1) - a > big) | (s > 3.4e38)
        with np.errstate(all="ignore"):
            c = np.where(s[..., None] > 0, np.rint((z - a[..., None]) / np.where(s > 0, s, 1.0)[..., None]), 0.0)
        c = np.where(bad[..., None], 0.0, c)
        assert ((c >= 0) & (c <= n)).all()
        code[..., g * GROUP:g * GROUP + y.shape[-1]] = c.astype(np.uint8)
        step[..., g] = np.where(bad, np.nan, s)
        lo[..., g] = np.where(bad, np.nan, a)
    return code, step, lo


def quantise_exact(x: np.ndarray, bits: int):
    """One group x [<= 32] in rational arithmetic -> codes, step, lo (exact in float64)."""
    n = 2 ** bits - 1
    xs = [Fraction(float(v)) for v in x]

    def grid(v: Fraction, up: bool) -> Fraction:
        if v == 0:
            return v
        e = 0
        while Fraction(2) ** e > abs(v):
            e -= 1
        while Fraction(2) ** (e + 1) <= abs(v):
            e += 1
        unit = Fraction(2) ** (max(e, -126) - 7)
        q = v / unit
        fl = q.numerator // q.denominator
        return (fl if not up or q == fl else fl + 1) * unit

    lo = grid(min(xs), False)
    step = grid((max(xs) - lo) / n, True)
    codes = [0 if step == 0 else round((v - lo) / step) for v in xs]      # round(): ties to even
    return np.array(codes, np.uint8), float(step), float(lo)


def held(x: np.ndarray, bits: int) -> np.ndarray:
    """What the memory stands for after x [..., D] has been pushed."""
    code, step, lo = quantise64(x, bits)
    v = lo[..., None] + step[..., None] * code.reshape(step.shape + (GROUP,))
    return v.reshape(code.shape)[..., : x.shape[-1]]


def parse(rows: torch.Tensor, D: int, bits: int):
    """Rows [..., row bytes] of a QuantMemory as (k codes, k step, k lo), (v codes, v step, v lo), and the bf16 left
    over after the G groups' parameters (one group's zeros where G is odd)."""
    G = (D + GROUP - 1) // GROUP
    r = rows.cpu()
    n = 4 * G * bits
    par = r[..., 2 * n:2 * n + 8 * (G + G % 2)].contiguous().view(torch.bfloat16).double().numpy()
    par = par.reshape(par.shape[:-1] + (-1, 4))

    def codes(c):
        c = c.numpy()
        return c if bits == 8 else np.stack((c & 15, c >> 4), -1).reshape(c.shape[:-1] + (-1,))

    return ((codes(r[..., :n]), par[..., :G, 0], par[..., :G, 1]),
            (codes(r[..., n:2 * n]), par[..., :G, 2], par[..., :G, 3]), par[..., G:, :])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def attend64(q, k, v, u, vb, r, C, scale=None):
    """Relative attention in 64 bits.  q [B, L, H, D]; k, v [B, K, H, D], the last L keys the
    segment's own; r [n_rows, H, >= D] as the kernel gets it.  Returns out [B, L, H, D] and the
    largest scale (|q+u|.|k| + |q+v|.|r|) over the visible pairs, which bounds what relative errors
    of the products add to a score."""
    B, L, H, D = q.shape
    K = k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    delta = K - L + np.arange(L)[:, None] - np.arange(K)[None]
    row = np.clip(delta, 0, C)
    out, size = np.empty((B, L, H, D)), 0.0
    for b in range(B):
        for h in range(H):
            qu, qv = q[b, :, h] + u[h], q[b, :, h] + vb[h]
            s = (qu @ k[b, :, h].T + np.take_along_axis(qv @ r[:, h, :D].T, row, 1)) * scale
            big = (np.abs(qu) @ np.abs(k[b, :, h]).T
                   + np.take_along_axis(np.abs(qv) @ np.abs(r[:, h, :D]).T, row, 1)) * scale
            size = max(size, float(big[delta >= 0].max()))
            s = np.where(delta < 0, -np.inf, s)
            p = np.exp(s - s.max(-1, keepdims=True))
            out[b, :, h] = (p / p.sum(-1, keepdims=True)) @ v[b, :, h]
    return out, size


def decode_tolerance(ref, size, vmax, dtype):
    """|out - ref| allowed of the on-chip kernel, elementwise.  The output's own rounding is half a
    step, eps/2 of the value.  A product is off by at most 2^-16 of its size (the coarsest operand is
    held as two bf16 parts, 16 bits) plus the fp32 summation of up to 256 terms, 256 * 2^-24 = 2^-16:
    a score is off by ds <= 2^-15 size, and the softmax turns that into 2 ds max|v|.  The weights and
    their sums are held to 2^-16 likewise: 2 * 2^-16 max|v| more.  fp32: the operands keep 22 bits and
    the summation bound stays: ds <= 2^-16 size."""
    ds = (2.0 ** -16 if dtype == torch.float32 else 2.0 ** -15) * size
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + (2 * ds + 2.0 ** -15) * vmax


def segment_tolerance(q, k, v, u, vb, r, C, ref):
    """|out - ref| allowed of the tensor-core kernels over the memory read back, elementwise.  They round
    c(q+u), c(q+v), k', the position term, the weights and v' to 16 bits, each by at most bf16's 2^-8 of
    its value (uniform: a deviation of 2^-8 / sqrt(3)), independently (in fp16, a bound eight times too
    wide).  Errors of a score's products add in
    squares, s2 = scale^2 [2 sum (q+u)^2 k^2 + sum (q+v)^2 r^2 + ((q+v).r)^2]; a score's error moves the
    output by p_j (v_j - out), a weight's and a value's by p_j v_j each.  Six deviations of the sum, and
    half a step of the output's own rounding, 2^-8 of its value."""
    B, L, H, D = q.shape
    K = k.shape[1]
    delta = K - L + np.arange(L)[:, None] - np.arange(K)[None]
    row = np.clip(delta, 0, C)
    tol = np.empty((B, L, H, D))
    for b in range(B):
        for h in range(H):
            qu, qv, kk, vv, rr = q[b, :, h] + u[h], q[b, :, h] + vb[h], k[b, :, h], v[b, :, h], r[:, h, :D]
            bd = np.take_along_axis(qv @ rr.T, row, 1)
            s = (qu @ kk.T + bd) * D ** -0.5
            s2 = (2 * (qu ** 2) @ (kk ** 2).T + np.take_along_axis((qv ** 2) @ (rr ** 2).T, row, 1) + bd ** 2) / D
            s = np.where(delta < 0, -np.inf, s)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o = ref[b, :, h]
            w = p ** 2 * s2
            var = w @ vv ** 2 - 2 * (w @ vv) * o + w.sum(-1, keepdims=True) * o ** 2 + 2 * (p ** 2) @ vv ** 2
            tol[b, :, h] = 2.0 ** -8 * np.abs(o) + 6 * 2.0 ** -8 / np.sqrt(3) * np.sqrt(np.maximum(var, 0))
    return tol
