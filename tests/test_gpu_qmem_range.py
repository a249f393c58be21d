"""GPU tests of txl_rel_attn_qmem on values of unlike size: infinities and NaN, elements far above or
below the rest of their head or group of channels.  References in 64 bits over what the memory stands for."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from qmem_common import attend64, decode_tolerance, f64, quantise64
from test_gpu_qmem_attn import Call

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


def attend(q, k, v, u, vb, r, C):
    """out [B, L, H, D] by the formula, and s2 as segment_tolerance counts it: out_i is a sum over the keys
    that query i sees, so that what it does not see may be anything.  Also the variance var of an output
    whose operands, position terms and weights each deviate by 1 of their value, independently (values that
    are not finite apart)."""
    B, L, H, D = q.shape
    K = k.shape[1]
    delta = K - L + np.arange(L)[:, None] - np.arange(K)[None]
    seen, row = delta >= 0, np.clip(delta, 0, C)
    out, var = np.empty((B, L, H, D)), np.empty((B, L, H, D))

    def finite(x):
        return np.where(np.isfinite(x), x, 0.0)

    with np.errstate(all="ignore"):
        for b in range(B):
            for h in range(H):
                qu, qv, kk, vv, rr = q[b, :, h] + u[h], q[b, :, h] + vb[h], k[b, :, h], v[b, :, h], r[:, h, :D]
                s = (qu @ kk.T + np.take_along_axis(qv @ rr.T, row, 1)) * D ** -0.5
                s = np.where(seen, s, -np.inf)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o = p @ finite(vv)
                for j, d in np.argwhere(~np.isfinite(vv)):
                    o[:, d] = np.where(seen[:, j], o[:, d] + p[:, j] * vv[j, d], o[:, d])
                out[b, :, h] = o
                p, o, vv = finite(p), finite(o), finite(vv)
                qu, qv, kk, rr = finite(qu), finite(qv), finite(kk), finite(rr)
                bd = np.take_along_axis(qv @ rr.T, row, 1)
                s2 = (2 * (qu ** 2) @ (kk ** 2).T + np.take_along_axis((qv ** 2) @ (rr ** 2).T, row, 1) + bd ** 2) / D
                w = p ** 2 * s2
                var[b, :, h] = w @ vv ** 2 - 2 * (w @ vv) * o + w.sum(-1, keepdims=True) * o ** 2 + 2 * (p ** 2) @ vv ** 2
    return out, np.maximum(var, 0)


def check(call, rows=slice(None)):
    """NaN and infinities where the formula has them; elsewhere at most six deviations of operands, position
    terms and weights rounded to bf16 (2^-8 of the value, uniform: 2^-8 / sqrt(3)) and the output's own
    rounding, half a step, 2^-8 of its value: what any of the segment kernels keeps."""
    ref, var = attend(*call.operands_as_given(), call.C)
    ref, var, out = ref[:, rows], var[:, rows], f64(call.out)[:, rows]
    assert np.array_equal(np.isnan(out), np.isnan(ref)), np.argwhere(np.isnan(out) != np.isnan(ref))[:5]
    inf = np.isinf(ref)
    assert np.array_equal(np.isinf(out), inf) and np.array_equal(out[inf], ref[inf])
    ok = np.isfinite(ref)
    err = np.abs(np.where(ok, out, 0) - np.where(ok, ref, 0))
    tol = 2.0 ** -8 * np.abs(np.where(ok, ref, 0)) + 6 * 2.0 ** -8 / np.sqrt(3) * np.sqrt(var)
    assert (err <= tol)[ok].all(), float((err / np.maximum(tol, 1e-300))[ok].max())


class Ranged(Call):
    def operands_as_given(self):
        """As operands(), with r's channels as they are (its padding is not read)."""
        q, k, v, u, vb, _ = self.operands()
        return q, k, v, u, vb, f64(self.r[..., :self.dims[3]])

    def push_again(self, txl, wp):
        M = self.mem.M
        self.mem.restore((wp - self.kh.shape[1]) % M, 0)
        txl.qmem_push(self.mem, self.kh.cuda(), self.vh.cuda())

    def go(self, txl):
        self.run(txl)
        torch.cuda.synchronize()


def segment(txl, D, L=40, M=200, bits=8, dtype="bf16", C=1000, **kw):
    return Ranged(txl, 2, 2, D, L, M, M, 9, C, bits, dtype, **kw)


WHERE = ["q", "first own key", "first own value", "position row", "clamped position row", "memory key", "memory value"]


@pytest.mark.parametrize("value", [INF, -INF, NAN], ids=str)
@pytest.mark.parametrize("D", [64, 96])
@pytest.mark.parametrize("where", WHERE)
def test_segment_values_that_are_not_finite(txl, where, D, value):
    """One element that is not finite and that every query sees (of q: its own row) does to a bf16 segment
    what the formula says, and nothing to the other heads and entries."""
    call = segment(txl, D, C=100 if where.startswith("clamped") else 1000)
    if where == "q":
        call.q[1, 20, 0, 3] = value
    elif where == "first own key":
        call.k[1, 0, 0, 3] = value
    elif where == "first own value":
        call.v[1, 0, 0, 3] = value
    elif where == "position row":
        call.r[3, 1, 5] = value
    elif where == "clamped position row":
        call.r[100, 1, 5] = value
    else:
        (call.kh if where == "memory key" else call.vh)[1, 77, 0, 3] = value
        call.push_again(txl, 9)
    call.go(txl)
    check(call)


@pytest.mark.parametrize("D", [64, 96])
@pytest.mark.parametrize("where", ["memory", "own"])
def test_segment_large_key_in_a_channel_without_query(txl, where, D):
    """A key of 2^17 in a channel where the queries are 0: scores of ordinary size."""
    call = segment(txl, D)
    call.q[..., 40], call.u[:, 40], call.vb[:, 40] = 0, 0, 0
    if where == "own":
        call.k[0, 0, 0, 40] = 2.0 ** 17
    else:
        call.kh[0, 33, 0, 40] = 2.0 ** 17
        call.push_again(txl, 9)
    call.go(txl)
    check(call)


@pytest.mark.parametrize("D", [64, 96])
def test_segment_large_position_in_a_channel_without_query(txl, D):
    call = segment(txl, D)
    call.q[..., 40], call.u[:, 40], call.vb[:, 40] = 0, 0, 0
    call.r[7, 0, 40] = 2.0 ** 17
    call.go(txl)
    check(call)


@pytest.mark.parametrize("D", [64, 96])
@pytest.mark.parametrize("what", ["k", "v"])
def test_segment_large_values_that_no_query_sees_yet(txl, what, D):
    """Own keys or values of 2^40 behind position 30: the queries before them do not see them."""
    call = segment(txl, D)
    getattr(call, what)[:, 30:] *= 2.0 ** 40
    call.go(txl)
    check(call, slice(0, 30))


@pytest.mark.parametrize("D", [64, 96])
@pytest.mark.parametrize("octaves,score", [(34, -40.0), (23, -16.0)])
def test_segment_large_value_with_little_weight(txl, D, octaves, score):
    """A position whose value is 2^octaves times the others' and whose weight is about e^score of theirs."""
    call = segment(txl, D)
    q = call.q[:, :1, :].float() + call.u
    call.q.copy_(call.q[:, :1].clone().expand_as(call.q))
    t = score * D ** 0.5 / (q ** 2).sum(-1, keepdim=True)
    call.kh[:, 50] = (q * t)[:, 0].cpu().to(call.dtype)
    call.vh[:, 50] *= 2.0 ** octaves
    call.push_again(txl, 9)
    call.go(txl)
    check(call)


@pytest.mark.parametrize("D", [64, 96])
def test_segment_value_channels_of_unlike_size(txl, D):
    """Channels 32 .. 63 of the values 2^40 times smaller than the others."""
    call = segment(txl, D)
    call.vh[..., 32:64] *= 2.0 ** -40
    call.v[..., 32:64] *= 2.0 ** -40
    call.push_again(txl, 9)
    call.go(txl)
    check(call)


@pytest.mark.parametrize("B,H,L,D", [(40, 8, 20, 64), (30, 4, 300, 41), (3, 2, 200, 96)])
def test_segment_heads_of_either_kind(txl, B, H, L, D):
    """Heads with a large key, large values or an infinity between ordinary ones, more of them than multiprocessors."""
    call = Ranged(txl, B, H, D, L, 60, 60, 9, 1000, 8, "bf16")
    call.q[..., 20], call.u[:, 20], call.vb[:, 20] = 0, 0, 0
    g = torch.Generator().manual_seed(B)
    kind = torch.randint(0, 6, (B, H), generator=g)
    for b, h in torch.argwhere(kind < 3).tolist():
        if kind[b, h] == 0:
            call.kh[b, 33, h, 20] = 2.0 ** 17
        elif kind[b, h] == 1:
            call.v[b, L // 2, h] *= 2.0 ** 20
        else:
            call.v[b, 0, h, 3] = INF
    call.push_again(txl, 9)
    call.go(txl)
    check(call)


@pytest.mark.parametrize("D", [41, 64, 96])
def test_segment_heads_of_either_kind_without_a_loadable_table(txl, D):
    """The same where r's rows do not start on 16-byte boundaries."""
    call = segment(txl, D)
    flat = torch.empty(call.r.numel() + 1, dtype=torch.bfloat16, device="cuda")
    flat[1:].copy_(call.r.reshape(-1))
    call.r = flat[1:].view(call.r.shape)
    call.v[0, 5, 1] *= 2.0 ** 20
    call.go(txl)
    check(call)


@pytest.mark.parametrize("L", [50, 300])
@pytest.mark.parametrize("D", [24, 64, 96])
@pytest.mark.parametrize("key,value", [(NAN, INF), (INF, NAN), (-INF, -INF), (3e38, -3e38)], ids=str)
def test_segment_sees_no_later_key(txl, key, value, D, L):
    """Keys and values of the segment that are NaN, infinite or at the end of bf16's range reach the queries from
    their position on, and no query before it (positions from 3/5 and 4/5 of the segment on)."""
    call = segment(txl, D, L=L, hs=D + 1, shift=1)
    call.v[:, 3 * L // 5:] = value
    call.v[0, 7 * L // 10, 0] = -value
    call.k[:, 4 * L // 5:] = key
    call.go(txl)
    # (scores past fp32's range are not compared)
    check(call, slice(0, 4 * L // 5) if key == 3e38 else slice(None))


@pytest.mark.parametrize("D", [64, 96])
def test_segment_values_that_are_not_finite_apart_in_the_segment(txl, D):
    """One element each, in different tiles, channels and heads."""
    call = segment(txl, D, L=400)
    call.v[0, 100, 0, 3], call.v[0, 300, 0, 3], call.v[0, 130, 0, D - 1] = INF, -INF, NAN
    call.v[1, 399, 1, 0] = INF
    call.v[0, 50, 1], call.v[0, 390, 1, 7] = 3e38, INF
    call.k[1, 200, 0, 5] = NAN
    call.go(txl)
    check(call)


def groups_within(call, bound):
    """The error's norm over each group of 32 channels against the result's."""
    ref, _ = attend(*call.operands_as_given(), call.C)
    out = f64(call.out)
    for d in range(0, ref.shape[-1], 32):
        e, n = np.linalg.norm((out - ref)[..., d:d + 32]), np.linalg.norm(ref[..., d:d + 32])
        assert e <= bound * n, (d, e / n)


# fp32: the bound of test_fp32_keeps_its_bits.  bf16: the output's rounding, at most 2^-8 / sqrt(3) of its value,
# and sums of 15 bits, whose 2^-15 is far below the rest of 2^-8.
GROUP_BOUND = {"f32": 2.0 ** -19, "bf16": 2.0 ** -8}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("octaves", [10, 16, 30])
@pytest.mark.parametrize("L", [1, 4, 16])
@pytest.mark.parametrize("bits", [4, 8])
def test_value_groups_of_unlike_size(txl, bits, L, octaves, dtype):
    """A group of 32 channels whose values are 2^octaves times smaller than the other's keeps its own bits."""
    for D in (64, 128):
        call = Ranged(txl, 2, 2, D, L, 900, 900, 9, 500, bits, dtype)
        for x in (call.vh, call.v):
            x[..., 32:64] *= 2.0 ** -octaves
        call.push_again(txl, 9)
        call.go(txl)
        groups_within(call, GROUP_BOUND[dtype])


@pytest.mark.parametrize("L", [1, 4, 16])
@pytest.mark.parametrize("bits", [4, 8])
def test_one_position_of_large_values_and_little_weight(txl, bits, L):
    """Its value is 2^16 times the others' and its weight some 2^-16: the others keep their bits."""
    call = Ranged(txl, 1, 2, 64, L, 4000, 4000, 9, 500, bits, "f32")
    q = call.q[:, :1].float() + call.u
    call.q.copy_(call.q[:, :1].clone().expand_as(call.q))
    t = -11.0 * 8 / (q ** 2).sum(-1, keepdim=True)
    call.kh[:, 50] = (q * t)[:, 0].cpu()
    call.vh[:, 50] *= 2.0 ** 16
    call.push_again(txl, 9)
    call.go(txl)
    groups_within(call, GROUP_BOUND["f32"])


@pytest.mark.parametrize("L", [1, 4, 16])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("octaves", [10, 20])
def test_query_groups_of_unlike_size(txl, octaves, bits, L):
    """Queries of a group of 32 channels 2^octaves times smaller than the other's, keys as much larger."""
    call = Ranged(txl, 2, 2, 64, L, 900, 900, 9, 500, bits, "f32")
    for x in (call.q, call.u, call.vb):
        x[..., 32:] *= 2.0 ** -octaves
    for x in (call.kh, call.k):
        x[..., 32:] *= 2.0 ** octaves
    call.push_again(txl, 9)
    call.go(txl)
    groups_within(call, GROUP_BOUND["f32"])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D", [41, 64, 96, 128])
def test_segments_keep_fp16s_bits(txl, D, bits):
    """Ordinary values: operands, position terms and weights deviate by fp16's 2^-11 / sqrt(3) of their value at
    most, twice that with the argument of the exponential, and the output by its own rounding, 2^-8 / sqrt(3) at
    most.  In the norm over all outputs the two add in squares.  (Rounding the operands to bf16 comes to
    four times what fp16 is allowed here.)"""
    call = Ranged(txl, 2, 3, D, 100, 700, 700, 9, 500, bits, "bf16")
    call.go(txl)
    ref, var = attend(*call.operands_as_given(), call.C)
    most = np.sqrt(((2.0 ** -8 / np.sqrt(3) * ref) ** 2 + (2 * 2.0 ** -11 / np.sqrt(3)) ** 2 * var).sum())
    assert np.linalg.norm(f64(call.out) - ref) <= most


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("c", [(2, 3, 64, 100, 1500), (1, 2, 128, 33, 700), (2, 1, 41, 17, 3000)])
def test_fp32_segments_keep_their_bits(txl, c, bits):
    """Products and sums in fp32, sums of at most 64 terms joined: each off by less than 2^-24 times sqrt(64) of
    its size; the exponential by 2^-22: a term of the output by less than 2^-20, and a factor of two for the sums."""
    B, H, D, L, M = c
    call = Ranged(txl, B, H, D, L, M, M, 5, 1000, bits, "f32")
    call.go(txl)
    ref, _ = attend(*call.operands_as_given(), call.C)
    assert np.linalg.norm(f64(call.out) - ref) <= 2.0 ** -19 * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [2, 4, 9, 16])
@pytest.mark.parametrize("key,value", [(NAN, INF), (INF, NAN), (3e38, -3e38)], ids=str)
def test_few_queries_see_no_later_key(txl, key, value, L, dtype):
    """Up to 16 queries: what an own key or value holds reaches the queries from its position on."""
    for M in (0, 100, 1500):
        call = Ranged(txl, 2, 2, 64, L, M, M, 7 if M else 0, 1000, 4, dtype)
        n = (L + 1) // 2
        call.v[:, n:] = value
        call.k[:, n:] = key
        call.go(txl)
        check(call, slice(0, n) if key == 3e38 else slice(None))


@pytest.mark.parametrize("value", [INF, -INF, NAN], ids=str)
@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L,M", [(1, 1200), (3, 200), (16, 600), (1, 150)])
def test_few_queries_values_that_are_not_finite(txl, L, M, dtype, where, value):
    """As test_segment_values_that_are_not_finite for up to 16 queries, with the position terms in a kernel of their own
    and in the attention kernel."""
    call = Ranged(txl, 2, 2, 64, L, M, M, 9, 100 if where.startswith("clamped") else 2000, 4, dtype)
    if where == "q":
        call.q[1, L // 2, 0, 3] = value
    elif where == "first own key":
        call.k[1, 0, 0, 3] = value
    elif where == "first own value":
        call.v[1, 0, 0, 3] = value
    elif where == "position row":
        call.r[3, 1, 5] = value
    elif where == "clamped position row":
        call.r[100, 1, 5] = value
    else:
        (call.kh if where == "memory key" else call.vh)[1, 77, 0, 3] = value
        call.push_again(txl, 9)
    call.go(txl)
    check(call)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("octaves", [12, 40])
@pytest.mark.parametrize("L", [1, 4, 16])
@pytest.mark.parametrize("bits", [4, 8])
def test_one_position_with_a_step_far_above_the_others(txl, bits, L, octaves, dtype):
    """One element of 2^octaves makes its group's step there that large: the group's sums are off by no more than
    2^-12 (fp32: 2^-14) of the weighted steps.  (bf16: one product is aligned to the position's, whose code counts as
    1024 at most, and drops what lies 24 bits below: 2^-14 of its weighted step.  fp32: the centred codes of at most 128
    cancel against lo + 128 step, 2^-17, in a sum of some ten terms per lane.  Weights 2^-33 below the largest are
    lost: 900 of them times 255 come to 2^-15.)"""
    call = Ranged(txl, 2, 2, 64, L, 900, 900, 9, 500, bits, dtype)
    call.vh[:, 50, :, 5] = 2.0 ** octaves
    call.push_again(txl, 9)
    call.go(txl)
    q, k, v, u, vb, r = call.operands_as_given()
    step = quantise64(f64(call.vh), bits)[1].repeat(32, -1)
    weighted, _ = attend(q, k, np.concatenate((step, np.zeros_like(v[:, -L:])), 1), u, vb, r, call.C)
    ref, size = attend64(q, k, v, u, vb, r, call.C)
    rest = np.delete(v, 50, 1)
    tol = decode_tolerance(ref, size, np.abs(rest).max(), call.dtype)
    # (what an error of the scores makes of that position's value is its weight times that error times the value)
    ds = (2.0 ** -16 if dtype == "f32" else 2.0 ** -15) * size
    at = np.abs(v[:, 50:51])
    p = weighted / np.maximum(step[:, 50:51], 1e-300)
    tol = tol + 4 * ds * np.minimum(p, 1.0) * at + 2.0 ** (-14 if dtype == "f32" else -12) * weighted
    err = np.abs(f64(call.out) - ref)
    assert (err <= tol).all(), float((err / tol).max())
