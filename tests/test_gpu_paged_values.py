"""GPU tests of the paged memory's attention where keys, values and positions' rows hold what is not finite, over long
memories and wide tables, against the 64-bit restatement in paged_common.py."""
from __future__ import annotations

import math

import pytest
import torch

from paged_common import Pages, attend
from test_gpu_paged import new

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


def check_against(mem, ref, out, before, q, u, vb, r, C, counts=None):
    """Outputs, and what every slot's weight gained, against the restatement (`ref` after the push)."""
    want, tol, got, got_tol = attend(ref, q.cpu(), u, vb, r, C, counts)
    live = ~torch.isnan(want)
    assert ((out.cpu().double() - want).abs() <= tol)[live].all()
    if before is not None:
        w = mem.weight.cpu().double() - before.double()
        # the sum over heads and queries is added once, in fp32: half a step of the old and of the new weight
        assert ((w - got).abs() <= got_tol + 2.0 ** -23 * (before.double() + got) + 1e-30).all()
    mem.check()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 3, 12])
@pytest.mark.parametrize("long", [False, True])
def test_weights_beside_a_key_that_scores_minus_infinity(txl, dtype, T, long):
    """A seen key with an infinite component scores -inf: it weighs nothing, and the others' weights are finite."""
    ref = Pages(2, 2, 64, [9000, 500] if long else [37, 90], 64, dtype, room=T)
    q, k, v, u, vb, r = new(2, T, 2, 64, dtype, 4, 50)
    q[..., 5] = 2.0 + 0.01 * torch.arange(T, device="cuda")[None, :, None]      # (and u is no less than -1.5)
    u[:, 5] = u[:, 5].clamp(min=-1.0)
    out_of = [ref.at(0, 20), ref.at(1, 31)]
    for p, row in out_of:
        ref.k[p, :, row, 5] = -math.inf
        ref.v[p, 0, row, 7] = math.inf                        # (nor does its value count)
    mem = ref.to_gpu(txl)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 50, 49, out, accumulate=True)
    ref.push(k.cpu(), v.cpu())
    before = ref.weight.clone()
    for p, row in out_of:
        ref.pos[p, row] = 1 << 30                              # the same as a key that no query sees
        ref.k[p, :, row, 5] = ref.v[p, 0, row, 7] = 0.0
    check_against(mem, ref, out, before, q, u, vb, r, 49)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 3, 12])
@pytest.mark.parametrize("long", [False, True])
def test_a_distance_whose_row_is_minus_infinity(txl, dtype, T, long):
    """A row of r with an infinite component scores -inf: keys at that distance weigh nothing."""
    ref = Pages(2, 2, 64, [9000, 500] if long else [37, 90], 64, dtype, room=T)
    q, k, v, u, vb, r = new(2, T, 2, 64, dtype, 4, 50)
    q[..., 5] = 2.0 + 0.01 * torch.arange(T, device="cuda")[None, :, None]
    vb[:, 5] = vb[:, 5].clamp(min=-1.0)
    cut = r.clone()
    cut[17, :, 5] = -math.inf
    mem = ref.to_gpu(txl)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), cut.cuda(), 50, 49, out, accumulate=True)
    # the restatement takes a query at a time: one key of each sequence is at that distance
    ref.push(k.cpu(), v.cpu())
    before, pos = ref.weight.clone(), ref.pos.clone()
    want, gain, gain_tol = [], 0.0, 0.0
    nxt = ref.next_pos.clone()
    for i in range(T):
        at = nxt - T + i
        ref.pos.copy_(pos)
        for b in range(2):
            p, row = ref.index(b, int(ref.length[b]))
            hit = pos[p, row] == at[b] - 17
            ref.pos[p[hit], row[hit]] = 1 << 30
        ref.next_pos.copy_(at + 1)
        o, tol, got, got_tol = attend(ref, q[:, i:i + 1].cpu(), u, vb, r, 49)
        want.append((o, tol))
        # (a sum over T queries where the restatement sums one: T times the bound of its additions)
        gain, gain_tol = gain + got, gain_tol + got_tol + got * 2 * T * 2.0 ** -23
    o = out.cpu().double()
    for i, (y, tol) in enumerate(want):
        assert ((o[:, i:i + 1] - y).abs() <= tol).all(), i
    w = mem.weight.cpu().double() - before.double()
    assert ((w - gain).abs() <= gain_tol + 2.0 ** -23 * (before.double() + gain) + 1e-30).all()
    mem.check()
