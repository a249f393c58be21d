"""GPU tests of 4-bit weights and the products with them, against the 64-bit restatement in paged_common.py."""
from __future__ import annotations

import math

import pytest
import torch

from paged_common import q4

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


def weights(k, n, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(k, n, generator=g) * (0.2 + torch.rand(n, generator=g)) + 0.3 * torch.randn(1, n, generator=g)).to(BF)


def rounded(held):
    return held.float().to(BF)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("k,n", [(1, 1), (64, 16), (100, 17), (129, 40), (410, 123), (512, 256)])
def test_what_the_codes_stand_for(txl, k, n, group):
    W = weights(k, n, seed=k)
    w = txl.QuantWeight.quantise(W.cuda(), group)
    *_, held = q4(W, group)
    # lo + step c fits fp32 to half a step of it, then one rounding to bf16: equal but where fp32's rounding decides a tie
    got = w.expand().cpu().double()
    assert ((got - held).abs() <= (2.0 ** -8) * held.abs() + 2.0 ** -23 * held.abs()).all()
    assert (got == rounded(held).double()).double().mean() > 0.999


@pytest.mark.parametrize("kind", ["constant", "zeros", "tiny", "huge", "steps", "nan", "inf"])
def test_groups_of_every_kind(txl, kind):
    k, n, group = 96, 20, 32
    W = weights(k, n, seed=5)
    if kind == "constant":
        W[:32] = W[:1]
    elif kind == "zeros":
        W.zero_()
    elif kind == "tiny":
        W = (W.float() * 2.0 ** -130).to(BF)
    elif kind == "huge":
        W = (W.float() / W.float().abs().max() * 1.6e38).to(BF)
    elif kind == "steps":                                       # 0 .. 15 exactly, and halves between (ties)
        W = (torch.arange(k * n).view(k, n) % 31 / 2).to(BF)
        W[::32], W[1::32] = 0.0, 15.0
    elif kind == "nan":
        W[40, 3] = math.nan
    else:
        W[70, 5], W[8, 6] = math.inf, -math.inf
    code, step, lo, held = q4(W, group)
    w = txl.QuantWeight.quantise(W.cuda(), group)
    got = w.expand().cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(held))
    ok = ~torch.isnan(held)
    assert ((got - held).abs()[ok] <= (2.0 ** -8 + 2.0 ** -23) * held.abs()[ok] + 2.0 ** -133).all()
    if kind in ("nan", "inf"):
        y = txl.linear_q4(torch.ones(2, k, dtype=BF, device="cuda"), w).cpu()
        assert torch.equal(torch.isnan(y), torch.isnan(held).any(0).expand(2, n))


def check_product(txl, m, k, n, group, x=None, w=None, W=None, Y=None, **kw):
    W = weights(k, n, seed=k + n) if W is None else W
    w = txl.QuantWeight.quantise(W.cuda(), group) if w is None else w
    if x is None:
        x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(BF).cuda()
    y = txl.linear_q4(x, w, Y, **kw)
    _, step, lo, held = q4(W, group)
    xd = x.cpu().double()
    want = xd @ held
    # fp32 sums of products with 128 + c, and of the correction: 2^-24 of the terms' size for each of k / 16 + 8 sums
    each = torch.repeat_interleave(step.abs() * 143 + lo.abs() + 128 * step, group, 0)[:k]
    size = xd.abs() @ each
    tol = 2.0 ** -8 * want.abs() + size * (k / 16 + 16) * 2.0 ** -24
    if m > 128 and x.data_ptr() % 16 == 0 and x.stride(0) % 8 == 0:        # (the weights are rounded to bf16 first)
        tol += 2.0 ** -8 * (xd.abs() @ held.abs())
    err = (y.cpu().double() - want).abs()
    assert (err <= tol).all(), float((err / tol).max())
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 2, 5, 8, 9, 16, 17, 40, 64, 128, 129, 200])
def test_rows(txl, m, group):
    check_product(txl, m, 256, 144, group)


@pytest.mark.parametrize("k,n", [(1, 1), (31, 5), (63, 16), (65, 17), (410, 1230), (1000, 33), (4096, 64), (64, 4096)])
@pytest.mark.parametrize("m", [1, 7, 13])
def test_shapes(txl, m, k, n):
    check_product(txl, m, k, n, 64)


@pytest.mark.parametrize("m", [3, 150])
def test_layouts(txl, m):
    """Rows of x and y that start anywhere; nothing is written beside y."""
    k, n = 200, 90
    g = torch.Generator().manual_seed(1)
    for off, pad in ((0, 0), (8, 8), (1, 3), (0, 1)):
        store = torch.full((m, k + off + pad), math.nan, dtype=BF, device="cuda")
        x = store[:, off:off + k]
        x.copy_(torch.randn(m, k, generator=g))
        ys = torch.full((m, n + 5), 7.0, dtype=BF, device="cuda")
        check_product(txl, m, k, n, 64, x=x, Y=ys[:, 2:2 + n])
        assert (ys[:, :2] == 7).all() and (ys[:, 2 + n:] == 7).all()


def test_a_weight_larger_than_32_bit_offsets_of_its_entries(txl):
    """n k = 2.2e9 entries: columns at the far end."""
    k, n = 1024, 2 ** 21
    W = torch.zeros(k, n, dtype=BF, device="cuda")
    part = weights(k, 32, seed=2)
    W[:, -32:] = part.cuda()
    w = txl.QuantWeight.quantise(W, 64)
    del W
    x = torch.randn(3, k, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    y = txl.linear_q4(x, w)
    alone = txl.linear_q4(x, txl.QuantWeight.quantise(part.cuda(), 64))
    assert (y[:, :-32] == 0).all() and torch.equal(y[:, -32:], alone)


def test_refusals_of_the_binding(txl):
    W = weights(64, 32).cuda()
    w = txl.QuantWeight.quantise(W)
    x = torch.zeros(150, 64, dtype=BF, device="cuda")
    for args, kw, error in (((x[:, :32], w), {}, ValueError), ((x.float(), w), {}, TypeError), ((x.t(), w), {}, ValueError),
                            ((x.cpu(), w), {}, ValueError), ((x, w, torch.zeros(150, 31, dtype=BF, device="cuda")), {}, ValueError),
                            ((x, w), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), txl.TxlError),
                            ((x, w), dict(err_flag=torch.zeros(1, device="cuda")), ValueError)):
        with pytest.raises(error):
            txl.linear_q4(*args, **kw)
    for bad in (dict(group=16), dict(W=W.float()), dict(W=W.cpu()), dict(W=W.t())):
        with pytest.raises((ValueError, TypeError)):
            txl.QuantWeight.quantise(**{**dict(W=W, group=64), **bad})
    with pytest.raises(ValueError):
        txl.QuantWeight(w.data[:-1], 64, 32, 64)
    with pytest.raises(ValueError):
        w.expand(torch.zeros(64, 33, dtype=BF, device="cuda"))


def test_not_finite_x(txl):
    x = torch.ones(3, 128, dtype=BF, device="cuda")
    x[1, 5] = math.inf
    y = txl.linear_q4(x, txl.QuantWeight.quantise(weights(128, 24).cuda()))
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[2]).all() and not torch.isfinite(y[1]).any()


def test_captured_on_another_stream_with_a_workspace(txl):
    W = weights(128, 64)
    w = txl.QuantWeight.quantise(W.cuda())
    x = torch.zeros(150, 128, dtype=BF, device="cuda")
    y = torch.zeros(150, 64, dtype=BF, device="cuda")
    ws = torch.empty(txl.linear_q4_workspace_size(150, w), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    txl.linear_q4(x, w, y, workspace=ws, stream=side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        txl.linear_q4(x, w, y, workspace=ws)
        txl.linear_q4(x[:5], w, y[:5])
    x.copy_(torch.randn(150, 128, generator=torch.Generator().manual_seed(3)))
    g.replay()
    torch.cuda.synchronize()
    few, all_ = y[:5].clone(), y[5:].clone()
    assert torch.equal(few, check_product(txl, 5, 128, 64, 64, x=x[:5], W=W))
    assert torch.equal(all_, check_product(txl, 150, 128, 64, 64, x=x, W=W)[5:])


def test_the_readmes_token_step(txl):
    """The README's step runs over many tokens, and its memory stays within its bound."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md"), encoding="utf-8").read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "def token_step" in c]
    assert len(code) == 1
    scope = {}
    exec(code[0], scope)
    B, H, D, d_model, keep = 3, 2, 32, 64, 40
    g = torch.Generator().manual_seed(0)
    w_qkv, w_o = (txl.QuantWeight.quantise(torch.randn(*s, generator=g).mul(0.1).to(BF).cuda()) for s in ((d_model, 3 * H * D), (H * D, d_model)))
    u, vb = torch.zeros(H, D, device="cuda"), torch.zeros(H, D, device="cuda")
    r = torch.randn(200, H, D, generator=g).to(BF).cuda()
    mem = txl.PagedMemory.empty(B, 30, 16, H, D)
    for t in range(150):
        h = torch.randn(B, d_model, generator=g).to(BF).cuda()
        y = scope["token_step"](h, mem, w_qkv, w_o, u, vb, r, 199, keep)
        assert y.shape == h.shape
    mem.check()
    assert torch.isfinite(y.float()).all() and mem.next_pos.tolist() == [150] * B and max(mem.reserved) < keep + 64
    assert mem.length.tolist() == mem.reserved


def test_a_generated_tokens_layer_step(txl):
    """4-bit projections around the paged attention, against the same in 64 bits from the layer's rounded parts."""
    B, H, D, d_model, n_rows = 3, 4, 32, 128, 80
    g = torch.Generator().manual_seed(0)
    Wqkv, Wo = (torch.randn(*s, generator=g).mul(0.1).to(BF) for s in ((d_model, 3 * H * D), (H * D, d_model)))
    w_in, w_out = txl.QuantWeight.quantise(Wqkv.cuda()), txl.QuantWeight.quantise(Wo.cuda())
    from paged_common import Pages, attend
    ref = Pages(B, H, D, [50, 3, 0], 16, BF, room=4)
    mem = ref.to_gpu(txl)
    u, vb = torch.zeros(H, D), torch.zeros(H, D)
    r = torch.randn(n_rows, H, D, generator=g).to(BF)
    for t in range(4):
        h = torch.randn(B, d_model, generator=g).to(BF).cuda()
        q, k, v = txl.linear_q4(h, w_in).view(B, 1, 3, H, D).unbind(2)
        a = torch.empty(B, 1, H, D, dtype=BF, device="cuda")
        txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), n_rows, n_rows - 1, a, accumulate=True)
        y = txl.linear_q4(a.view(B, H * D), w_out)
        ref.push(k.cpu(), v.cpu())
        want, tol, *_ = attend(ref, q.cpu(), u, vb, r, n_rows - 1)
        assert ((a.cpu().double() - want).abs() <= tol).all()
        assert torch.equal(y, check_product(txl, B, H * D, d_model, 64, x=a.view(B, H * D), W=Wo))
    mem.check()
