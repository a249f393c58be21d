"""GPU tests of products with 4-bit weights at the ends of the range: a finite product is finite, whatever its parts are."""
from __future__ import annotations

import math

import pytest
import torch

from paged_common import q4
from test_gpu_linear_q4 import weights

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


def check(txl, x, W, group):
    """Y where it fits bf16, against 64 bits; the tolerance counts fp32 sums of the kernel's terms and one rounding."""
    m, k = x.shape
    y = txl.linear_q4(x, txl.QuantWeight.quantise(W.cuda(), group)).cpu().double()
    _, step, lo, held = q4(W, group)
    xd = x.cpu().double()
    want = xd @ held
    each = torch.repeat_interleave(step.abs() * 143 + lo.abs() + 128 * step, group, 0)[:k]
    tol = 2.0 ** -8 * want.abs() + (xd.abs() @ each) * (k / 16 + 16) * 2.0 ** -24
    fits = want.abs() + tol < torch.finfo(BF).max
    assert fits.double().mean() > 0.5
    err = (y - want).abs()
    assert (err[fits] <= tol[fits]).all(), (int((~torch.isfinite(y[fits])).sum()), float((err / tol)[fits].max()))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m", [1, 5, 13, 40])
@pytest.mark.parametrize("size", [2.0 ** 118, 1e37, 1.6e38, 3e38])
def test_large_weights(txl, m, group, size):
    """Steps up to 4e37: 128 steps are beyond fp32, and so are sums that cancel against the minimum's."""
    k, n = 300, 70
    W = weights(k, n, seed=group)
    W = (W.double() / W.double().abs().max() * size).to(BF)
    g = torch.Generator().manual_seed(m)
    check(txl, (torch.randn(m, k, generator=g) * 2.0 ** -7).to(BF).cuda(), W, group)


@pytest.mark.parametrize("m", [3, 16, 150])
def test_large_x(txl, m):
    """x up to 1e38 against weights of 1e-3; rows that start anywhere, so that 150 of them go through the codes too."""
    k, n = 260, 50
    g = torch.Generator().manual_seed(m)
    W = (torch.randn(k, n, generator=g) * 1e-3).to(BF)
    store = torch.empty(m, k + 1, dtype=BF, device="cuda")
    x = store[:, 1:]
    x.copy_((torch.randn(m, k, generator=g) * 3e37).to(BF))
    check(txl, x, W, 64)


def test_one_large_column_among_others(txl):
    """What is computed again leaves the columns and rows beside it as they are without it."""
    k, n, m = 512, 96, 6
    W = weights(k, n, seed=9)
    x = (torch.randn(m, k, generator=torch.Generator().manual_seed(2)) * 2.0 ** -7).to(BF).cuda()
    plain = txl.linear_q4(x, txl.QuantWeight.quantise(W.cuda()))
    big = W.clone()
    big[:, 37] = (W[:, 37].float() * 2.0 ** 125).to(BF)
    y = txl.linear_q4(x, txl.QuantWeight.quantise(big.cuda()))
    others = [c for c in range(n) if c != 37]
    assert torch.equal(y[:, others], plain[:, others])
    check(txl, x, big, 64)


def test_not_a_number_stays_in_its_row_and_column(txl):
    """An infinite x, a NaN among the weights: what the product of them with finite numbers is, and nothing beside it."""
    k, n, m = 200, 40, 4
    W = weights(k, n, seed=4)
    W[150, 11] = math.nan
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(5)).to(BF)
    x[2, 77] = -math.inf
    y = txl.linear_q4(x.cuda(), txl.QuantWeight.quantise(W.cuda())).cpu().double()
    *_, held = q4(W, 64)
    want = x.double() @ held
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    inf = torch.isinf(want)
    assert bool(inf[2].any()) and torch.equal(y[inf], want[inf])


def test_no_rows(txl):
    """A step with no sequence in it."""
    w = txl.QuantWeight.quantise(weights(64, 24).cuda())
    assert txl.linear_q4(torch.empty(0, 64, dtype=BF, device="cuda"), w).shape == (0, 24)
    y = torch.empty(0, 24, dtype=BF, device="cuda")
    assert txl.linear_q4(torch.empty(0, 64, dtype=BF, device="cuda"), w, y) is y
