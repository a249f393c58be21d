"""GPU tests of the paged memory's page table on the host and the device: no sequences, tables with gaps, tables wider than what
sequences hold, and long memories, against the 64-bit restatement in paged_common.py."""
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


# ------------------------------------------------------------------------------------ nothing to do
@pytest.mark.parametrize("dtype", [BF, F])
def test_a_memory_of_no_sequences(txl, dtype):
    """Every call of a batch that has become empty does nothing."""
    mem = txl.PagedMemory.empty(0, 4, 16, 2, 64, dtype=dtype)
    q, k, v, u, vb, r = new(0, 3, 2, 64, dtype, 1, 10)
    mem.reserve(3)
    txl.paged_push(mem, k, v)
    out = torch.empty_like(q)
    assert txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 10, 9, out, accumulate=True) is out
    txl.paged_evict(mem, 2)
    mem.trim()
    mem.check()
    assert mem.reserved == [] and mem.free_pages == 4


# ------------------------------------------------------------------------------------ what is not read
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_queries_past_a_sequences_count_are_not_read(txl, dtype, T):
    """NaN in every row of q that no sequence has: the workspace, which holds all that is made of q, shows none of it."""
    ref = Pages(3, 2, 64, [40, 7, 100], 16, dtype, room=T)
    q, k, v, u, vb, r = new(3, T, 2, 64, dtype, 4, 60)
    counts = torch.tensor([1, 0, T], dtype=torch.int32)
    for b in range(3):
        q[b, int(counts[b]):] = math.nan
    mem = ref.to_gpu(txl)
    ws = torch.zeros((txl.rel_attn_paged_workspace_size(q, mem, 60, True) + 3) // 4, device="cuda")
    out = torch.full_like(q, 5.0)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 60, 59, out, counts=counts.cuda(), accumulate=True, workspace=ws)
    assert not torch.isnan(ws).any()
    ref.push(k.cpu(), v.cpu(), counts)
    check_against(mem, ref, out, ref.weight.clone(), torch.nan_to_num(q), u, vb, r, 59, counts)
