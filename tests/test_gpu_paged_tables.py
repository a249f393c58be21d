"""GPU tests of the paged memory's page table on the host and the device: no sequences, tables with gaps, tables wider than what
sequences hold, and long memories, against the 64-bit restatement in paged_common.py."""
from __future__ import annotations

import pytest
import torch

from test_gpu_paged import new

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m

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
