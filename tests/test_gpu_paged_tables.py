"""GPU tests of the paged memory's page table on the host and the device: no sequences, tables with gaps, tables wider than what
sequences hold, and long memories, against the 64-bit restatement in paged_common.py."""
from __future__ import annotations

import math

import pytest
import torch

from paged_common import Pages, attend
from test_gpu_paged import check_memory, new

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


# ------------------------------------------------------------------------------------ gaps
def test_a_gap_in_a_row_stays_where_it_is(txl):
    """A page that a table lacks in front of others: what the host writes for any sequence leaves the others' slots alone."""
    from transformer_xl_relative_gb300 import native
    L, n = 16, 12
    mem = txl.PagedMemory.empty(1, n, L, 2, 64)
    _, k, v, u, vb, r = new(2, 60, 2, 64, BF, 1, 80)
    table = torch.full((2, 6), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor([5, 3, 7])
    table[1, :1] = 2
    i32 = dict(dtype=torch.int32, device="cuda")
    whole = txl.PagedMemory(mem.k, mem.v, mem.pos, mem.weight, table.cuda(), torch.zeros(2, **i32), torch.zeros(2, **i32))
    txl.paged_push(whole, k[:, :48], v[:, :48], counts=torch.tensor([48, 9], **i32))
    table[0, 1] = -1                                           # positions 16 .. 31 are lost
    mem = txl.PagedMemory(mem.k, mem.v, mem.pos, mem.weight, table.cuda(), whole.length.clone(), whole.next_pos.clone())
    assert mem.free_pages == n - 3 and mem.reserved == [48, 9]
    mem.reserve([0, 20])
    assert mem.table[0].tolist() == [5, -1, 7, -1, -1, -1] and mem.table[1, :2].min() >= 0
    mem.reserve([1, 0])
    row = mem.table[0].tolist()
    assert row[:3] == [5, -1, 7] and row[3] >= 0 and row[4:] == [-1, -1] and mem.free_pages == n - 5
    q, kn, vn, *_ = new(2, 1, 2, 64, BF, 2, 1)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, kn, vn, u.cuda(), vb.cuda(), r.cuda(), 80, 79, out)
    with pytest.raises(txl.TxlError) as e:
        mem.check()
    assert e.value.status == native.TXL_ERR_PAGE
    ref = Pages(2, 2, 64, [48, 9], L, BF, room=48)
    for b, m in ((0, 48), (1, 9)):
        for s in range(m):
            p, at = ref.at(b, s)
            ref.k[p, :, at], ref.v[p, :, at], ref.pos[p, at] = k[b, s].cpu(), v[b, s].cpu(), s
    ref.push(kn.cpu(), vn.cpu())
    for s in range(16, 32):
        p, at = ref.at(0, s)
        ref.pos[p, at] = 1 << 30                               # seen by nobody
    want, tol, *_ = attend(ref, q.cpu(), u, vb, r, 79)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    # neither eviction (which leaves a sequence with a gap as it is), nor trim, nor release moves or frees what is not there
    txl.paged_evict(mem, 20)
    assert mem.length.tolist() == [49, 10] and mem.reserved[0] == 49
    mem.trim()
    assert mem.table[0].tolist() == row and mem.reserved == [49, 10]
    mem.release(0)
    assert (mem.table[0] == -1).all() and mem.free_pages == n - 1 and sorted(mem._free) == sorted(set(range(n)) - {int(mem.table[1, 0])})


def test_a_gap_behind_the_length_is_filled(txl):
    """No position is lost there: the next pages of the sequence come from the pool, those behind the gap are free."""
    mem = txl.PagedMemory.empty(1, 8, 16, 2, 64)
    table = torch.tensor([[6, -1, 3, 99]], dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    mem = txl.PagedMemory(mem.k, mem.v, mem.pos, mem.weight, table, torch.tensor([10], **i32), torch.tensor([10], **i32))
    assert mem.free_pages == 7 and mem.reserved == [10]
    mem.reserve(30)
    row = mem.table[0].tolist()
    assert row[0] == 6 and len({*row[:3]}) == 3 and min(row[:3]) >= 0 and row[3] == -1 and mem.free_pages == 5
    _, k, v, *_ = new(1, 30, 2, 64, BF, 1, 1)
    txl.paged_push(mem, k, v)
    mem.check()
    assert mem.length.tolist() == [40]


def test_a_page_listed_twice_is_free_once(txl):
    """Behind the length a row may list a page that it has already: the pool gets it back once."""
    mem = txl.PagedMemory.empty(1, 4, 16, 2, 64)
    table = torch.tensor([[2, 2, 1], [0, -1, -1]], dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    mem = txl.PagedMemory(mem.k, mem.v, mem.pos, mem.weight, table, torch.tensor([9, 9], **i32), torch.tensor([9, 9], **i32))
    assert mem.free_pages == 1
    mem.trim()
    assert mem.table[0].tolist() == [2, -1, -1] and mem.free_pages == 2
    mem = txl.PagedMemory(mem.k, mem.v, mem.pos, mem.weight, table.copy_(torch.tensor([[2, 2, 1], [0, -1, -1]])), mem.length, mem.next_pos)
    mem.release(0)
    assert mem.free_pages == 3 and sorted(mem._free) == [1, 2, 3]


# ------------------------------------------------------------------------------------ tables wider than the pool
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 3, 9])
@pytest.mark.parametrize("D,page_len", [(64, 16), (41, 48), (128, 64)])
def test_weights_over_a_wide_table(txl, dtype, T, D, page_len):
    """Every row of the table could hold the pool: what scores take follows the pool, and weights are what they were."""
    ref = Pages(4, 3, D, [300, 0, 70, 16], page_len, dtype, room=T, spare=5, first=[400, 0, 71, 16])
    n = ref.k.shape[0]
    narrow = ref.table.clone()
    ref.table = torch.cat((narrow, torch.full((4, n - narrow.shape[1]), -1, dtype=torch.int32)), 1)
    q, k, v, u, vb, r = new(4, T, 3, D, dtype, 3, 120)
    counts = torch.tensor([T, max(1, T - 1), 0, T], dtype=torch.int32)
    wide = ref.to_gpu(txl)
    ref.table = narrow
    slim = ref.to_gpu(txl)
    outs, before = [], None
    ref.push(k.cpu(), v.cpu(), counts)
    before = ref.weight.clone()
    for mem in (wide, slim):
        out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
        txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 120, 119, out, counts=counts.cuda(), accumulate=True)
        outs.append(out)
        check_against(mem, ref, out, before, q, u, vb, r, 119, counts)
    assert torch.equal(*outs) and torch.equal(wide.weight, slim.weight)
    need = txl.rel_attn_paged_workspace_size(q, wide, 120, True) - txl.rel_attn_paged_workspace_size(q, wide, 120, False)
    assert need <= (n * page_len + 4) * 3 * T * 4 + 64


def test_a_missing_page_in_a_wide_table(txl):
    """A slot without a page has no score: the others' weights are right, and nothing is written for it."""
    ref = Pages(2, 2, 64, [100, 60], 16, BF, room=3, spare=5)
    n = ref.k.shape[0]
    narrow = ref.table.clone()
    ref.table = torch.cat((narrow, torch.full((2, n - narrow.shape[1]), -1, dtype=torch.int32)), 1)
    q, k, v, u, vb, r = new(2, 3, 2, 64, BF, 3, 120)
    mem = ref.to_gpu(txl)
    mem.table[0, 2] = -7
    ref.table = narrow
    out = torch.empty_like(q)
    ws = torch.zeros(txl.rel_attn_paged_workspace_size(q, mem, 120, True) + 64, dtype=torch.uint8, device="cuda")
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 120, 119, out, accumulate=True, workspace=ws)
    with pytest.raises(txl.TxlError):
        mem.check()
    assert (ws[-64:] == 0).all()
    ref.push(k.cpu(), v.cpu())
    before = ref.weight.clone()
    for s in range(32, 48):
        p, row = ref.at(0, s)
        ref.pos[p, row] = 1 << 30
    check_against(mem, ref, out, before, q, u, vb, r, 119)


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


# ------------------------------------------------------------------------------------ long memories
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype,T,D", [(BF, 1, 8), (BF, 2, 8), (BF, 16, 8), (F, 1, 8), (F, 3, 8)])
def test_shares_of_many_tiles_of_a_pair(txl, dtype, T, D, wide):
    """Pairs enough that a block takes more than 32 tiles a warp of one pair: a warp looks for its pages again and again."""
    B, H, n = 16, 16, 6016
    ref = Pages(B, H, D, [n - b % 3 for b in range(B)], 64, dtype, room=T, order=True)
    q, k, v, u, vb, r = new(B, T, H, D, dtype, 4, 400)
    if wide:                                                   # (rows that could hold the pool: scores by the pool's slots)
        ref.table = torch.cat((ref.table, torch.full((B, ref.k.shape[0] - ref.table.shape[1]), -1, dtype=torch.int32)), 1)
    mem = ref.to_gpu(txl)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 400, 399, out, accumulate=True)
    ref.push(k.cpu(), v.cpu())
    check_against(mem, ref, out, ref.weight.clone(), q, u, vb, r, 399)


@pytest.mark.parametrize("D,T", [(64, 1), (64, 4), (64, 6), (64, 16), (128, 1), (128, 5)])
def test_shares_of_many_tiles_of_shared_pages(txl, D, T):
    """The same for rings of other depths and blocks of other sizes: many sequences read one sequence's pages, of which each
    attends with queries of its own."""
    B, H, n = 48, 16, 6016
    ref = Pages(1, H, D, [n], 64, BF, order=True)
    mem1 = ref.to_gpu(txl)
    wide = lambda x: x.cuda().expand(B, *x.shape[1:]).contiguous()
    mem = txl.PagedMemory(mem1.k, mem1.v, mem1.pos, mem1.weight, wide(ref.table), wide(ref.length[None])[:, 0].contiguous(),
                          wide(ref.next_pos[None])[:, 0].contiguous())
    q, _, _, u, vb, r = new(B, T, H, D, BF, 4, 400)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, None, None, u.cuda(), vb.cuda(), r.cuda(), 400, 399, out)
    for b in (0, 17, B - 1):
        want, tol, *_ = attend(ref, q[b:b + 1].cpu(), u, vb, r, 399)
        assert ((out[b:b + 1].cpu().double() - want).abs() <= tol).all(), b
    mem.check()


def test_evict_more_than_shared_memory_holds(txl):
    """70000 slots of a sequence: a block of the cluster makes keys anew that its shared memory has no room for."""
    for recent, kind in ((1000, "random"), (0, "few")):
        ref = Pages(2, 1, 8, [70001, 300], 64, BF, first=[80000, 300], seed=recent)
        if kind == "few":
            ref.weight.copy_((ref.weight * 3).floor())
        mem = ref.to_gpu(txl)
        txl.paged_evict(mem, 30011, recent)
        ref.evict(30011, recent)
        check_memory(mem, ref)
