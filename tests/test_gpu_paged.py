"""GPU tests of the paged memory: pushes, the relative attention over it, the attention weights it adds up, and
evictions, against the 64-bit restatement in paged_common.py."""
from __future__ import annotations

import math

import pytest
import torch

from paged_common import Pages, attend

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


def same(a, b):
    return torch.equal(torch.nan_to_num(a.cpu(), nan=7e7), torch.nan_to_num(b.cpu(), nan=7e7))


def check_memory(mem, ref, weight=True):
    """Everything but the weights bit for bit."""
    assert same(mem.k, ref.k) and same(mem.v, ref.v)
    assert same(mem.pos, ref.pos) and same(mem.length, ref.length) and same(mem.next_pos, ref.next_pos)
    if weight:
        assert same(mem.weight, ref.weight)
    mem.check()


def new(B, T, H, D, dtype, seed, n_rows, layout="dense", ld_r=None):
    """q, k, v [B, T, H, D] in the given layout, u, vb, r."""
    g = torch.Generator().manual_seed(seed)

    def one():
        x = torch.randn(B, T, H, D, generator=g).to(dtype)
        if layout == "dense":
            return x.cuda()
        if layout == "padded":                       # rows of a multiple of 16 bytes
            s = torch.full((B, T, H, (D + 7) // 8 * 8 + 8), math.nan, dtype=dtype, device="cuda")
            s[..., :D] = x.cuda()
            return s[..., :D]
        if layout == "odd":                          # rows that start anywhere
            s = torch.full((B, T, H, D + 3), math.nan, dtype=dtype, device="cuda")[..., 1:1 + D]
            s.copy_(x.cuda())
            return s
        s = torch.empty(H, B, T, D, dtype=dtype, device="cuda").permute(1, 2, 0, 3)     # heads outermost
        s.copy_(x.cuda())
        return s

    q, k, v = one(), one(), one()
    u, vb = (0.3 * torch.randn(H, D, generator=g) for _ in range(2))
    ld = ld_r or (D + 7) // 8 * 8
    r = torch.full((n_rows, H, ld), math.nan, dtype=dtype)
    r[..., :D] = torch.randn(n_rows, H, D, generator=g).to(dtype)
    return q, k, v, u, vb, r


def step(txl, ref, T, C, n_rows, seed=1, counts=None, layout="dense", accumulate=False, pushed=False, scale=None, ld_r=None,
         q_scale=1.0):
    """One rel_attn_paged call against the restatement."""
    B, H, D, dtype = ref.B, ref.H, ref.D, ref.dtype
    q, k, v, u, vb, r = new(B, T, H, D, dtype, seed, n_rows, layout, ld_r)
    q.mul_(q_scale)
    mem = ref.to_gpu(txl)
    cnt = torch.tensor(counts, dtype=torch.int32) if counts is not None else None
    ref.push(k.cpu(), v.cpu(), cnt)
    if pushed:
        txl.paged_push(mem, k, v, counts=None if cnt is None else cnt.cuda())
    before = ref.weight.clone()
    out = torch.full((B, T, H, D), 5.0, dtype=dtype, device="cuda") if layout == "dense" else torch.full_like(q, 5.0)
    txl.rel_attn_paged(q, mem, *((None, None) if pushed else (k, v)), u.cuda(), vb.cuda(), r.cuda(), n_rows, C, out,
                       scale=scale or 0.0, counts=None if cnt is None else cnt.cuda(), accumulate=accumulate)
    want, tol, got, got_tol = attend(ref, q.cpu(), u, vb, r, C, cnt, scale)
    alone = torch.isnan(want)
    o = out.cpu().double()
    assert (o[alone] == 5.0).all()
    err = (o - want).abs()
    assert (err[~alone] <= tol[~alone]).all(), float((err / tol)[~alone].max())
    check_memory(mem, ref, weight=not accumulate)
    if accumulate:
        w = mem.weight.cpu().double() - before.double()
        bound = got_tol + 2.0 ** -23 * (before.double() + got) + 1e-30
        assert ((w - got).abs() <= bound).all(), float(((w - got).abs() / bound).max())
    return out


# ------------------------------------------------------------------------------------ pushes
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("layout", ["dense", "padded", "odd", "heads"])
@pytest.mark.parametrize("D,page_len", [(41, 16), (64, 48)])
def test_push(txl, dtype, layout, D, page_len):
    ref = Pages(3, 2, D, [0, 15, 70], page_len, dtype, room=40)
    _, k, v, *_ = new(3, 37, 2, D, dtype, 2, 1, layout)
    mem = ref.to_gpu(txl)
    counts = torch.tensor([37, 0, 20], dtype=torch.int32)
    txl.paged_push(mem, k, v, counts=counts.cuda())
    ref.push(k.cpu(), v.cpu(), counts)
    txl.paged_push(mem, k[:, :3], v[:, :3])
    ref.push(k[:, :3].cpu(), v[:, :3].cpu())
    check_memory(mem, ref)


def test_push_long_and_counts_out_of_range(txl):
    ref = Pages(2, 3, 128, [5, 0], 32, BF, room=3000)
    _, k, v, *_ = new(2, 2500, 3, 128, BF, 3, 1)
    mem = ref.to_gpu(txl)
    txl.paged_push(mem, k, v, counts=torch.tensor([-4, 99999], dtype=torch.int32, device="cuda"))
    ref.push(k.cpu(), v.cpu(), torch.tensor([0, 2500]))
    check_memory(mem, ref)


def test_push_without_room_leaves_the_sequence(txl):
    from transformer_xl_relative_gb300 import native
    ref = Pages(3, 2, 32, [10, 14, 3], 16, BF, room=4)
    ref.table[2, 1] = 1000                                   # no page
    _, k, v, *_ = new(3, 20, 2, 32, BF, 3, 1)
    mem = ref.to_gpu(txl)
    txl.paged_push(mem, k, v, counts=torch.tensor([6, 19, 14], dtype=torch.int32, device="cuda"))
    ref.push(k.cpu(), v.cpu(), torch.tensor([6, 0, 0]))      # 14 + 19 > 32 slots; slot 16 has no page
    with pytest.raises(txl.TxlError) as e:
        mem.check()
    assert e.value.status == native.TXL_ERR_PAGE
    check_memory(mem, ref)


@pytest.mark.parametrize("T", [1, 2])
def test_every_bit_enters(txl, T):
    """A push copies bits: the payloads of NaN and the sign of zero too, and rows end in zeros."""
    ref = Pages(1, 2, 41, [20], 16, BF, room=T)
    mem = ref.to_gpu(txl)
    bits = (torch.arange(T * 2 * 41, dtype=torch.int32) * 37 % 65536 - 32768).to(torch.int16)
    bits[::3] = torch.tensor([0x7fc1, 0x7f81, -1, -32768] * 100, dtype=torch.int16)[: len(bits[::3])]
    k = bits.view(BF).view(1, T, 2, 41).cuda()
    q, _, v, u, vb, r = new(1, T, 2, 41, BF, 1, 30)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 30, 29, out)
    for t in range(T):
        p, row = ref.at(0, 20 + t)
        assert torch.equal(mem.k[p, :, row].cpu().view(torch.int16), k[0, t].cpu().view(torch.int16))
        assert torch.equal(mem.v[p, :, row].cpu().view(torch.int16), v[0, t].cpu().view(torch.int16))
        whole = torch.as_strided(mem.k, (*mem.k.shape[:3], 48), mem.k.stride())
        assert (whole[p, :, row, 41:] == 0).all()


# ------------------------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("D", [1, 8, 31, 32, 41, 64, 80, 96, 128])
@pytest.mark.parametrize("T", [1, 9])
def test_widths(txl, dtype, D, T):
    ref = Pages(3, 2, D, [0, 33, 200], 16, dtype, room=T, seed=D)
    step(txl, ref, T, C=100, n_rows=101, accumulate=D in (41, 128))


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16])
def test_query_counts(txl, dtype, T):
    ref = Pages(4, 3, 64, [0, 1, 150, 47], 32, dtype, room=T, seed=T)
    step(txl, ref, T, C=60, n_rows=61, counts=[T, T // 2, 0, max(1, T - 1)], accumulate=True)


@pytest.mark.parametrize("page_len", [16, 48, 64, 1024])
@pytest.mark.parametrize("layout", ["padded", "odd", "heads"])
def test_pages_and_layouts(txl, page_len, layout):
    ref = Pages(2, 4, 41, [333, 90], page_len, BF, room=3)
    step(txl, ref, 3, C=1000, n_rows=400, layout=layout, ld_r=43, accumulate=True)


@pytest.mark.parametrize("dtype", [BF, F])
def test_positions_in_any_order_with_gaps(txl, dtype):
    ref = Pages(3, 2, 64, [100, 217, 16], 16, dtype, room=4, first=[500, 218, 4000])
    step(txl, ref, 4, C=300, n_rows=301, accumulate=True)


def test_a_position_table_shorter_than_the_clamp(txl):
    ref = Pages(2, 2, 64, [100, 30], 16, BF, room=2)
    step(txl, ref, 2, C=1 << 30, n_rows=20)
    ref = Pages(2, 2, 64, [100, 30], 16, BF, room=2)
    step(txl, ref, 2, C=0, n_rows=50)


def test_positions_pushed_before(txl):
    ref = Pages(3, 2, 64, [100, 0, 31], 16, BF, room=5)
    step(txl, ref, 5, C=50, n_rows=51, counts=[5, 3, 0], pushed=True, accumulate=True, scale=0.3)


@pytest.mark.parametrize("dtype", [BF, F])
def test_one_sharp_key(txl, dtype):
    """Scores of some hundreds: the softmax is one key's, and exponents run over their whole range."""
    ref = Pages(2, 2, 64, [700, 40], 64, dtype, room=1)
    step(txl, ref, 1, C=30, n_rows=31, q_scale=40.0, accumulate=True)


def test_many_ragged_sequences(txl):
    """More (sequence, head) pairs than blocks, lengths from none on: shares cut pairs anywhere."""
    B = 200
    lens = [(b * 37) % 130 for b in range(B)]
    ref = Pages(B, 5, 64, lens, 16, BF, room=2, seed=5)
    step(txl, ref, 2, C=64, n_rows=65, counts=[b % 3 for b in range(B)], accumulate=True)


@pytest.mark.parametrize("dtype,D,T", [(BF, 64, 1), (BF, 128, 16), (F, 64, 1)])
def test_a_long_sequence(txl, dtype, D, T):
    """One pair over every block: as many parts as there are blocks are joined."""
    ref = Pages(1, 1, D, [9000], 128, dtype, room=T, seed=9)
    step(txl, ref, T, C=9100, n_rows=9050, accumulate=True)


def test_no_visible_position(txl):
    """Queries whose positions lie before every key's, and queries of an empty memory: zeros."""
    ref = Pages(2, 2, 64, [20, 0], 16, BF, room=0)
    ref.pos += 1000
    mem = ref.to_gpu(txl)
    q, _, _, u, vb, r = new(2, 2, 2, 64, BF, 1, 10)
    out = torch.full_like(q, 5.0)
    w = mem.weight.clone()
    txl.rel_attn_paged(q, mem, None, None, u.cuda(), vb.cuda(), r.cuda(), 10, 9, out, accumulate=True)
    assert (out == 0).all() and torch.equal(mem.weight, w)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("long", [False, True])
def test_what_a_query_does_not_see_does_not_reach_it(txl, dtype, bad, long):
    """Unused slots, and the keys and values of later tokens, hold infinities and NaN."""
    B, H, D, T = 2, 2, 64, 3
    lens = [9000, 4500] if long else [37, 90]
    ref = Pages(B, H, D, lens, 64, dtype, room=40)
    for b in range(B):
        for s in list(range(lens[b] + T, lens[b] + 35)):
            p, row = ref.at(b, s)
            ref.k[p, :, row] = ref.v[p, :, row] = bad
    q, k, v, u, vb, r = new(B, T, H, D, dtype, 4, 50)
    k[:, 2, :, 3], v[:, 2, 0] = bad, bad
    mem = ref.to_gpu(txl)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 50, 49, out)
    ref.push(k.cpu(), v.cpu())
    want, tol, *_ = attend(ref, q.cpu(), u, vb, r, 49)
    o = out.cpu().double()
    assert ((o - want).abs() <= tol)[:, :2].all()
    # the last query sees them: nothing finite comes of a score that is NaN, or of an infinite value
    if math.isnan(bad):
        assert torch.isnan(o[:, 2]).all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_a_seen_infinite_value(txl, dtype):
    """An infinite value that a query does see makes that channel infinite and no other."""
    ref = Pages(1, 1, 64, [50], 16, dtype, room=1)
    p, row = ref.at(0, 20)
    ref.v[p, 0, row, 7] = math.inf
    q, k, v, u, vb, r = new(1, 1, 1, 64, dtype, 4, 60)
    mem = ref.to_gpu(txl)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 60, 59, out)
    o = out.cpu().flatten()
    assert o[7] == math.inf and torch.isfinite(o[:7]).all() and torch.isfinite(o[8:]).all()


def test_a_page_that_is_missing(txl):
    """Slots without a page count as not there, and the memory says so."""
    from transformer_xl_relative_gb300 import native
    ref = Pages(1, 2, 64, [100], 16, BF, room=1)
    q, k, v, u, vb, r = new(1, 1, 2, 64, BF, 4, 60)
    mem = ref.to_gpu(txl)
    mem.table[0, 2] = -7
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 60, 59, out)
    with pytest.raises(txl.TxlError) as e:
        mem.check()
    assert e.value.status == native.TXL_ERR_PAGE
    ref.push(k.cpu(), v.cpu())
    for s in range(32, 48):
        p, row = ref.at(0, s)
        ref.pos[p, row] = 1 << 30                            # seen by nobody
    want, tol, *_ = attend(ref, q.cpu(), u, vb, r, 59)
    assert ((out.cpu().double() - want).abs() <= tol).all()


def test_a_token_without_room_leaves_the_sequence(txl):
    """One token a sequence, whose pages the kernel itself finds missing: outputs, lengths and weights as they were."""
    from transformer_xl_relative_gb300 import native
    for T in (1, 2):
        ref = Pages(3, 2, 64, [31, 32, 5], 16, BF, room=0)        # (32 slots each)
        q, k, v, u, vb, r = new(3, T, 2, 64, BF, 4, 60)
        mem = ref.to_gpu(txl)
        mem.table[2, 0] = -1
        out = torch.full_like(q, 5.0)
        before = mem.weight.clone()
        txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 60, 59, out, accumulate=True)
        with pytest.raises(txl.TxlError) as e:
            mem.check()
        assert e.value.status == native.TXL_ERR_PAGE
        counts = torch.tensor([1 if T == 1 else 0, 0, 0])
        ref.push(k.cpu(), v.cpu(), counts)
        assert (out[1:] == 5).all()
        assert torch.equal(mem.length.cpu(), ref.length) and torch.equal(mem.next_pos.cpu(), ref.next_pos)
        if T == 1:
            want, tol, got, got_tol = attend(ref, q.cpu(), u, vb, r, 59, counts)
            assert ((out.cpu().double() - want).abs() <= tol)[0].all()
            mine = ref.table[0].long()
            w = mem.weight.cpu()[mine] - torch.where(ref.weight[mine] == 0, ref.weight[mine], before.cpu()[mine])
            assert ((w - got[mine]).abs() <= got_tol[mine] + 2.0 ** -22 * (1 + got[mine])).all()
        others = ref.table[1:].flatten().long()
        assert torch.equal(mem.weight[others.cuda()], before[others.cuda()])


@pytest.mark.parametrize("dtype", [BF, F])
def test_tokens_whose_second_page_is_missing(txl, dtype):
    """Sixteen tokens that begin in a page the sequence has and end in one it lacks: it is left as it was."""
    from transformer_xl_relative_gb300 import native
    ref = Pages(3, 2, 64, [25, 25, 16], 16, dtype, room=16)
    q, k, v, u, vb, r = new(3, 16, 2, 64, dtype, 4, 60)
    mem = ref.to_gpu(txl)
    mem.table[1, 2] = -1
    out = torch.full_like(q, 5.0)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 60, 59, out)
    with pytest.raises(txl.TxlError) as e:
        mem.check()
    assert e.value.status == native.TXL_ERR_PAGE
    counts = torch.tensor([16, 0, 16], dtype=torch.int32)
    ref.push(k.cpu(), v.cpu(), counts)
    check_memory(mem, ref, weight=False)
    assert (out[1] == 5).all()
    want, tol, *_ = attend(ref, q.cpu(), u, vb, r, 59, counts)
    assert ((out.cpu().double() - want).abs() <= tol)[[0, 2]].all()


@pytest.mark.parametrize("dtype", [BF, F])
def test_calls_one_after_another(txl, dtype):
    """Calls of different sizes queued without a pause leave what they leave with a pause after each."""
    T = [4, 1, 16, 2, 1, 1, 8, 3, 16, 1, 5, 4]
    ref = Pages(5, 4, 64, [700, 33, 0, 250, 1400], 16, dtype, room=sum(T))
    args = [new(5, t, 4, 64, dtype, 7 + i, 300) for i, t in enumerate(T)]
    dev = [[x.cuda() for x in a] for a in args]
    left = []
    for pause in (True, False):
        mem = ref.to_gpu(txl)
        outs = [torch.full_like(a[0], 5.0) for a in dev]
        ws = torch.empty(txl.rel_attn_paged_workspace_size(dev[2][0], mem, 300, True), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for (q, k, v, u, vb, r), out in zip(dev, outs):
            txl.rel_attn_paged(q, mem, k, v, u, vb, r, 300, 299, out, accumulate=True, workspace=ws)
            if pause:
                torch.cuda.synchronize()
        mem.check()
        left.append([x.clone() for x in (mem.k, mem.v, mem.pos, mem.weight, mem.length, mem.next_pos, *outs)])
    assert all(same(a, b) for a, b in zip(*left))


def test_as_many_sequences_as_a_memory_holds(txl):
    """B = 4096 at the widest head and most tokens: the blocks' shared memory at its largest."""
    B, T = 4096, 16
    ref = Pages(4, 1, 128, [20, 0, 33, 7], 16, BF, room=T)
    q, k, v, u, vb, r = new(4, T, 1, 128, BF, 4, 60)
    mem4 = ref.to_gpu(txl)
    pick = torch.tensor([0, 1, 2, 3])
    at = torch.tensor([0, 1000, 2222, 4095])
    wide = lambda x: torch.zeros(B, *x.shape[1:], dtype=x.dtype, device="cuda").index_copy_(0, at.cuda(), x.cuda()[pick.cuda()])
    mem = txl.PagedMemory(mem4.k, mem4.v, mem4.pos, mem4.weight, wide(ref.table), wide(ref.length), wide(ref.next_pos))
    counts = torch.zeros(B, dtype=torch.int32)
    counts[at] = T
    out = torch.full((B, T, 1, 128), 5.0, dtype=BF, device="cuda")
    txl.rel_attn_paged(wide(q), mem, wide(k), wide(v), u.cuda(), vb.cuda(), r.cuda(), 60, 59, out, counts=counts.cuda(), accumulate=True)
    ref.push(k.cpu(), v.cpu())
    want, tol, *_ = attend(ref, q.cpu(), u, vb, r, 59)
    o = out.cpu()
    assert ((o[at].double() - want).abs() <= tol).all()
    idle = torch.ones(B, dtype=torch.bool)
    idle[at] = False
    assert (o[idle] == 5).all()
    assert torch.equal(mem.length.cpu()[at], ref.length) and int(mem.length.sum()) == int(ref.length.sum())
    mem.check()


@pytest.mark.parametrize("T", [1, 3])
def test_infinite_keys_and_values_in_a_long_memory(txl, T):
    """A seen infinite value in a pair of many parts, and a query that is not a number beside one that is."""
    ref = Pages(2, 2, 64, [9000, 40], 64, BF, room=T)
    p, row = ref.at(0, 4321)
    ref.v[p, 1, row, 9] = -math.inf
    q, k, v, u, vb, r = new(2, T, 2, 64, BF, 4, 60)
    q[1, 0, 0, 5] = math.nan
    mem = ref.to_gpu(txl)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 60, 59, out)
    o = out.cpu().double()
    assert (o[0, :, 1, 9] == -math.inf).all() and torch.isnan(o[1, 0, 0]).all()
    ref.v[p, 1, row, 9] = 0.0
    ref.push(k.cpu(), v.cpu())
    want, tol, *_ = attend(ref, q.cpu(), u, vb, r, 59)
    ok = torch.isfinite(o) & ~torch.isnan(want)
    assert int((~ok).sum()) == T + 64 and ((o - want).abs() <= tol)[ok].all()


def test_the_same_bits_every_time(txl):
    ref = Pages(5, 3, 64, [1000, 3, 2222, 0, 517], 16, BF, room=4)
    q, k, v, u, vb, r = new(5, 4, 3, 64, BF, 4, 600)
    outs = []
    for _ in range(4):
        mem = ref.to_gpu(txl)
        out = torch.empty_like(q)
        txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 600, 599, out, accumulate=True)
        outs.append((out, mem.weight))
    for out, w in outs[1:]:
        assert torch.equal(out, outs[0][0]) and torch.equal(w, outs[0][1])


def test_offsets_past_32_bits(txl):
    """Pages whose first element lies past 2^32 (bf16 elements of one pool)."""
    H, D, page_len, n = 16, 128, 128, 17000                   # 4.4e9 elements a pool
    mem = txl.PagedMemory.empty(1, n, page_len, H, D, max_pages=4)
    ref = Pages(1, H, D, [300], page_len, BF, room=2, spare=0)
    for i in range(int(ref.table.shape[1])):
        far, p = n - 1 - 2 * i, int(ref.table[0, i])
        mem.k[far], mem.v[far] = ref.k[p].cuda(), ref.v[p].cuda()
        mem.pos[far], mem.weight[far] = ref.pos[p].cuda(), ref.weight[p].cuda()
        mem.table[0, i] = far
    mem.length.copy_(ref.length)
    mem.next_pos.copy_(ref.next_pos)
    q, k, v, u, vb, r = new(1, 2, H, D, BF, 4, 320)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 320, 319, out, accumulate=True)
    ref.push(k.cpu(), v.cpu())
    want, tol, *_ = attend(ref, q.cpu(), u, vb, r, 319)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    pages = [(n - 1 - 2 * i, int(p)) for i, p in enumerate(ref.table[0])]
    for far, p in pages:                                      # (the sums of weights have their own test)
        ref.weight[p] = mem.weight[far].cpu()
    txl.paged_evict(mem, 200, 50)
    ref.evict(200, 50)
    for far, p in pages:
        assert same(mem.k[far], ref.k[p]) and same(mem.v[far], ref.v[p]) and same(mem.pos[far], ref.pos[p])
    assert int(mem.length[0]) == 200
    mem.check()


# ------------------------------------------------------------------------------------ eviction
def evict(txl, ref, keep, recent):
    mem = ref.to_gpu(txl)
    txl.paged_evict(mem, keep, recent)
    ref.evict(keep, recent)
    check_memory(mem, ref)
    return mem


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (40, 0), (64, 64), (100, 30), (299, 100), (300, 300)])
def test_evict(txl, dtype, keep, recent):
    ref = Pages(4, 3, 41, [300, 0, 64, 150], 16, dtype, first=[300, 0, 900, 151], seed=keep)
    evict(txl, ref, keep, recent)


@pytest.mark.parametrize("kind", ["equal", "two", "zeros", "infinite", "nan", "negative", "close"])
def test_evict_ties(txl, kind):
    """Equal weights leave in the order of their positions; NaN leaves last."""
    ref = Pages(2, 1, 8, [2500, 700], 32, BF, seed=3)
    g = torch.Generator().manual_seed(1)
    u = torch.rand(ref.weight.shape, generator=g)
    if kind == "equal":
        ref.weight.fill_(0.25)
    elif kind == "two":
        ref.weight.copy_(torch.where(u < 0.5, 1.0, 2.0))
    elif kind == "zeros":
        ref.weight.copy_(torch.where(u < 0.3, 0.0, torch.where(u < 0.6, -0.0, u)))
    elif kind == "infinite":
        ref.weight.copy_(torch.where(u < 0.5, math.inf, u))
    elif kind == "nan":
        ref.weight.copy_(torch.where(u < 0.7, math.nan, torch.where(u < 0.8, math.inf, u)))
    elif kind == "negative":
        ref.weight.copy_(u - 0.5)
    else:
        ref.weight.copy_(1.0 + (u * 8).floor() * 2.0 ** -23)
    evict(txl, ref, 333, 100)


def test_evict_long(txl):
    ref = Pages(2, 1, 64, [20000, 7001], 128, BF, seed=4)
    evict(txl, ref, 5000, 512)


def test_evict_again_and_missing_pages(txl):
    from transformer_xl_relative_gb300 import native
    ref = Pages(2, 2, 32, [200, 200], 16, BF, first=[400, 400])
    mem = ref.to_gpu(txl)
    for keep in (150, 150, 90, 17):
        txl.paged_evict(mem, keep, 10)
        ref.evict(keep, 10)
        check_memory(mem, ref)
    mem.table[1, 0] = 9999
    txl.paged_evict(mem, 10, 5)
    kept = int(ref.length[1])
    with pytest.raises(txl.TxlError) as e:
        mem.check()
    assert e.value.status == native.TXL_ERR_PAGE
    assert mem.length.tolist() == [10, kept]


def test_room_after_an_eviction(txl):
    """No sequence has room for more than it kept; what was reserved and not pushed is reserved again."""
    mem = txl.PagedMemory.empty(1, 8, 16, 2, 64)
    x = torch.randn(1, 60, 2, 64, device="cuda").to(BF)
    mem.reserve(70)
    txl.paged_push(mem, x, x)
    txl.paged_evict(mem, 64, 8)
    assert mem.reserved == [64] and mem.length.tolist() == [60] and mem.free_pages == 3
    txl.paged_evict(mem, 20, 8)
    assert mem.reserved == [20] and mem.length.tolist() == [20] and mem.free_pages == 3
    mem.trim()
    assert mem.reserved == [20] and mem.free_pages == 6
    mem.reserve(60)
    txl.paged_push(mem, x, x)
    assert mem.length.tolist() == [80] and mem.next_pos.tolist() == [120]
    mem.check()


# ------------------------------------------------------------------------------------ a run of them
def test_generation_with_a_bounded_memory(txl):
    """Prompts, tokens and evictions through the public entry points, pages from the memory's own pool, against the
    restatement; the weights of the restatement follow the device's (their own test bounds them)."""
    B, H, D, L = 3, 4, 64, 16
    mem = txl.PagedMemory.empty(B, 40, L, H, D, max_pages=12)
    ref = Pages(B, H, D, [0] * B, L, BF, room=12 * L, spare=4)
    n_rows = 400
    prompts = torch.tensor([90, 20, 57], dtype=torch.int32)
    _, k, v, u, vb, r = new(B, 90, H, D, BF, 1, n_rows)
    mem.reserve(prompts.tolist())
    txl.paged_push(mem, k, v, counts=prompts.cuda())
    ref.push(k.cpu(), v.cpu(), prompts)
    for t in range(60):
        q, k, v, *_ = new(B, 2, H, D, BF, 10 + t, 1)
        counts = torch.tensor([2, t % 3 % 2, 1], dtype=torch.int32)
        mem.reserve(2)
        out = torch.zeros_like(q)
        txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), n_rows, n_rows - 1, out, counts=counts.cuda(),
                           accumulate=True)
        ref.push(k.cpu(), v.cpu(), counts)
        want, tol, *_ = attend(ref, q.cpu(), u, vb, r, n_rows - 1, counts)
        live = ~torch.isnan(want)
        assert ((out.cpu().double() - want).abs() <= tol)[live].all(), t
        if t % 20 == 19:
            host = mem.table.cpu()
            for b in range(B):
                n = int(ref.length[b])
                p, row = ref.index(b, n)
                s = torch.arange(n)
                ref.weight[p, row] = mem.weight.cpu()[host[b, s // L].long(), s % L]
            txl.paged_evict(mem, 64, 16)
            ref.evict(64, 16)
            mem.trim()
            assert mem.free_pages == 40 - sum((int(n) + L - 1) // L for n in ref.length)
        assert torch.equal(mem.length.cpu(), ref.length) and torch.equal(mem.next_pos.cpu(), ref.next_pos)
    mem.check()
    free = mem.free_pages
    mem.release(0)
    assert mem.length.tolist()[0] == 0 and mem.free_pages > free and (mem.table[0] == -1).all()
    with pytest.raises(ValueError):
        mem.reserve(10 ** 6)
    with pytest.raises(ValueError):
        mem.reserve([1, 2])
    with pytest.raises(ValueError):
        mem.release(3)


def test_shared_pages(txl):
    """Two sequences read one prefix; the page that both have is free when both have gone."""
    mem = txl.PagedMemory.empty(1, 6, 16, 2, 64)
    _, k, v, *_ = new(1, 32, 2, 64, BF, 1, 1)
    mem.reserve(32)
    txl.paged_push(mem, k, v)
    pages = mem.table[0, :2].tolist()
    table = torch.tensor([pages + [5], pages + [-1]], dtype=torch.int32, device="cuda")
    both = txl.PagedMemory(mem.k, mem.v, mem.pos, mem.weight, table, mem.length.repeat(2), mem.next_pos.repeat(2))
    assert both.free_pages == 3
    q, kn, vn, u, vb, r = new(2, 1, 2, 64, BF, 2, 40)
    q[1], kn[1], vn[1] = q[0], kn[0], vn[0]
    both.reserve(1)
    out = torch.empty_like(q)
    txl.rel_attn_paged(q, both, kn, vn, u.cuda(), vb.cuda(), r.cuda(), 40, 39, out)
    both.check()
    assert torch.equal(out[0], out[1])
    both.release(0)
    assert both.free_pages == 3                              # (its own page; the other sequence took one)
    both.release(1)
    assert both.free_pages == 6


def test_refusals_of_the_binding(txl):
    mem = txl.PagedMemory.empty(2, 4, 16, 2, 64)
    q, k, v, u, vb, r = new(2, 1, 2, 64, BF, 2, 40)
    u, vb, r = u.cuda(), vb.cuda(), r.cuda()
    out = torch.empty_like(q)
    good = dict(q=q, mem=mem, k_new=k, v_new=v, u=u, v_bias=vb, r=r, n_rows=40, clamp_len=39, out=out)
    for bad, error in ((dict(v_new=None), ValueError), (dict(k_new=k.float()), TypeError), (dict(q=q.float()), TypeError),
                       (dict(u=u.double()), TypeError), (dict(u=u[:1]), ValueError), (dict(n_rows=41), ValueError),
                       (dict(r=r[:, :1]), ValueError), (dict(out=out[:1]), ValueError), (dict(q=q.cpu()), ValueError),
                       (dict(counts=torch.zeros(2, device="cuda")), ValueError),
                       (dict(counts=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError),
                       (dict(workspace=torch.empty(8, dtype=torch.uint8)), ValueError),
                       (dict(q=q.transpose(1, 3), out=out.transpose(1, 3)), ValueError), (dict(clamp_len=-1), txl.TxlError),
                       (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), txl.TxlError)):
        with pytest.raises(error):
            txl.rel_attn_paged(**{**good, **bad})
    for bad, error in ((dict(k_new=k[:1], v_new=v[:1]), ValueError), (dict(v_new=v.float()), TypeError),
                       (dict(k_new=k.cpu(), v_new=v.cpu()), ValueError),
                       (dict(k_new=k.transpose(2, 3), v_new=v.transpose(2, 3)), ValueError)):
        with pytest.raises(error):
            txl.paged_push(**{**dict(mem=mem, k_new=k, v_new=v), **bad})
    for keep, recent in ((0, 0), (3, 4), (3, -1)):
        with pytest.raises(txl.TxlError):
            txl.paged_evict(mem, keep, recent)
    for kw in (dict(table=mem.table.long()), dict(length=mem.length[:1]), dict(pos=mem.pos[:, :8]), dict(weight=mem.pos)):
        with pytest.raises(ValueError):
            txl.PagedMemory(**{**dict(k=mem.k, v=mem.v, pos=mem.pos, weight=mem.weight, table=mem.table, length=mem.length,
                                      next_pos=mem.next_pos), **kw})
    mem.check()
    assert mem.length.tolist() == [0, 0]


def test_captured_and_replayed(txl):
    """A captured step replays over lengths that grow on the device, and two graphs share a workspace."""
    B, H, D = 2, 2, 64
    ref = Pages(B, H, D, [40, 7], 16, BF, room=20)
    mem = ref.to_gpu(txl)
    q, k, v, u, vb, r = new(B, 1, H, D, BF, 1, 64)
    u, vb, r = u.cuda(), vb.cuda(), r.cuda()
    out = torch.zeros_like(q)
    ws = torch.empty(txl.rel_attn_paged_workspace_size(q, mem, 64, True), dtype=torch.uint8, device="cuda")
    state = [t.clone() for t in (mem.k, mem.v, mem.pos, mem.weight, mem.length, mem.next_pos)]
    run = lambda acc: txl.rel_attn_paged(q, mem, k, v, u, vb, r, 64, 63, out, accumulate=acc, workspace=ws)
    run(True)                                                 # (kernels prepared before the capture)
    graphs = []
    for acc in (True, False):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(acc)
        graphs.append(g)
    for t, s in zip((mem.k, mem.v, mem.pos, mem.weight, mem.length, mem.next_pos), state):
        t.copy_(s)
    for i in range(8):
        for t, seed in ((q, 3 * i), (k, 3 * i + 1), (v, 3 * i + 2)):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(seed)))
        graphs[i % 2].replay()
        ref.push(k.cpu(), v.cpu())
        want, tol, *_ = attend(ref, q.cpu(), u.cpu(), vb.cpu(), r.cpu(), 63)
        assert ((out.cpu().double() - want).abs() <= tol).all(), i
    assert mem.length.tolist() == [48, 15]


def test_on_another_stream(txl):
    ref = Pages(2, 2, 64, [300, 20], 16, BF, room=3)
    q, k, v, u, vb, r = new(2, 3, 2, 64, BF, 1, 64)
    u, vb, r = u.cuda(), vb.cuda(), r.cuda()
    mem = ref.to_gpu(txl)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    txl.rel_attn_paged(q, mem, k, v, u, vb, r, 64, 63, out, accumulate=True, stream=side)
    txl.paged_push(mem, k[:, :0], v[:, :0], stream=side)
    txl.paged_evict(mem, 250, 20, stream=side)
    side.synchronize()
    ref.push(k.cpu(), v.cpu())
    want, tol, *_ = attend(ref, q.cpu(), u.cpu(), vb.cpu(), r.cpu(), 63)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert mem.length.tolist() == [250, 23]
