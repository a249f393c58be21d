"""GPU tests of the paged memory and the 4-bit weights as a serving loop uses them: captured at once, replayed together, idle
batches, and positions at the end of their range."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

from paged_common import Pages, attend
from test_gpu_paged import check_memory, new, same

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


FIRST_CALLS = """
import sys
sys.path.insert(0, %r)
import torch
import transformer_xl_relative_gb300 as txl
T = int(sys.argv[1])
g = torch.Generator(device="cuda").manual_seed(0)
draw = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
mem = txl.PagedMemory.empty(2, 20, 16, 2, 64)
mem.reserve(90)
k, v, q, kn, vn, r = draw(2, 90 - T, 2, 64), draw(2, 90 - T, 2, 64), draw(2, T, 2, 64), draw(2, T, 2, 64), draw(2, T, 2, 64), draw(100, 2, 64)
u = torch.zeros(2, 64, device="cuda")
W, x = draw(128, 48), draw(2 * T, 128)
out, y = torch.zeros_like(q), torch.zeros(2 * T, 48, device="cuda").bfloat16()
data = torch.zeros(txl.native.load().txl_q4_bytes(128, 48, 64), dtype=torch.uint8, device="cuda")
w = txl.QuantWeight(data, 128, 48, 64)
state = mem.k, mem.v, mem.pos, mem.weight, mem.length, mem.next_pos
start = [t.clone() for t in state]

def step():
    txl.paged_push(mem, k, v)
    txl.rel_attn_paged(q, mem, kn, vn, u, u, r, 100, 99, out, accumulate=True)
    txl.paged_evict(mem, 40, 10)
    txl.linear_q4(x, w, y)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
w2 = txl.QuantWeight.quantise(W)
data.copy_(w2.data)
seen = []
for run in (graph.replay, graph.replay, step):
    for t, s in zip(state, start):
        t.copy_(s)
    run()
    torch.cuda.synchronize()
    mem.check()
    seen.append([t.clone() for t in (*state, out, y)])
assert mem.length.tolist() == [40, 40] and mem.next_pos.tolist() == [90, 90]
assert float(out.float().abs().sum()) > 0 and float(y.float().abs().sum()) > 0
assert all(torch.equal(a, b) for s in seen[1:] for a, b in zip(seen[0], s))
print("same")
"""


@pytest.mark.parametrize("T", [1, 5])
def test_the_first_calls_of_a_process_may_be_captured(txl, T):
    """A push, tokens, an eviction and a product in one graph, replayed and called: the same bits."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALLS % root, str(T)], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "same" in p.stdout, p.stderr[-2000:]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 4])
def test_no_sequence_has_a_token(txl, dtype, T):
    """Every count is 0: nothing changes, and the next call finds the memory in order."""
    ref = Pages(3, 2, 64, [40, 0, 17], 16, dtype, room=2 * T)
    mem = ref.to_gpu(txl)
    q, k, v, u, vb, r = new(3, T, 2, 64, dtype, 4, 60)
    u, vb, r = u.cuda(), vb.cuda(), r.cuda()
    out = torch.full_like(q, 5.0)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    txl.paged_push(mem, k, v, counts=none)
    for acc in (False, True):
        txl.rel_attn_paged(q, mem, k, v, u, vb, r, 60, 59, out, counts=none, accumulate=acc)
        txl.rel_attn_paged(q, mem, None, None, u, vb, r, 60, 59, out, counts=none, accumulate=acc)
    assert (out == 5).all()
    check_memory(mem, ref)
    txl.rel_attn_paged(q, mem, k, v, u, vb, r, 60, 59, out)
    ref.push(k.cpu(), v.cpu())
    want, tol, *_ = attend(ref, q.cpu(), u.cpu(), vb.cpu(), r.cpu(), 59)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    check_memory(mem, ref)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("T", [1, 3, 16])
def test_the_last_positions(txl, dtype, T):
    """Positions up to 2^31 - 33: distances, pushes and evictions are those of the same sequence at the beginning."""
    ref = Pages(2, 2, 64, [70, 33], 16, dtype, room=T, first=[90, 33])
    q, k, v, u, vb, r = new(2, T, 2, 64, dtype, 4, 60)
    last = 2 ** 31 - 33 - 90 - T + 1
    got = []
    for shift in (0, last):
        ref.pos += shift
        ref.next_pos += shift
        mem = ref.to_gpu(txl)
        ref.pos -= shift
        ref.next_pos -= shift
        out = torch.empty_like(q)
        txl.rel_attn_paged(q, mem, k, v, u.cuda(), vb.cuda(), r.cuda(), 60, 59, out, accumulate=True)
        assert (mem.next_pos.cpu() - shift).tolist() == [90 + T, 33 + T]
        txl.paged_evict(mem, 30, 12)
        mem.check()
        used = ref.table.flatten().long().cuda()
        got.append((out, mem.k, mem.v, mem.pos[used].cpu() - shift, mem.weight, mem.length))
    assert all(same(a, b) for a, b in zip(*got))
