"""GPU tests of txl_rel_attn_qmem: relative attention over a quantised memory, against 64-bit
arithmetic over what the memory stands for, and the run of push and attention that generates."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gpu_common import ld_r_for
from qmem_common import attend64, decode_tolerance, f64, held, segment_tolerance

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


class Call:
    """Inputs of one call: the pushed history, the segment, biases and position rows."""

    def __init__(self, txl, B, H, D, L, M, valid, wp, C, bits, dtype, seed=0, hs=None, shift=0):
        self.dims, self.C, self.bits, self.dtype = (B, L, H, D), C, bits, DT[dtype]
        g = torch.Generator().manual_seed(seed + 17 * L + M + D)
        gain = 0.5 + 1.5 * torch.rand(H, D, generator=g)
        self.kh, self.vh = ((randn(g, B, valid, H, D) * gain).to(self.dtype) for _ in range(2))
        self.q, self.k, self.v = (self.place(randn(g, B, L, H, D), hs, shift) for _ in range(3))
        self.u, self.vb = (0.3 * randn(g, H, D).cuda() for _ in range(2))
        self.n_rows = min(M + L, C + 1)
        self.r = torch.full((self.n_rows, H, ld_r_for(D)), float("nan"), dtype=self.dtype, device="cuda")
        self.r[..., :D] = (0.7 * randn(g, self.n_rows, H, D)).to(self.dtype).cuda()
        self.mem = None
        if M > 0:
            self.mem = txl.QuantMemory.empty(B, M, H, D, bits=bits)
            self.mem.rows.fill_(0xFF)                  # slots that are not valid hold NaN parameters
            self.mem.restore((wp - valid) % M, 0)
            if valid:
                txl.qmem_push(self.mem, self.kh.cuda(), self.vh.cuda())
            assert self.mem.state() == (wp, valid)
        self.out = self.place(torch.full((B, L, H, D), float("nan")), hs, shift)

    def place(self, x, hs, shift):
        B, T, H, D = x.shape
        hs = hs or D
        flat = torch.full((B * T * H * hs + shift,), float("nan"), dtype=self.dtype, device="cuda")
        y = flat[shift:].view(B, T, H, hs)[..., :D]
        y.copy_(x.to(self.dtype))
        return y

    def run(self, txl, **kw):
        return txl.rel_attn_qmem(self.q, self.mem, self.k, self.v, self.u, self.vb, self.r, self.n_rows, self.C,
                                 self.out, **kw)

    def operands(self):
        k = np.concatenate((held(f64(self.kh), self.bits), f64(self.k)), 1)
        v = np.concatenate((held(f64(self.vh), self.bits), f64(self.v)), 1)
        return f64(self.q), k, v, f64(self.u), f64(self.vb), np.nan_to_num(f64(self.r))

    def reference(self, scale=None):
        x = self.operands()
        ref, size = attend64(*x, self.C, scale)
        return ref, size, float(np.abs(x[2]).max())


def check(call, scale=None):
    ref, size, vmax = call.reference(scale)
    err = np.abs(f64(call.out) - ref)
    tol = decode_tolerance(ref, size, vmax, call.dtype)
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


def check_segment(call):
    ref, _, _ = call.reference()
    tol = segment_tolerance(*call.operands(), call.C, ref)
    err = np.abs(f64(call.out) - ref)
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


DECODE = [
    # B, H, D, L, M, valid, wp, C, dtype, head stride, elements off alignment
    (1, 1, 64, 1, 1, 1, 0, 5, "bf16", None, 0),             # two keys in all
    (2, 3, 64, 1, 100, 100, 0, 1000, "bf16", None, 0),
    (2, 3, 64, 1, 1000, 1000, 37, 300, "bf16", None, 0),    # wrapped ring, clamp inside
    (3, 2, 64, 1, 700, 1, 699, 1000, "bf16", None, 0),      # one valid position
    (2, 2, 64, 1, 50, 0, 0, 1000, "bf16", None, 0),         # an empty memory: the query sees itself
    (1, 2, 64, 4, 0, 0, 0, 1000, "bf16", None, 0),          # no memory at all
    (2, 2, 64, 1, 900, 900, 5, 0, "bf16", None, 0),         # every distance clamps to 0
    (9, 2, 64, 1, 333, 300, 200, 100, "bf16", None, 0),     # more batch entries than a block takes
    (5, 3, 64, 2, 513, 513, 511, 400, "bf16", None, 0),
    (3, 2, 64, 3, 600, 599, 1, 1000, "bf16", None, 0),
    (2, 2, 64, 4, 640, 640, 128, 1000, "bf16", None, 0),
    (2, 2, 64, 5, 257, 257, 0, 1000, "bf16", None, 0),
    (2, 1, 64, 8, 257, 200, 3, 100, "bf16", None, 0),
    (1, 2, 64, 9, 300, 300, 77, 1000, "bf16", None, 0),
    (2, 1, 64, 16, 530, 530, 529, 200, "bf16", None, 0),
    (1, 2, 128, 1, 2100, 2100, 1000, 1000, "bf16", None, 0),
    (2, 2, 128, 3, 130, 130, 7, 1000, "bf16", None, 0),
    (1, 1, 128, 16, 300, 300, 0, 50, "bf16", None, 0),
    (4, 2, 41, 1, 300, 290, 5, 1000, "bf16", 48, 0),        # odd D, heads 48 apart
    (2, 2, 41, 3, 300, 300, 5, 100, "bf16", None, 1),       # odd D, dense, off alignment
    (2, 2, 33, 1, 65, 65, 64, 1000, "bf16", None, 0),
    (1, 2, 32, 2, 64, 64, 0, 1000, "bf16", None, 0),
    (1, 3, 1, 1, 40, 40, 3, 1000, "bf16", None, 0),
    (2, 2, 96, 1, 150, 150, 149, 1000, "bf16", None, 0),
    (1, 2, 80, 7, 90, 90, 30, 1000, "bf16", None, 0),
    (1, 2, 8, 8, 8, 8, 3, 16, "f32", None, 0),
    (2, 2, 64, 1, 777, 500, 600, 64, "f32", None, 0),
    (2, 1, 41, 5, 300, 300, 5, 1000, "f32", None, 1),
    (1, 2, 128, 16, 200, 200, 5, 1000, "f32", None, 0),
    (4, 1, 64, 1, 40, 40, 5, 1000, "f32", None, 0),
    (1, 2, 64, 1, 40003, 40000, 12345, 1000, "bf16", None, 0),     # the largest clusters
    (1, 1, 64, 6, 9000, 9000, 8999, 8000, "bf16", None, 0),
    (1, 1, 128, 1, 3329, 3329, 17, 1000, "bf16", None, 0),         # the last ranks of a cluster without keys
    (1, 1, 64, 16, 3400, 3393, 17, 3000, "bf16", None, 0),
    (9, 2, 64, 16, 70, 70, 11, 1000, "bf16", None, 0),             # more (entry, query) pairs than a block takes
    (9, 1, 128, 9, 70, 66, 11, 50, "bf16", None, 0),
    (1, 2, 96, 6, 333, 331, 100, 97, "bf16", None, 0),
    (2, 2, 64, 1, 301, 301, 100, 98, "bf16", None, 1),             # distances beyond the table, off alignment
    (2, 2, 64, 2, 302, 299, 100, 99, "bf16", None, 1),
    (2, 1, 41, 3, 303, 303, 302, 101, "bf16", 47, 1),
    (1, 2, 72, 4, 5000, 5000, 4321, 100, "f32", 76, 0),
    (2, 2, 64, 1, 255, 255, 100, 1000, "bf16", None, 0),           # position terms in the attention kernel
    (2, 2, 64, 1, 256, 256, 100, 1000, "bf16", None, 0),           # and not
    (2, 2, 128, 8, 248, 240, 100, 230, "bf16", None, 0),
    (1, 2, 41, 16, 4000, 4000, 77, 210, "bf16", None, 1),          # clamped except the last range
    (1, 2, 64, 2, 20000, 19999, 77, 60, "bf16", None, 0),
    (1, 2, 64, 1, 255, 255, 100, 1000, "f32", None, 0),
    (1, 2, 64, 1, 256, 256, 100, 1000, "f32", None, 0),
    (2, 2, 64, 16, 600, 600, 100, 500, "f32", None, 0),            # 32 pairs of (entry, query)
    (3, 1, 96, 11, 400, 400, 100, 380, "f32", None, 1),            # 33
    (2, 1, 33, 16, 3000, 3000, 77, 30, "f32", None, 1),
]
IDS = ["B%dH%dD%d_L%dM%dv%dwp%dC%d_%s_hs%s_s%d" % c for c in DECODE]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("c", DECODE, ids=IDS)
def test_few_queries_match_64_bits(txl, c, bits):
    B, H, D, L, M, valid, wp, C, dtype, hs, shift = c
    call = Call(txl, B, H, D, L, M, valid, wp, C, bits, dtype, hs=hs, shift=shift)
    assert txl.rel_attn_qmem_path(call.q, call.mem, call.k, call.v, call.r, call.out) == 5
    call.run(txl)
    torch.cuda.synchronize()
    check(call)
    if hs:                                                  # the gaps between heads stay
        gap = torch.as_strided(call.out, (B, L, H - 1, hs - D), call.out.stride(), call.out.storage_offset() + D)
        assert torch.isnan(gap).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("c", [(10, 2, 64, 3, 358), (2, 2, 8, 8, 1377), (1, 2, 128, 1, 4653), (1, 3, 41, 7, 8938)])
def test_fp32_keeps_its_bits(txl, c, bits):
    """The parts of q and of the weights are off by 2^-23 of themselves, the exponential by 2^-22: a term of the
    sums by less than 2^-20.  The sums average such errors, and the codes are centred, so that terms do not cancel
    more than the values themselves do; another factor of two is for the roundings of the sums."""
    B, H, D, L, M = c
    call = Call(txl, B, H, D, L, M, M, 5, 1000, bits, "f32")
    call.run(txl)
    torch.cuda.synchronize()
    ref, _, _ = call.reference()
    assert np.linalg.norm(f64(call.out) - ref) <= 2.0 ** -19 * np.linalg.norm(ref)


def test_a_given_scale(txl):
    call = Call(txl, 2, 2, 64, 1, 200, 200, 9, 1000, 4, "bf16")
    call.run(txl, scale=0.31)
    torch.cuda.synchronize()
    check(call, scale=0.31)


@pytest.mark.parametrize("factor", [1e-30, 1e-6, 1e4, 1e25, 1e33])
@pytest.mark.parametrize("bits", [4, 8])
def test_values_of_any_magnitude(txl, bits, factor):
    """The output scales with the values, whatever their size (the softmax does not see them)."""
    call = Call(txl, 2, 2, 64, 1, 300, 300, 9, 1000, bits, "f32")
    call.vh, call.v = call.vh * factor, call.v * factor
    call.mem.restore((9 - 300) % 300, 0)
    txl.qmem_push(call.mem, call.kh.cuda(), call.vh.cuda())
    call.run(txl)
    torch.cuda.synchronize()
    check(call)


def test_steps_that_differ_by_many_orders(txl):
    """A position with a huge value step and no weight beside positions of small steps that carry it,
    before and after them in the memory."""
    for first in (True, False):
        call = Call(txl, 1, 1, 64, 1, 400, 400, 0, 1000, 4, "f32")
        j = 3 if first else 390
        q = f64(call.q)[0, 0, 0] + f64(call.u)[0]
        call.kh[0, j, 0] = torch.from_numpy(-q * 40 / np.linalg.norm(q)).float()     # a score far below the rest
        call.vh[0, j, 0] *= 1e6
        call.mem.restore(0, 0)
        txl.qmem_push(call.mem, call.kh.cuda(), call.vh.cuda())
        call.run(txl)
        torch.cuda.synchronize()
        ref, size, _ = call.reference()
        # that position's weight is below 2^-40; the others' values are below 16
        tol = decode_tolerance(ref, size, 16.0, torch.float32)
        assert (np.abs(f64(call.out) - ref) <= tol).all()


def test_large_scores(txl):
    """Scores of some hundreds: the running maximum moves, weights underflow."""
    call = Call(txl, 2, 2, 64, 2, 500, 500, 123, 1000, 8, "f32")
    call.q.mul_(40.0)
    call.run(txl)
    torch.cuda.synchronize()
    ref, size, vmax = call.reference()
    # ds = 2^-16 size is no longer small: the weights move by at most e^(2 ds) - 1
    ds = 2.0 ** -16 * size
    tol = 2.0 ** -24 * np.abs(ref) + (2 * np.expm1(2 * ds) + 2.0 ** -15) * vmax
    assert (np.abs(f64(call.out) - ref) <= tol).all()


def test_a_group_of_nan_reaches_only_what_it_should(txl):
    """A NaN value group makes its 32 output channels NaN, a NaN key the whole row; other heads and
    batch entries stay exact."""
    call = Call(txl, 3, 2, 64, 1, 100, 100, 11, 1000, 4, "bf16")
    call.vh[0, 40, 1, 33] = float("nan")
    call.kh[1, 7, 0, 2] = float("inf")
    call.mem.restore(11, 0)
    txl.qmem_push(call.mem, call.kh.cuda(), call.vh.cuda())
    call.run(txl)
    torch.cuda.synchronize()
    out = f64(call.out)
    assert np.isnan(out[0, 0, 1, 32:]).all() and np.isnan(out[1, 0, 0]).all()
    call.vh[0, 40, 1, 33] = 0.0
    call.kh[1, 7, 0, 2] = 0.0
    ref, size, vmax = call.reference()
    tol = decode_tolerance(ref, size, vmax, call.dtype)
    ok = np.abs(out - ref) <= tol
    assert ok[0, :, 0].all() and ok[0, 0, 1, :32].all() and ok[1, :, 1].all() and ok[2].all()


SEGMENT = [
    # B, H, D, L, M, valid, wp, C, dtype, expected path
    (2, 2, 64, 128, 128, 128, 0, 1000, "bf16", 1),
    (2, 2, 41, 50, 90, 80, 7, 60, "bf16", 1),               # dense odd rows: copied for TMA
    (1, 2, 24, 33, 700, 700, 650, 1000, "bf16", 1),
    (1, 1, 96, 140, 1000, 990, 3, 500, "bf16", 1),
    (40, 8, 64, 20, 30, 30, 29, 1000, "bf16", 1),           # more heads than multiprocessors
    (1, 3, 64, 200, 300, 250, 77, 150, "bf16", 1),          # a ring write pointer no tile divides
    (1, 2, 64, 17, 40, 40, 39, 1000, "bf16", 1),
    (2, 2, 128, 100, 130, 130, 7, 1000, "bf16", 1),
    (1, 2, 64, 40, 64, 0, 5, 1000, "bf16", 1),              # nothing valid yet
    (1, 2, 64, 40, 0, 0, 0, 1000, "bf16", 1),
    (1, 2, 41, 30, 50, 50, 13, 1000, "f32", 6),
    (2, 2, 64, 32, 64, 64, 1, 1000, "f32", 6),              # whole tiles
    (1, 3, 64, 33, 1000, 990, 77, 300, "f32", 6),           # eight ranks, one query in the last tile
    (3, 2, 128, 17, 129, 129, 128, 50, "f32", 6),
    (1, 1, 8, 100, 300, 300, 299, 0, "f32", 6),
    (2, 1, 96, 65, 200, 1, 150, 1000, "f32", 6),
    (1, 2, 24, 70, 64, 0, 5, 1000, "f32", 6),               # nothing valid yet
    (1, 2, 64, 95, 0, 0, 0, 40, "f32", 6),
    (20, 8, 33, 20, 30, 30, 29, 1000, "f32", 6),            # more heads than multiprocessors
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("c", SEGMENT, ids=["B%dH%dD%d_L%dM%dv%dwp%dC%d_%s_p%d" % c for c in SEGMENT])
def test_segments_match_64_bits(txl, c, bits):
    """Longer segments: the fused kernels over the expanded memory in bf16, a kernel of its own for fp32."""
    B, H, D, L, M, valid, wp, C, dtype, path = c
    call = Call(txl, B, H, D, L, M, valid, wp, C, bits, dtype)
    assert txl.rel_attn_qmem_path(call.q, call.mem, call.k, call.v, call.r, call.out) == path
    call.run(txl)
    torch.cuda.synchronize()
    if dtype == "f32":
        check(call)
    else:
        check_segment(call)


def test_fp32_segment_sees_no_later_key(txl):
    """Keys and values of the segment that are NaN or infinite reach the queries from their position on."""
    call = Call(txl, 1, 2, 64, 50, 200, 200, 9, 1000, 4, "f32", hs=65, shift=1)
    ref, size, vmax = call.reference()
    call.k[:, 40:] = float("nan")
    call.v[:, 35:] = float("inf")
    call.run(txl)
    torch.cuda.synchronize()
    out = f64(call.out)
    tol = decode_tolerance(ref, size, vmax, call.dtype)
    assert (np.abs(out - ref) <= tol)[:, :35].all()
    assert np.isinf(out[:, 35:40]).all() and np.isnan(out[:, 40:]).all()


@pytest.mark.parametrize("factor", [1e-30, 1e-5, 1e5, 1e30])
def test_segment_values_of_any_magnitude(txl, factor):
    """V is held in fp16 in units taken from the data, so its size does not matter."""
    call = Call(txl, 2, 2, 64, 40, 300, 300, 9, 1000, 4, "bf16")
    call.vh = (call.vh * factor).to(torch.bfloat16)
    call.v.mul_(factor)
    call.mem.restore((9 - 300) % 300, 0)
    txl.qmem_push(call.mem, call.kh.cuda(), call.vh.cuda())
    call.run(txl)
    torch.cuda.synchronize()
    check_segment(call)


@pytest.mark.parametrize("factor", [1e-30, 1e-5, 1e5, 1e30])
def test_segment_keys_of_any_magnitude(txl, factor):
    """K likewise, with queries that bring the scores back to size."""
    call = Call(txl, 2, 2, 64, 40, 300, 300, 9, 1000, 8, "bf16")
    call.kh = (call.kh * factor).to(torch.bfloat16)
    call.k.mul_(factor)
    call.q.div_(factor)
    call.u.div_(factor)
    call.vb.div_(factor)
    call.r.mul_(factor)
    call.mem.restore((9 - 300) % 300, 0)
    txl.qmem_push(call.mem, call.kh.cuda(), call.vh.cuda())
    call.run(txl)
    torch.cuda.synchronize()
    check_segment(call)


@pytest.mark.parametrize("row", [0, 37, 138])
def test_segment_one_large_position_row(txl, row):
    """A table whose rows are all small but one."""
    call = Call(txl, 3, 2, 64, 40, 100, 100, 9, 1000, 4, "bf16")
    call.r.mul_(2.0 ** -20)
    call.r[row] *= 2.0 ** 20
    call.run(txl)
    torch.cuda.synchronize()
    check_segment(call)


def test_segment_with_an_unaligned_position_table(txl):
    call = Call(txl, 1, 2, 64, 40, 100, 100, 9, 1000, 8, "bf16")
    flat = torch.empty(call.r.numel() + 1, dtype=torch.bfloat16, device="cuda")
    flat[1:].copy_(call.r.reshape(-1))
    call.r = flat[1:].view(call.r.shape)
    assert txl.rel_attn_qmem_path(call.q, call.mem, call.k, call.v, call.r, call.out) == 1
    call.run(txl)
    torch.cuda.synchronize()
    check_segment(call)


@pytest.mark.parametrize("bits", [4, 8])
def test_generation_over_a_quantised_memory(txl, bits):
    """A prompt segment, then tokens one, three and one at a time, each attended before it is pushed;
    the ring wraps on the way.  Every output against the concatenated history in 64 bits."""
    B, H, D, M, C = 2, 2, 64, 48, 40
    g = torch.Generator().manual_seed(4)
    u, vb = (0.3 * randn(g, H, D).cuda() for _ in range(2))
    r = (0.7 * randn(g, C + 1, H, D)).bfloat16().cuda()
    mem = txl.QuantMemory.empty(B, M, H, D, bits=bits)
    kh, vh = [], []
    for step, L in enumerate([40] + [1] * 6 + [3] * 3 + [1] * 4 + [20] + [1] * 3):
        q, k, v = (randn(g, B, L, H, D).bfloat16() for _ in range(3))
        out = torch.empty(B, L, H, D, dtype=torch.bfloat16, device="cuda")
        txl.rel_attn_qmem(q.cuda(), mem, k.cuda(), v.cuda(), u, vb, r, C + 1, C, out)
        txl.qmem_push(mem, k.cuda(), v.cuda())
        torch.cuda.synchronize()
        hist = [np.concatenate([held(f64(x), bits) for x in h] + [f64(cur)], 1)[:, -(M + L):] if h else f64(cur)
                for h, cur in ((kh, k), (vh, v))]
        x = (f64(q), hist[0], hist[1], f64(u), f64(vb), f64(r), C)
        ref, size = attend64(*x)
        tol = decode_tolerance(ref, size, np.abs(hist[1]).max(), torch.bfloat16) if L <= 16 \
            else segment_tolerance(*x, ref)
        assert (np.abs(f64(out) - ref) <= tol).all(), step
        kh.append(k)
        vh.append(v)


def test_two_streams_and_repeated_calls_agree(txl):
    """Calls on two streams at once give what each gives alone, and the same call twice the same bits."""
    calls = [Call(txl, 4, 4, 64, 1, 1500, 1500, 100, 1000, 4, "bf16", seed=1),
             Call(txl, 2, 4, 128, 2, 900, 800, 3, 100, 8, "bf16", seed=2)]
    alone = []
    for c in calls:
        c.run(txl)
        torch.cuda.synchronize()
        alone.append(c.out.clone())
        c.out.fill_(float("nan"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for c, s in zip(calls, streams):
            c.run(txl, stream=s)
    torch.cuda.synchronize()
    for c, a in zip(calls, alone):
        assert torch.equal(c.out, a)


@pytest.mark.parametrize("L", [1, 16, 30])
def test_replayed_from_a_graph(txl, L):
    call = Call(txl, 2, 2, 64, L, 300, 300, 31, 1000, 4, "bf16")
    ws = torch.empty(max(16, txl.rel_attn_qmem_workspace_size(call.q, call.mem)), dtype=torch.uint8, device="cuda")
    call.run(txl, workspace=ws)
    torch.cuda.synchronize()
    first = call.out.clone()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call.run(txl, workspace=ws)
    q2 = call.q.flip(0).clone()
    for q, turned in ((call.q.clone(), False), (q2, True)):
        call.q.copy_(q)
        call.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        if not turned:
            assert torch.equal(call.out, first)
        check(call) if L <= 16 else check_segment(call)


FIRST_CALL = """
import sys, torch
sys.path.insert(0, %r)
import transformer_xl_relative_gb300 as txl
B, H, D, M, L, C = 1, 2, 64, 200, int(sys.argv[1]), 1000
k, q = (torch.randn(B, max(M, L), H, D, device="cuda").bfloat16() for _ in range(2))
u = torch.zeros(H, D, device="cuda")
r = torch.randn(M + L, H, D, device="cuda").bfloat16()
mem = txl.QuantMemory.empty(B, M, H, D)
outs = [torch.empty(B, L, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
ws = torch.empty(txl.rel_attn_qmem_workspace_size(q[:, :L], mem) + 1048576, dtype=torch.uint8, device="cuda")
g = torch.cuda.CUDAGraph()
def step(out):
    mem.restore(0, 0)
    txl.qmem_push(mem, k[:, :M], q[:, :M])
    txl.rel_attn_qmem(q[:, :L], mem, k[:, :L], k[:, :L], u, u, r, M + L, C, out, workspace=ws)
with torch.cuda.graph(g):
    step(outs[0])
mem.rows.zero_()
g.replay()
torch.cuda.synchronize()
step(outs[1])
torch.cuda.synchronize()
assert torch.equal(*outs) and torch.isfinite(outs[0]).all()
print("same")
"""


@pytest.mark.parametrize("L", [1, 40])
def test_the_first_call_of_a_process_may_be_captured(txl, L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", FIRST_CALL % root, str(L)], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and "same" in p.stdout, p.stderr[-2000:]


def test_workspaces_and_flags_elsewhere_are_refused(txl):
    call = Call(txl, 1, 2, 64, 1, 100, 100, 0, 1000, 4, "bf16")
    need = txl.rel_attn_qmem_workspace_size(call.q, call.mem)
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(need)):
        with pytest.raises(ValueError):
            call.run(txl, workspace=bad)
    for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int64, device="cuda"),
                torch.zeros(0, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            call.run(txl, err_flag=bad)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    call.run(txl, err_flag=flag)
    torch.cuda.synchronize()
    assert flag.item() == 0
    check(call)


def test_the_output_may_replace_the_queries(txl):
    for L in (1, 3, 16):
        call = Call(txl, 2, 2, 64, L, 3000, 3000, 50, 1000, 4, "bf16")
        ref, size, vmax = call.reference()
        call.out = call.q
        call.run(txl)
        torch.cuda.synchronize()
        assert (np.abs(f64(call.out) - ref) <= decode_tolerance(ref, size, vmax, call.dtype)).all()


def test_a_memory_past_four_gigabytes(txl):
    """64-bit offsets: 2 heads of 40 million slots, the valid ones at the far end of each."""
    M, D, bits, C = 40_000_000, 64, 8, 50
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    g = torch.Generator().manual_seed(9)
    rows = torch.empty(1, 2, M, 144, dtype=torch.uint8, device="cuda")
    mem = txl.QuantMemory(rows, D, bits, wp=M - 40, valid=0)
    kh, vh = (randn(g, 1, 100, 2, D).bfloat16() for _ in range(2))
    txl.qmem_push(mem, kh.cuda(), vh.cuda())
    q, k, v = (randn(g, 1, 1, 2, D).bfloat16() for _ in range(3))
    u, vb = (0.3 * randn(g, 2, D).cuda() for _ in range(2))
    r = (0.7 * randn(g, C + 1, 2, D)).bfloat16().cuda()
    out = torch.empty(1, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    txl.rel_attn_qmem(q.cuda(), mem, k.cuda(), v.cuda(), u, vb, r, C + 1, C, out)
    torch.cuda.synchronize()
    kk = np.concatenate((held(f64(kh), bits), f64(k)), 1)
    vv = np.concatenate((held(f64(vh), bits), f64(v)), 1)
    ref, size = attend64(f64(q), kk, vv, f64(u), f64(vb), f64(r), C)
    assert (np.abs(f64(out) - ref) <= decode_tolerance(ref, size, np.abs(vv).max(), torch.bfloat16)).all()
