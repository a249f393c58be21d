"""GPU tests of the quantised K/V memory: txl_qmem_push and txl_qmem_read against the definition in
64-bit and rational arithmetic.  Codes and parameters are compared exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from qmem_common import f64, held, parse, quantise64, quantise_exact

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def txl():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import transformer_xl_relative_gb300 as m
    return m


def tensor(shape, dtype, seed, layout="dense"):
    """[B, T, H, D] on the device in one of the layouts callers use."""
    B, T, H, D = shape
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, H, D, generator=g).to(DT[dtype]).cuda()
    if layout == "dense":
        return x
    if layout == "padded":                             # heads a multiple of 8 elements apart
        hs = (D + 7) // 8 * 8 + 8
        store = torch.full((B, T, H, hs), float("nan"), dtype=x.dtype, device="cuda")
    elif layout == "headmajor":                        # [B, H, T, D] storage
        store = torch.empty(B, H, T, D, dtype=x.dtype, device="cuda").permute(0, 2, 1, 3)
    elif layout == "shifted":                          # one element off 16-byte alignment
        flat = torch.full((B * T * H * D + 9,), float("nan"), dtype=x.dtype, device="cuda")
        store = flat[1:1 + B * T * H * D].view(B, T, H, D)
    view = store[..., :D]
    view.copy_(x)
    return view


def fresh(txl, B, M, H, D, bits, wp=0, valid=0, fill=0xA5):
    """A memory whose rows hold a pattern, so that untouched bytes show."""
    mem = txl.QuantMemory.empty(B, M, H, D, bits=bits)
    mem.rows.fill_(fill)
    mem.restore(wp, valid)
    return mem


def expect_slots(mem, x, which, slots, bits):
    """Codes and parameters of x [B, n, H, D] in the given slots."""
    code, step, lo = quantise64(f64(x).transpose(0, 2, 1, 3), bits)
    k, v, rest = parse(mem.rows[:, :, slots], x.shape[-1], bits)
    got = k if which == "k" else v
    np.testing.assert_array_equal(got[0], code)
    np.testing.assert_array_equal(got[1], step)
    np.testing.assert_array_equal(got[2], lo)
    assert (rest == 0).all()


PUSH = [
    # B, H, D, L, M, wp, dtype, layout
    (2, 3, 64, 7, 16, 0, "bf16", "dense"),
    (1, 1, 64, 1, 1, 0, "bf16", "dense"),              # one slot
    (2, 2, 64, 1, 9, 8, "bf16", "headmajor"),          # one token into the last slot
    (2, 2, 41, 20, 24, 13, "bf16", "padded"),          # wraps, odd D
    (2, 2, 41, 20, 24, 13, "f32", "shifted"),
    (1, 3, 128, 50, 33, 5, "bf16", "dense"),           # more positions than slots
    (1, 2, 128, 33, 33, 32, "f32", "dense"),
    (3, 2, 1, 5, 6, 2, "bf16", "dense"),
    (1, 2, 31, 5, 6, 2, "f32", "headmajor"),
    (1, 2, 33, 5, 6, 2, "bf16", "shifted"),
    (1, 2, 80, 9, 10, 4, "bf16", "dense"),
    (2, 2, 96, 9, 10, 4, "f32", "padded"),
    (1, 2, 24, 300, 301, 77, "bf16", "shifted"),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("c", PUSH, ids=["B%dH%dD%d_L%dM%dwp%d_%s_%s" % c for c in PUSH])
def test_push_holds_the_definition(txl, c, bits):
    B, H, D, L, M, wp, dtype, layout = c
    k, v = tensor((B, L, H, D), dtype, 1, layout), tensor((B, L, H, D), dtype, 2, layout)
    mem = fresh(txl, B, M, H, D, bits, wp, valid=min(2, M))
    txl.qmem_push(mem, k, v)
    torch.cuda.synchronize()
    n = min(L, M)
    slots = [(wp + t) % M for t in range(L - n, L)]
    expect_slots(mem, k[:, L - n:], "k", slots, bits)
    expect_slots(mem, v[:, L - n:], "v", slots, bits)
    assert mem.state() == ((wp + L) % M, min(min(2, M) + L, M))
    rest = [s for s in range(M) if s not in slots]
    if rest:
        assert (mem.rows[:, :, rest] == 0xA5).all()


def special_groups():
    """Groups where rounding, range or cancellation goes to an edge (fp32 values)."""
    rng = np.random.default_rng(5)
    f = np.float32
    out = []
    out.append(np.zeros(32, f))
    out.append(np.full(32, 1.7, f))                                    # constant, not a bf16 value
    out.append(np.full(32, -3.0, f))
    out.append(np.array([-0.0, 0.0] * 16, f))
    for n in (15, 255):                                                # exact ties, every one of them
        out.append(((np.arange(32) % n) + 0.5).astype(f) * f(0.25) + np.where(np.arange(32) == 0, -0.125, 0).astype(f))
        t = (np.arange(32) * (n / 31)).astype(f)
        t[0], t[1] = 0, n
        t[2:] = np.floor(t[2:]) + 0.5
        out.append(t)
        out.append(np.nextafter(t, f(0)).astype(f))                    # one step off the ties
        out.append(np.nextafter(t, f(1e9)).astype(f))
        u = t.copy()
        u[0] = f(-1e-30)                                               # the minimum vanishes in x - lo
        out.append(u)
        u = t.copy()
        u[0] = f(1e-30)
        out.append(u)
    out.append((rng.standard_normal(32) * 1e-42).astype(f))            # subnormals
    out.append((rng.standard_normal(32) * 1e-37).astype(f))
    out.append((rng.standard_normal(32) * 5e37).astype(f))
    out.append(np.array([1e38, -1e38] + [1e-30] * 30, f))
    out.append(np.array([1.0 + 2.0 ** -23] + [1.0] * 31, f))           # the smallest range above 1
    out.append(np.array([1.0 - 2.0 ** -24] + [1.0] * 31, f))
    out.append(np.exp(rng.uniform(-60, 60, 32)).astype(f))             # many magnitudes
    out.append((np.exp(rng.uniform(-20, 20, 32)) * rng.choice([-1, 1], 32)).astype(f))
    for _ in range(40):
        out.append((rng.standard_normal(32) * np.exp(rng.uniform(-40, 40))).astype(f))
        # multiples of a bf16 step around a bf16 minimum: many exact ties
        st = f(rng.integers(128, 256)) * f(2.0) ** f(rng.integers(-20, 20))
        out.append((rng.integers(0, 31, 32) * st * f(0.5) - st).astype(f))
    return np.stack(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
def test_push_at_the_edges(txl, dtype, bits):
    x = torch.from_numpy(special_groups()).to(DT[dtype])
    n = x.shape[0]
    ref = [quantise_exact(row, bits) for row in x.double().numpy()]
    k = x.view(1, n, 1, 32).cuda()
    mem = fresh(txl, 1, n, 1, 32, bits)
    txl.qmem_push(mem, k, k)
    torch.cuda.synchronize()
    for codes, steps, los in parse(mem.rows[0, 0], 32, bits)[:2]:
        for i, (code, step, lo) in enumerate(ref):
            assert steps[i, 0] == step and los[i, 0] == lo, (i, steps[i], step, los[i], lo)
            np.testing.assert_array_equal(codes[i], code, err_msg=str((i, x[i])))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
def test_groups_that_are_not_finite_read_back_as_nan(txl, dtype, bits):
    big = float(torch.finfo(DT[dtype]).max)
    x = torch.randn(1, 8, 1, 64, generator=torch.Generator().manual_seed(3))
    x[0, 0, 0, 5] = float("nan")
    x[0, 1, 0, 40] = float("inf")
    x[0, 2, 0, 0] = float("-inf")
    x[0, 3, 0, 0], x[0, 3, 0, 1] = big, -big          # the range is not finite
    x = x.to(DT[dtype]).cuda()
    mem = fresh(txl, 1, 8, 1, 64, bits)
    txl.qmem_push(mem, x, x.flip(1))
    k = torch.zeros(1, 8, 1, 64, dtype=torch.float32, device="cuda")
    v = torch.zeros_like(k)
    txl.qmem_read(mem, 0, 8, k, v)
    k, v = f64(k)[0, :, 0], f64(v)[0, ::-1, 0]
    want = {(0, 0), (1, 1), (2, 0), (3, 0)}
    for t in range(8):
        for g in range(2):
            for y in (k, v):
                part = y[t, 32 * g:32 * g + 32]
                if (t, g) in want:
                    assert np.isnan(part).all()
                else:
                    np.testing.assert_array_equal(part, held(f64(x)[0, t, 0], bits)[32 * g:32 * g + 32].astype(np.float32))


READ = [
    # B, H, D, M, valid, wp, j0, n, dtype out, layout
    (2, 3, 64, 40, 40, 0, 0, 40, "bf16", "dense"),
    (2, 3, 64, 40, 33, 17, 7, 33, "f32", "dense"),     # wraps, partly valid
    (1, 2, 41, 20, 20, 19, 3, 11, "bf16", "padded"),
    (1, 2, 41, 20, 20, 19, 3, 1, "f32", "shifted"),
    (2, 1, 128, 9, 9, 4, 8, 1, "bf16", "headmajor"),
    (1, 2, 96, 300, 300, 123, 0, 300, "bf16", "shifted"),
    (1, 2, 1, 5, 5, 2, 1, 3, "f32", "dense"),
]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("c", READ, ids=["B%dH%dD%d_M%dv%dwp%d_j%dn%d_%s_%s" % c for c in READ])
def test_read_returns_what_is_held(txl, c, bits):
    """The value lo + step c rounded once: fp32 within half a step of fp32; bf16 within half a step of
    bf16 and one of fp32 (the fused multiply-add rounds to fp32 first)."""
    B, H, D, M, valid, wp, j0, n, dtype, layout = c
    k, v = tensor((B, valid, H, D), "bf16", 1), tensor((B, valid, H, D), "bf16", 2)
    mem = fresh(txl, B, M, H, D, bits, (wp - valid) % M)
    txl.qmem_push(mem, k, v)
    assert mem.state() == (wp % M, valid)
    ko, vo = tensor((B, n, H, D), dtype, 3, layout), tensor((B, n, H, D), dtype, 4, layout)
    txl.qmem_read(mem, j0, n, ko, vo)
    torch.cuda.synchronize()
    f = j0 - (M - valid)
    for got, x in ((ko, k), (vo, v)):
        ref = held(f64(x), bits)[:, f:f + n]
        tol = (torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -23) * np.abs(ref)
        assert (np.abs(f64(got) - ref) <= tol).all()
    if layout == "padded":                             # the gaps between heads stay
        store = torch.as_strided(ko, (B, n, H, ko.stride(2) - D), ko.stride(), ko.storage_offset() + D)
        assert torch.isnan(store[:, :, :-1]).all()


def test_a_memory_past_four_gigabytes(txl):
    """Offsets of rows need 64 bits: 2 heads of 40 million slots of 144 bytes."""
    M, D, bits = 40_000_000, 64, 8
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    rows = torch.empty(1, 2, M, 144, dtype=torch.uint8, device="cuda")
    mem = txl.QuantMemory(rows, D, bits, wp=M - 40, valid=0)
    k, v = tensor((1, 100, 2, D), "bf16", 1), tensor((1, 100, 2, D), "bf16", 2)
    txl.qmem_push(mem, k, v)
    assert mem.state() == (60, 100)
    ko, vo = torch.empty_like(k).float(), torch.empty_like(v).float()
    txl.qmem_read(mem, M - 100, 100, ko, vo)
    torch.cuda.synchronize()
    for got, x in ((ko, k), (vo, v)):
        np.testing.assert_allclose(f64(got), held(f64(x), bits), rtol=2.0 ** -23)


def test_push_and_read_replayed_from_a_graph(txl):
    """A captured push writes the slots it was captured with; the inputs may change between replays."""
    B, H, D, L, M, bits = 2, 2, 64, 5, 12, 4
    mem = fresh(txl, B, M, H, D, bits, wp=10)
    k, v = tensor((B, L, H, D), "bf16", 1), tensor((B, L, H, D), "bf16", 2)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        txl.qmem_push(mem, k, v)
        mem.restore(10, 0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            txl.qmem_push(mem, k, v)
            txl.qmem_read(mem, M - L, L, ko, vo)
    torch.cuda.synchronize()
    for seed in (7, 8):
        k.copy_(tensor((B, L, H, D), "bf16", seed))
        v.copy_(tensor((B, L, H, D), "bf16", seed + 10))
        g.replay()
        torch.cuda.synchronize()
        for got, x in ((ko, k), (vo, v)):
            ref = held(f64(x), bits)
            assert (np.abs(f64(got) - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref)).all()
