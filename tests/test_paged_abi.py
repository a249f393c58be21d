"""CPU tests of the paged memory's and the 4-bit weights' entry points: what they refuse, before anything is launched, and
the workspaces that they ask for."""
import ctypes
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 40          # an aligned address that is never dereferenced (host-side checks only)


@pytest.fixture(scope="module")
def native():
    spec = importlib.util.spec_from_file_location(
        "txl_build", os.path.join(ROOT, "transformer_xl_relative_gb300", "_build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.build()
    from transformer_xl_relative_gb300 import native as n
    n.load()
    return n


def paged(native, **kw):
    f = dict(k=FAKE, v=FAKE, pos=FAKE, weight=FAKE, table=FAKE, length=FAKE, next_pos=FAKE, scratch=FAKE, err_flag=None,
             B=2, H=4, D=41, ld=48, n_pages=10, page_len=16, max_pages=5, dtype=1)
    f.update(kw)
    return native.TxlPaged(*[f[n] for n, _ in native.TxlPaged._fields_])


BAD_MEMORIES = [
    (dict(B=-1), "INVALID_ARG"), (dict(H=0), "INVALID_ARG"), (dict(D=0), "INVALID_ARG"), (dict(ld=40), "INVALID_ARG"),
    (dict(n_pages=-1), "INVALID_ARG"), (dict(page_len=0), "INVALID_ARG"), (dict(max_pages=-1), "INVALID_ARG"),
    (dict(dtype=2), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(weight=None), "INVALID_ARG"),
    (dict(table=None), "INVALID_ARG"), (dict(length=None), "INVALID_ARG"), (dict(scratch=None), "INVALID_ARG"),
    (dict(D=129, ld=136), "UNSUPPORTED"), (dict(page_len=24), "UNSUPPORTED"), (dict(B=4097), "UNSUPPORTED"),
    (dict(H=65536), "UNSUPPORTED"), (dict(ld=65544), "UNSUPPORTED"), (dict(n_pages=1 << 28), "UNSUPPORTED"), (dict(max_pages=1 << 28), "UNSUPPORTED"),
    (dict(ld=44), "ALIGNMENT"), (dict(k=FAKE + 8), "ALIGNMENT"), (dict(pos=FAKE + 4), "ALIGNMENT"),
    (dict(length=FAKE + 2), "ALIGNMENT"), (dict(err_flag=FAKE + 1), "ALIGNMENT"),
]


def status(native, name):
    return getattr(native, "TXL_ERR_" + name)


def push(native, mem, T=3, k=FAKE, v=FAKE, counts=None):
    V = native.TxlView
    return native.load().txl_paged_push(ctypes.byref(mem) if mem is not None else None, ctypes.byref(V(k, 1, 1, 1)),
                                        ctypes.byref(V(v, 1, 1, 1)), T, counts, None)


def attn(native, mem, T=2, clamp=5, n_rows=6, q=FAKE, k=FAKE, v=FAKE, out=FAKE, counts=0, u=FAKE, vb=FAKE, r=FAKE, ld_r=48,
         ws=FAKE, nbytes=1 << 40, accumulate=0):
    args = native.PAGED_ARGS.pack(T, clamp, n_rows, accumulate, 0.0, ctypes.addressof(mem) if mem is not None else 0,
                                  q, 1, 1, 1, k, 1, 1, 1, v, 1, 1, 1, out, 1, 1, 1, counts, u, vb, r, ld_r, ws, nbytes, 0)
    return native.load().txl_rel_attn_paged(args)


@pytest.mark.parametrize("change,name", BAD_MEMORIES)
def test_memories_that_are_refused(native, change, name):
    mem = paged(native, **change)
    assert push(native, mem) == status(native, name)
    assert attn(native, mem) == status(native, name)
    assert native.load().txl_paged_evict(ctypes.byref(mem), 4, 0, FAKE, 1 << 40, None) == status(native, name)


def test_nothing_to_do(native):
    lib = native.load()
    assert push(native, paged(native), T=0) == native.TXL_OK
    assert push(native, paged(native, B=0)) == native.TXL_OK
    assert attn(native, paged(native), T=0) == native.TXL_OK
    assert attn(native, paged(native, B=0)) == native.TXL_OK
    assert lib.txl_paged_evict(ctypes.byref(paged(native)), 80, 0, None, 0, None) == native.TXL_OK   # holds 80 at most
    w = native.TxlQ4(FAKE, 64, 64, 64)
    assert lib.txl_linear_q4(0, ctypes.byref(w), FAKE, 64, FAKE, 64, None, 0, None, None) == native.TXL_OK


def test_calls_that_are_refused(native):
    mem = paged(native)
    invalid, unsupported, alignment, workspace = (status(native, n) for n in ("INVALID_ARG", "UNSUPPORTED", "ALIGNMENT",
                                                                              "WORKSPACE"))
    assert push(native, None) == invalid and push(native, mem, T=-1) == invalid and push(native, mem, k=None) == invalid
    assert push(native, mem, counts=FAKE + 2) == alignment and push(native, mem, k=FAKE + 1) == alignment
    assert push(native, paged(native, dtype=0, ld=44), v=FAKE + 2) == alignment
    for kw in (dict(T=-1), dict(clamp=-1), dict(n_rows=0), dict(q=0), dict(out=0), dict(k=0), dict(v=0), dict(u=0),
               dict(vb=0), dict(r=0), dict(ld_r=40)):
        assert attn(native, mem, **kw) == invalid, kw
    assert attn(native, None) == invalid
    assert attn(native, mem, T=17) == unsupported and attn(native, mem, ld_r=1 << 30) == unsupported
    assert attn(native, mem, n_rows=(1 << 31) - 1, clamp=(1 << 31) - 1) == unsupported
    for kw in (dict(q=FAKE + 1), dict(r=FAKE + 1), dict(u=FAKE + 2), dict(counts=FAKE + 1), dict(ws=FAKE + 8)):
        assert attn(native, mem, **kw) == alignment, kw
    need = native.load().txl_rel_attn_paged_workspace_size(ctypes.byref(mem), 2, 6, 0)
    assert need > 0 and attn(native, mem, nbytes=need - 1) == workspace and attn(native, mem, ws=0) == workspace
    more = native.load().txl_rel_attn_paged_workspace_size(ctypes.byref(mem), 2, 6, 1)
    assert more >= need + 2 * 4 * 2 * 80 * 4 and attn(native, mem, nbytes=more - 1, accumulate=1) == workspace
    lib = native.load()
    for keep, recent in ((0, 0), (-3, 0), (5, -1), (5, 6)):
        assert lib.txl_paged_evict(ctypes.byref(mem), keep, recent, FAKE, 1 << 40, None) == invalid
    need = lib.txl_paged_evict_workspace_size(ctypes.byref(mem))
    assert lib.txl_paged_evict(ctypes.byref(mem), 5, 1, FAKE, need - 1, None) == workspace
    assert lib.txl_paged_evict(ctypes.byref(mem), 5, 1, FAKE + 4, need, None) == alignment


def test_workspaces_of_shapes_that_are_refused(native):
    lib = native.load()
    mem = paged(native)
    assert lib.txl_rel_attn_paged_workspace_size(None, 1, 1, 0) == 0
    for T, n in ((0, 1), (17, 1), (1, 0), (1, -5)):
        assert lib.txl_rel_attn_paged_workspace_size(ctypes.byref(mem), T, n, 0) == 0
    assert lib.txl_paged_evict_workspace_size(None) == 0


def test_four_bit_weights(native):
    lib = native.load()
    assert lib.txl_q4_bytes(64, 64, 64) == 2048 + 256
    assert lib.txl_q4_bytes(410, 1230, 64) == 20 * 7 * 2048 + 20 * 7 * 256
    assert lib.txl_q4_bytes(65, 65, 32) == 2 * 2 * 2048 + 2 * 3 * 256
    for k, n, g in ((0, 1, 64), (1, 0, 64), (1, 1, 16), (1, 1, 0), ((1 << 21) + 1, 1, 64), (1, (1 << 21) + 1, 64)):
        assert lib.txl_q4_bytes(k, n, g) == 0
        w = native.TxlQ4(FAKE, k, n, g)
        assert lib.txl_q4_quantise(ctypes.byref(w), FAKE, 1 << 22, None) == native.TXL_ERR_INVALID_ARG
    w = native.TxlQ4(FAKE, 64, 32, 64)
    call = lambda m=1, w=w, X=FAKE, ldx=64, Y=FAKE, ldy=32, ws=None, size=0: lib.txl_linear_q4(
        m, ctypes.byref(w), X, ldx, Y, ldy, ws, size, None, None)
    assert call(m=-1) == native.TXL_ERR_INVALID_ARG and call(X=None) == native.TXL_ERR_INVALID_ARG
    assert call(ldx=63) == native.TXL_ERR_INVALID_ARG and call(ldy=31) == native.TXL_ERR_INVALID_ARG
    assert call(w=native.TxlQ4(None, 64, 32, 64)) == native.TXL_ERR_INVALID_ARG
    assert call(w=native.TxlQ4(FAKE + 8, 64, 32, 64)) == native.TXL_ERR_ALIGNMENT
    assert call(X=FAKE + 1) == native.TXL_ERR_ALIGNMENT and call(m=(1 << 19) + 1) == native.TXL_ERR_UNSUPPORTED
    assert lib.txl_linear_q4_workspace_size(128, ctypes.byref(w)) == 0
    need = lib.txl_linear_q4_workspace_size(129, ctypes.byref(w))
    assert need == 64 * 32 * 2
    assert call(m=129) == native.TXL_ERR_WORKSPACE and call(m=129, ws=FAKE, size=need - 1) == native.TXL_ERR_WORKSPACE
    assert call(m=129, ws=FAKE + 2, size=need) == native.TXL_ERR_ALIGNMENT
    assert lib.txl_q4_quantise(ctypes.byref(w), FAKE, 31, None) == native.TXL_ERR_INVALID_ARG
    assert lib.txl_q4_quantise(ctypes.byref(w), FAKE + 1, 32, None) == native.TXL_ERR_ALIGNMENT
    assert lib.txl_q4_expand(ctypes.byref(w), None, 32, None) == native.TXL_ERR_INVALID_ARG


def test_the_binding_refuses_what_is_not_on_a_device(native):
    import torch
    import transformer_xl_relative_gb300 as txl
    with pytest.raises(ValueError):
        txl.PagedMemory.empty(2, 4, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        txl.QuantWeight.quantise(torch.zeros(64, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        txl.QuantWeight.quantise(torch.zeros(64, 64))


def test_what_an_earlier_kernel_may_write_is_not_read_through_the_read_only_path():
    """The kernels may start before those in front of them have ended: nothing they read is read-only while they run."""
    import re
    csrc = os.path.join(ROOT, "transformer_xl_relative_gb300", "csrc")
    for name in ("txl_paged.cu", "txl_paged.cuh", "txl_paged_attn.cu", "txl_linear_q4.cu"):
        text = re.sub(r"//.*", "", open(os.path.join(csrc, name), encoding="utf-8").read())
        assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", text), name
