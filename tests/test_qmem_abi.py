"""CPU tests of the quantised memory's entry points: sizes, kernel selection and refusals.  Nothing
here launches a kernel (every call is rejected, has nothing to do, or decides a path)."""
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


def qmem(native, B=2, M=128, H=4, D=64, bits=4, wp=0, valid=None, rows=FAKE):
    return native.TxlQmem(rows, B, M, H, D, bits, wp, M if valid is None else valid)


def dense(native, B, T, H, D, ptr=FAKE):
    return native.TxlView(ptr, T * H * D, H * D, D)


def test_row_sizes(native):
    """G groups take G * bits / 2 units of codes and ceil(G / 2) of parameters; never a multiple of eight."""
    row = native.load().txl_qmem_row_bytes
    assert row(64, 4) == 80 and row(64, 8) == 144 and row(41, 4) == 80
    assert row(32, 4) == 48 and row(1, 8) == 80
    assert row(96, 4) == 144 and row(96, 8) == 224                  # 8 units become 9; 14
    assert row(128, 4) == 160 and row(128, 8) == 288
    for bad in ((0, 4), (129, 4), (64, 3), (-1, 8)):
        assert row(*bad) == 0


MEM_ERRORS = [
    (dict(bits=5), "TXL_ERR_UNSUPPORTED"), (dict(D=129), "TXL_ERR_UNSUPPORTED"),
    (dict(rows=None), "TXL_ERR_INVALID_ARG"), (dict(wp=128), "TXL_ERR_INVALID_ARG"),
    (dict(wp=-1), "TXL_ERR_INVALID_ARG"), (dict(valid=129), "TXL_ERR_INVALID_ARG"),
    (dict(valid=-1), "TXL_ERR_INVALID_ARG"), (dict(M=-1, valid=0), "TXL_ERR_INVALID_ARG"),
    (dict(M=0, valid=1), "TXL_ERR_INVALID_ARG"), (dict(B=-1), "TXL_ERR_INVALID_ARG"),
    (dict(H=0), "TXL_ERR_INVALID_ARG"), (dict(D=0), "TXL_ERR_INVALID_ARG"),
    (dict(rows=FAKE + 8), "TXL_ERR_ALIGNMENT"),
    (dict(B=65536), "TXL_ERR_UNSUPPORTED"), (dict(H=65536), "TXL_ERR_UNSUPPORTED"),
]


@pytest.mark.parametrize("change,status", MEM_ERRORS, ids=["-".join(map(str, c)) + "-" + s for c, s in MEM_ERRORS])
def test_a_bad_memory_is_refused_everywhere(native, change, status):
    lib, want = native.load(), getattr(native, status)
    m = qmem(native, **change)
    before = (m.wp, m.valid)
    x = dense(native, 2, 8, 4, 64)
    assert lib.txl_qmem_push(ctypes.byref(m), ctypes.byref(x), ctypes.byref(x), 8, 1, None) == want
    assert (m.wp, m.valid) == before
    assert lib.txl_qmem_read(ctypes.byref(m), 0, 8, ctypes.byref(x), ctypes.byref(x), 1, None) == want
    q = dense(native, 2, 1, 4, 64)
    vs = [ctypes.byref(q)] * 2
    assert lib.txl_rel_attn_qmem_path(2, 1, 4, 64, ctypes.byref(q), ctypes.byref(m), *vs, FAKE, 64, ctypes.byref(q),
                                      1) == -want
    assert lib.txl_rel_attn_qmem(2, 1, 4, 64, 10, ctypes.byref(q), ctypes.byref(m), *vs, FAKE, FAKE, FAKE, 64, 11, 0.0,
                                 ctypes.byref(q), 1, None, 0, None, None) == want


def test_push_and_read_refusals(native):
    lib, E = native.load(), native
    m, x = qmem(native), dense(native, 2, 8, 4, 64)
    null = native.TxlView(None, 1, 1, 1)
    p = ctypes.byref
    assert lib.txl_qmem_push(None, p(x), p(x), 8, 1, None) == E.TXL_ERR_INVALID_ARG
    assert lib.txl_qmem_push(p(m), p(null), p(x), 8, 1, None) == E.TXL_ERR_INVALID_ARG
    assert lib.txl_qmem_push(p(m), p(x), p(x), -1, 1, None) == E.TXL_ERR_INVALID_ARG
    assert lib.txl_qmem_push(p(m), p(x), p(x), 8, 2, None) == E.TXL_ERR_INVALID_ARG
    assert lib.txl_qmem_push(p(m), p(x), p(x), 0, 1, None) == E.TXL_OK              # nothing to do
    empty = qmem(native, M=0)
    assert lib.txl_qmem_push(p(empty), p(x), p(x), 8, 1, None) == E.TXL_OK
    m = qmem(native, M=100, valid=60)
    for j0, n in ((39, 1), (99, 2), (40, 61), (-1, 1), (50, -1), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert lib.txl_qmem_read(p(m), j0, n, p(x), p(x), 1, None) == E.TXL_ERR_INVALID_ARG, (j0, n)
    assert lib.txl_qmem_read(p(m), 100, 0, p(x), p(x), 1, None) == E.TXL_OK
    assert lib.txl_qmem_read(p(m), 40, 1, p(null), p(x), 1, None) == E.TXL_ERR_INVALID_ARG
    assert lib.txl_qmem_read(p(m), 40, 1, p(x), p(x), 7, None) == E.TXL_ERR_INVALID_ARG


def attn(native, B=2, L=1, H=4, D=64, C=10, n_rows=11, dtype=1, ws=None, ws_bytes=0, u=FAKE, r=FAKE, ld_r=None, m=None,
         null=None):
    q = [dense(native, B, max(L, 1), H, D) for _ in range(4)]
    if null is not None:
        q[null] = native.TxlView(None, 1, 1, 1)
    p = ctypes.byref
    m = qmem(native) if m is None else m
    return native.load().txl_rel_attn_qmem(B, L, H, D, C, p(q[0]), p(m), p(q[1]), p(q[2]), u, FAKE, r, ld_r or D, n_rows,
                                           0.0, p(q[3]), dtype, ws, ws_bytes, None, None)


def test_attention_refusals(native):
    E = native
    assert attn(native, C=-1) == E.TXL_ERR_INVALID_ARG
    assert attn(native, n_rows=10) == E.TXL_ERR_INVALID_ARG                # distances 0 .. C need C + 1 rows
    assert attn(native, C=2 ** 31 - 1, n_rows=128) == E.TXL_ERR_INVALID_ARG   # M + L = 129 of them otherwise
    assert attn(native, u=None) == E.TXL_ERR_INVALID_ARG
    assert attn(native, r=None) == E.TXL_ERR_INVALID_ARG
    assert attn(native, ld_r=63) == E.TXL_ERR_INVALID_ARG
    assert attn(native, dtype=3) == E.TXL_ERR_INVALID_ARG
    assert attn(native, L=-1) == E.TXL_ERR_INVALID_ARG
    assert attn(native, D=130) == E.TXL_ERR_UNSUPPORTED
    for i in range(4):
        assert attn(native, null=i) == E.TXL_ERR_INVALID_ARG
    assert attn(native, B=3) == E.TXL_ERR_INVALID_ARG                      # the memory holds two entries
    assert attn(native, H=3) == E.TXL_ERR_INVALID_ARG
    assert attn(native, D=32) == E.TXL_ERR_INVALID_ARG
    assert attn(native, L=0) == E.TXL_OK
    big = qmem(native, M=2 ** 31 - 1, valid=5)
    assert attn(native, m=big) == E.TXL_ERR_UNSUPPORTED                    # M + L past 32 bits
    assert attn(native, m=qmem(native, M=2 ** 31 - 4097, valid=5)) == E.TXL_ERR_UNSUPPORTED
    assert attn(native, m=qmem(native, M=2 ** 31 - 4098, valid=5)) == E.TXL_ERR_WORKSPACE   # the first that is taken


def test_calls_need_their_workspace(native):
    lib, E = native.load(), native
    m = qmem(native)
    p = ctypes.byref
    need = ((2 * 128 + 3 * 17) * 2 + 128 + 17) * 4 * 64 * 2 + 2 * 4 * 144
    assert lib.txl_rel_attn_qmem_workspace_size(2, 17, 4, 64, p(m), 1) == need
    assert lib.txl_rel_attn_qmem_workspace_size(2, 17, 4, 64, p(m), 0) == 0
    assert lib.txl_rel_attn_qmem_workspace_size(2, 16, 4, 64, p(m), 1) == 2 * 4 * 16 * (148 + 1) * 4
    assert lib.txl_rel_attn_qmem_workspace_size(2, 1, 4, 64, None, 1) == 2 * 4 * 1 * (4 + 1) * 4
    assert lib.txl_rel_attn_qmem_workspace_size(2, 17, 4, 64, None, 1) == 0
    assert lib.txl_rel_attn_qmem_workspace_size(2, 17, 4, 41, p(qmem(native, D=41)), 1) == (need - 1152) // 64 * 48 + 1152
    assert attn(native, L=17) == E.TXL_ERR_WORKSPACE
    assert attn(native, L=1) == E.TXL_ERR_WORKSPACE
    assert attn(native, L=1, ws=FAKE, ws_bytes=2 * 4 * 1 * (132 + 1) * 4 - 1) == E.TXL_ERR_WORKSPACE
    assert attn(native, L=17, ws=FAKE, ws_bytes=need - 1) == E.TXL_ERR_WORKSPACE
    assert attn(native, L=17, ws=FAKE + 8, ws_bytes=need) == E.TXL_ERR_WORKSPACE


def test_path_selection(native):
    def path(L=1, D=64, dtype=1, m=None, ptr=FAKE, ld_r=None):
        m = qmem(native, D=D) if m is None else m
        q = dense(native, 2, L, 4, D, ptr)
        p = ctypes.byref
        return native.load().txl_rel_attn_qmem_path(2, L, 4, D, p(q), p(m), p(q), p(q), FAKE, ld_r or D, p(q), dtype)

    assert path() == 5 and path(L=16) == 5 and path(L=16, dtype=0) == 5 and path(D=41) == 5
    assert path(L=17) == 1                                             # read back, fused tcgen05 kernel
    assert path(L=200, m=qmem(native, M=300, wp=77, valid=250)) == 1   # whatever the ring's write pointer
    assert path(L=200, dtype=0) == 6                                   # fp32: CUDA cores
    assert path(L=200, D=41, ld_r=48) == 1                             # dense 82-byte rows are copied
    assert path(L=200, ptr=FAKE + 2) == 1                              # and so are misaligned ones
    assert path(L=200, m=qmem(native, valid=0)) == 1


def test_python_checks():
    import torch

    import transformer_xl_relative_gb300 as txl
    rows = torch.zeros(1, 2, 8, 80, dtype=torch.uint8)
    for bad in (lambda: txl.QuantMemory(rows, 64, 5), lambda: txl.QuantMemory(rows, 129, 4),
                lambda: txl.QuantMemory(rows, 64, 8), lambda: txl.QuantMemory(rows[0], 64, 4),
                lambda: txl.QuantMemory(rows.float(), 64, 4), lambda: txl.QuantMemory(rows.transpose(1, 2), 64, 4),
                lambda: txl.QuantMemory(rows, 64, 4)):                # the last: not on a CUDA device
        with pytest.raises(ValueError):
            bad()


def test_the_struct_form_reads_its_arguments(native):
    """txl_rel_attn_qmem_call with the packed arguments of the binding: the statuses of the long form."""
    q = (FAKE, 1 * 4 * 64, 4 * 64, 64)
    m = qmem(native)

    def call(B=2, n_rows=11, dtype=1, ws=FAKE, ws_bytes=1 << 20, r=FAKE, ld_r=64, L=1, mem=None, C=10):
        a = native.QMEM_ARGS.pack(B, L, 4, 64, C, n_rows, dtype, 0.0, *q, *q, *q, *q,
                                  ctypes.addressof(m) if mem is None else mem, FAKE, FAKE, r, ld_r, ws, ws_bytes, 0, 0)
        return native.load().txl_rel_attn_qmem_call(a)

    assert native.load().txl_rel_attn_qmem_call(None) == native.TXL_ERR_INVALID_ARG
    assert call(L=0) == native.TXL_OK
    assert call(B=3) == native.TXL_ERR_INVALID_ARG
    assert call(n_rows=10) == native.TXL_ERR_INVALID_ARG
    assert call(C=-1) == native.TXL_ERR_INVALID_ARG
    assert call(dtype=9) == native.TXL_ERR_INVALID_ARG
    assert call(r=0) == native.TXL_ERR_INVALID_ARG
    assert call(ld_r=63) == native.TXL_ERR_INVALID_ARG
    assert call(ws=0) == native.TXL_ERR_WORKSPACE
    assert call(ws=FAKE + 4) == native.TXL_ERR_WORKSPACE
    assert call(ws_bytes=100) == native.TXL_ERR_WORKSPACE


def test_the_struct_forms_of_push_and_read(native):
    """txl_qmem_push_call and txl_qmem_read_call with the packed arguments of the binding: the statuses of
    the long forms."""
    x = (FAKE, 1 * 4 * 64, 4 * 64, 64)
    m = qmem(native, valid=100)
    lib = native.load()

    def args(mem=None, k=x, v=x, j0=0, n=0, dtype=1):
        return native.QMEM_KV_ARGS.pack(ctypes.addressof(m) if mem is None else mem, *k, *v, j0, n, dtype, 0)

    for f in (lib.txl_qmem_push_call, lib.txl_qmem_read_call):
        assert f(None) == native.TXL_ERR_INVALID_ARG
        assert f(args(mem=0)) == native.TXL_ERR_INVALID_ARG
        assert f(args(k=(0, *x[1:]))) == native.TXL_ERR_INVALID_ARG
        assert f(args(v=(0, *x[1:]))) == native.TXL_ERR_INVALID_ARG
        assert f(args(n=-1, j0=28)) == native.TXL_ERR_INVALID_ARG
        assert f(args(dtype=9, j0=28)) == native.TXL_ERR_INVALID_ARG
        assert f(args(j0=28)) == native.TXL_OK                              # nothing to do
    assert lib.txl_qmem_read_call(args(j0=27)) == native.TXL_ERR_INVALID_ARG     # not valid yet
    assert lib.txl_qmem_read_call(args(j0=128, n=1)) == native.TXL_ERR_INVALID_ARG
