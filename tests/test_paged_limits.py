"""CPU tests of the paged memory's and the 4-bit weights' entry points at the ends of their ranges: empty batches, the most
slots, and workspaces against what a memory holds."""
import ctypes

import pytest

from test_paged_abi import FAKE, attn, native, paged, push  # noqa: F401  (`native` is the fixture)


def test_no_rows_through_the_codes(native):  # noqa: F811
    """An empty tensor has no address: a product of no rows is done all the same, and the shape is still checked."""
    lib = native.load()
    w = native.TxlQ4(FAKE, 64, 32, 64)
    call = lambda **kw: lib.txl_linear_q4(*{**dict(m=0, w=ctypes.byref(w), X=None, ldx=64, Y=None, ldy=32, ws=None, size=0,
                                                   err=None, stream=None), **kw}.values())
    assert call() == native.TXL_OK
    assert call(ldx=63) == native.TXL_ERR_INVALID_ARG and call(ldy=31) == native.TXL_ERR_INVALID_ARG
    assert call(m=1) == native.TXL_ERR_INVALID_ARG and call(m=1, X=FAKE) == native.TXL_ERR_INVALID_ARG
    assert call(w=ctypes.byref(native.TxlQ4(None, 64, 32, 64))) == native.TXL_ERR_INVALID_ARG


def test_no_sequences(native):  # noqa: F811
    """A memory of no sequences, whose tensors have no addresses."""
    mem = paged(native, B=0, table=None, length=None, next_pos=None)
    assert push(native, mem, T=3, k=None, v=None) == native.TXL_OK
    assert attn(native, mem, q=0, k=0, v=0, out=0) == native.TXL_OK
    assert push(native, mem, T=-1, k=None, v=None) == native.TXL_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["n_pages", "max_pages"])
def test_the_most_slots(native, name):  # noqa: F811
    """Slots are counted in 32 bits, ahead of the last one too: the last 2^20 below 2^31 are refused, before any launch."""
    mem = paged(native, page_len=1 << 20, **{name: (1 << 11) - 1})
    for st in (push(native, mem), attn(native, mem),
               native.load().txl_paged_evict(ctypes.byref(mem), 4, 0, FAKE, 1 << 40, None)):
        assert st == native.TXL_ERR_UNSUPPORTED
    # one page less is taken: the call ends at the workspace, which is the next thing that it looks at
    mem = paged(native, page_len=1 << 20, **{name: (1 << 11) - 2})
    assert attn(native, mem, ws=0) == native.TXL_ERR_WORKSPACE
    assert push(native, paged(native), T=(1 << 31) - (1 << 20)) == native.TXL_ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [1, 2, 16])
@pytest.mark.parametrize("B,n_pages,page_len,max_pages", [(32, 2112, 64, 2112), (8, 10, 16, 10), (4096, 5000, 16, 300), (3, 100, 32, 4)])
def test_scores_take_no_more_than_the_memory_has_slots(native, T, B, n_pages, page_len, max_pages):  # noqa: F811
    """The scores that `accumulate` keeps: one for each head, query and slot, of the pool or of all rows of the table, whichever
    are fewer (a wide table, as an empty memory has by default, does not multiply the pool by the batch)."""
    mem = paged(native, B=B, n_pages=n_pages, page_len=page_len, max_pages=max_pages)
    size = native.load().txl_rel_attn_paged_workspace_size
    scores = size(ctypes.byref(mem), T, 6, 1) - size(ctypes.byref(mem), T, 6, 0)
    slots = min(n_pages, B * max_pages) * page_len
    assert 0 <= scores - (slots + B) * 4 * T * 4 < 64            # (a log-sum-exp for each head and query of a sequence)
