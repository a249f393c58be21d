"""Python binding of libtxl.so over torch CUDA tensors.

Argument marshalling only: every function converts tensors to pointers and element strides and
calls the C ABI of the same name; all computation happens in the library's CUDA kernels.  Torch
provides device memory and streams.  Tensors are [B, T, H, D] views whose last dimension is
contiguous; r is [n_rows, H, ld_r].
"""
from __future__ import annotations

import ctypes

import torch

from . import native
from .native import TxlMem, TxlPaged, TxlQ4, TxlQmem, TxlView, check

_DTYPES = {torch.float32: native.TXL_F32, torch.bfloat16: native.TXL_BF16}


def _lib():
    return native.load()


def dtype_code(t: torch.Tensor) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError("libtxl computes in float32 or bfloat16, got %s" % t.dtype) from None


def view(t: torch.Tensor) -> TxlView:
    """[B, T, H, D] tensor with contiguous D -> txl_view."""
    if t.dim() != 4:
        raise ValueError("expected a [B, T, H, D] tensor, got shape %s" % (tuple(t.shape),))
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("the last (d) dimension must be contiguous")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    return TxlView(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _raw_stream(stream, device: int) -> int:
    """cudaStream_t of `stream`, or of the current stream of CUDA device `device`."""
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


def _on_device(device: int, call, args):
    """call(args) with CUDA device `device` current (the library launches on the current device)."""
    if device == torch._C._cuda_getDevice():
        return call(args)
    with torch.cuda.device(device):
        return call(args)


class Memory:
    """K/V memory of M positions per batch entry (FIFO ring, or a plain contiguous memory).

    ``k`` and ``v`` are [B, M, H, D] tensors (same strides).  ``wp``/``valid`` follow txl_mem:
    logical memory key j lives in slot (wp + j) mod M and is valid iff j >= M - valid.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, wp: int = 0, valid: int = 0):
        if k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must share shape, strides and dtype")
        self.k, self.v = k, v
        B, M, H, D = k.shape
        self._c = TxlMem(k.data_ptr() if M else None, v.data_ptr() if M else None,
                         k.stride(0), k.stride(1), k.stride(2), B, M, H, D, dtype_code(k), wp, valid)

    @classmethod
    def empty(cls, B, M, H, D, dtype=torch.bfloat16, device="cuda", head_stride=None):
        hs = head_stride or D
        store = torch.zeros(B, M, H, hs, dtype=dtype, device=device)
        store2 = torch.zeros(B, M, H, hs, dtype=dtype, device=device)
        return cls(store[..., :D], store2[..., :D], 0, 0)

    @classmethod
    def full(cls, k: torch.Tensor, v: torch.Tensor):
        """A contiguous memory, oldest position first, every slot valid."""
        return cls(k, v, 0, k.shape[1])

    @property
    def M(self) -> int:
        return self._c.M

    @property
    def wp(self) -> int:
        return self._c.wp

    @property
    def valid(self) -> int:
        return self._c.valid

    def state(self):
        """Host ring state (wp, valid): with the buffers, everything needed to resume."""
        return self._c.wp, self._c.valid

    def restore(self, wp: int, valid: int) -> None:
        self._c.wp, self._c.valid = int(wp), int(valid)

    @property
    def c_struct(self) -> TxlMem:
        return self._c


def rel_pos_gen(W_R: torch.Tensor, r: torch.Tensor, n_rows: int, d_model: int, n_head: int,
                d_head: int, stream=None) -> torch.Tensor:
    """r[delta, h, d] = sum_m R_delta[m] W_R[m, h*d_head + d] for delta < n_rows (txl_rel_pos_gen)."""
    if W_R.dim() != 2 or W_R.stride(1) != 1 or r.dim() != 3 or r.stride(2) != 1:
        raise ValueError("W_R must be [d_model, ld_w] and r [n_rows, H, ld_r] with unit last stride")
    if r.stride(1) * n_head != r.stride(0) and r.shape[0] > 1:
        raise ValueError("r rows must be n_head * ld_r elements apart")
    st = _lib().txl_rel_pos_gen(n_rows, d_model, n_head, d_head, W_R.data_ptr(), W_R.stride(0),
                                r.data_ptr(), r.stride(1), dtype_code(W_R), _stream(stream))
    check(st, "txl_rel_pos_gen")
    return r


def _attn_args(q, mem, k_cur, v_cur, r, out):
    B, L, H, D = q.shape
    memc = ctypes.byref(mem.c_struct) if mem is not None else None
    return (B, L, H, D), memc, view(q), view(k_cur), view(v_cur), view(out)


def rel_attn_fwd(q: torch.Tensor, mem: Memory | None, k_cur: torch.Tensor, v_cur: torch.Tensor,
                 u: torch.Tensor, v_bias: torch.Tensor, r: torch.Tensor, n_rows: int,
                 clamp_len: int, out: torch.Tensor, scale: float = 0.0,
                 err_flag: torch.Tensor | None = None, stream=None, lse: torch.Tensor | None = None) -> torch.Tensor:
    """One relative-attention call over [memory ++ current] (txl_rel_attn_fwd).  With `lse` (fp32
    [B, L, H]) the call also saves every row's log-sum-exp for rel_attn_bwd (txl_rel_attn_fwd_lse)."""
    (B, L, H, D), memc, vq, vk, vv, vo = _attn_args(q, mem, k_cur, v_cur, r, out)
    if u.dtype != torch.float32 or v_bias.dtype != torch.float32:
        raise TypeError("u and v_bias are fp32 [H, D]")
    if not (u.is_contiguous() and v_bias.is_contiguous()):
        raise ValueError("u and v_bias must be contiguous [H, D]")
    ef = err_flag.data_ptr() if err_flag is not None else None
    if lse is not None:
        _check_lse(lse, B, L, H)
        st = _lib().txl_rel_attn_fwd_lse(
            B, L, H, D, int(clamp_len), ctypes.byref(vq), memc, ctypes.byref(vk), ctypes.byref(vv),
            u.data_ptr(), v_bias.data_ptr(), r.data_ptr(), r.stride(1), int(n_rows), float(scale),
            ctypes.byref(vo), lse.data_ptr(), dtype_code(q), None, 0, ef, _stream(stream))
        check(st, "txl_rel_attn_fwd_lse")
        return out
    st = _lib().txl_rel_attn_fwd(
        B, L, H, D, int(clamp_len), ctypes.byref(vq), memc, ctypes.byref(vk), ctypes.byref(vv),
        u.data_ptr(), v_bias.data_ptr(), r.data_ptr(), r.stride(1), int(n_rows), float(scale),
        ctypes.byref(vo), dtype_code(q), None, 0, ef, _stream(stream))
    check(st, "txl_rel_attn_fwd")
    return out


def _check_lse(lse: torch.Tensor, B: int, L: int, H: int) -> None:
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, L, H) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, L, H] tensor")


def rel_attn_decode_workspace_size(q: torch.Tensor, mem: Memory | None) -> int:
    """Bytes of workspace rel_attn_decode needs (txl_rel_attn_decode_workspace_size)."""
    B, L, H, D = q.shape
    memc = ctypes.byref(mem.c_struct) if mem is not None else None
    return int(_lib().txl_rel_attn_decode_workspace_size(B, L, H, D, memc))


def rel_attn_decode(q: torch.Tensor, mem: Memory | None, k_cur: torch.Tensor, v_cur: torch.Tensor,
                    u: torch.Tensor, v_bias: torch.Tensor, r: torch.Tensor, n_rows: int,
                    clamp_len: int, out: torch.Tensor, scale: float = 0.0,
                    workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of 1..16 queries per (b, h) over a long memory, keys split across CTAs
    (txl_rel_attn_decode).  Without `workspace`, a device buffer of the required size is taken
    from torch's allocator for the call."""
    (B, L, H, D), memc, vq, vk, vv, vo = _attn_args(q, mem, k_cur, v_cur, r, out)
    if u.dtype != torch.float32 or v_bias.dtype != torch.float32:
        raise TypeError("u and v_bias are fp32 [H, D]")
    if not (u.is_contiguous() and v_bias.is_contiguous()):
        raise ValueError("u and v_bias must be contiguous [H, D]")
    need = rel_attn_decode_workspace_size(q, mem)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    nbytes = workspace.numel() * workspace.element_size()
    st = _lib().txl_rel_attn_decode(
        B, L, H, D, int(clamp_len), ctypes.byref(vq), memc, ctypes.byref(vk), ctypes.byref(vv),
        u.data_ptr(), v_bias.data_ptr(), r.data_ptr(), r.stride(1), int(n_rows), float(scale),
        ctypes.byref(vo), dtype_code(q), workspace.data_ptr(), nbytes, _stream(stream))
    check(st, "txl_rel_attn_decode")
    return out


def rel_attn_path(q, mem, k_cur, v_cur, r, out) -> int:
    """1 = fused tcgen05 kernel, 2 = SIMT kernel (txl_rel_attn_path)."""
    (B, L, H, D), memc, vq, vk, vv, vo = _attn_args(q, mem, k_cur, v_cur, r, out)
    return _lib().txl_rel_attn_path(B, L, H, D, ctypes.byref(vq), memc, ctypes.byref(vk),
                                    ctypes.byref(vv), r.data_ptr(), r.stride(1), ctypes.byref(vo),
                                    dtype_code(q))


def rel_attn_decode_path(q, mem, k_cur, v_cur, r, out) -> int:
    """1 = fused tcgen05 kernel, 4 = split-key decode kernels (txl_rel_attn_decode_path)."""
    (B, L, H, D), memc, vq, vk, vv, vo = _attn_args(q, mem, k_cur, v_cur, r, out)
    return _lib().txl_rel_attn_decode_path(B, L, H, D, ctypes.byref(vq), memc, ctypes.byref(vk),
                                           ctypes.byref(vv), r.data_ptr(), r.stride(1), ctypes.byref(vo),
                                           dtype_code(q))


def rel_attn_bwd_path(q, mem, k_cur, v_cur, r, out, d_out, g: dict) -> int:
    """1 = tcgen05 gradient kernel, 2 = mma.sync, 3 = SIMT (txl_rel_attn_bwd_path), for the gradient
    buffers g (as rel_attn_bwd returns them: dq, dk_cur, dv_cur, dr)."""
    (B, L, H, D), memc, vq, vk, vv, vo = _attn_args(q, mem, k_cur, v_cur, r, out)
    vg = view(d_out)
    return _lib().txl_rel_attn_bwd_path(B, L, H, D, ctypes.byref(vq), memc, ctypes.byref(vk), ctypes.byref(vv),
                                        r.data_ptr(), r.stride(1), ctypes.byref(vo), ctypes.byref(vg),
                                        g["dq"].data_ptr(), g["dk_cur"].data_ptr(), g["dv_cur"].data_ptr(),
                                        g["dr"].data_ptr(), dtype_code(q))


def mem_push(mem: Memory, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> Memory:
    """Append k_new/v_new [B, L, H, D] to the FIFO memory (txl_mem_push)."""
    vk, vv = view(k_new), view(v_new)
    st = _lib().txl_mem_push(ctypes.byref(mem.c_struct), ctypes.byref(vk), ctypes.byref(vv),
                             k_new.shape[1], _stream(stream))
    check(st, "txl_mem_push")
    return mem


def _rows2d(t: torch.Tensor, what: str):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("%s must be a 2-D tensor with unit column stride" % what)
    return t.data_ptr(), t.stride(0)


def linear(X: torch.Tensor, W: torch.Tensor, Y: torch.Tensor | None = None,
           err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W for bf16 X [m, k] and W [k, n] (txl_linear); Y [m, n] is allocated if not given."""
    m, k = X.shape
    k2, n = W.shape
    if k2 != k:
        raise ValueError("inner dimensions differ")
    if Y is None:
        Y = torch.empty(m, n, dtype=X.dtype, device=X.device)
    px, ldx = _rows2d(X, "X")
    pw, ldw = _rows2d(W, "W")
    py, ldy = _rows2d(Y, "Y")
    st = _lib().txl_linear(m, n, k, px, ldx, pw, ldw, py, ldy, dtype_code(X),
                           err_flag.data_ptr() if err_flag is not None else None, _stream(stream))
    check(st, "txl_linear")
    return Y


def rel_attn_layer_workspace_size(B: int, L: int, H: int, D: int) -> int:
    """Bytes of workspace rel_attn_layer needs (txl_rel_attn_layer_workspace_size)."""
    return int(_lib().txl_rel_attn_layer_workspace_size(B, L, H, D))


def rel_attn_layer(h: torch.Tensor, mem: Memory | None, W_qkv: torch.Tensor, W_o: torch.Tensor,
                   u: torch.Tensor, v_bias: torch.Tensor, r: torch.Tensor, n_rows: int, clamp_len: int,
                   n_head: int, d_head: int, y: torch.Tensor | None = None, scale: float = 0.0,
                   workspace: torch.Tensor | None = None, err_flag: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """One attention-layer step over hidden states h [B, L, d_model] (txl_rel_attn_layer): the
    projections, the relative attention over [memory ++ segment], the output projection, and the
    push of the segment's keys and values into `mem`.  Returns y [B, L, d_model]."""
    B, L, d_model = h.shape
    if h.stride(2) != 1 or (B > 1 and h.stride(0) != L * h.stride(1)):
        raise ValueError("h must be [B, L, d_model] with rows b*L + t evenly spaced")
    if u.dtype != torch.float32 or v_bias.dtype != torch.float32:
        raise TypeError("u and v_bias are fp32 [H, D]")
    if not (u.is_contiguous() and v_bias.is_contiguous() and W_qkv.is_contiguous() and W_o.is_contiguous()):
        raise ValueError("u, v_bias, W_qkv and W_o must be contiguous")
    if y is None:
        y = torch.empty(B, L, d_model, dtype=h.dtype, device=h.device)
    if y.stride(2) != 1 or (B > 1 and y.stride(0) != L * y.stride(1)):
        raise ValueError("y must be [B, L, d_model] with rows b*L + t evenly spaced")
    need = rel_attn_layer_workspace_size(B, L, n_head, d_head)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=h.device)
    nbytes = workspace.numel() * workspace.element_size()
    memc = ctypes.byref(mem.c_struct) if mem is not None else None
    st = _lib().txl_rel_attn_layer(
        B, L, n_head, d_head, d_model, int(clamp_len), h.data_ptr(), h.stride(1), memc, W_qkv.data_ptr(),
        W_o.data_ptr(), u.data_ptr(), v_bias.data_ptr(), r.data_ptr(), r.stride(1), int(n_rows), float(scale),
        y.data_ptr(), y.stride(1), workspace.data_ptr(), nbytes,
        err_flag.data_ptr() if err_flag is not None else None, _stream(stream))
    check(st, "txl_rel_attn_layer")
    return y


def rel_attn_layer_fused_workspace_size(B: int, L: int, H: int, D: int) -> int:
    """Bytes of workspace rel_attn_layer_fused needs (txl_rel_attn_layer_fused_workspace_size)."""
    return int(_lib().txl_rel_attn_layer_fused_workspace_size(B, L, H, D))


def rel_attn_layer_fused(h: torch.Tensor, mem: Memory, mem_len: int, W_qkv: torch.Tensor, W_o: torch.Tensor,
                         u: torch.Tensor, v_bias: torch.Tensor, r: torch.Tensor, n_rows: int, clamp_len: int,
                         n_head: int, d_head: int, y: torch.Tensor | None = None, scale: float = 0.0,
                         workspace: torch.Tensor | None = None, err_flag: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """The layer step of rel_attn_layer with the memory push folded into the projection
    (txl_rel_attn_layer_fused): `mem` is a ring of at least mem_len + L slots (Memory.empty(B,
    slots, H, D)) holding a memory of mem_len positions.  Returns y [B, L, d_model]."""
    B, L, d_model = h.shape
    if h.stride(2) != 1 or (B > 1 and h.stride(0) != L * h.stride(1)):
        raise ValueError("h must be [B, L, d_model] with rows b*L + t evenly spaced")
    if u.dtype != torch.float32 or v_bias.dtype != torch.float32:
        raise TypeError("u and v_bias are fp32 [H, D]")
    if not (u.is_contiguous() and v_bias.is_contiguous() and W_qkv.is_contiguous() and W_o.is_contiguous()):
        raise ValueError("u, v_bias, W_qkv and W_o must be contiguous")
    if y is None:
        y = torch.empty(B, L, d_model, dtype=h.dtype, device=h.device)
    if y.stride(2) != 1 or (B > 1 and y.stride(0) != L * y.stride(1)):
        raise ValueError("y must be [B, L, d_model] with rows b*L + t evenly spaced")
    need = rel_attn_layer_fused_workspace_size(B, L, n_head, d_head)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=h.device)
    nbytes = workspace.numel() * workspace.element_size()
    st = _lib().txl_rel_attn_layer_fused(
        B, L, n_head, d_head, d_model, int(clamp_len), h.data_ptr(), h.stride(1), ctypes.byref(mem.c_struct),
        int(mem_len), W_qkv.data_ptr(), W_o.data_ptr(), u.data_ptr(), v_bias.data_ptr(), r.data_ptr(), r.stride(1),
        int(n_rows), float(scale), y.data_ptr(), y.stride(1), workspace.data_ptr(), nbytes,
        err_flag.data_ptr() if err_flag is not None else None, _stream(stream))
    check(st, "txl_rel_attn_layer_fused")
    return y


def rel_attn_bwd(q: torch.Tensor, mem: Memory | None, k_cur: torch.Tensor, v_cur: torch.Tensor,
                 u: torch.Tensor, v_bias: torch.Tensor, r: torch.Tensor, n_rows: int, clamp_len: int,
                 out: torch.Tensor, d_out: torch.Tensor, scale: float = 0.0,
                 workspace: torch.Tensor | None = None, stream=None, lse: torch.Tensor | None = None) -> dict:
    """Gradients of one rel_attn_fwd call for the upstream gradient d_out (txl_rel_attn_bwd; with
    `lse`, the statistics rel_attn_fwd saved for this call, txl_rel_attn_bwd_lse).
    Returns fp32 tensors dq, dk_cur, dv_cur [B, L, H, D], du, dv_bias [H, D], dr [n_rows, H, D]."""
    (B, L, H, D), memc, vq, vk, vv, vo = _attn_args(q, mem, k_cur, v_cur, r, out)
    vg = view(d_out)
    if u.dtype != torch.float32 or v_bias.dtype != torch.float32:
        raise TypeError("u and v_bias are fp32 [H, D]")
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {"dq": torch.empty(B, L, H, D, **f32), "dk_cur": torch.empty(B, L, H, D, **f32),
         "dv_cur": torch.empty(B, L, H, D, **f32), "du": torch.empty(H, D, **f32),
         "dv_bias": torch.empty(H, D, **f32), "dr": torch.empty(n_rows, H, D, **f32)}
    need = int(_lib().txl_rel_attn_bwd_workspace_size(B, L, H, D))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if lse is not None:
        _check_lse(lse, B, L, H)
    st = _lib().txl_rel_attn_bwd_lse(
        B, L, H, D, int(clamp_len), ctypes.byref(vq), memc, ctypes.byref(vk), ctypes.byref(vv),
        u.data_ptr(), v_bias.data_ptr(), r.data_ptr(), r.stride(1), int(n_rows), float(scale),
        ctypes.byref(vo), ctypes.byref(vg), lse.data_ptr() if lse is not None else None,
        g["dq"].data_ptr(), g["dk_cur"].data_ptr(), g["dv_cur"].data_ptr(),
        g["du"].data_ptr(), g["dv_bias"].data_ptr(), g["dr"].data_ptr(), dtype_code(q), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream))
    check(st, "txl_rel_attn_bwd_lse" if lse is not None else "txl_rel_attn_bwd")
    return g


def rel_pos_bwd(dr: torch.Tensor, d_model: int, dW_R: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dW_R [d_model, H*D] = sum_delta R_delta^T dr[delta] for fp32 dr [n_rows, H, D] (txl_rel_pos_bwd)."""
    n_rows, H, D = dr.shape
    if not dr.is_contiguous() or dr.dtype != torch.float32:
        raise ValueError("dr must be a contiguous fp32 [n_rows, H, D] tensor")
    if dW_R is None:
        dW_R = torch.empty(d_model, H * D, dtype=torch.float32, device=dr.device)
    st = _lib().txl_rel_pos_bwd(n_rows, d_model, H, D, dr.data_ptr(), dW_R.data_ptr(), dW_R.stride(0),
                                _stream(stream))
    check(st, "txl_rel_pos_bwd")
    return dW_R


def rel_attn_table_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, u: torch.Tensor,
                       v_bias: torch.Tensor, r_table: torch.Tensor, max_len: int, out: torch.Tensor,
                       key_mask: torch.Tensor | None = None, scale: float = 0.0, stream=None) -> torch.Tensor:
    """The learned-table variant (txl_rel_attn_table_fwd): bidirectional attention over q, k, v
    [B, L, H, D] with the position vector of a pair read from r_table [2 max_len - 1, H, ld_r] at
    clamp(i - j + max_len - 1); key_mask [B, L] uint8 (0 = masked) or None."""
    B, L, H, D = q.shape
    if u.dtype != torch.float32 or v_bias.dtype != torch.float32:
        raise TypeError("u and v_bias are fp32 [H, D]")
    if key_mask is not None and (key_mask.dtype != torch.uint8 or not key_mask.is_contiguous()):
        raise TypeError("key_mask must be a contiguous uint8 [B, L] tensor")
    vq, vk, vv, vo = view(q), view(k), view(v), view(out)
    st = _lib().txl_rel_attn_table_fwd(
        B, L, H, D, int(max_len), ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(vv), u.data_ptr(),
        v_bias.data_ptr(), r_table.data_ptr(), r_table.stride(1),
        key_mask.data_ptr() if key_mask is not None else None, float(scale), ctypes.byref(vo), dtype_code(q),
        _stream(stream))
    check(st, "txl_rel_attn_table_fwd")
    return out


def rel_attn_table_path(q, k, v, r_table, max_len: int, out, key_mask=None) -> int:
    """1 = persistent tcgen05 kernel, 3 = mma.sync tensor-core kernel, 2 = CUDA-core kernel
    (txl_rel_attn_table_path)."""
    B, L, H, D = q.shape
    vq, vk, vv, vo = view(q), view(k), view(v), view(out)
    return _lib().txl_rel_attn_table_path(
        B, L, H, D, int(max_len), ctypes.byref(vq), ctypes.byref(vk), ctypes.byref(vv), r_table.data_ptr(),
        r_table.stride(1), key_mask.data_ptr() if key_mask is not None else None, ctypes.byref(vo), dtype_code(q))


class QuantMemory:
    """K/V memory of M positions per batch entry held as 4- or 8-bit codes (txl_qmem): groups of 32
    channels of a head share a bf16 step and minimum.  ``rows`` is uint8 [B, H, M, row bytes], a position
    and head's k codes, v codes and parameters; ``wp``/``valid`` as in Memory.  Filled by qmem_push, read
    by rel_attn_qmem and qmem_read."""

    def __init__(self, rows: torch.Tensor, D: int, bits: int, wp: int = 0, valid: int = 0):
        row = self.row_bytes(D, bits)
        if rows.dim() != 4 or rows.shape[3] != row or rows.dtype != torch.uint8 or not rows.is_contiguous():
            raise ValueError("a quantised memory of d_head %d holds contiguous uint8 [B, H, M, %d]" % (D, row))
        if not rows.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        B, H, M, _ = rows.shape
        self.rows, self.device, self._bhd = rows, rows.get_device(), (B, H, D)
        self._c = TxlQmem(rows.data_ptr() if M else None, B, M, H, D, bits, int(wp), int(valid))
        self.address = ctypes.addressof(self._c)          # of the C struct, for calls that take it as a number

    @staticmethod
    def row_bytes(D: int, bits: int) -> int:
        """Bytes a position and head take (txl_qmem_row_bytes)."""
        row = int(_lib().txl_qmem_row_bytes(D, bits))
        if row == 0:
            raise ValueError("bits must be 4 or 8 and D in 1..128")
        return row

    @classmethod
    def empty(cls, B, M, H, D, bits=4, device="cuda"):
        return cls(torch.zeros(B, H, M, cls.row_bytes(D, bits), dtype=torch.uint8, device=device), D, bits)

    @property
    def M(self) -> int:
        return self._c.M

    @property
    def wp(self) -> int:
        return self._c.wp

    @property
    def valid(self) -> int:
        return self._c.valid

    def state(self):
        """Host ring state (wp, valid): with the buffers, everything needed to resume."""
        return self._c.wp, self._c.valid

    def restore(self, wp: int, valid: int) -> None:
        self._c.wp, self._c.valid = int(wp), int(valid)

    @property
    def c_struct(self) -> TxlQmem:
        return self._c


def _qmem_kv(mem: QuantMemory, k: torch.Tensor, v: torch.Tensor, j0: int, T: int, stream) -> bytes:
    """The packed txl_qmem_kv_args of k and v [B, T, H, D] of the memory's shape and device."""
    shape, dev, dtype = (*mem._bhd[:1], T, *mem._bhd[1:]), mem.device, k.dtype
    if k.shape != shape or v.shape != shape:
        raise ValueError("expected [B, T, H, D] = %s, got %s and %s" % (shape, tuple(k.shape), tuple(v.shape)))
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("tensors must live on the memory's device")
    if dtype != v.dtype:
        raise TypeError("k and v must share a dtype")
    (k0, k1, k2, k3), (v0, v1, v2, v3) = k.stride(), v.stride()
    if (k3 != 1 or v3 != 1) and shape[3] > 1:
        raise ValueError("the last (d) dimension must be contiguous")
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError("libtxl computes in float32 or bfloat16, got %s" % dtype)
    return native.QMEM_KV_ARGS.pack(mem.address, k.data_ptr(), k0, k1, k2, v.data_ptr(), v0, v1, v2, j0, T, code,
                                    _raw_stream(stream, dev))


def qmem_push(mem: QuantMemory, k_new: torch.Tensor, v_new: torch.Tensor, stream=None) -> QuantMemory:
    """Quantise k_new/v_new [B, L, H, D] into the FIFO memory (txl_qmem_push)."""
    args = _qmem_kv(mem, k_new, v_new, 0, k_new.shape[1], stream)
    check(_on_device(mem.device, _lib().txl_qmem_push_call, args), "txl_qmem_push")
    return mem


def qmem_read(mem: QuantMemory, j0: int, n: int, k_out: torch.Tensor, v_out: torch.Tensor, stream=None):
    """What the memory's logical positions j0 .. j0+n-1 (oldest first, all valid) stand for, into
    k_out/v_out [B, n, H, D] (txl_qmem_read)."""
    args = _qmem_kv(mem, k_out, v_out, j0, n, stream)
    check(_on_device(mem.device, _lib().txl_qmem_read_call, args), "txl_qmem_read")
    return k_out, v_out


def rel_attn_qmem_workspace_size(q: torch.Tensor, mem: QuantMemory | None) -> int:
    """Bytes of workspace rel_attn_qmem needs (txl_rel_attn_qmem_workspace_size)."""
    B, L, H, D = q.shape
    memc = ctypes.byref(mem.c_struct) if mem is not None else None
    return int(_lib().txl_rel_attn_qmem_workspace_size(B, L, H, D, memc, dtype_code(q)))


def _qattn_refusal(q, mem, k_cur, v_cur, u, v_bias, r, n_rows, out, dev):
    """Raises what is wrong with the arguments of rel_attn_qmem (called when something is)."""
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    if q.dtype not in _DTYPES:
        raise TypeError("libtxl computes in float32 or bfloat16, got %s" % q.dtype)
    H, D = q.shape[2:]
    for t in (k_cur, v_cur, out):
        if t.shape != q.shape or t.dtype != q.dtype or t.get_device() != dev:
            raise ValueError("q, k_cur, v_cur and out must share shape, dtype and device")
    for t in (u, v_bias):
        if t.dtype != torch.float32:
            raise TypeError("u and v_bias are fp32 [H, D]")
        if t.shape != (H, D) or not t.is_contiguous() or t.get_device() != dev:
            raise ValueError("u and v_bias must be contiguous [H, D] on the queries' device")
    if mem is not None and mem.device != dev:
        raise ValueError("tensors must live on the memory's device")
    if any(t.stride(3) != 1 for t in (q, k_cur, v_cur, out)) and D > 1:
        raise ValueError("the last (d) dimension must be contiguous")
    raise ValueError("r must be [n_rows, H, ld_r] of the queries' dtype and device, rows H * ld_r apart")


def rel_attn_qmem(q: torch.Tensor, mem: QuantMemory | None, k_cur: torch.Tensor, v_cur: torch.Tensor,
                  u: torch.Tensor, v_bias: torch.Tensor, r: torch.Tensor, n_rows: int, clamp_len: int,
                  out: torch.Tensor, scale: float = 0.0, workspace: torch.Tensor | None = None,
                  err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Relative attention over [quantised memory ++ current segment] (txl_rel_attn_qmem).  Without
    `workspace`, a device buffer of the required size is taken from torch's allocator for the call."""
    shape, dtype, dev = q.shape, q.dtype, q.get_device()
    B, L, H, D = shape
    (q0, q1, q2, q3), (k0, k1, k2, k3), (v0, v1, v2, v3), (o0, o1, o2, o3) = (
        q.stride(), k_cur.stride(), v_cur.stride(), out.stride())
    rs, rt = r.shape, r.stride()
    if not (dev >= 0 and dtype in _DTYPES and k_cur.shape == shape and v_cur.shape == shape and out.shape == shape
            and k_cur.dtype == dtype and v_cur.dtype == dtype and out.dtype == dtype and r.dtype == dtype
            and k_cur.get_device() == dev and v_cur.get_device() == dev and out.get_device() == dev
            and u.get_device() == dev and v_bias.get_device() == dev and r.get_device() == dev
            and u.dtype == torch.float32 and v_bias.dtype == torch.float32
            and u.shape == (H, D) and v_bias.shape == (H, D) and u.is_contiguous() and v_bias.is_contiguous()
            and (D == 1 or q3 == k3 == v3 == o3 == 1) and (mem is None or mem.device == dev)
            and len(rs) == 3 and rs[0] >= n_rows and rs[1] == H and rs[2] >= D and rt[2] == 1
            and (rs[0] <= 1 or rt[0] == H * rt[1])):
        _qattn_refusal(q, mem, k_cur, v_cur, u, v_bias, r, n_rows, out, dev)
    if workspace is None:
        # from the pool of the stream that will use it, so that it is not reused before it has been
        need = max(rel_attn_qmem_workspace_size(q, mem), 16)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(dev):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and live on the queries' device")
    if err_flag is not None and (err_flag.get_device() != dev or err_flag.dtype != torch.int32 or err_flag.numel() < 1):
        raise ValueError("err_flag must be an int32 on the queries' device")
    args = native.QMEM_ARGS.pack(
        B, L, H, D, clamp_len, n_rows, _DTYPES[dtype], scale, q.data_ptr(), q0, q1, q2, k_cur.data_ptr(), k0, k1, k2,
        v_cur.data_ptr(), v0, v1, v2, out.data_ptr(), o0, o1, o2, mem.address if mem is not None else 0, u.data_ptr(),
        v_bias.data_ptr(), r.data_ptr(), rt[1], workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        err_flag.data_ptr() if err_flag is not None else 0, _raw_stream(stream, dev))
    check(_on_device(dev, _lib().txl_rel_attn_qmem_call, args), "txl_rel_attn_qmem")
    return out


def rel_attn_qmem_path(q, mem, k_cur, v_cur, r, out) -> int:
    """5 = the kernel that multiplies the codes (up to 16 queries), 6 = the fp32 one of longer segments, 1 = the
    expanded memory, then the tcgen05 kernels (txl_rel_attn_qmem_path)."""
    B, L, H, D = q.shape
    memc = ctypes.byref(mem.c_struct) if mem is not None else None
    vq, vk, vv, vo = view(q), view(k_cur), view(v_cur), view(out)
    return _lib().txl_rel_attn_qmem_path(B, L, H, D, ctypes.byref(vq), memc, ctypes.byref(vk), ctypes.byref(vv),
                                         r.data_ptr(), r.stride(1), ctypes.byref(vo), dtype_code(q))


class PagedMemory:
    """K/V memory of B sequences of different lengths in pages of one pool (txl_paged).

    ``k``/``v`` are [n_pages, H, page_len, D] (rows padded to 16 bytes), ``pos`` int32 and ``weight`` fp32 [n_pages,
    page_len], ``table`` int32 [B, max_pages], ``length`` and ``next_pos`` int32 [B], all on one device: slot s of
    sequence b is row s % page_len of page table[b, s // page_len].  Filled by paged_push and rel_attn_paged, cut by
    paged_evict.  The host gives pages to sequences: reserve before positions are pushed, release for a sequence that has
    ended, trim for pages that an eviction left empty.

    A table may lack pages that a sequence's length spans: those slots count as not there, and their entries stay as they
    are (-1) when pages are reserved or freed.  Behind the length a sequence has the pages up to the first missing one."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor, weight: torch.Tensor, table: torch.Tensor,
                 length: torch.Tensor, next_pos: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be [n_pages, H, page_len, D] of one shape, layout and dtype")
        if not k.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        n, H, page_len, D = k.shape
        ld = k.stride(2)
        if k.stride(3) != 1 or k.stride(1) != page_len * ld or (n > 1 and k.stride(0) != H * page_len * ld):
            raise ValueError("pages must be dense [n_pages, H, page_len, ld], the first D of each row")
        dev = k.get_device()
        for t, shape, dtype, what in ((pos, (n, page_len), torch.int32, "pos"), (weight, (n, page_len), torch.float32, "weight"),
                                      (table, None, torch.int32, "table"), (length, table.shape[:1], torch.int32, "length"),
                                      (next_pos, table.shape[:1], torch.int32, "next_pos")):
            if t.dtype != dtype or not t.is_contiguous() or t.get_device() != dev or (
                    t.dim() != 2 if shape is None else t.shape != torch.Size(shape)):
                raise ValueError("%s must be a contiguous %s%s on the pages' device"
                                 % (what, dtype, "" if shape is None else " " + str(list(shape))))
        self.k, self.v, self.pos, self.weight = k, v, pos, weight
        self.table, self.length, self.next_pos, self.device = table, length, next_pos, dev
        B, most = table.shape
        self._scratch = torch.zeros(B * (H + 1) + 2, dtype=torch.int32, device=k.device)     # the last is err_flag
        at = self._scratch.data_ptr()
        self._c = TxlPaged(k.data_ptr(), v.data_ptr(), pos.data_ptr(), weight.data_ptr(), table.data_ptr(),
                           length.data_ptr(), next_pos.data_ptr(), at, at + 4 * (B * (H + 1) + 1), B, H, D, ld, n, page_len, most, dtype_code(k))
        self.address = ctypes.addressof(self._c)
        self._shape, self._dtype = (B, H, D), k.dtype
        self._room = length.tolist()                                               # positions that room was asked for
        self._rows = []                                                            # pages of every sequence, -1: missing
        for row, room in zip(table.tolist(), self._room):
            row = [p if 0 <= p < n else -1 for p in row]
            end = min(most, (max(room, 0) + page_len - 1) // page_len)
            while end < most and row[end] >= 0:
                end += 1
            self._rows.append(row[:end])
        self._gaps = [-1 in row for row in self._rows]
        used = {p for row in self._rows for p in row}
        self._free = [p for p in range(n - 1, -1, -1) if p not in used]

    @classmethod
    def empty(cls, B, n_pages, page_len, H, D, max_pages=None, dtype=torch.bfloat16, device="cuda"):
        """An empty memory; a sequence may hold up to max_pages pages (all of them by default).  paged_evict's workspace
        is four bytes for each position that the B rows of the table could hold: give max_pages where sequences are bounded."""
        unit = 16 // torch.empty(0, dtype=dtype).element_size()
        ld = (D + unit - 1) // unit * unit
        k, v = (torch.zeros(n_pages, H, page_len, ld, dtype=dtype, device=device)[..., :D] for _ in range(2))
        i32 = dict(dtype=torch.int32, device=device)
        return cls(k, v, torch.zeros(n_pages, page_len, **i32), torch.zeros(n_pages, page_len, device=device),
                   torch.full((B, n_pages if max_pages is None else max_pages), -1, **i32),
                   torch.zeros(B, **i32), torch.zeros(B, **i32))

    @property
    def c_struct(self) -> TxlPaged:
        return self._c

    @property
    def page_len(self) -> int:
        return self._c.page_len

    @property
    def reserved(self) -> list:
        """Positions that every sequence has room for: its length, and what was reserved and not pushed."""
        return list(self._room)

    @property
    def free_pages(self) -> int:
        """Pages that no sequence has."""
        return len(self._free)

    def reserve(self, positions) -> None:
        """Pages for `positions` more positions of every sequence (an int, or one of each).  A pushed position must
        have been reserved; one that was reserved and then not pushed keeps its room until trim.  Raises, and changes
        nothing, when the pool or a sequence's row of the table is too small.  The table changes on the current stream
        (as it does in release and trim)."""
        B = self._shape[0]
        more = [positions] * B if isinstance(positions, int) else [int(x) for x in positions]
        if len(more) != B or min(more, default=0) < 0:
            raise ValueError("reserve takes a number of positions, or one for each sequence")
        L = self.page_len
        want = [(r + m + L - 1) // L - len(p) if m else 0 for r, m, p in zip(self._room, more, self._rows)]
        if any(w > 0 and len(p) + w > self._c.max_pages for w, p in zip(want, self._rows)):
            raise ValueError("a sequence takes at most %d pages" % self._c.max_pages)
        if sum(w for w in want if w > 0) > len(self._free):
            raise ValueError("the pool has %d free pages" % len(self._free))
        for p, w in zip(self._rows, want):
            p.extend(self._free.pop() for _ in range(w))
        self._room = [r + m for r, m in zip(self._room, more)]
        if any(w > 0 for w in want):
            self._write_table()

    def _give_back(self, b: int, kept: int) -> None:
        """Sequence b keeps its first `kept` pages; the others are free (but for those it shares)."""
        gone, self._rows[b] = self._rows[b][kept:], self._rows[b][:kept]
        self._gaps[b] = self._gaps[b] and -1 in self._rows[b]
        used = {p for row in self._rows for p in row} if gone else ()
        self._free.extend(p for p in dict.fromkeys(reversed(gone)) if p >= 0 and p not in used)

    def release(self, b: int) -> None:
        """Sequence b has ended: it is empty, and its pages are free."""
        if not 0 <= b < len(self._rows):
            raise ValueError("the memory has %d sequences" % len(self._rows))
        self._give_back(b, 0)
        self._room[b] = 0
        self._write_table()
        with torch.cuda.device(self.device):
            self.length[b] = 0
            self.next_pos[b] = 0

    def trim(self) -> None:
        """Frees the pages that hold no position (reads the lengths: waits for the device)."""
        self._room = self.length.tolist()
        L = self.page_len
        for b, n in enumerate(self._room):
            self._give_back(b, (n + L - 1) // L)
        self._write_table()

    def check(self) -> None:
        """Raises if a call met a slot without a page since the last check (waits for the device)."""
        with torch.cuda.device(self.device):
            flag = int(self._scratch[-1])
            self._scratch[-1] = 0
        check(flag, "paged memory")

    def _write_table(self) -> None:
        most = self._c.max_pages
        host = torch.tensor([p + [-1] * (most - len(p)) for p in self._rows], dtype=torch.int32).view(self.table.shape)
        with torch.cuda.device(self.device):
            self.table.copy_(host)


def _paged_counts(mem: PagedMemory, counts) -> int:
    if counts is None:
        return 0
    if counts.dtype != torch.int32 or counts.shape != mem._shape[:1] or not counts.is_contiguous() or counts.get_device() != mem.device:
        raise ValueError("counts must be a contiguous int32 [B] on the memory's device")
    return counts.data_ptr()


def paged_push(mem: PagedMemory, k_new: torch.Tensor, v_new: torch.Tensor, counts: torch.Tensor | None = None,
               stream=None) -> PagedMemory:
    """New positions of every sequence into its reserved pages (txl_paged_push): rows t < counts[b] (int32 [B], all
    T without it) of k_new, v_new [B, T, H, D]."""
    (B, H, D), dev, dtype, shape = mem._shape, mem.device, mem._dtype, k_new.shape
    if len(shape) != 4 or shape[0] != B or shape[2] != H or shape[3] != D or v_new.shape != shape:
        raise ValueError("expected k_new and v_new [%d, T, %d, %d]" % (B, H, D))
    if k_new.dtype != dtype or v_new.dtype != dtype:
        raise TypeError("k_new and v_new must have the memory's dtype")
    if k_new.get_device() != dev or v_new.get_device() != dev:
        raise ValueError("tensors must live on the memory's device")
    (k0, k1, k2, k3), (v0, v1, v2, v3) = k_new.stride(), v_new.stride()
    if (k3 != 1 or v3 != 1) and D > 1:
        raise ValueError("the last (d) dimension must be contiguous")
    args = native.PAGED_PUSH_ARGS.pack(mem.address, k_new.data_ptr(), k0, k1, k2, v_new.data_ptr(), v0, v1, v2,
                                       _paged_counts(mem, counts), _raw_stream(stream, dev), shape[1])
    check(_on_device(dev, _lib().txl_paged_push_call, args), "txl_paged_push")
    return mem


def rel_attn_paged_workspace_size(q: torch.Tensor, mem: PagedMemory, n_rows: int, accumulate: bool = False) -> int:
    """Bytes of workspace rel_attn_paged needs (txl_rel_attn_paged_workspace_size)."""
    return int(_lib().txl_rel_attn_paged_workspace_size(ctypes.byref(mem._c), q.shape[1], int(n_rows), int(accumulate)))


def _paged_refusal(q, mem, k_new, v_new, u, v_bias, r, n_rows, out):
    """Raises what is wrong with the arguments of rel_attn_paged (called when something is)."""
    B, H, D = mem._shape
    given = [t for t in (q, k_new, v_new, out) if t is not None]
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new come together")
    if any(t.dtype != mem._dtype for t in (*given, r)):
        raise TypeError("q, k_new, v_new, r and out must have the memory's dtype")
    if u.dtype != torch.float32 or v_bias.dtype != torch.float32:
        raise TypeError("u and v_bias are fp32 [H, D]")
    if any(t.get_device() != mem.device for t in (*given, u, v_bias, r)):
        raise ValueError("tensors must live on the memory's device")
    if any(t.dim() != 4 or t.shape != q.shape for t in given) or (q.shape[0], *q.shape[2:]) != (B, H, D):
        raise ValueError("q, k_new, v_new and out must be [%d, T, %d, %d]" % (B, H, D))
    if any(t.shape != (H, D) or not t.is_contiguous() for t in (u, v_bias)):
        raise ValueError("u and v_bias must be contiguous [H, D]")
    if any(t.stride(3) != 1 for t in given) and D > 1:
        raise ValueError("the last (d) dimension must be contiguous")
    raise ValueError("r must be [n_rows, H, ld_r], rows H * ld_r apart")


def rel_attn_paged(q: torch.Tensor, mem: PagedMemory, k_new: torch.Tensor | None, v_new: torch.Tensor | None,
                   u: torch.Tensor, v_bias: torch.Tensor, r: torch.Tensor, n_rows: int, clamp_len: int,
                   out: torch.Tensor, scale: float = 0.0, counts: torch.Tensor | None = None, accumulate: bool = False,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Relative attention of 1..16 new tokens a sequence over a paged memory (txl_rel_attn_paged): pushes k_new, v_new
    [B, T, H, D] into their reserved pages (or takes the last positions as pushed already, both None), then attends;
    rows past counts[b] (int32 [B]) are left alone.  With `accumulate`, every slot's weight grows by the attention it
    receives.  Without `workspace`, a device buffer of the required size is taken from torch's allocator for the call."""
    shape, dtype, dev = q.shape, q.dtype, mem.device
    B, H, D = mem._shape
    own = k_new is not None
    rs, rt = r.shape, r.stride()
    if not (len(shape) == 4 and shape[0] == B and shape[2] == H and shape[3] == D and out.shape == shape
            and own == (v_new is not None) and (not own or (k_new.shape == shape and v_new.shape == shape
                                                            and k_new.dtype == dtype and v_new.dtype == dtype
                                                            and k_new.get_device() == dev and v_new.get_device() == dev
                                                            and (D == 1 or k_new.stride(3) == v_new.stride(3) == 1)))
            and dtype == mem._dtype and out.dtype == dtype and r.dtype == dtype
            and q.get_device() == dev and out.get_device() == dev and r.get_device() == dev
            and u.get_device() == dev and v_bias.get_device() == dev
            and u.dtype == torch.float32 and v_bias.dtype == torch.float32
            and u.shape == (H, D) and v_bias.shape == (H, D) and u.is_contiguous() and v_bias.is_contiguous()
            and (D == 1 or q.stride(3) == out.stride(3) == 1)
            and len(rs) == 3 and rs[0] >= n_rows and rs[1] == H and rs[2] >= D and rt[2] == 1
            and (rs[0] <= 1 or rt[0] == H * rt[1])):
        _paged_refusal(q, mem, k_new, v_new, u, v_bias, r, n_rows, out)
    n = _paged_counts(mem, counts)
    if workspace is None:
        # from the pool of the stream that will use it, so that it is not reused before it has been
        need = max(rel_attn_paged_workspace_size(q, mem, min(n_rows, clamp_len + 1), accumulate), 16)
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(dev):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and live on the memory's device")
    none = (0, 0, 0, 0)
    args = native.PAGED_ARGS.pack(
        shape[1], clamp_len, n_rows, bool(accumulate), scale, mem.address, q.data_ptr(), *q.stride()[:3],
        *((k_new.data_ptr(), *k_new.stride()[:3], v_new.data_ptr(), *v_new.stride()[:3]) if own else none + none),
        out.data_ptr(), *out.stride()[:3], n, u.data_ptr(), v_bias.data_ptr(), r.data_ptr(), rt[1], workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, dev))
    check(_on_device(dev, _lib().txl_rel_attn_paged, args), "txl_rel_attn_paged")
    return out


def paged_evict_workspace_size(mem: PagedMemory) -> int:
    """Bytes of workspace paged_evict needs (txl_paged_evict_workspace_size)."""
    return int(_lib().txl_paged_evict_workspace_size(ctypes.byref(mem._c)))


def paged_evict(mem: PagedMemory, keep: int, recent: int = 0, workspace: torch.Tensor | None = None,
                stream=None) -> PagedMemory:
    """Cut every sequence to `keep` positions (txl_paged_evict): the last `recent` ones and those of the largest
    weight stay.  The pages stay with their sequences (PagedMemory.trim frees them), and no sequence counts as having
    room reserved for more than `keep` positions: reserve again what was reserved and is not pushed yet.  A sequence that
    lacks a page is left as it is."""
    dev = mem.device
    if workspace is None:
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(dev):
            workspace = torch.empty(max(paged_evict_workspace_size(mem), 16), dtype=torch.uint8, device=mem.k.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and live on the memory's device")
    raw, size = _raw_stream(stream, dev), workspace.numel() * workspace.element_size()
    st = _on_device(dev, lambda _: _lib().txl_paged_evict(ctypes.byref(mem._c), int(keep), int(recent), workspace.data_ptr(),
                                                          size, raw), None)
    check(st, "txl_paged_evict")
    keep = int(keep)
    mem._room = [x if x < keep or gap else keep for x, gap in zip(mem._room, mem._gaps)]
    return mem


class QuantWeight:
    """A matrix W [k, n] as 4-bit codes (txl_q4): groups of 32, 64 or 128 entries of a column share a bf16 step and
    minimum.  Multiplied by linear_q4."""

    def __init__(self, data: torch.Tensor, k: int, n: int, group: int):
        need = int(_lib().txl_q4_bytes(k, n, group))
        if need == 0:
            raise ValueError("4-bit weights are [k, n] with k, n >= 1 in groups of 32, 64 or 128")
        if data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() != need or not data.is_cuda:
            raise ValueError("4-bit weights of [%d, %d] in groups of %d take %d bytes of a CUDA device" % (k, n, group, need))
        self.data, self.shape, self.group, self.device = data, (k, n), group, data.get_device()
        self._c = TxlQ4(data.data_ptr(), k, n, group)
        self.address = ctypes.addressof(self._c)

    @classmethod
    def quantise(cls, W: torch.Tensor, group: int = 64, stream=None):
        """The codes of bf16 W [k, n] (txl_q4_quantise)."""
        p, ld = _rows2d(W, "W")
        if W.dtype != torch.bfloat16:
            raise TypeError("linear_q4 computes in bfloat16, got %s" % W.dtype)
        if not W.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        size = int(_lib().txl_q4_bytes(W.shape[0], W.shape[1], group))
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(W.get_device()):
            w = cls(torch.empty(size, dtype=torch.uint8, device=W.device), W.shape[0], W.shape[1], group)
        raw = _raw_stream(stream, w.device)
        check(_on_device(w.device, lambda _: _lib().txl_q4_quantise(ctypes.byref(w._c), p, ld, raw), None), "txl_q4_quantise")
        return w

    def expand(self, W: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """What the codes stand for, as bf16 [k, n] (txl_q4_expand)."""
        if W is None:
            with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(self.device):
                W = torch.empty(self.shape, dtype=torch.bfloat16, device=self.data.device)
        p, ld = _rows2d(W, "W")
        if W.dtype != torch.bfloat16 or tuple(W.shape) != self.shape or W.get_device() != self.device:
            raise ValueError("W must be bfloat16 [%d, %d] on the weights' device" % self.shape)
        raw = _raw_stream(stream, self.device)
        check(_on_device(self.device, lambda _: _lib().txl_q4_expand(ctypes.byref(self._c), p, ld, raw), None), "txl_q4_expand")
        return W


def linear_q4_workspace_size(m: int, w: QuantWeight) -> int:
    """Bytes of workspace linear_q4 needs for m rows (txl_linear_q4_workspace_size)."""
    return int(_lib().txl_linear_q4_workspace_size(int(m), ctypes.byref(w._c)))


def linear_q4(X: torch.Tensor, w: QuantWeight, Y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              err_flag: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X W for bf16 X [m, k] and 4-bit W [k, n] (txl_linear_q4); Y [m, n] is allocated if not given, and so is the
    workspace where many rows need one."""
    dev, (k, n), shape = w.device, w.shape, X.shape
    if len(shape) != 2 or shape[1] != k or X.dtype != torch.bfloat16 or X.get_device() != dev:
        _q4_refusal(X, w)
    m, (ldx, x1) = shape[0], X.stride()
    need = linear_q4_workspace_size(m, w) if m > 16 and workspace is None else 0
    if Y is None or need:
        with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(dev):
            if Y is None:
                Y = torch.empty(m, n, dtype=X.dtype, device=X.device)
            if need:
                workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    if Y.shape != (m, n) or Y.dtype != torch.bfloat16 or Y.get_device() != dev:
        raise ValueError("Y must be bfloat16 [%d, %d] on the weights' device" % (m, n))
    ldy, y1 = Y.stride()
    if (x1 != 1 and k > 1) or (y1 != 1 and n > 1):
        raise ValueError("X and Y must have unit column stride")
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and live on the weights' device")
    if err_flag is not None and (err_flag.get_device() != dev or err_flag.dtype != torch.int32 or err_flag.numel() < 1):
        raise ValueError("err_flag must be an int32 on the weights' device")
    pw, size = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (0, 0)
    args = native.Q4_ARGS.pack(w.address, X.data_ptr(), ldx if m > 1 else (k + 7) // 8 * 8, Y.data_ptr(), ldy if m > 1 else n,
                               pw, size, err_flag.data_ptr() if err_flag is not None else 0, _raw_stream(stream, dev), m)
    check(_on_device(dev, _lib().txl_linear_q4_call, args), "txl_linear_q4")
    return Y


def _q4_refusal(X, w):
    """Raises what is wrong with X of linear_q4 (called when something is)."""
    if X.dim() != 2:
        raise ValueError("X must be a 2-D tensor with unit column stride")
    if X.shape[1] != w.shape[0]:
        raise ValueError("inner dimensions differ")
    if X.dtype != torch.bfloat16:
        raise TypeError("linear_q4 computes in bfloat16, got %s" % X.dtype)
    raise ValueError("tensors must live on the weights' device")


def selftest_wait_timeout(err_flag: torch.Tensor, timeout_us: int, stream=None) -> None:
    st = _lib().txl_selftest_wait_timeout(err_flag.data_ptr(), int(timeout_us), _stream(stream))
    check(st, "txl_selftest_wait_timeout")


def version() -> int:
    return _lib().txl_version()
