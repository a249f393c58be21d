"""The README's example over a quantised memory runs, and computes what its calls compute."""
import os
import re

import numpy as np
import pytest
import torch

from qmem_common import attend64, f64, held

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_layer_over_a_quantised_memory():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    code = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "def layer_step" in c]
    assert len(code) == 1
    scope = {}
    exec(code[0], scope)
    txl, B, H, D, d_model, M, C = scope["txl"], 2, 2, 64, 128, 48, 40
    g = torch.Generator().manual_seed(3)
    W_qkv, W_o, W_R = ((torch.randn(d_model, n, generator=g) * d_model ** -0.5).bfloat16().cuda()
                       for n in (3 * H * D, d_model, H * D))
    u, vb = (0.3 * torch.randn(H, D, generator=g).cuda() for _ in range(2))
    r = torch.empty(C + 1, H, D, dtype=torch.bfloat16, device="cuda")
    txl.rel_pos_gen(W_R, r, C + 1, d_model, H, D)
    mem = txl.QuantMemory.empty(B, M, H, D, bits=8)
    hist, pushed = [], 0
    for L in (40, 1, 1, 3, 20, 1):
        h = torch.randn(B, L, d_model, generator=g).bfloat16().cuda()
        y = scope["layer_step"](h, mem, W_qkv, W_o, u, vb, r, C)
        pushed += L
        assert y.shape == h.shape and mem.valid == min(pushed, M)
        q, k, v = (f64(x) for x in txl.linear(h.view(B * L, d_model), W_qkv).view(B, L, 3, H, D).unbind(2))
        keys, values = (np.concatenate([held(x[i], 8) for x in hist] + [cur], 1)[:, -(M + L):]
                        for i, cur in ((0, k), (1, v)))
        a, _ = attend64(q, keys, values, f64(u), f64(vb), f64(r), C)
        ref = a.reshape(B, L, H * D) @ f64(W_o)
        # the attention's output and the layer's are bf16 (2^-8 of their value at most), the first's operands 16 bits
        assert np.linalg.norm(f64(y) - ref) <= 3 * 2.0 ** -8 * np.linalg.norm(ref)
        hist.append((k, v))
