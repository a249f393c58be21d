"""The kernels of the quantised memory start before the kernels in front of them have ended, so what those may write (the
memory's rows, q, k, v, r, the workspace) is not read through the read-only path, which wants data that nobody
writes while a kernel runs: __ldg is left to the biases."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "transformer_xl_relative_gb300", "csrc")


def test_only_the_biases_take_the_read_only_path():
    for name in ("txl_qmem.cu", "txl_qmem_attn.cu", "txl_qmem_seg.cu", "txl_rows.cuh", "txl_attn_common.cuh"):
        text = re.sub(r"//.*", "", open(os.path.join(CSRC, name), encoding="utf-8").read())
        assert not re.search(r"__ldg\((?!p\.(u|vb) )|ld\.global\.nc|__restrict__", text), name
    for name in ("txl_attn_persist.cu", "txl_attn_tc.cu"):
        text = open(os.path.join(CSRC, name), encoding="utf-8").read()
        assert not re.search(r"__ldg\([^;]*\b(units|un)\b", text), name
