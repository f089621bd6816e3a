"""Edges of the attention entry points on the GPU, against the fp64 oracle.

Tolerances are those of Case.check unless a test derives its own.
"""
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- windows
WINDOWS = [  # dtype, heads, kv heads, lens, query tokens; queries before the first token among them
    ("bf16", 1, 1, [5, 90, 0], [10, 3, 1]),             # rows 4, 8 and 16 of the split kernel
    ("bf16", 6, 2, [2, 40, 33], [5, 2, 1]),
    ("f32", 2, 1, [3, 70], [9, 2]),
    ("bf16", 8, 2, [10, 300, 1], [64, 20, 30]),         # the prompt kernel
    ("bf16", 4, 4, [1, 700, 200], [150, 300, 0]),
]


@pytest.mark.parametrize("i", range(len(WINDOWS)))
@pytest.mark.parametrize("window", ["int_max", "int_max - 2", "2^30", "table", "table - 1", "table + 1"])
def test_windows_as_wide_as_any_number(i, window):
    """A window counts back from positions that may lie before the first token:
    the widest of an int must act as none, beside requests of the usual kind."""
    dtype, heads, kv, lens, qs = WINDOWS[i]
    c = Case(200 + i, dtype, heads, kv, 128, 16, lens, qs)
    cap = c.table.shape[1] * 16
    c.window = {"int_max": 2 ** 31 - 1, "int_max - 2": 2 ** 31 - 3, "2^30": 1 << 30, "table": cap,
                "table - 1": cap - 1, "table + 1": cap + 1}[window]
    c.cfg.window = c.window
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    c.window = c.cfg.window = 0                         # no request has as many tokens
    c.run()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
