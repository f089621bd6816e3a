"""A bounded wait of the attention kernels for many rows that runs out: the call
comes back with MOE_ERR_TIMEOUT, nothing faults or hangs, and the next call, with
the limit restored, is right."""
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from test_gpu_attn import Case
from test_gpu_attn_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("shared", [False, True])
def test_wait_limit_runs_out_then_the_next_call_is_right(shared, D):
    if shared:
        c = Shared(130, "bf16", 16, 2, D, 64, [1400 + 9 * i for i in range(16)], [1] * 16, [0, 16], [1390])
        call, ws = c.shared, c.sws
    else:
        c = Case(131, "bf16", 16, 2, D, 64, [1400, 700], [60, 40])
        call, ws = c.run, c.ws
    try:
        B.set_wait_limit_ns(4)
        call()
        rc, flags = B.moe_get_status(ws)
        assert rc == 6 and flags & B.DEV_TIMEOUT, (rc, flags)
    finally:
        B.set_wait_limit_ns(0)
    torch.cuda.synchronize()
    call()
    assert B.moe_get_status(ws) == (0, 0)
    c.check()
