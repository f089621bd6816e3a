"""Groups of requests that are larger than the caller says. Tolerances are those of test_gpu_attn_shared."""
import pytest

from expert_moe_layer_gb300 import binding as B
from test_gpu_attn_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,n,most", [("bf16", 3, 2), ("bf16", 20, 19), ("f32", 3, 1)])
@pytest.mark.parametrize("told", [0, 31, 32, 90])
def test_a_group_of_too_many_tokens_is_flagged_whatever_its_prefix(dtype, n, most, told):
    lens = [100 + i for i in range(n)]
    for max_group in (most, n):
        c = Shared(110, dtype, 8, 2, 64, 16, lens, [1] * n, [0, n], [96], told=[told], max_group=max_group)
        c.shared()
        assert c.status() == ((5, B.DEV_BAD_SEGMENT) if max_group < n else (0, 0))
        c.check()


def test_a_group_of_too_many_tokens_does_not_end_the_sharing_of_others():
    lens = [130 + i for i in range(30)]
    c = Shared(111, "bf16", 8, 2, 128, 16, lens, [1] * 30, [0, 10, 30], [96, 128], max_group=19)
    c.shared()
    assert c.status() == (5, B.DEV_BAD_SEGMENT)
    c.check()
    # requests without queries do not count
    qs = [1] * 19 + [0] * 11
    c = Shared(112, "bf16", 8, 2, 128, 16, lens, qs, [0, 10, 30], [0, 20], max_group=10)
    c.shared()
    assert c.status() == (0, 0)
    c.check()
