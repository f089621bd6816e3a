"""Shared prefixes of many groups, and groups that are larger than the caller says.
Tolerances are those of test_gpu_attn_shared."""
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from test_gpu_attn_shared import Shared

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups", [64, 65, 100])
@pytest.mark.parametrize("D,heads,kv,q", [(128, 16, 1, 1), (256, 16, 2, 2), (64, 8, 2, 3)])
def test_many_groups_whose_rows_take_the_prompt_kernel(D, heads, kv, q, groups):
    """Up to 64 groups the prefix kernel sums up its list itself, of more it takes
    the plan's. Groups of no, one and many requests, prefixes of none to several
    tiles, full and half-filled row tiles, beside one another."""
    sizes, prefixes = [4, 1, 0, 9, 17, 5, 2, 40], [96, 0, 31, 32, 160, 293, 130, 64, 256]
    lens, qs, bounds, prefix = [], [], [0], []
    for g in range(groups):
        n, p = sizes[g % 8], prefixes[g % 9]
        prefix.append(p)
        lens += [p + q + (3 * i + g) % 11 for i in range(n)]
        qs += [1 + (i + g) % q for i in range(n)]
        bounds.append(bounds[-1] + n)
    c = Shared(100 + groups + D, "bf16", heads, kv, D, 32, lens, qs, bounds, prefix)
    assert c.max_group * heads // kv >= 64          # rows from which on it is that kernel
    c.shared()
    assert c.status() == (0, 0)
    c.check()
    first = c.out.clone(), c.lse.clone()
    c.out.fill_(1.0)
    c.sws.fill_(0xff)
    c.shared()
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


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
