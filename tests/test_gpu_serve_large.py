"""Norms, page calls and shared prefixes whose offsets pass 32 bits. Tolerances are
those of test_gpu_serve and test_gpu_attn_shared."""
import numpy as np
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from oracle import serve_oracle as S
from test_gpu_attn_shared import Shared
from test_gpu_serve import TORCH, _f64, _norm_check, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,act,res", [(270_000, 8192, "bf16", "bf16"), (270_000, 8191, "bf16", "bf16"),
                                         (140_000, 16384, "bf16", "f32"), (1 << 24, 130, "bf16", "bf16")])
def test_norm_rows_whose_elements_pass_32_bits(T, H, act, res):
    gen = torch.Generator("cuda").manual_seed(T)
    rand = lambda dt: torch.randn(T, H, device="cuda", dtype=TORCH[dt], generator=gen)  # noqa: E731
    y, x, gate = rand(act), rand(res), rand(act)
    w = torch.randn(H, device="cuda", generator=gen)
    cfg = B.make_norm_config(H, "rms", act, res, True, "linear", 0.6, 0.0, 1e-5)
    xo, h = torch.full_like(x, 7), torch.full_like(y, 7)
    B.moe_norm(cfg, T, y, x, w, None, gate, w, None, xo, h)
    edge = (1 << 31) // H
    rows = [0, 1, edge // 2, edge - 1, edge, edge + 1, T - 2, T - 1]
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    r, want, dr, dh = S.norm(_f64(x[rows]), _f64(y[rows]), True, _f64(w), None, _f64(gate[rows]), False,
                             _f64(w), None, False, f32(0.6), 0.0, f32(1e-5))
    _norm_check(xo[rows], r, dr, res)
    _norm_check(h[rows], want, dh, act)
    assert not (h == 7).all(dim=1).any()                     # no row is left out


def test_pages_whose_bytes_pass_32_bits():
    pages, kv, dim, page = 300_000, 8, 128, 16
    cfg = B.make_attn_config(kv, kv, dim, page)
    caches = [torch.empty(pages, kv, page * dim * 9 // 8, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert caches[0].numel() > 1 << 32
    gen = torch.Generator("cuda").manual_seed(1)
    ends = [0, 3, 116_508, 233_016, pages - 2, pages - 1]    # the second 2^31 bytes begin near 116508
    for c in caches:
        for p in ends:
            c[p].random_(0, 256, generator=gen)
    f = B.make_kv_caches(cfg, caches)
    dst = [pages - 3, pages - 4, 1, pages - 5, 2, 233_015]
    B.moe_kv_copy_pages(cfg, f, f, len(ends), ints(ends), ints(dst))
    for c in caches:
        assert torch.equal(c[dst], c[ends])
    # a shared page that is copied, and the pages in use moved to the front
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    held, refs = ints([0, 0]), torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[pages - 6:] = 0
    pool = B.make_kv_pool(cfg, table, held, refs, f)
    ws = torch.empty(B.kv_pool_workspace_size(cfg, pool, 2), dtype=torch.uint8, device="cuda")
    B.moe_kv_reserve(cfg, pool, 1, ints([0]), ints([0]), ints([20]), ws)
    assert table[0].tolist() == [pages - 6, pages - 5, -1, -1]
    B.moe_kv_fork(cfg, pool, 1, ints([0]), ints([1]), ints([20]), ws)
    B.moe_kv_reserve(cfg, pool, 1, ints([1]), ints([20]), ints([21]), ws)
    assert B.moe_get_status(ws) == (0, 0) and table[1].tolist() == [pages - 6, pages - 4, -1, -1]
    for c in caches:
        assert torch.equal(c[pages - 4], c[pages - 5])
    refs[:pages - 6] = 0
    before = [[c[int(p)].clone() for p in table[1, :2]] for c in caches]
    used = ints([0])
    B.moe_kv_compact(cfg, pool, used, ws)
    assert B.moe_get_status(ws) == (0, 0)
    assert used.item() == 3 and table[:, :2].tolist() == [[0, 1], [0, 2]] and refs[:4].tolist() == [2, 1, 1, 0]
    for c, b in zip(caches, before):
        assert torch.equal(c[0], b[0]) and torch.equal(c[2], b[1])


@pytest.mark.parametrize("dtype,n", [("bf16", 3), ("bf16", 20), ("f32", 3)])
def test_shared_prefixes_on_pages_past_32_bits(dtype, n):
    c = Shared(120, dtype, 8, 2, 128, 16, [300 + i for i in range(n)], [1] * n, [0, n], [290])
    small, size = c.cache, c.cache[0].numel()
    more = (5 << 30) // size
    c.cache = torch.empty(more + small.shape[0], *small.shape[1:], dtype=torch.uint8, device="cuda")
    c.cache[more:] = small
    c.d["table"] += torch.where(c.d["table"] >= 0, more, 0).int()
    c.shared()
    assert c.status() == (0, 0)
    c.check()
