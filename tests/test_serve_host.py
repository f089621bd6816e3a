"""Shared pages and norms without a GPU: the oracles against hand-made checks,
and the refusals of the C ABI and of the binding."""
import ctypes

import numpy as np
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from oracle import serve_oracle as S

CFG = dict(num_heads=8, num_kv_heads=2, head_dim=64, page_size=16)
FAKE = 1 << 20
BIG = 1 << 40


# ---------------------------------------------------------------- the oracles
def test_pool_oracle_by_hand():
    o = S.Pool(np.full((3, 4), -1, np.int32), np.zeros(3, np.int32), np.zeros(6, np.int32), 16,
               [np.arange(6)[:, None].repeat(2, 1)])
    assert o.reserve([1], [0], [20]) == 0 and o.table[1].tolist() == [0, 1, -1, -1]
    assert o.fork([1, 1], [0, 2], [20, 16]) == 0
    assert o.refs.tolist() == [3, 2, 0, 0, 0, 0]
    assert o.reserve([0], [20], [21]) == 0                 # the partly filled page becomes its own
    assert o.table[0, :2].tolist() == [0, 2] and o.caches[0][2, 0] == 1
    assert o.refs.tolist() == [3, 1, 1, 0, 0, 0]
    assert o.release([1, 1], [16, 40]) == 0 and o.refs.tolist() == [3, 0, 1, 0, 0, 0]
    assert o.compact() == (2, 0)
    assert o.table[0, :2].tolist() == [0, 1] and o.refs.tolist() == [3, 1, 0, 0, 0, 0]
    assert o.caches[0][1, 0] == 1
    assert o.reserve([0, 2], [64, 16], [64, 64]) == S.NO_PAGE    # 2 of the 4 free pages, 3 more do not fit
    assert o.reserve([1, 2], [16, 64], [33, 64]) == S.NO_PAGE and o.held.tolist() == [4, 3, 1]
    assert o.fork([0], [0], [1]) == S.BAD_ROW


def test_norm_oracle_by_hand():
    x = np.array([[3.0, -3.0, 3.0, -3.0]])
    r, h, dr, dh = S.norm(x, eps=1e-12)
    np.testing.assert_allclose(h, [[1, -1, 1, -1]])
    r, h, _, _ = S.norm(x + 5, y=np.ones((1, 4)), layer=True, scale=2.0, offset=1.0, pre_w=np.ones(4), eps=1e-12)
    np.testing.assert_allclose(r, x + 7)
    np.testing.assert_allclose(h, [[2, -2, 2, -2]])
    assert (dr >= 0).all() and (dh < 1e-4).all()


def test_norm_bound_covers_fp32_and_is_tight():
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=(2, 50, 300)).astype(np.float32)
    r, h, dr, dh = S.norm(x, y, post=True, layer=True, gate=y, sigmoid=True)
    f = lambda v: ((v - v.mean(-1, keepdims=True)) / np.sqrt(v.var(-1, keepdims=True) + np.float32(1e-6)))  # noqa: E731
    r32 = x + f(y) / (1 + np.exp(-y))
    assert r32.dtype == np.float32
    assert (np.abs(r32 - r) <= dr).all() and (np.abs(f(r32) - h) <= dh).all()
    assert (dh < 2e-5 * (1 + np.abs(h))).all()


# ------------------------------------------------------------------- the ABI
def _caches(n=2, pages=20, pointer=FAKE):
    array = (ctypes.c_void_p * max(n, 1))(*[pointer] * n)
    c = B.KvCaches(n, pages, array)
    c.keep = array
    return c


def _pool(rows=4, width=8, table=FAKE, held=FAKE, refs=FAKE, **kw):
    c = _caches(**kw)
    p = B.KvPool(table, held, refs, rows, width, c)
    p.keep = c
    return p


POOLS = [
    (dict(), 0), (dict(rows=0), 1), (dict(rows=(1 << 18) + 1), 1), (dict(width=0), 1),
    (dict(width=(1 << 20) + 1), 1), (dict(table=None), 1), (dict(held=FAKE + 2), 1), (dict(refs=FAKE + 4), 0), (dict(refs=FAKE + 1), 1),
    (dict(n=0), 1), (dict(n=257), 1), (dict(pages=0), 1), (dict(pages=(1 << 30) + 1), 1),
    (dict(pointer=None), 1), (dict(pointer=FAKE + 8), 1),
]


@pytest.mark.parametrize("kw,expect", POOLS)
def test_pools_are_checked(kw, expect):
    cfg, pool = B.make_attn_config(**CFG), _pool(**kw)
    L, c, p = B.lib(), ctypes.byref(cfg), ctypes.byref(pool)
    assert (B.kv_pool_workspace_size(cfg, pool, 3) == 0) == (expect != 0)
    # n = 0 (and a workspace too small) return before any CUDA call
    assert L.moe_kv_fork(c, p, 0, None, None, None, None, 0, None) == expect
    assert L.moe_kv_reserve(c, p, 0, None, None, None, None, 0, None) == expect
    assert L.moe_kv_release(c, p, 0, None, None, None, 0, None) == expect
    assert L.moe_kv_compact(c, p, None, None, 0, None) == (expect or 3)


def test_items_of_pool_calls_are_checked():
    cfg, pool = B.make_attn_config(**CFG), _pool()
    L, c, p = B.lib(), ctypes.byref(cfg), ctypes.byref(pool)
    need = B.kv_pool_workspace_size(cfg, pool, 3)
    for n in (-1, (1 << 18) + 1):
        assert B.kv_pool_workspace_size(cfg, pool, n) == 0
        assert L.moe_kv_fork(c, p, n, FAKE, FAKE, FAKE, None, 0, None) == 1
        assert L.moe_kv_reserve(c, p, n, FAKE, FAKE, FAKE, FAKE, BIG, None) == 1
        assert L.moe_kv_release(c, p, n, FAKE, None, None, 0, None) == 1
    for bad in (None, FAKE + 2):
        assert L.moe_kv_fork(c, p, 3, bad, FAKE, FAKE, None, 0, None) == 1
        assert L.moe_kv_fork(c, p, 3, FAKE, bad, FAKE, None, 0, None) == 1
        assert L.moe_kv_fork(c, p, 3, FAKE, FAKE, bad, None, 0, None) == 1
        assert L.moe_kv_reserve(c, p, 3, None, bad, FAKE, FAKE, BIG, None) == 1
        assert L.moe_kv_reserve(c, p, 3, None, FAKE, bad, FAKE, BIG, None) == 1
    assert L.moe_kv_reserve(c, p, 5, None, FAKE, FAKE, FAKE, BIG, None) == 1     # rows 0 .. 4 of 4
    assert L.moe_kv_release(c, p, 5, None, None, None, 0, None) == 1
    assert L.moe_kv_reserve(c, p, 3, None, FAKE, FAKE, FAKE, need - 1, None) == 3
    assert L.moe_kv_reserve(c, p, 3, None, FAKE, FAKE, None, need, None) == 3
    assert L.moe_kv_fork(c, p, 3, FAKE, FAKE, FAKE, FAKE, 3, None) == 3
    assert L.moe_kv_release(c, p, 3, FAKE, FAKE + 1, FAKE, 4, None) == 1
    assert L.moe_kv_compact(c, p, FAKE + 1, FAKE, BIG, None) == 1
    assert L.moe_kv_fork(c, None, 3, FAKE, FAKE, FAKE, None, 0, None) == 1
    bad = B.make_attn_config(**{**CFG, "head_dim": 96})
    assert L.moe_kv_fork(ctypes.byref(bad), p, 0, None, None, None, None, 0, None) == 2
    bad = B.make_attn_config(**{**CFG, "page_size": 20})
    assert L.moe_kv_compact(ctypes.byref(bad), p, None, FAKE, BIG, None) == 1


def test_copies_of_pages_are_checked():
    cfg, a, b = B.make_attn_config(**CFG), _caches(), _caches(pages=9)
    L, c = B.lib(), ctypes.byref(cfg)
    call = lambda f, t, n, s=FAKE, d=FAKE, ws=None, size=0: L.moe_kv_copy_pages(  # noqa: E731
        c, ctypes.byref(f), ctypes.byref(t), n, s, d, ws, size, None)
    assert call(a, b, 0) == 0
    assert call(a, _caches(n=3), 0) == 1 and call(_caches(n=0), b, 0) == 1 and call(a, _caches(pages=0), 0) == 1
    assert call(a, b, -1) == 1 and call(a, b, 2, s=None) == 1 and call(a, b, 2, d=FAKE + 1) == 1
    assert call(a, b, 2, ws=FAKE, size=2) == 3
    assert L.moe_kv_copy_pages(c, None, ctypes.byref(b), 2, FAKE, FAKE, None, 0, None) == 1


@pytest.mark.parametrize("kw,expect", [
    (dict(), 0), (dict(kind="layer", act_dtype="f32", residual_dtype="bf16", gate="sigmoid"), 0),
    (dict(hidden_size=1), 0), (dict(hidden_size=0), 1), (dict(hidden_size=16385), 2),
    (dict(eps=0.0), 1), (dict(eps=float("inf")), 1), (dict(residual_scale=float("nan")), 1),
    (dict(weight_offset=float("inf")), 1),
])
def test_validate_norm_config(kw, expect):
    assert B.validate_norm_config(B.make_norm_config(**{"hidden_size": 64, **kw})) == expect


def test_norm_arguments_are_checked():
    cfg = B.make_norm_config(64)
    L, c = B.lib(), ctypes.byref(cfg)

    def call(T=2, y=FAKE, ys=64, x=2 * FAKE, xs=64, pw=None, pb=None, g=None, gt=0, gc=1, nw=None, nb=None,
             xo=3 * FAKE, h=4 * FAKE, ws=None, size=0):
        return L.moe_norm(c, T, y, ys, x, xs, pw, pb, g, gt, gc, nw, nb, xo, h, ws, size, None)

    assert call(T=0, x=None) == 0
    for kw in (dict(T=-1), dict(T=(1 << 24) + 1), dict(x=None), dict(xo=None, h=None), dict(ys=63), dict(xs=-64),
               dict(xs=BIG), dict(y=FAKE + 1), dict(x=FAKE + 1), dict(pw=FAKE + 4), dict(nb=FAKE + 8),
               dict(xo=FAKE + 2), dict(h=FAKE + 2), dict(g=FAKE + 1), dict(g=FAKE, gc=2), dict(g=FAKE, gt=-1),
               dict(y=None), dict(y=None, xo=None, pw=FAKE), dict(y=None, xo=None, g=FAKE),
               dict(x=3 * FAKE, xs=80), dict(y=4 * FAKE, ys=80), dict(h=2 * FAKE), dict(xo=FAKE),
               dict(xo=4 * FAKE)):
        assert call(**kw) == 1, kw
    assert call(ws=FAKE, size=3) == 3
    assert L.moe_norm(None, *[0] * 16, None) == 1


def test_shared_attention_arguments_are_checked():
    cfg = B.make_attn_config(**CFG)
    L, c = B.lib(), ctypes.byref(cfg)
    size = lambda *a: B.kv_attention_shared_workspace_size(cfg, *a)  # noqa: E731
    for bad in ((-1, 4, 1, 1, 4), (4, -1, 1, 1, 4), (4, 4, -1, 1, 4), (4, 4, 1, -1, 4), (4, 4, 1, 1, -1),
                (4, (1 << 18) + 1, 1, 1, 4), (4, 4, 1, (1 << 18) + 1, 4)):
        assert size(*bad) == 0
    need = size(4, 4, 1, 1, 4)
    assert need > 4 * 4 * 8 * 64 and size(4, 4, 1, 1, 400) > need      # (the prompt kernel's pieces)
    # without groups, with a window, or with many rows per request: as moe_kv_attention
    assert size(4, 4, 1, 0, 0) == B.kv_attention_workspace_size(cfg, 4, 4, 1)
    assert size(4, 128, 32, 1, 128) == B.kv_attention_workspace_size(cfg, 4, 128, 32)
    w = B.make_attn_config(**CFG, window=9)
    assert B.kv_attention_shared_workspace_size(w, 4, 4, 1, 1, 4) == B.kv_attention_workspace_size(w, 4, 4, 1)

    def call(seqs=4, T=4, mq=1, groups=1, mg=4, q=FAKE, ts=512, hs=64, offs=None, lens=FAKE, table=FAKE, mp=8,
             go=FAKE, pl=FAKE, cache=FAKE, pages=9, out=FAKE, lse=None, ws=FAKE, size=need, cfg=c):
        return L.moe_kv_attention_shared(cfg, seqs, T, mq, groups, mg, q, ts, hs, offs, lens, table, mp, go, pl,
                                         cache, pages, out, lse, ws, size, None)

    assert call(T=0, seqs=0, q=None) == 0
    for kw in (dict(groups=-1), dict(mg=-1), dict(mg=0), dict(go=None), dict(pl=None), dict(go=FAKE + 2),
               dict(pl=FAKE + 1), dict(q=None), dict(q=FAKE + 8), dict(ts=509), dict(hs=60), dict(seqs=3),
               dict(lens=None), dict(table=None), dict(mp=0), dict(mp=(1 << 20) + 1), dict(cache=None),
               dict(pages=0), dict(out=FAKE + 4), dict(lse=FAKE + 2), dict(mq=0), dict(T=-1)):
        assert call(**kw) == 1, kw
    assert call(size=need - 1) == 3 and call(ws=None) == 3 and call(ws=FAKE + 8) == 3
    assert call(groups=0, go=None, pl=None, size=8) == 3
    bad = B.make_attn_config(**{**CFG, "head_dim": 96})
    assert call(cfg=ctypes.byref(bad)) == 2


def test_binding_refuses_wrong_tensors():
    cfg = B.make_attn_config(**CFG)
    with pytest.raises(ValueError, match="at least one"):
        B.make_kv_caches(cfg, [])
    with pytest.raises(ValueError, match="torch.uint8"):
        B.make_kv_caches(cfg, [torch.zeros(3, 2, 1152)])
    with pytest.raises(ValueError, match="device tensors"):
        B.make_kv_caches(cfg, [torch.zeros(3, 2, 1152, dtype=torch.uint8)])
    with pytest.raises(ValueError, match="torch.int32"):
        B.make_kv_pool(cfg, torch.zeros(3, 4), None, None, _caches())
    n = B.make_norm_config(64)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    for y, match in ((x.float(), "bfloat16"), (x[:1], "shape"), (x, "device tensors")):
        with pytest.raises(ValueError, match=match):
            B.moe_norm(n, 2, y, x, None, None, None, None, None, None, x)
    for g, match in ((x.float(), "bfloat16"), (x[:, :7], "device"), (x, "device")):
        with pytest.raises(ValueError, match=match):
            B._gate(g, n, 2)
