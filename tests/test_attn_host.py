"""The attention entry points without a GPU: the oracle against hand-made
checks, the config and argument checks of the C ABI, and the binding's."""
import ctypes
import math

import numpy as np
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from oracle import attn_oracle as A

OK = dict(num_heads=32, num_kv_heads=8, head_dim=128, page_size=64, rotary_dim=128,
          rope_positions=4096)
FAKE = 1 << 20


def _cfg(**kw):
    return B.make_attn_config(**{**OK, **kw})


# ---------------------------------------------------------------- the oracle
def test_e4m3_values_are_torchs():
    b = torch.arange(256, dtype=torch.uint8)
    np.testing.assert_array_equal(A.E4M3, b.view(torch.float8_e4m3fn).double().numpy())


def test_nearest_even_against_brute_force():
    rng = np.random.default_rng(0)
    x = np.concatenate([np.abs(rng.normal(size=500)) * 4, (A.LEVELS[1:] + A.LEVELS[:-1]) / 2, [9.0]])
    for v, i in zip(x, A.nearest_even(x, A.LEVELS)):
        d = np.abs(A.LEVELS - v)
        best = np.flatnonzero(d == d.min())
        assert i == (best[0] if len(best) == 1 else [b for b in best if b % 2 == 0][0])


def test_quantise_reaches_the_top_level_and_packs_both_ways():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 16, 2, 64)).astype(np.float32)
    x[0, 0, 0, :16] = 0
    x[0, 1, 0, 3] = np.nan
    x[0, 2, 0, 5] = np.inf
    codes, s = A.quantise(x)
    assert np.abs(codes).max() == 6 and (codes[0, 0, 0, :16] == 0).all() and codes[0, 1, 0, 3] == 0
    assert s[0, 2, 0, 0] == 0x7e and codes[0, 2, 0, 5] == 6
    cache = A.pack_cache((codes, s), (codes, s), 16)
    assert cache.shape == (3, 2, 16 * 64 * 9 // 8)
    for c2, s2 in A.unpack_cache(cache, 16, 64):
        np.testing.assert_array_equal(c2, codes)
        np.testing.assert_array_equal(s2, s)


def test_rotation_keeps_scores_relative():
    """q at p and k at p - 7 score the same for every p."""
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(2, 1, 1, 64))
    t = A.rope_table(np.arange(5000), 64, 1e4)
    for inter in (False, True):
        s = [float(np.sum(A.rotate(q, [p], t, 64, inter, dtype=np.float64)
                          * A.rotate(k, [p - 7], t, 64, inter, dtype=np.float64)))
             for p in (7, 100, 4999)]
        assert max(s) - min(s) < 1e-10
        back = A.rotate(A.rotate(q, [4999], t, 64, inter, dtype=np.float64), [4999], t, 64, inter,
                        inverse=True, dtype=np.float64)
        np.testing.assert_allclose(back, q, atol=1e-12)


def test_scaled_frequencies_meet_their_ends():
    f, _ = A.frequencies(128, 1e4)
    p, _ = A.frequencies(128, 1e4, kind="parts", factor=8, original=8192)
    y, gain = A.frequencies(128, 1e4, kind="yarn", factor=8, original=8192)
    for x in (p, y):
        assert x[0] == f[0] and math.isclose(x[-1], f[-1] / 8) and (x <= f).all()
    assert math.isclose(gain, 1 + 0.1 * math.log(8))
    n, _ = A.frequencies(128, 1e4, kind="ntk", factor=8)
    assert math.isclose(n[-1], f[-1] / 8)


def test_attention_oracle_against_a_dense_mask():
    rng = np.random.default_rng(3)
    n, m, w = 11, 4, 5
    q, k, v = rng.normal(size=(m, 4, 64)), rng.normal(size=(n, 2, 64)), rng.normal(size=(n, 2, 64))
    out, lse, _, _ = A.attention(q, k, v, n, 0.125, w)
    x = np.einsum("mhd,nhd->mhn", q, k.repeat(2, axis=1)) * 0.125
    pos, key = n - m + np.arange(m)[:, None], np.arange(n)
    x[~np.broadcast_to(((key <= pos) & (key > pos - w))[:, None], x.shape)] = -np.inf
    e = np.exp(x)
    np.testing.assert_allclose(lse, np.log(e.sum(-1)))
    np.testing.assert_allclose(out, np.einsum("mhn,nhd->mhd", e / e.sum(-1, keepdims=True),
                                              v.repeat(2, axis=1)))
    out, lse, _, _ = A.attention(q, k, v, 2, 0.125)      # two queries before the first token
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()


# ------------------------------------------------------------------ the ABI
@pytest.mark.parametrize("kw,expect", [
    (dict(), 0), (dict(num_heads=1, num_kv_heads=1), 0), (dict(act_dtype="f32"), 0),
    (dict(rotary_dim=0, rope_positions=0), 0), (dict(rotary_dim=2), 0),
    (dict(head_dim=80, rotary_dim=80), 0), (dict(head_dim=512), 0), (dict(window=1), 0),
    (dict(num_heads=30), 1), (dict(num_heads=0), 1), (dict(num_kv_heads=0), 1),
    (dict(head_dim=0), 1), (dict(head_dim=127), 1), (dict(page_size=8), 1),
    (dict(page_size=48), 1), (dict(page_size=512), 1), (dict(rotary_dim=3), 1),
    (dict(rotary_dim=130), 1), (dict(rotary_dim=-2), 1), (dict(rope_positions=0), 1),
    (dict(window=-1), 1), (dict(softmax_scale=float("nan")), 1), (dict(softmax_scale=-1.0), 1),
    (dict(k_scale=0.0), 1), (dict(k_scale=1e-45), 1), (dict(v_scale=float("inf")), 1),
    (dict(head_dim=514), 2), (dict(num_heads=1024), 2),
])
def test_validate_attn_config(kw, expect):
    assert B.validate_attn_config(_cfg(**kw)) == expect


def test_page_bytes_and_workspace_sizes():
    assert B.kv_page_bytes(_cfg()) == 8 * 64 * 128 * 9 // 8
    assert B.kv_page_bytes(_cfg(head_dim=80, rotary_dim=0)) == 0
    assert B.kv_page_bytes(_cfg(page_size=3)) == 0
    assert B.kv_attention_workspace_size(_cfg(), 4, 4, 1) > 0
    for args in ((-1, 4, 1), (4, -1, 1), (4, 4, -1), (4, (1 << 18) + 1, 1), ((1 << 18) + 1, 4, 1)):
        assert B.kv_attention_workspace_size(_cfg(), *args) == 0
    assert B.kv_attention_workspace_size(_cfg(head_dim=96, rotary_dim=0), 4, 4, 1) == 0


def _call(name, cfg, args):
    return getattr(B.lib(), name)(ctypes.byref(cfg), *args)


def _refused(name, cfg, good, changes):
    """Each change of one argument of a good call gives its status."""
    for i, value, status in changes:
        args = list(good)
        args[i] = value
        assert _call(name, cfg, args) == status, (name, i, value)


def test_rope_table_refusals():
    sc = lambda **kw: ctypes.byref(B.make_rope_scaling(**kw))  # noqa: E731
    good = [8, FAKE, sc(), FAKE, None, 0, None]
    _refused("moe_rope_table", _cfg(), good, [
        (0, -1, 1), (0, (1 << 24) + 1, 1), (1, FAKE + 2, 1), (3, None, 1), (3, FAKE + 4, 1),
        (2, None, 1), (2, sc(base=1.0), 1), (2, sc(base=float("inf")), 1),
        (2, sc(kind="linear", factor=0.5), 1), (2, sc(kind="parts", factor=2), 1),
        (2, sc(kind="yarn", factor=2, original_positions=100, slow_turns=9, fast_turns=3), 1),
        (2, sc(attention_factor=-1.0), 1)])
    assert _call("moe_rope_table", _cfg(rotary_dim=0), good) == 1
    assert _call("moe_rope_table", _cfg(rotary_dim=2), [8, FAKE, sc(kind="ntk", factor=2), FAKE,
                                                       None, 0, None]) == 1
    assert _call("moe_rope_table", _cfg(), [8, FAKE, sc(), FAKE, FAKE, 3, None]) == 3
    assert _call("moe_rope_table", _cfg(), [0, None, sc(), None, None, 0, None]) == 0


def test_rope_refusals():
    good = [4, 32, FAKE, 4096, 128, FAKE, FAKE, 0, FAKE * 2, None, 0, None]
    _refused("moe_rope", _cfg(), good, [
        (0, -1, 1), (0, (1 << 18) + 1, 1), (1, 0, 1), (1, 513, 1), (2, None, 1), (2, FAKE + 1, 1),
        (3, -1, 1), (4, 64, 1), (4, -128, 1), (5, None, 1), (6, None, 1), (6, FAKE + 4, 1),
        (8, None, 1), (8, FAKE + 2, 1), (9, FAKE + 2, 3)])
    # in place, but the rows are not contiguous
    assert _call("moe_rope", _cfg(), [4, 32, FAKE, 8192, 128, FAKE, FAKE, 0, FAKE, None, 0, None]) == 1
    assert _call("moe_rope", _cfg(), [0] + [1] + [None] + [0, 0] + [None, None, 0, None, None, 0, None]) == 0


def test_rope_ignores_the_head_counts():
    cfg = _cfg(num_heads=3, num_kv_heads=2)
    assert B.validate_attn_config(cfg) == 1
    assert _call("moe_rope", cfg, [0, 1, None, 0, 0, None, None, 0, None, None, 0, None]) == 0
    assert _call("moe_rope_table", cfg, [0, None, ctypes.byref(B.make_rope_scaling()), None, None,
                                         0, None]) == 0
    assert _call("moe_kv_read", cfg, [0, None, None, 0, None, None, None, 0, None]) == 1


def test_append_and_read_refusals():
    good = [4, FAKE, 4096, 128, FAKE, 1024, 128, FAKE, 1024, 128, FAKE, FAKE, FAKE, FAKE * 2, FAKE,
            10, None, 0, None]
    _refused("moe_kv_append", _cfg(), good, [
        (0, -1, 1), (4, None, 1), (5, -1, 1), (6, 100, 1), (7, None, 1), (7, FAKE + 1, 1),
        (10, None, 1), (11, None, 1), (11, FAKE + 4, 1), (12, None, 1), (13, None, 1),
        (14, None, 1), (14, FAKE + 8, 1), (15, 0, 1), (15, 1 << 40, 1), (16, FAKE + 1, 3)])
    assert _call("moe_kv_append", _cfg(head_dim=96, rotary_dim=96), good) == 2
    assert _call("moe_kv_append", _cfg(), [0] + [None, 0, 0] * 3 + [None] * 5 + [0, None, 0, None]) == 0
    good = [4, FAKE, FAKE, 10, FAKE, FAKE, None, 0, None]
    _refused("moe_kv_read", _cfg(), good, [
        (0, -1, 1), (1, None, 1), (2, None, 1), (3, 0, 1), (4, None, 1), (5, FAKE + 8, 1)])
    assert _call("moe_kv_read", _cfg(head_dim=80, rotary_dim=0), good) == 2


def test_attention_refusals():
    cfg = _cfg()
    need = B.kv_attention_workspace_size(cfg, 2, 4, 2)
    good = [2, 4, 2, FAKE, 4096, 128, FAKE, FAKE, FAKE, 8, FAKE, 10, FAKE, FAKE, FAKE, need, None]
    _refused("moe_kv_attention", cfg, good, [
        (0, -1, 1), (0, 0, 1), (1, -1, 1), (2, 0, 1), (3, None, 1), (3, FAKE + 8, 1), (4, 4100, 1),
        (5, 129, 1), (5, 64, 1), (6, None, 1), (7, None, 1), (8, None, 1), (9, 0, 1),
        (9, (1 << 20) + 1, 1), (10, None, 1), (10, FAKE + 8, 1), (11, 0, 1), (12, None, 1),
        (13, FAKE + 2, 1), (14, None, 3), (14, FAKE + 8, 3), (15, need - 1, 3)])
    assert _call("moe_kv_attention", _cfg(head_dim=80, rotary_dim=0), good) == 2
    assert _call("moe_kv_attention", cfg, [0, 0, 0] + [None, 0, 0] + [None] * 3 + [0, None, 0] +
                 [None] * 3 + [0, None]) == 0


def test_binding_checks_types_shapes_and_devices():
    cfg = _cfg()
    q = torch.zeros(4, 32, 128, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        B.moe_rope(cfg, 4, q, pos, None, q)
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        B.moe_rope(cfg, 4, q.float(), pos, None, q)
    with pytest.raises(ValueError, match="must have shape"):
        B.moe_kv_append(cfg, 5, q, q, q, pos, pos, None, q, q)
    with pytest.raises(ValueError, match="must be torch.int64"):
        B._typed("slots", pos, "i64", (4,))
    with pytest.raises(KeyError):
        B.make_attn_config(8, 8, 128, act_dtype="f16")
