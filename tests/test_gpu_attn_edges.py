"""Edges of the attention entry points on the GPU, against the fp64 oracle.

Tolerances are those of Case.check unless a test derives its own.
"""
import decimal
import math
import random

import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from oracle import attn_oracle as A
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


# --------------------------------------------------------- scores of fp32 layers
def _one_key(D, heads, q):
    """fp32 queries [heads, D] of one kv head over a single cached key whose
    channels are all 6: the denominator is 1 and lse is the score itself."""
    cfg = B.make_attn_config(heads, 1, D, 16, "f32")
    k = torch.full((1, 1, D), 6.0, device="cuda")
    cache = torch.zeros(1, 1, 16 * D * 9 // 8, dtype=torch.uint8, device="cuda")
    B.moe_kv_append(cfg, 1, None, k, k, None, torch.zeros(1, dtype=torch.int64, device="cuda"), None,
                    None, cache)
    out, lse = torch.empty(1, heads, D, device="cuda"), torch.empty(1, heads, device="cuda")
    ws = torch.empty(B.kv_attention_workspace_size(cfg, 1, 1, 1), dtype=torch.uint8, device="cuda")
    B.moe_kv_attention(cfg, 1, 1, 1, q[None].cuda(), None, torch.ones(1, dtype=torch.int32, device="cuda"),
                       torch.zeros(1, 1, dtype=torch.int32, device="cuda"), cache, out, lse, ws)
    assert B.moe_get_status(ws) == (0, 0)
    # the weight is p over itself: p as two f16, the exponential and the sums (test_gpu_attn's terms)
    assert ((out.double() - 6).abs() <= 6 * (2.0 ** -24 + 2.0 ** -21 + 32 * 2.0 ** -23 + 2.0 ** -21)).all()
    score = 6.0 * q.double().sum(1) * D ** -0.5
    reach = 6.0 * q.double().abs().sum(1) * D ** -0.5
    return lse[0].double().cpu(), score, reach


def _score_bound(D, score, reach):
    """Of the score, relative to the sum of |q k|, in units of 2^-23: the queries
    are held in 22 bits (2); 32 channels at a time go through the matrix unit, the
    high terms in two steps that lose up to 2 each, the low terms 2^-11 of that
    (4.5); D/32 - 1 fp32 additions (half of that). Of lse: the gain, the maximum,
    the base, the logarithm's sum and the factor to natural units round once each
    (2.5, with the factor's own error 3), and the exponential and the logarithm add
    2^-21."""
    return 2.0 ** -23 * ((6.5 + (D / 32 - 1) / 2) * reach + 3 * score.abs()) + 2.0 ** -21


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 4, 8])
def test_f32_scores_do_not_lose_their_small_parts(D, heads):
    """One channel carries the score; one channel of every other 16 adds a little
    whose high and low halves both end just below a bit of the running sum."""
    q = torch.zeros(heads, D, dtype=torch.float64)
    ulp = 2.0 ** -13                          # of 6 * 172 in fp32
    for h in range(heads):
        small = (1025 + 2 * h) * 2.0 ** -15   # f16; 6 * small is half an ulp over whole ones
        q[h, 4:D // 4:4] = small + 0.74 / 6 * ulp
    q[:, 0] = 172.0
    q = (q * 2.0 ** 3).float()                # scores of several hundred
    got, score, reach = _one_key(D, heads, q)
    assert ((got - score).abs() <= _score_bound(D, score, reach)).all(), \
        ((got - score) / (2.0 ** -23 * reach)).tolist()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_f32_scores_of_large_queries(D):
    gen = torch.Generator().manual_seed(D)
    q = torch.randn(8, D, generator=gen).abs() * 100
    q[4:] *= torch.randn(4, D, generator=gen).sign()
    got, score, reach = _one_key(D, 8, q)
    assert ((got - score).abs() <= _score_bound(D, score, reach)).all(), \
        ((got - score) / (2.0 ** -23 * reach)).tolist()


# -------------------------------------------------------------------- append
APPENDS = [  # dtype, T, heads, kv heads, D, R, elements before the rows: each rotation kernel, few and many tokens
    ("bf16", 9, 4, 2, 128, 64, 0), ("bf16", 700, 24, 8, 128, 128, 0),
    ("bf16", 9, 4, 2, 128, 66, 0), ("bf16", 700, 24, 8, 128, 34, 0),
    ("bf16", 9, 4, 2, 64, 64, 1), ("f32", 11, 3, 1, 256, 256, 0), ("f32", 11, 3, 1, 64, 30, 0),
]


def _append_inputs(dtype, T, heads, kv, D, R, skew, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    cfg = B.make_attn_config(heads, kv, D, 16, dtype, R, "half", 50)
    flat = torch.randn(skew + T * (heads + 2 * kv) * D, generator=gen, device="cuda").to(dt)
    rows = flat[skew:].view(T, heads + 2 * kv, D)
    table = torch.randn(50, R, generator=gen, device="cuda")
    pos = torch.randint(0, 50, (T,), generator=gen, device="cuda", dtype=torch.int32)
    pages = T // 16 + 2
    slots = torch.randperm(pages * 16, generator=gen, device="cuda")[:T]
    cache = torch.zeros(pages, kv, 16 * D * 9 // 8, dtype=torch.uint8, device="cuda")
    return cfg, rows[:, :heads], rows[:, heads:heads + kv], rows[:, heads + kv:], pos, slots, table, cache


@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append_skips_the_queries_of_a_bad_slot(i):
    """A slot of -1 takes a token's queries alone; one outside the cache nothing."""
    cfg, q, k, v, pos, slots, table, cache = _append_inputs(*APPENDS[i], seed=i)
    T = q.shape[0]
    want = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    B.moe_rope(cfg, T, q, pos, table, want)
    good = cache.clone()
    B.moe_kv_append(cfg, T, None, k, v, pos, slots, table, None, good)
    slots[1], slots[3], slots[T - 1], slots[5] = -2, cache.shape[0] * 16, 1 << 40, -1
    out = torch.full_like(want, 5.0)
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    B.moe_kv_append(cfg, T, q, k, v, pos, slots, table, out, cache, ws)
    assert B.moe_get_status(ws) == (5, B.DEV_BAD_SLOT)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[[1, 3, T - 1]] = True
    assert (out[bad] == 5).all()
    assert torch.equal(out[~bad], want[~bad])
    # the other tokens' keys and values, and nothing else
    again = torch.zeros_like(cache)
    keep = ~bad
    keep[5] = False
    n = int(keep.sum())
    B.moe_kv_append(cfg, n, None, k[keep], v[keep], pos[keep], slots[keep], table, None, again)
    assert torch.equal(cache, again) and not torch.equal(cache, good)


@pytest.mark.parametrize("i", range(len(APPENDS)))
def test_append_rotates_queries_in_place(i):
    cfg, q, k, v, pos, slots, table, cache = _append_inputs(*APPENDS[i], seed=50 + i)
    T = q.shape[0]
    want = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    B.moe_kv_append(cfg, T, q, k, v, pos, slots, table, want, cache)
    own, again = q.contiguous().clone(), torch.zeros_like(cache)
    B.moe_kv_append(cfg, T, own, k, v, pos, slots, table, own, again)
    assert torch.equal(own, want) and torch.equal(again, cache)


# --------------------------------------------------------------------- table
@pytest.mark.parametrize("base,original,scaled", [(4.0, 131072.0, False), (1e4, 4.0, True),
                                                  (1e4, 1e12, False), (1e6, 0.5, True)])
@pytest.mark.parametrize("R", [64, 96, 128])
def test_yarn_whose_ramp_lies_on_one_side_of_the_pairs(base, original, scaled, R):
    """Every pair turns more than 32 times in the original context and keeps its
    frequency, or less than once and is slowed down by the factor. Positions are
    small, so that fp64 angles are exact to 2^-45: the table's bound is its series'
    2^-29 and 2^-29 of the angle that is cut off, two roundings of the fractions,
    one of the gain and of its product, all on values up to the gain."""
    n, factor = 200, 8.0
    f = base ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)
    turns = original * f / (2 * math.pi)
    assert (turns < 1).all() if scaled else (turns > 32).all()
    a = torch.arange(n, dtype=torch.float64)[:, None] * (f / factor if scaled else f)
    gain = 0.1 * math.log(factor) + 1
    want = gain * torch.cat([a.cos(), a.sin()], 1)
    cfg = B.make_attn_config(1, 1, 128, rotary_dim=R, rope_positions=n)
    out = torch.empty(n, R, device="cuda")
    B.moe_rope_table(cfg, n, None, B.make_rope_scaling(base, "yarn", factor, original), out)
    assert ((out.double().cpu() - want).abs() <= 4 * 2.0 ** -24 * gain).all()


PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("R,base", [(64, 1e4), (128, 1e6), (96, 1e4), (34, 5e5)])
def test_table_at_far_positions(R, base):
    """Against angles reduced with 60 digits. The table's own bound is that of the
    test above. A frequency is fp64's power (2^-52), its turns a division by a
    rounded 2 pi (2^-53 and 2^-54) cut to 2^-64, and its exponent is rounded, which
    ln(base) multiplies: the position multiplies all of them."""
    pos = [0, 1, -1, 4095, 131071, 1 << 20, (1 << 20) - 1, 16777213, -16777213, 1 << 27, 2 ** 31 - 1, -2 ** 31]
    cfg = B.make_attn_config(1, 1, 128, rotary_dim=R, rope_positions=len(pos))
    out = torch.empty(len(pos), R, device="cuda")
    B.moe_rope_table(cfg, len(pos), torch.tensor(pos, dtype=torch.int32, device="cuda"),
                     B.make_rope_scaling(base), out)
    got = out.double().cpu()
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        f = [decimal.Decimal(base) ** (decimal.Decimal(-2 * i) / R) for i in range(R // 2)]
        for r, p in enumerate(pos):
            for i in range(R // 2):
                turns = p * f[i] / (2 * PI)
                a = float((turns - turns.to_integral_value()) * 2 * PI)
                exponent = 2 * i / R * math.log(base) * 2.0 ** -53
                tol = 4 * 2.0 ** -24 + abs(p) * (float(f[i]) * (2.0 ** -51 + exponent) + 7 * 2.0 ** -64)
                assert abs(got[r, i] - math.cos(a)) <= tol, (p, i)
                assert abs(got[r, R // 2 + i] - math.sin(a)) <= tol, (p, i)


# ------------------------------------------------------------ far ends of scales
@pytest.mark.parametrize("dtype,D,lens,qs", [("bf16", 128, [40, 3], [1, 1]), ("bf16", 128, [300, 90], [70, 64]),
                                             ("bf16", 256, [100], [80]), ("f32", 64, [40, 70], [2, 1])])
@pytest.mark.parametrize("ks,scale", [(1e-20, 0.0), (1.0, 1e-30), (1e-30, 1e-8)])
def test_zero_queries_under_tiny_scales(dtype, D, lens, qs, ks, scale):
    """A row of zeros scores 0 everywhere whatever the scales: the mean of the
    values, and the logarithm of the keys' number; masked keys stay masked."""
    c = Case(370, dtype, 2, 2, D, 16, lens, qs, ks=ks, scale=scale)
    c.q[:, 0] = 0
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()


# ------------------------------------------------------------- large batches
def _batch(seed, n, most, queries):
    """n requests: lengths 0 to `most`, query counts of `queries`, empty ones among both."""
    rng = random.Random(seed)
    lens = [rng.choice([0, 1, 15, 16, 17, rng.randint(0, most), rng.randint(0, most)]) for _ in range(n)]
    qs = [rng.choice(queries) for _ in range(n)]
    lens[0], qs[0], qs[-1] = most, max(queries), 0
    return lens, qs


BATCHES = [  # dtype, heads, kv heads, D, page, requests, longest, query counts, window
    # every CTA of the split kernel plans up to 256 requests itself, 128 at a time
    ("bf16", 2, 1, 128, 16, 128, 90, [1], 0), ("bf16", 2, 1, 128, 16, 129, 90, [1, 0], 0),
    ("bf16", 2, 2, 64, 32, 256, 70, [1, 2, 0], 0),
    # more are planned by the kernel before it, 1024 at a time: each type, rows of 4, 8 and 16
    ("bf16", 2, 1, 128, 16, 257, 90, [1, 0], 0), ("bf16", 6, 1, 128, 16, 300, 60, [1], 20),
    ("bf16", 6, 1, 128, 64, 300, 60, [1, 2, 0], 0), ("bf16", 2, 2, 64, 16, 1025, 50, [1, 0], 0),
    ("bf16", 7, 1, 64, 16, 260, 300, [1], 0), ("bf16", 12, 1, 64, 16, 260, 90, [1, 3], 0),
    ("bf16", 2, 1, 256, 16, 270, 60, [1, 0], 0), ("bf16", 8, 1, 256, 16, 270, 60, [1, 0], 0),
    ("bf16", 5, 1, 256, 16, 270, 60, [1, 3], 9),
    ("f32", 2, 1, 128, 16, 2100, 40, [1, 0], 0), ("f32", 6, 1, 128, 16, 300, 60, [1, 2], 0),
    ("f32", 2, 2, 64, 16, 300, 90, [1, 2, 0], 0), ("f32", 8, 1, 64, 16, 270, 60, [1], 30),
    ("f32", 2, 1, 256, 16, 300, 60, [1, 0], 0), ("f32", 4, 1, 256, 32, 270, 60, [1, 2], 0),
    # the prompt kernel: requests and row tiles beyond a round of its plan
    ("bf16", 2, 1, 128, 16, 1025, 60, [1, 0, 2, 40], 0), ("bf16", 1, 1, 64, 16, 2100, 90, [1, 0, 64], 20),
    ("bf16", 4, 2, 256, 16, 1030, 50, [1, 0, 33], 0),
]


@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_large_batches(i):
    dtype, heads, kv, D, page, n, most, queries, window = BATCHES[i]
    lens, qs = _batch(i, n, most, queries)
    c = Case(300 + i, dtype, heads, kv, D, page, lens, qs, window).run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()
    out, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(1.0)
    c.run()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


def test_large_batch_of_long_and_short_requests():
    """Segments cut over many CTAs between hundreds that fit into one."""
    lens, qs = _batch(50, 400, 200, [1])
    for b in (3, 200, 398):
        lens[b] = 6000
    c = Case(350, "bf16", 4, 2, 128, 64, lens, qs).run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()


def test_prompt_of_more_row_tiles_than_a_round_of_the_plan():
    """8300 query tokens of a group of 32: 1038 row tiles of one request."""
    c = Case(351, "bf16", 32, 1, 64, 64, [8300, 40], [8300, 2]).run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check(rows=[0, 1, 7, 8, 1000, 4095, 4096, 8190, 8191, 8192, 8199, 8200, 8299])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_f32_rows_of_four_and_eight(D):
    for heads, lens, qs in ((1, [3000, 1], [4, 1]), (4, [3000, 20], [1, 1]), (8, [2000, 7], [1, 0]),
                            (3, [100, 40], [5, 3])):
        c = Case(360 + heads, "f32", heads, 1, D, 32, lens, qs).run()
        assert B.moe_get_status(c.ws) == (0, 0)
        c.check()


# ---------------------------------------------------- layouts and strange rows
MIXED = [  # dtype, heads, kv heads, D, page, lens, query tokens, window: rows of 4, 8, 16, and the prompt kernel
    ("bf16", 2, 1, 128, 16, [50, 9], [2, 2], 0), ("bf16", 4, 1, 64, 32, [50, 9], [2, 1], 0),
    ("bf16", 3, 1, 128, 64, [500, 70], [5, 4], 0), ("f32", 2, 1, 128, 16, [90, 9], [4, 3], 0),
    ("bf16", 2, 1, 256, 16, [70], [6], 30), ("bf16", 4, 2, 128, 16, [700, 90], [200, 40], 0),
    ("bf16", 4, 2, 64, 256, [700, 90], [200, 40], 50), ("bf16", 2, 2, 256, 32, [300, 90], [130, 70], 0),
]


@pytest.mark.parametrize("i", range(len(MIXED)))
def test_rows_of_nan_and_infinity_concern_themselves_alone(i):
    """Padding rows of a captured batch hold anything."""
    dtype, heads, kv, D, page, lens, qs, window = MIXED[i]
    c = Case(400 + i, dtype, heads, kv, D, page, lens, qs, window)
    strange = [r for r in range(max(qs)) if r % 3 == 1]
    for b in range(len(lens)):
        for n, r in enumerate(r for r in strange if r < qs[b]):
            c.q[c.offs[b] + r] = [float("nan"), float("inf"), -float("inf")][n % 3]
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check(rows=[r for r in range(max(qs)) if r % 3 != 1])
    assert torch.isnan(c.out[c.offs[0] + 1]).all()      # a query of NaN says so


@pytest.mark.parametrize("i", range(len(MIXED)))
def test_queries_whose_heads_come_first(i):
    """[heads, tokens, channels] in memory: the token stride is the smaller one."""
    dtype, heads, kv, D, page, lens, qs, window = MIXED[i]
    c = Case(420 + i, dtype, heads, kv, D, page, lens, qs, window).run()
    out, lse = c.out.clone(), c.lse.clone()
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    c.out.fill_(1.0)
    c.run()
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("i", range(len(MIXED)))
def test_tokens_of_bad_pages_are_left_out(i):
    """The first, a middle and the last page of a request, below and beyond the
    cache; queries are compared with attention over the tokens that are left."""
    dtype, heads, kv, D, page, lens, qs, window = MIXED[i]
    c = Case(440 + i, dtype, heads, kv, D, page, lens, qs)
    n, q = lens[0], qs[0]
    used = -(-n // page)
    bad = sorted({0, used // 2, used - 1}) if used > 3 else [0]
    for p, v in zip(bad, (-1, c.cache.shape[0], 2 ** 31 - 1)):
        c.d["table"][0, p] = v
    c.run()
    assert B.moe_get_status(c.ws) == (5, B.DEV_BAD_PAGE)
    c.check(only=range(1, len(lens)))
    keep = torch.tensor([t for t in range(n) if t // page not in bad])
    qd, out, lse = c.q.double().cpu().numpy(), c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
    for r in sorted({0, 1, q // 2, q - 1}):
        k = keep[keep <= n - q + r].numpy()
        if not len(k):
            assert (out[r] == 0).all() and (lse[r] == -math.inf).all()
            continue
        ref, l, size, reach = A.attention(qd[r:r + 1], c.k[0][k], c.v[0][k], len(k), c.scale)
        ds, sums = (D / 16 + 4) * 2.0 ** -23 * reach, (n / 16 + 32) * 2.0 ** -23
        p = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21
        tol = c.u * abs(ref) + size * (2 * ds[..., None] + p + sums + 2.0 ** -21)
        assert (abs(out[r:r + 1] - ref) <= tol).all(), r
        assert (abs(lse[r:r + 1] - l) <= ds + sums + 2.0 ** -20 + 2.0 ** -23 * abs(l)).all(), r


@pytest.mark.parametrize("dtype,heads,D", [("bf16", 64, 64), ("bf16", 512, 128), ("bf16", 130, 256),
                                           ("f32", 512, 64), ("bf16", 63, 128)])
def test_single_tokens_of_very_wide_groups(dtype, heads, D):
    """One kv head under up to 512 query heads, one token each: without offsets."""
    c = Case(460, dtype, heads, 1, D, 16, [100, 0, 1, 333], [1] * 4).run(offs=False)
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()
    want = c.out.clone()
    c.out.fill_(1.0)
    B.moe_kv_attention(c.cfg, 4, 4, 1, c.q, c.d["offs"], c.d["lens"], c.d["table"], c.cache, c.out, None, c.ws)
    assert torch.equal(c.out, want)
