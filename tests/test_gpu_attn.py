"""Rotary positions, the 4-bit paged cache and attention over it, on the GPU,
against the fp64 oracle.

Tolerances, with u = finfo(type).eps / 2 of the output type:
  table      the argument of sincospi is rounded once and corrected, its
             result is within 2 ulp, the gain rounds once: 4 * 2^-24 * gain
  rope       two products and their sum in fp32, then one rounding:
             3 * 2^-24 * (|a c| + |b s|) + u * |out|
  append     codes and scales are equal (the oracle does the same fp32 steps)
  attention  with A = sum_j p_j |v_j| and S = the largest sum |q k| * scale:
             the scores of one tile come from D/16 matrix steps, each rounding
             or truncating at 2^-23 of S (and for fp32 queries, split into two
             f16, 2^-22 of S): ds = (D/16 + 4) * 2^-23 * S, twice (numerator
             and denominator); p as f16 adds 2^-11 (as two f16 2^-21); sums
             over tiles and pieces 2^-23 each, and the exponentials 2^-21:
             |out - ref| <= u |ref| + A * (2 ds + 2^-11 or 2^-21 + (n/16 + 32) 2^-23 + 2^-21)
             |lse - ref| <= ds + (n/16 + 32) 2^-23 + 2^-20 + 2^-23 |ref|
"""
import numpy as np
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rows(rng, T, heads, D, dtype, slack=0, scale=1.0):
    """A [T, heads, D] slice of wider rows, with NaN around it."""
    x = torch.from_numpy(rng.normal(size=(T, heads + 2 * slack, D)).astype(np.float32) * scale)
    x = x.to(TORCH[dtype])
    x[:, :slack] = float("nan")
    x[:, slack + heads:] = float("nan")
    return x.cuda()[:, slack:slack + heads]


# -------------------------------------------------------------------- table
@pytest.mark.parametrize("R,n,kind", [(2, 5, "none"), (64, 2048, "none"), (128, 777, "linear"),
                                      (96, 300, "ntk"), (128, 1000, "parts"), (128, 999, "yarn"),
                                      (512, 33, "yarn"), (66, 1, "none")])
@pytest.mark.parametrize("far", [False, True])
def test_table(R, n, kind, far):
    rng = np.random.default_rng(n)
    pos = rng.integers(-(1 << 31), 1 << 31, n).astype(np.int32) if far else None
    kw = dict(kind=kind, factor=8.0, original=4096.0)
    cfg = B.make_attn_config(1, 1, 512, rotary_dim=R, rope_positions=n)
    out = torch.full((n + 1, R), 7.0, device="cuda")
    B.moe_rope_table(cfg, n, None if pos is None else torch.from_numpy(pos).cuda(),
                     B.make_rope_scaling(1e4, kind, 8.0, 4096.0), out[:n])
    want = A.rope_table(np.arange(n) if pos is None else pos, R, 1e4, **kw)
    _, gain = A.frequencies(R, 1e4, **kw)
    # frequencies agree to about 2^-52, which far positions multiply
    slack = 4 * 2.0 ** -24 * gain + (2.0 ** 31 * 2.0 ** -50 if far else 0)
    assert np.abs(_f64(out[:n]) - want).max() <= slack
    assert (out[n] == 7).all()


# --------------------------------------------------------------------- rope
ROPE = [  # dtype, T, heads, D, R, layout, slack heads
    ("bf16", 1, 1, 128, 128, "half", 0), ("bf16", 7, 5, 128, 64, "interleaved", 3),
    ("bf16", 33, 8, 64, 64, "half", 1), ("f32", 5, 3, 256, 256, "half", 2),
    ("f32", 9, 2, 64, 32, "interleaved", 0), ("bf16", 4, 3, 80, 80, "half", 1),
    ("bf16", 3, 2, 128, 66, "half", 1), ("f32", 3, 2, 128, 30, "interleaved", 1),
    ("bf16", 2, 2, 128, 0, "half", 1), ("f32", 6, 1, 512, 2, "half", 0),
    ("bf16", 1100, 16, 128, 96, "half", 4), ("bf16", 2, 3, 18, 10, "half", 0),
    ("bf16", 900, 24, 128, 128, "interleaved", 2),
    ("bf16", 1000, 20, 128, 66, "half", 1), ("bf16", 1000, 20, 128, 98, "interleaved", 1),
    ("f32", 700, 16, 256, 200, "half", 1), ("f32", 40, 5, 256, 34, "half", 0),
    ("bf16", 37, 5, 64, 2, "half", 2), ("bf16", 9, 3, 48, 46, "half", 0), ("f32", 3, 2, 64, 62, "half", 1),
]


@pytest.mark.parametrize("dtype,T,heads,D,R,layout,slack", ROPE)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dtype, T, heads, D, R, layout, slack, inverse):
    rng = np.random.default_rng(T * D + R)
    n = 500
    x = _rows(rng, T, heads, D, dtype, slack)
    pos = rng.integers(0, n, T).astype(np.int32)
    table = torch.from_numpy(A.rope_table(np.arange(n), max(R, 2), 1e4).astype(np.float32)).cuda()
    cfg = B.make_attn_config(heads, heads, D, act_dtype=dtype, rotary_dim=R, rope_layout=layout,
                             rope_positions=n if R else 0)
    out = torch.full((T, heads, D), 9.0, dtype=TORCH[dtype], device="cuda")
    args = (torch.from_numpy(pos).cuda(), table) if R else (None, None)
    B.moe_rope(cfg, T, x, *args, out, inverse=inverse)
    xs, tb = _f64(x), _f64(table)
    want = A.rotate(xs, pos, tb, R, layout == "interleaved", inverse, dtype=np.float64)
    # |a c| + |b s|: of non-negative inputs, the larger of the two turns
    size = np.maximum(*(np.abs(A.rotate(np.abs(xs), pos, np.abs(tb), R, layout == "interleaved",
                                        inv, np.float64)) for inv in (False, True)))
    u = torch.finfo(TORCH[dtype]).eps / 2
    assert (np.abs(_f64(out) - want) <= 3 * 2.0 ** -24 * size + u * np.abs(want)).all()
    if R < D:
        np.testing.assert_array_equal(_f64(out)[..., R:], xs[..., R:])
    # in place gives the same bits
    y = x.contiguous()
    B.moe_rope(cfg, T, y, *args, y, inverse=inverse)
    assert torch.equal(y, out)


def test_rope_inverse_is_the_gradient():
    """d/dx <w, rope(x)> is rope's inverse of w: by differences, and linearly."""
    rng = np.random.default_rng(5)
    cfg = B.make_attn_config(2, 2, 64, act_dtype="f32", rotary_dim=64, rope_positions=64)
    t = torch.from_numpy(A.rope_table(np.arange(64), 64, 1e4).astype(np.float32)).cuda()
    pos = torch.tensor([3, 63, 0], dtype=torch.int32, device="cuda")
    x, w = _rows(rng, 3, 2, 64, "f32"), _rows(rng, 3, 2, 64, "f32")
    run = lambda v, inv: (lambda o: (B.moe_rope(cfg, 3, v, pos, t, o, inverse=inv), o)[1])(torch.empty_like(v))  # noqa: E731
    grad = _f64(run(w, True))
    for i in (0, 17, 63):
        d = torch.zeros_like(x)
        d[1, 1, i] = 0.5
        diff = (_f64(run(x + d, False)) - _f64(run(x - d, False)))
        # the two runs round their outputs (magnitudes up to 8) at 2^-24 each
        assert abs((diff * _f64(w)).sum() - grad[1, 1, i]) < 4 * 128 * 8 * 2.0 ** -24


# ----------------------------------------------------------- append and read
APPEND = [  # dtype, T, heads, kv heads, D, R, layout, page, k_scale
    ("bf16", 1, 8, 2, 128, 128, "half", 16, 1.0), ("bf16", 37, 6, 3, 64, 32, "interleaved", 32, 0.5),
    ("f32", 20, 4, 1, 256, 256, "half", 64, 1.0), ("bf16", 19, 4, 4, 128, 66, "half", 16, 3.0),
    ("f32", 11, 2, 2, 64, 30, "interleaved", 128, 0.7), ("bf16", 8, 2, 1, 128, 0, "half", 16, 1.0),
    ("bf16", 700, 32, 8, 128, 128, "half", 64, 1.0),
    ("bf16", 600, 40, 8, 128, 64, "interleaved", 256, 1.0),
    ("bf16", 700, 24, 8, 128, 98, "half", 64, 1.0), ("bf16", 500, 24, 8, 64, 46, "interleaved", 16, 1.0),
    ("f32", 90, 6, 2, 256, 250, "half", 32, 1.0),
]


@pytest.mark.parametrize("dtype,T,heads,kv,D,R,layout,page,ks", APPEND)
def test_append_and_read(dtype, T, heads, kv, D, R, layout, page, ks):
    rng = np.random.default_rng(T + D)
    n, pages = 300, T // page + 3
    cfg = B.make_attn_config(heads, kv, D, page, dtype, R, layout, n if R else 0, k_scale=ks,
                             v_scale=2.0)
    table = A.rope_table(np.arange(n), max(R, 2), 1e4).astype(np.float32)
    pos = rng.integers(0, n, T).astype(np.int32)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    q = _rows(rng, T, heads, D, dtype, 1)
    k = _rows(rng, T, kv, D, dtype, 2, scale=30.0)
    v = _rows(rng, T, kv, D, dtype, 1, scale=1e-3 if T == 37 else 1.0)
    k[0, 0, :16] = 0
    v[-1, -1, 3] = float("nan")
    if T > 1:
        slots[T // 2] = -1
    before = rng.integers(0, 256, (pages, kv, page * D * 9 // 8)).astype(np.uint8)
    cache = torch.from_numpy(before).cuda()
    q_out = torch.full((T, heads, D), 5.0, dtype=TORCH[dtype], device="cuda")
    ws = torch.full((4,), 77, dtype=torch.uint8, device="cuda")
    dpos, dtab = (torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda()) if R else (None, None)
    dslots = torch.from_numpy(slots).cuda()
    B.moe_kv_append(cfg, T, q, k, v, dpos, dslots, dtab, q_out, cache, ws)
    assert B.moe_get_status(ws) == (0, 0)

    inter = layout == "interleaved"
    rounded = lambda x: torch.from_numpy(x).to(TORCH[dtype]).float().numpy()  # noqa: E731
    kr = rounded(A.rotate(k.float().cpu().numpy(), pos, table, R, inter))
    (kc, k8), (vc, v8) = A.quantise(kr, ks), A.quantise(v.float().cpu().numpy(), 2.0)
    got = cache.cpu().numpy()
    (gk, gk8), (gv, gv8) = A.unpack_cache(got, page, D)
    (bk, bk8), (bv, bv8) = A.unpack_cache(before, page, D)
    for t, s in enumerate(slots):
        if s >= 0:
            p, r = divmod(int(s), page)
            bk[p, r], bk8[p, r], bv[p, r], bv8[p, r] = kc[t], k8[t], vc[t], v8[t]
    for a, b in ((gk, bk), (gk8, bk8), (gv, bv), (gv8, bv8)):   # and nothing else changed
        np.testing.assert_array_equal(a, b)
    want_q = rounded(A.rotate(q.float().cpu().numpy(), pos, table, R, inter))
    np.testing.assert_array_equal(q_out.float().cpu().numpy(), want_q)

    ko, vo = torch.full_like(k.contiguous(), 3.0), torch.full_like(v.contiguous(), 3.0)
    B.moe_kv_read(cfg, T, dslots, cache, ko, vo, ws)
    assert B.moe_get_status(ws) == (0, 0)
    live = (slots >= 0)[:, None, None]
    f = lambda c, s, g: torch.from_numpy(np.where(live, A.stored_values(c, s).astype(np.float32) * np.float32(g), 0)).to(TORCH[dtype]).double().numpy()  # noqa: E731
    np.testing.assert_array_equal(_f64(ko), f(kc, k8, ks))
    np.testing.assert_array_equal(_f64(vo), f(vc, v8, 2.0))
    # keys alone: no queries in the launch
    again = torch.from_numpy(before).cuda()
    B.moe_kv_append(cfg, T, None, k, v, dpos, dslots, dtab, None, again)
    assert torch.equal(again, cache)


def test_bad_positions_and_slots_are_flagged_and_skipped():
    rng = np.random.default_rng(8)
    cfg = B.make_attn_config(2, 2, 64, 16, rotary_dim=64, rope_positions=10)
    t = torch.from_numpy(A.rope_table(np.arange(10), 64, 1e4).astype(np.float32)).cuda()
    x = _rows(rng, 4, 2, 64, "bf16")
    ws = torch.zeros(4, dtype=torch.uint8, device="cuda")
    out = torch.full((4, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([0, 10, -1, 9], dtype=torch.int32, device="cuda")
    B.moe_rope(cfg, 4, x, pos, t, out, ws=ws)
    assert B.moe_get_status(ws) == (5, B.DEV_BAD_POSITION)
    assert (out[1:3] == 5).all() and not (out[0] == 5).all() and not (out[3] == 5).all()
    cache = torch.zeros(2, 2, 16 * 64 * 9 // 8, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([32, 1, 2, -2], dtype=torch.int64, device="cuda")
    B.moe_kv_append(cfg, 4, None, x, x, pos, slots, t, None, cache, ws)
    assert B.moe_get_status(ws) == (5, B.DEV_BAD_POSITION | B.DEV_BAD_SLOT)
    assert (cache == 0).all()
    k, v = torch.ones_like(x), torch.ones_like(x)
    B.moe_kv_read(cfg, 4, slots, cache, k, v, ws)
    assert B.moe_get_status(ws) == (5, B.DEV_BAD_SLOT) and (k == 0).all() and (v == 0).all()
    B.moe_kv_read(cfg, 4, slots.clamp(0, 31), cache, k, v, ws)      # the next call clears the word
    assert B.moe_get_status(ws) == (0, 0)


# ---------------------------------------------------------------- attention
class Case:
    """Requests over a shuffled cache: values for the oracle, device tensors."""

    def __init__(self, seed, dtype, heads, kv, D, page, lens, qs, window=0, ks=1.0, vs=1.0,
                 scale=0.0, spare=2, q_scale=1.5):
        rng = np.random.default_rng(seed)
        self.lens, self.qs, self.window, self.page, self.D, self.kv = lens, qs, window, page, D, kv
        self.cfg = B.make_attn_config(heads, kv, D, page, dtype, window=window, k_scale=ks,
                                      v_scale=vs, softmax_scale=scale)
        self.scale = scale or D ** -0.5
        self.u = torch.finfo(TORCH[dtype]).eps / 2
        self.dtype = dtype
        counts = [-(-n // page) for n in lens]
        pages = sum(counts) + spare
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(counts + [1]) + 1), -7, np.int32)
        # memory that no token was stored to: NaN scales everywhere
        raw = np.full((pages, page, kv, D // 16), 0x7f, np.uint8)
        k8, v8 = raw.copy(), raw.copy() | 0x80
        kc, vc = np.full((pages, page, kv, D), 6.0), np.full((pages, page, kv, D), -6.0)
        self.k, self.v, at = [], [], 0
        for b, n in enumerate(lens):
            ids = order[at:at + counts[b]]
            at += counts[b]
            self.table[b, :counts[b]] = ids
            k, v = (rng.normal(size=(n, kv, D)).astype(np.float32) for _ in range(2))
            (c1, s1), (c2, s2) = A.quantise(k, ks), A.quantise(v, vs)
            self.k.append(A.stored_values(c1, s1, ks))
            self.v.append(A.stored_values(c2, s2, vs))
            for t in range(n):
                p, r = ids[t // page], t % page
                kc[p, r], k8[p, r], vc[p, r], v8[p, r] = c1[t], s1[t], c2[t], s2[t]
        self.cache = torch.from_numpy(A.pack_cache((kc, k8), (vc, v8), page)).cuda()
        self.T = sum(qs)
        self.q = _rows(rng, self.T, heads, D, dtype, 1, scale=q_scale)
        self.offs = np.concatenate([[0], np.cumsum(qs)]).astype(np.int32)
        self.d = dict(offs=torch.from_numpy(self.offs).cuda(), table=torch.from_numpy(self.table).cuda(),
                      lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        self.max_q = max(qs + [1])
        self.ws = torch.full((B.kv_attention_workspace_size(self.cfg, len(lens), self.T, self.max_q),),
                             0xff, dtype=torch.uint8, device="cuda")
        self.out = torch.full((self.T, heads, D), 3.0, dtype=TORCH[dtype], device="cuda")
        self.lse = torch.full((self.T, heads), 3.0, device="cuda")

    def run(self, stream=None, offs=True):
        B.moe_kv_attention(self.cfg, len(self.lens), self.T, self.max_q, self.q,
                           self.d["offs"] if offs else None, self.d["lens"], self.d["table"],
                           self.cache, self.out, self.lse, self.ws, stream=stream)
        return self

    def check(self, rows=None, only=None, peaked=False):
        q, out, lse = _f64(self.q), _f64(self.out), _f64(self.lse)
        for b, n in enumerate(self.lens):
            if only is not None and b not in only:
                continue
            sl = slice(self.offs[b], self.offs[b + 1])
            take = np.arange(self.qs[b]) if rows is None else np.array([r for r in rows if r < self.qs[b]], int)
            parts = [A.attention(q[sl][i:i + 1], self.k[b], self.v[b], n - self.qs[b] + 1 + i,
                                 self.scale, self.window) for i in take]
            for i, (ref, l, size, reach) in zip(take, parts):
                # fp32 queries in two f16, or exact bf16 ones
                ds = (self.D / 16 + 4) * 2.0 ** -23 * reach
                sums = (n / 16 + 32) * 2.0 ** -23
                p = 2.0 ** -11 if self.dtype == "bf16" else 2.0 ** -21
                tol = self.u * np.abs(ref) + size * (2 * ds[..., None] + p + sums + 2.0 ** -21)
                if peaked:  # weights far below the largest one fall under f16's last bit
                    tol += 2.0 ** -31 * np.abs(self.v[b]).sum(0).repeat(ref.shape[1] // self.kv, axis=0)
                err = np.abs(out[sl][i:i + 1] - ref)
                assert (err <= tol).all(), (b, i, (err - tol).max(), err.max())
                seen = np.isfinite(l)
                got = lse[sl][i:i + 1]
                assert (np.isneginf(got) == ~seen).all(), (b, i)
                assert (np.abs(got - l)[seen] <= (ds + sums + 2.0 ** -20 + 2.0 ** -23 * np.abs(l))[seen]).all()
        return self


ATTN = [  # dtype, heads, kv heads, D, page, lens, query tokens, window
    ("bf16", 2, 1, 128, 16, [1], [1], 0),
    ("bf16", 8, 8, 128, 16, [1, 15, 16, 17, 33], [1] * 5, 0),
    ("bf16", 16, 2, 128, 64, [5, 64, 65, 129], [1] * 4, 0),
    ("bf16", 5, 1, 64, 32, [100, 31], [1, 1], 0),
    ("bf16", 12, 4, 256, 128, [300, 7], [1, 1], 0),
    ("bf16", 16, 1, 128, 16, [77], [1], 0),
    ("bf16", 32, 1, 64, 256, [500, 3], [1, 1], 0),
    ("bf16", 4, 2, 128, 16, [0, 9, 0], [1, 1, 1], 0),
    ("bf16", 6, 2, 128, 32, [40, 3, 90], [4, 5, 2], 0),
    ("bf16", 8, 1, 256, 16, [50], [3], 0),
    ("bf16", 8, 2, 128, 16, [200, 30, 64], [1, 1, 1], 50),
    ("bf16", 3, 1, 64, 16, [70, 20], [17, 20], 9),
    ("bf16", 8, 4, 128, 64, [150, 0, 64], [40, 0, 64], 0),
    ("f32", 4, 2, 64, 16, [45, 1, 16], [1, 1, 1], 0),
    ("f32", 8, 1, 128, 32, [90, 33], [5, 2], 20),
    ("f32", 2, 2, 256, 16, [64], [7], 0),
]


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention(i):
    dtype, heads, kv, D, page, lens, qs, window = ATTN[i]
    c = Case(i, dtype, heads, kv, D, page, lens, qs, window).run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_scales(dtype):
    c = Case(3, dtype, 4, 2, 128, 16, [61, 20], [2, 1], ks=0.37, vs=5.0, scale=0.2).run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()


@pytest.mark.parametrize("dtype,heads,kv,D", [("bf16", 8, 2, 128), ("bf16", 16, 1, 64), ("f32", 4, 1, 128)])
def test_attention_long_context_is_split_and_joined(dtype, heads, kv, D):
    c = Case(11, dtype, heads, kv, D, 64, [9000, 300, 1, 4100], [1, 1, 1, 1]).run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()
    first = (c.out.clone(), c.lse.clone())
    for _ in range(3):                           # the joining order is fixed
        c.run()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


def test_attention_peaked_scores_move_the_maximum():
    """Scores that grow along the context by far more than the lag allowed to
    the running maximum, and queries scaled up to bf16's far ends."""
    c = Case(12, "bf16", 2, 1, 128, 16, [400], [1], q_scale=40.0).run()
    c.check()
    for far in (2.0 ** 60, 2.0 ** -60):
        d = Case(13, "bf16", 2, 1, 128, 16, [50], [1], scale=0.1 / far)
        d.q.mul_(far)
        d.run().check()


def test_attention_queries_before_the_first_token():
    """More query tokens than cached tokens: the first ones see nothing."""
    c = Case(14, "bf16", 4, 2, 128, 16, [3, 20], [6, 4])
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0)
    assert (c.out[:3] == 0).all() and torch.isneginf(c.lse[:3]).all()
    c.check()


def test_attention_without_offsets_or_lse_and_on_another_stream():
    c = Case(15, "bf16", 8, 2, 128, 16, [90, 5, 33], [1, 1, 1]).run()
    want, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(1.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c.run(stream=s, offs=False)
    s.synchronize()
    assert torch.equal(c.out, want) and torch.equal(c.lse, lse)
    c.out.fill_(1.0)
    B.moe_kv_attention(c.cfg, 3, 3, 1, c.q, None, c.d["lens"], c.d["table"], c.cache, c.out, None, c.ws)
    assert torch.equal(c.out, want)


PROMPT = [  # heads, kv heads, D, page, lens, query tokens, window (bf16, >= 64 rows a request)
    (8, 2, 128, 16, [40], [40], 0),                      # one half, one tile
    (4, 1, 64, 64, [130], [50], 0),
    (2, 2, 128, 32, [300, 129, 128], [300, 129, 1], 0),  # two halves, several tiles
    (16, 2, 128, 64, [515, 20, 0, 90], [65, 20, 0, 33], 0),
    (5, 1, 64, 16, [400, 31], [100, 31], 0),             # a group of five: tokens cross halves
    (24, 1, 128, 128, [260], [30], 0),
    (4, 2, 128, 16, [700, 260], [200, 260], 70),         # window: first tile not the first page
    (8, 8, 64, 256, [1000], [600], 300),
    (3, 1, 128, 16, [33, 5], [60, 40], 0),               # queries before the first token
    (16, 16, 128, 64, [2050], [2050], 0),                # more units than SMs
    (4, 1, 128, 64, [9000], [16], 0),                    # few rows, long context: pieces are joined
    (8, 2, 64, 16, [5000, 700, 64], [70, 33, 16], 0),
    (6, 2, 128, 32, [3000], [150], 1000),
    (4, 2, 256, 16, [40, 333], [32, 33], 0),             # 256 channels: one half, tiles of 64 keys
    (8, 1, 256, 64, [1200], [40], 300),
    (2, 1, 256, 128, [70], [200], 0),
]


@pytest.mark.parametrize("i", range(len(PROMPT)))
def test_attention_prompt(i):
    heads, kv, D, page, lens, qs, window = PROMPT[i]
    c = Case(100 + i, "bf16", heads, kv, D, page, lens, qs, window)
    assert max(qs) * heads // kv >= 64
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0)
    rows = None if c.T * heads < 4000 else sorted({0, 1, 63, 64, 127, 128, 129, 255, 256, 257, 500, 1000, 2047, 2048, 2049})
    c.check(rows=rows)
    first = (c.out.clone(), c.lse.clone())
    c.out.fill_(1.0)
    c.run()
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


def test_attention_prompt_overlapping_offsets_stay_inside_the_tables():
    """Offsets that give many requests the same rows: flagged, and the requests
    that fit the list are computed."""
    B_ = 40
    c = Case(130, "bf16", 4, 1, 128, 16, [64] * B_, [64] + [0] * (B_ - 1))
    offs = [0, 64] * (B_ // 2) + [0]
    c.d["offs"].copy_(torch.tensor(offs, dtype=torch.int32))
    c.run()
    rc, flags = B.moe_get_status(c.ws)
    assert rc == 5 and flags & B.DEV_BAD_SEGMENT
    c.d["offs"].copy_(torch.from_numpy(c.offs))
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check()


def test_attention_prompt_peaked_scores_rescale():
    """Scores spread over hundreds: most weights are far below the largest. p is
    kept as f16 times at least 2^6 over the maximum, its last bit is 2^-24, so a
    weight is off by up to 2^-25 / 2^6 of the largest: sum_j |v_j| 2^-31 more."""
    c = Case(120, "bf16", 4, 2, 128, 16, [600], [150], q_scale=40.0).run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check(rows=range(0, 150, 7), peaked=True)


def test_attention_prompt_bad_pages():
    c = Case(121, "bf16", 4, 2, 128, 16, [200, 150], [70, 64])
    c.run()
    good = c.out.clone()
    c.d["table"][0, 3] = c.cache.shape[0]
    c.run()
    assert B.moe_get_status(c.ws) == (5, B.DEV_BAD_PAGE)
    assert torch.equal(c.out[70:], good[70:])
    keep = np.r_[0:48, 64:200]
    for i in (0, 5, 69):
        p = 200 - 70 + i
        k = keep[keep <= p]
        ref, _, size, _ = A.attention(_f64(c.q)[i:i + 1], c.k[0][k], c.v[0][k], len(k), c.scale)
        assert (np.abs(_f64(c.out)[i:i + 1] - ref) <= 2.0 ** -8 * np.abs(ref) + size * 2.0 ** -10).all()


def test_attention_prompt_wait_limit_runs_out_then_the_next_call_is_exact():
    c = Case(122, "bf16", 8, 2, 128, 64, [1500], [700])
    try:
        B.set_wait_limit_ns(4)
        c.run()
        rc, flags = B.moe_get_status(c.ws)
        assert rc == 6 and flags & B.DEV_TIMEOUT, (rc, flags)
    finally:
        B.set_wait_limit_ns(0)
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0)
    c.check(rows=(0, 300, 699))


def test_attention_flags_bad_pages_lengths_and_offsets():
    c = Case(16, "bf16", 4, 2, 128, 16, [40, 50, 60, 33], [1, 1, 1, 1])
    c.run()
    good = c.out.clone()
    c.d["table"][1, 2] = c.cache.shape[0]             # one page id past the cache
    c.run()
    assert B.moe_get_status(c.ws) == (5, B.DEV_BAD_PAGE)
    c.check(only=(0, 2, 3))
    # request 1 without the tokens of that page
    q, keep = _f64(c.q)[1:2], np.r_[0:32, 48:50]
    ref, _, size, _ = A.attention(q, c.k[1][keep], c.v[1][keep], len(keep), c.scale)
    assert (np.abs(_f64(c.out)[1:2] - ref) <= 2.0 ** -8 * np.abs(ref) + size * 2.0 ** -10).all()
    c.d["table"][1, 2] = -1
    c.d["lens"][3] = -5
    c.run()
    assert B.moe_get_status(c.ws) == (5, B.DEV_BAD_PAGE)
    assert (c.out[3] == 0).all() and torch.isneginf(c.lse[3]).all()
    c.d["table"].copy_(torch.from_numpy(c.table))
    c.d["lens"].copy_(torch.tensor(c.lens, dtype=torch.int32))
    for bad in ([0, 1, 2, 3, 5], [0, 2, 1, 3, 4], [-1, 1, 2, 3, 4], [0, 1, 3, 3, 4]):
        c.d["offs"].copy_(torch.tensor(bad, dtype=torch.int32))
        c.run()
        assert B.moe_get_status(c.ws)[1] & B.DEV_BAD_SEGMENT
    c.d["offs"].copy_(torch.from_numpy(c.offs))
    c.run()
    assert B.moe_get_status(c.ws) == (0, 0) and torch.equal(c.out, good)


def test_attention_length_beyond_the_table_is_clamped():
    c = Case(17, "bf16", 2, 1, 128, 16, [48], [1])
    table = c.d["table"][:, :3].contiguous()
    c.d["lens"].fill_(1000)
    B.moe_kv_attention(c.cfg, 1, 1, 1, c.q, c.d["offs"], c.d["lens"], table, c.cache, c.out, c.lse, c.ws)
    assert B.moe_get_status(c.ws) == (5, B.DEV_BAD_PAGE)
    c.check()


def test_attention_in_a_graph_follows_the_lengths():
    c = Case(18, "bf16", 8, 2, 128, 16, [300, 40], [1, 1])
    c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run()
    torch.cuda.synchronize()
    c.lens = [299, 17]
    c.d["lens"].copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.out.fill_(1.0)
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes: its last pages are appended to, read
    back and attended to."""
    rng = np.random.default_rng(19)
    cfg = B.make_attn_config(4, 2, 128, 64, rotary_dim=0)
    pages = (1 << 32) // B.kv_page_bytes(cfg) + 8
    cache = torch.zeros(pages, 2, 64 * 128 * 9 // 8, dtype=torch.uint8, device="cuda")
    n = 100
    slots = torch.arange(n, device="cuda") + (pages - 2) * 64
    k, v, q = (_rows(rng, n if h == 2 else 1, h, 128, "bf16") for h in (2, 2, 4))
    B.moe_kv_append(cfg, n, None, k, v, None, slots, None, None, cache)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    B.moe_kv_read(cfg, n, slots, cache, ko, vo)
    want = A.stored_values(*A.quantise(k.float().cpu().numpy()))
    np.testing.assert_array_equal(_f64(ko), want)
    assert not cache[:pages - 2].any()
    out = torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(B.kv_attention_workspace_size(cfg, 1, 1, 1), dtype=torch.uint8, device="cuda")
    B.moe_kv_attention(cfg, 1, 1, 1, q, None, torch.tensor([n], dtype=torch.int32, device="cuda"),
                       torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device="cuda"), cache,
                       out, None, ws)
    assert B.moe_get_status(ws) == (0, 0)
    ref, _, size, _ = A.attention(_f64(q), _f64(ko), _f64(vo), n, 128 ** -0.5)
    assert (np.abs(_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + size * 2.0 ** -10).all()


def test_debug_library_agrees():
    c = Case(20, "bf16", 8, 2, 128, 16, [70, 20], [1, 1]).run()
    want = c.out.clone()
    with B.debug_library():
        c.out.fill_(1.0)
        c.run()
        assert torch.equal(c.out, want)
