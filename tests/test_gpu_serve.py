"""Shared pages of a cache and norms around a block, on the GPU, against the
oracles. Page calls are exact. Norms: the oracle's bound on fp32 arithmetic plus
half a step of the output's type, finfo(type).eps / 2 of its value."""
import numpy as np
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from oracle import serve_oracle as S

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------- pages
class Pool:
    """A pool on the GPU beside its oracle."""

    def __init__(self, rows, width, pages, page=16, caches=2, kv=1, dim=64, seed=0, fill=True, skew=0):
        rng = np.random.default_rng(seed)
        self.cfg = B.make_attn_config(kv, kv, dim, page)
        size = page * dim * 9 // 8
        data = [rng.integers(0, 256, (pages, kv, size), dtype=np.uint8) for _ in range(caches)] if fill else []
        self.o = S.Pool(np.full((rows, width), -1, np.int32), np.zeros(rows, np.int32),
                        np.zeros(pages, np.int32), page, data)
        self.caches = ([torch.from_numpy(d).cuda() for d in data] if fill else
                       [torch.zeros(pages, kv, size, dtype=torch.uint8, device="cuda") for _ in range(caches)])
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages + skew, dtype=torch.int32, device="cuda")[skew:]
        self.pool = B.make_kv_pool(self.cfg, self.table, self.held, self.refs, self.caches)
        self.ws = torch.full((B.kv_pool_workspace_size(self.cfg, self.pool, 4096),), 0x5a,
                             dtype=torch.uint8, device="cuda")

    def load(self):
        """The oracle's state onto the GPU."""
        for t, a in ((self.table, self.o.table), (self.held, self.o.held), (self.refs, self.o.refs)):
            t.copy_(torch.from_numpy(a))

    def _flags(self, want):
        assert B.moe_get_status(self.ws) == (5 if want else 0, want)

    def fork(self, parents, children, tokens):
        B.moe_kv_fork(self.cfg, self.pool, len(parents), *map(ints, (parents, children, tokens)), self.ws)
        self._flags(self.o.fork(parents, children, tokens))

    def release(self, rows, keep=None):
        B.moe_kv_release(self.cfg, self.pool, len(rows), ints(rows), None if keep is None else ints(keep),
                         self.ws)
        self._flags(self.o.release(rows, [0] * len(rows) if keep is None else keep))

    def reserve(self, rows, start, end):
        B.moe_kv_reserve(self.cfg, self.pool, len(start), None if rows is None else ints(rows), ints(start),
                         ints(end), self.ws)
        self._flags(self.o.reserve(list(range(len(start))) if rows is None else rows, start, end))

    def compact(self):
        used = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        B.moe_kv_compact(self.cfg, self.pool, used, self.ws)
        n, flags = self.o.compact()
        self._flags(flags)
        assert used.item() == n

    def check(self):
        for name, t, a in (("held", self.held, self.o.held), ("table", self.table, self.o.table),
                           ("refs", self.refs, self.o.refs)):
            np.testing.assert_array_equal(t.cpu().numpy(), a, err_msg=name)
        for t, a in zip(self.caches, self.o.caches):
            assert np.array_equal(t.cpu().numpy(), a)


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def test_a_prompt_is_forked_written_to_released_and_compacted():
    p = Pool(rows=6, width=8, pages=40)
    p.reserve([2, 0], [0, 0], [70, 16])
    p.check()
    p.fork([2, 2, 0, 2], [1, 3, 4, 5], [70, 64, 16, 0])
    p.check()
    p.reserve(None, [16, 70, 70, 64, 16, 0], [17, 71, 72, 65, 50, 0])   # copies, fresh pages, nothing
    p.check()
    p.release([2, 0], [33, 0])
    p.check()
    p.compact()
    p.check()
    p.compact()                                                         # nothing left to move
    p.check()
    p.release(list(range(6)))
    p.check()
    assert not p.refs.any() and not p.held.any() and (p.table == -1).all()
    p.compact()
    p.check()


@pytest.mark.parametrize("pages", [1, 7, 8192, 8193, 20011])
@pytest.mark.parametrize("seed", range(3))
def test_random_runs(pages, seed):
    rng = np.random.default_rng(100 * pages + seed)
    rows, ps = int(rng.integers(2, 40)), 16
    width = max(2, min(40, pages // 4))
    p = Pool(rows, width, pages, ps, caches=1 if pages > 8000 else 3, kv=2 if pages < 100 else 1, seed=seed,
             skew=seed)
    # pages in use all over the pool, by no row that the calls below name
    p.o.refs[rng.random(pages) < (0.0 if pages < 10 else 0.6)] = 1
    p.load()
    for _ in range(12):
        n = int(rng.integers(1, 2 * rows))
        kind = rng.integers(0, 5)
        any_row = lambda m: [int(v) for v in rng.integers(-1, rows + 1, m)]  # noqa: E731
        if kind == 0:
            p.fork(any_row(n), any_row(n), [int(v) for v in rng.integers(-1, width * ps // 2, n)])
        elif kind == 1:
            p.release(any_row(n // 3 + 1), [int(v) for v in rng.integers(-1, width * ps + 9, n // 3 + 1)])
        elif kind == 4:
            p.compact()
        else:
            a = rng.integers(-1, width * ps // 2, n)
            b = a + rng.integers(-1, 90, n)
            p.reserve(any_row(n), [int(v) for v in a], [int(v) for v in b])
        p.check()


def test_too_few_pages_end_the_list():
    p = Pool(rows=5, width=10, pages=9)
    p.reserve(None, [0, 0, 0, 0, 0], [48, 70, 32, 5, 0])       # 3 of 9, 5 more, then 2 do not fit
    p.check()
    assert p.held.tolist() == [3, 5, 0, 0, 0]
    p.fork([0], [2], [40])
    p.reserve([2, 0], [40, 40], [41, 41])                      # both need one, one is left
    p.check()
    assert (p.table >= -1).all()                               # (no mark stays behind)


def test_sharers_of_a_page_each_get_their_own_and_it_is_free_afterwards():
    p = Pool(rows=4, width=4, pages=12)
    p.reserve([0], [0], [20])
    p.fork([0, 0, 0], [1, 2, 3], [20, 20, 20])
    p.reserve(None, [20] * 4, [21] * 4)
    p.check()
    assert p.refs.tolist()[:6] == [4, 0, 1, 1, 1, 1]
    p.reserve([3], [32], [33])                                 # takes page 1 again
    p.check()
    assert p.table[3].tolist() == [0, 5, 1, -1]


def test_rows_that_are_rewritten_from_an_earlier_token():
    """Every shared page from there on is replaced, the first alone is copied."""
    p = Pool(rows=3, width=150, pages=700)
    p.reserve([0], [0], [2400])
    p.fork([0, 0], [1, 2], [2400, 1200])
    p.reserve([1, 0], [100, 1195], [2400, 1300])
    p.check()


def test_pools_of_more_pages_than_chunks_of_the_smallest_size():
    """Nine million pages: chunks of twice the size, and moves across all of them."""
    rng = np.random.default_rng(3)
    n = 9_000_003
    p = Pool(rows=3, width=20, pages=n, caches=1, fill=False)
    p.o.refs[:] = rng.random(n) < 0.999
    p.load()
    p.reserve([1], [0], [300])
    p.check()
    p.o.refs[: n - 5000] = 0
    p.o.refs[p.o.table[1, :19]] = 1
    p.load()
    p.compact()
    p.check()


def test_bad_entries_and_counts_are_flagged_and_left():
    p = Pool(rows=3, width=4, pages=20)
    p.reserve([0], [0], [64])
    p.o.table[0, 1], p.o.table[0, 2] = 99, -5
    p.o.refs[p.o.table[0, 3]] = 0                               # held by a row, counted by none
    p.load()
    p.fork([0], [1], [40])
    p.check()
    p.release([1])
    p.check()
    p.release([0])
    p.check()
    p.o.refs[:] = 0
    p.o.refs[10:12] = 1
    p.o.table[2, :3], p.o.held[2] = [10, 15, 11], 3             # page 15 is free
    p.load()
    p.compact()
    p.check()


@pytest.mark.parametrize("start", [0, 20])
def test_bad_entries_between_pages_that_are_replaced(start):
    """Whatever stands in an entry, only pages of the pool are taken, counted or copied."""
    p = Pool(rows=3, width=16, pages=40)
    p.reserve([0], [0], [256])
    p.fork([0], [1], [256])
    for e, bad in ((0, -3), (2, -2), (4, -41), (6, -42), (8, -2 ** 31), (10, 2 ** 31 - 1), (12, -30), (13, 40)):
        p.o.table[1, e] = bad
    p.load()
    p.reserve([1], [start], [256])
    p.check()
    p.o.table[0, 3], p.o.table[0, 5] = -4, -2 ** 31 + 1         # of an item that finds too few pages
    p.o.refs[:] = np.maximum(p.o.refs, 1)
    p.load()
    p.reserve([0], [0], [256])
    p.check()


def test_page_calls_in_a_graph():
    """Captured once, replayed on other states: the same as eager calls."""
    p, q = (Pool(rows=8, width=12, pages=9000, seed=5) for _ in range(2))
    parents, children = ints([0, 1]), ints([4, 5])
    args = {id(x): [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 8, 8)] for x in (p, q)}

    def step(x):
        shared, start, end = args[id(x)]
        B.moe_kv_release(x.cfg, x.pool, 2, children, None, x.ws)
        B.moe_kv_fork(x.cfg, x.pool, 2, parents, children, shared, x.ws)
        B.moe_kv_reserve(x.cfg, x.pool, 8, None, start, end, x.ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(p)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(p)
    torch.cuda.synchronize()
    for x in (p, q):
        x.o.held[:], x.o.table[:], x.o.refs[:] = 0, -1, 0
        x.load()
    for i in range(6):
        a = [30 + 17 * i] * 2 + [0, 7 * i] + [0] * 4
        for x in (p, q):
            shared, start, end = args[id(x)]
            start.copy_(ints([min(v, 30 + 17 * max(i - 1, 0)) if i else 0 for v in a]))
            end.copy_(ints(a))
            shared.copy_(ints([0, 0] if i == 0 else [30 + 17 * (i - 1)] * 2))
        graph.replay()
        step(q)
        torch.cuda.synchronize()
        for u, v in zip((p.table, p.held, p.refs, *p.caches), (q.table, q.held, q.refs, *q.caches)):
            assert torch.equal(u, v)


@pytest.mark.parametrize("page,dim,kv,caches", [(16, 64, 1, 1), (64, 128, 3, 5), (256, 256, 2, 2),
                                                (32, 128, 1, 256)])
def test_copy_pages(page, dim, kv, caches):
    rng = np.random.default_rng(page + dim)
    cfg = B.make_attn_config(kv, kv, dim, page)
    size = page * dim * 9 // 8
    a = [torch.from_numpy(rng.integers(0, 256, (9, kv, size), dtype=np.uint8)).cuda() for _ in range(caches)]
    b = [torch.from_numpy(rng.integers(0, 256, (13, kv, size), dtype=np.uint8)).cuda() for _ in range(caches)]
    before = [t.clone() for t in b]
    src, dst = [8, 0, -1, 3, 9, -2, 2, 2], [12, 1, 5, -1, 0, 2, 13, 7]
    ws = torch.full((4,), 9, dtype=torch.uint8, device="cuda")
    f, t = B.make_kv_caches(cfg, a), B.make_kv_caches(cfg, b)
    B.moe_kv_copy_pages(cfg, f, t, 8, ints(src), ints(dst), ws)
    assert B.moe_get_status(ws) == (5, B.DEV_BAD_PAGE)
    for x, y, z in zip(a, b, before):
        z[12], z[1], z[7] = x[8], x[0], x[2]
        assert torch.equal(y, z)
    B.moe_kv_copy_pages(cfg, t, t, 2, ints([12, 1]), ints([4, 3]))       # within one pool
    for y, z in zip(b, before):
        z[4], z[3] = z[12], z[1]
        assert torch.equal(y, z)


# ---------------------------------------------------------------------- norms
NORMS = [  # T, H, act, residual, kind, post, gate, strided
    (1, 1, "bf16", "bf16", "rms", False, "none", False), (3, 7, "f32", "f32", "layer", True, "full", False),
    (5, 64, "bf16", "bf16", "rms", True, "channel", True), (9, 128, "bf16", "f32", "layer", False, "token", False),
    (1, 2048, "bf16", "bf16", "rms", False, "none", False), (77, 511, "bf16", "bf16", "layer", True, "full", False),
    (33, 513, "f32", "bf16", "rms", True, "token", True), (13, 520, "f32", "f32", "rms", False, "channel", False),
    (10, 4096, "bf16", "f32", "rms", True, "channel", True), (6, 5120, "f32", "f32", "layer", True, "full", False),
    (4, 16384, "bf16", "bf16", "layer", True, "full", False), (3, 16384, "f32", "f32", "rms", True, "none", True),
    (2, 16383, "bf16", "f32", "layer", True, "channel", False), (300, 1000, "bf16", "bf16", "rms", True, "full", True),
    (1000, 136, "f32", "bf16", "layer", False, "channel", False),
    # rows that lie anywhere: no tensor's begin like another's
    (7, 1000, "bf16", "f32", "rms", True, "full", 3), (9, 130, "f32", "bf16", "layer", True, "channel", 3),
    # many rows for each block, in every kernel
    (20000, 64, "bf16", "bf16", "rms", True, "channel", False), (8000, 256, "f32", "bf16", "layer", True, "full", False),
    (3000, 2048, "bf16", "f32", "layer", True, "full", True), (2500, 2056, "bf16", "bf16", "rms", False, "token", False),
    (2500, 1001, "bf16", "f32", "rms", True, "full", False), (20000, 99, "f32", "f32", "layer", True, "channel", False),
    (9000, 333, "bf16", "bf16", "rms", True, "full", 3), (1100, 4100, "bf16", "bf16", "rms", False, "none", False),
    (900, 12288, "bf16", "bf16", "rms", True, "channel", False), (400, 16383, "f32", "f32", "layer", True, "none", False),
    (2000, 1000, "f32", "bf16", "rms", False, "full", 3),
    (700, 4096, "bf16", "f32", "layer", False, "full", True), (640, 5120, "bf16", "bf16", "rms", False, "channel", False),
    (305, 1536, "bf16", "bf16", "layer", False, "full", False),
]


def _norm_case(T, H, act, res, kind, post, gate, strided, seed):
    rng = np.random.default_rng(seed)
    rand = lambda *s: rng.normal(size=s).astype(np.float32)  # noqa: E731

    def rows(dt, m):
        if not strided:
            return torch.from_numpy(m).to(TORCH[dt]).cuda()
        at, more = (8, 24) if strided is True else next(places)
        wide = torch.full((T, H + more), float("nan"), dtype=TORCH[dt], device="cuda")
        wide[:, at:at + H] = torch.from_numpy(m).to(TORCH[dt])
        return wide[:, at:at + H]

    places = iter([(3, 5), (2, 7)])
    y, x = rows(act, 3 * rand(T, H) + 0.3), rows(res, 2 * rand(T, H) - 1)
    w = {k: torch.from_numpy(rand(H)).cuda() for k in ("post_w", "pre_w", "post_b", "pre_b")}
    if kind == "rms":
        w["post_b"] = w["pre_b"] = None
    if not post:
        w["post_w"] = w["post_b"] = None
    g = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    g = None if g is None else torch.from_numpy(2 * rand(*g)).to(TORCH[act]).cuda()
    return y, x, w, g


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _norm_check(got, want, bound, dtype):
    u = torch.finfo(TORCH[dtype]).eps / 2
    tiny = torch.finfo(TORCH[dtype]).smallest_normal * u
    err = np.abs(_f64(got) - want)
    assert (err <= bound + u * (np.abs(want) + bound) + tiny).all(), np.nanmax(err - bound - u * np.abs(want))


@pytest.mark.parametrize("case", NORMS)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_norm(case, sigmoid):
    T, H, act, res, kind, post, gate, strided = case
    y, x, w, g = _norm_case(*case, seed=T * H)
    cfg = B.make_norm_config(H, kind, act, res, post, "sigmoid" if sigmoid else "linear", 0.6, 0.5, 1e-5)
    xo = torch.full((T + 1, H), 7.0, dtype=TORCH[res], device="cuda")
    h = torch.full((T + 1, H), 7.0, dtype=TORCH[act], device="cuda")
    args = (y, x, w["post_w"], w["post_b"], g, w["pre_w"], w["pre_b"])
    ws = torch.full((4,), 3, dtype=torch.uint8, device="cuda")
    B.moe_norm(cfg, T, *args, xo[:T], h[:T], ws)
    assert B.moe_get_status(ws) == (0, 0)
    k = dict(layer=kind == "layer", offset=0.5, eps=1e-5)
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    r, want, dr, dh = S.norm(_f64(x), _f64(y), post, _f64(w["post_w"]), _f64(w["post_b"]), _f64(g), sigmoid,
                             _f64(w["pre_w"]), _f64(w["pre_b"]), k["layer"], f32(0.6), 0.5, f32(1e-5))
    _norm_check(xo[:T], r, dr, res)
    _norm_check(h[:T], want, dh, act)
    assert (xo[T:] == 7).all() and (h[T:] == 7).all()
    # either output alone, and in place: the same bits
    one = torch.empty_like(xo[:T])
    B.moe_norm(cfg, T, *args[:5], None, None, one, None)
    assert torch.equal(one, xo[:T])
    two = torch.empty_like(h[:T])
    B.moe_norm(cfg, T, *args, None, two)
    assert torch.equal(two, h[:T])
    yc, xc = y.clone(memory_format=torch.contiguous_format), x.clone(memory_format=torch.contiguous_format)
    B.moe_norm(cfg, T, yc, xc, *args[2:], xc, yc)
    # (a contiguous row may take other chunks than a strided one: sums in another order)
    _norm_check(xc, r, dr, res)
    _norm_check(yc, want, dh, act)
    # without a block before
    _, want, _, dh = S.norm(_f64(x), pre_w=_f64(w["pre_w"]), pre_b=_f64(w["pre_b"]), **{**k, "eps": f32(1e-5)})
    B.moe_norm(cfg, T, None, x, None, None, None, w["pre_w"], w["pre_b"], None, two)
    _norm_check(two, want, dh, act)


def test_norm_rows_of_zeros_large_offsets_and_non_finite_rows():
    T, H = 6, 1024
    for kind in ("rms", "layer"):
        cfg = B.make_norm_config(H, kind, "f32", eps=1e-6)
        x = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
        x[0] = 0
        x[1] += 1e4                                   # a mean far larger than the deviation
        x[2, 5] = float("inf")
        x[3, 7] = float("nan")
        x[4] = 1e-30
        h = torch.empty_like(x)
        B.moe_norm(cfg, T, None, x, None, None, None, None, None, None, h)
        good = [0, 1, 4, 5]
        _, want, _, dh = S.norm(_f64(x)[good], layer=kind == "layer", eps=float(np.float32(1e-6)))
        _norm_check(h[good], want, dh, "f32")
        assert (h[0] == 0).all() and torch.isnan(h[2, 5]) and torch.isnan(h[3]).all()


def test_norm_of_heads_of_a_projection():
    """Rows need not be tokens: heads of 128 channels, in slices of a wider projection."""
    T, heads = 37, 12
    cfg = B.make_norm_config(128)
    qkv = torch.randn(T, heads + 4, 128, device="cuda").bfloat16()
    w = torch.randn(128, device="cuda")
    h = torch.empty(heads, T, 128, device="cuda", dtype=torch.bfloat16)
    for i in range(heads):
        B.moe_norm(cfg, T, None, qkv[:, i], None, None, None, w, None, None, h[i])
    _, want, _, dh = S.norm(_f64(qkv[:, :heads]).swapaxes(0, 1), pre_w=_f64(w), eps=float(np.float32(1e-6)))
    _norm_check(h, want, dh, "bf16")
