"""Attention of requests that share a prefix, on the GPU, against the fp64 oracle.

Tolerances are those of test_gpu_attn's Case.check: the sums over the prefix and
over the own keys, and their pieces, are added in fp32 like the tiles there (a
piece has four tiles of 32 keys at least, so that n / 16 counts more additions
than there are)."""
import numpy as np
import pytest
import torch

from expert_moe_layer_gb300 import binding as B
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


def _views(cache, page, D):
    """The keys' codes and scales and the values' of a cache: [pages, kv, page, n]."""
    at, out = 0, []
    for n in (page * D // 2, page * D // 16) * 2:
        out.append(cache[..., at:at + n].unflatten(-1, (page, n // page)))
        at += n
    return out


class Shared(Case):
    """Case whose requests groups[g] .. groups[g+1] - 1 have their first prefix[g]
    tokens in common: whole pages are shared, the page they end in is copied. The
    page table is wide enough for sharing to be taken up (or, not wide, is not)."""

    def __init__(self, seed, dtype, heads, kv, D, page, lens, qs, groups, prefix, told=None, max_group=None,
                 wide=True, **kw):
        super().__init__(seed, dtype, heads, kv, D, page, lens, qs, **kw)
        views = _views(self.cache, page, D)
        for g, p in enumerate(prefix):
            live = [b for b in range(groups[g], groups[g + 1]) if qs[b] > 0 and lens[b] >= p]
            for b in live[1:]:
                n, rest = divmod(p, page)
                a = live[0]
                self.table[b, :n] = self.table[a, :n]
                if rest:
                    for v in views:
                        v[int(self.table[b, n]), :, :rest] = v[int(self.table[a, n]), :, :rest]
                self.k[b][:p], self.v[b][:p] = self.k[a][:p], self.v[a][:p]
        if wide:
            more = 41e6 / (len(lens) * kv * page * D * 9 / 8) - self.table.shape[1]
            self.table = np.pad(self.table, ((0, 0), (0, max(0, int(more) + 1))), constant_values=-7)
        self.d["table"] = torch.from_numpy(self.table).cuda()
        self.G = len(prefix)
        self.d["groups"] = torch.tensor(groups if self.G else [0], dtype=torch.int32, device="cuda")
        self.d["prefix"] = torch.tensor(prefix if told is None else told, dtype=torch.int32, device="cuda")
        sizes = [int(self.offs[groups[g + 1]] - self.offs[groups[g]]) for g in range(self.G)]
        self.max_group = max(sizes + [1]) if max_group is None else max_group
        size = B.kv_attention_shared_workspace_size(self.cfg, len(lens), self.T, self.max_q, self.G,
                                                    self.max_group)
        self.sws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")

    def shared(self, stream=None, offs=True, lse=True):
        B.moe_kv_attention_shared(self.cfg, len(self.lens), self.T, self.max_q, self.G, self.max_group, self.q,
                                  self.d["offs"] if offs else None, self.d["lens"], self.d["table"],
                                  self.d["groups"], self.d["prefix"], self.cache, self.out,
                                  self.lse if lse else None, self.sws, stream=stream)
        return self

    def status(self):
        return B.moe_get_status(self.sws)


CASES = [  # dtype, heads, kv heads, D, page, lens, query tokens, groups, prefix
    ("bf16", 2, 1, 128, 16, [40, 41], [1, 1], [0, 2], [32]),                    # one tile shared
    ("bf16", 2, 1, 128, 16, [40, 41], [1, 1], [0, 2], [31]),                    # less than a tile: none
    ("bf16", 16, 2, 128, 16, [1001, 1064, 1003, 1032], [1] * 4, [0, 4], [1000]),
    ("bf16", 8, 8, 128, 64, [300] * 5, [1] * 5, [0, 5], [299]),                 # every key but their own
    ("bf16", 5, 1, 64, 32, [200, 100, 90, 64, 65, 66], [1, 2, 3, 1, 1, 1], [0, 3, 3, 6], [77, 500, 64]),
    ("bf16", 12, 4, 256, 128, [300, 277, 400], [2, 1, 4], [0, 3], [256]),
    ("bf16", 32, 8, 128, 64, [500, 3, 420, 410, 0, 450], [1, 1, 1, 0, 1, 1], [2, 6], [400]),  # outside; idle; with no key
    ("bf16", 32, 8, 128, 64, [500, 3, 420, 410, 0, 450], [1, 1, 1, 0, 0, 1], [2, 6], [400]),
    ("bf16", 4, 1, 64, 256, [900, 800, 1000], [3, 5, 1], [0, 3], [700]),
    ("f32", 4, 2, 64, 16, [145, 130, 116], [1, 1, 1], [0, 3], [100]),
    ("f32", 24, 4, 64, 32, [300, 250, 222, 90, 70], [3, 3, 2, 1, 3], [0, 3, 5], [215, 64]),
    ("f32", 6, 1, 256, 16, [150, 140], [2, 5], [0, 2], [128]),
    ("f32", 8, 2, 128, 64, [700, 701], [5, 1], [0, 1, 2], [640, 640]),          # groups of one: none
    # from 64 rows of a group on: the prompt kernel over the prefix
    ("bf16", 32, 8, 128, 64, [600 + 9 * i for i in range(16)], [1] * 16, [0, 16], [599]),
    ("bf16", 8, 2, 128, 16, [300 + i for i in range(70)], [1 + i % 3 for i in range(70)], [0, 33, 70], [290, 160]),
    ("bf16", 8, 1, 64, 32, [400] * 40, [4] * 40, [0, 40], [390]),               # 1280 rows, five row tiles
    ("bf16", 8, 2, 256, 128, [513 + i for i in range(20)], [1] * 20, [0, 20], [512]),
    ("bf16", 7, 7, 128, 32, [129, 200, 190], [30, 40, 50], [0, 3], [96]),
    ("bf16", 16, 1, 128, 16, [330] * 12, [7] * 12, [0, 12], [320]),             # 112 rows of a request
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_shared(i):
    c = Shared(i, *CASES[i]).shared()
    assert c.status() == (0, 0)
    c.check()
    first = c.out.clone(), c.lse.clone()
    c.out.fill_(1.0)
    c.shared()                                   # in a fixed order: the same bits
    assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


@pytest.mark.parametrize("dtype,heads,kv,D,n,q", [("bf16", 8, 2, 128, 5, 1), ("bf16", 16, 1, 64, 40, 1),
                                                  ("bf16", 8, 2, 256, 12, 2), ("f32", 4, 1, 128, 6, 2)])
def test_long_prefixes_are_cut_into_pieces(dtype, heads, kv, D, n, q):
    """Few row tiles over many tiles of keys: every row joins many pieces."""
    lens = [9000 + 37 * i for i in range(n)]
    c = Shared(60 + n, dtype, heads, kv, D, 64, lens, [q] * n, [0, n], [8990]).shared()
    assert c.status() == (0, 0)
    c.check()
    first = c.out.clone()
    for _ in range(3):
        c.shared()
        assert torch.equal(c.out, first)


@pytest.mark.parametrize("D,heads,kv,groups", [
    (128, 8, 4, [(2, 17, 31), (4, 45, 12), (2, 32, 23)]),            # pieces of one tile, of odd numbers
    (64, 8, 4, [(2, 17, 30), (2, 25, 25), (4, 45, 17), (2, 32, 9)]),
    (128, 16, 8, [(2, 17 + i % 9, 1 + i % 5) for i in range(30)]),   # several segments to a CTA
    (256, 8, 4, [(4, 45, 9), (2, 32, 12), (3, 43, 5)]),              # row tiles of 128 rows
])
def test_row_tiles_with_half_their_rows(D, heads, kv, groups):
    """Groups of (requests, query tokens of each, tiles of 128 prefix tokens) whose last
    row tile has no more than 128 of its 256 rows (or 128), beside full ones."""
    lens, qs, bounds, prefix = [], [], [0], []
    for g, (n, q, tiles) in enumerate(groups):
        prefix.append(128 * tiles - 32 * (g % 4))
        lens += [prefix[-1] + q + 5 * i for i in range(n)]
        qs += [q] * n
        bounds.append(bounds[-1] + n)
    c = Shared(90 + D, "bf16", heads, kv, D, 64, lens, qs, bounds, prefix).shared()
    assert c.status() == (0, 0)
    c.check()
    first = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.sws.fill_(0xff)
        c.shared()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


@pytest.mark.parametrize("dtype,n", [("bf16", 3), ("bf16", 20), ("f32", 3)])
def test_prefixes_reach_no_further_than_the_requests(dtype, n):
    """The prefix is cut to what every request has before its queries."""
    lens = [200 + i for i in range(n)]
    for told in (150, 199, 200, 5000, 2 ** 31 - 1):
        c = Shared(70, dtype, 8, 2, 128, 16, lens, [1] * n, [0, n], [150 if told == 150 else 199], told=[told])
        c.shared()
        assert c.status() == (0, 0)
        c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_and_peaked_scores(dtype):
    c = Shared(71, dtype, 8, 2, 128, 16, [261, 220, 300], [2, 1, 1], [0, 3], [200], ks=0.37, vs=5.0, scale=0.2)
    c.shared().check()
    c = Shared(72, dtype, 8, 2, 64, 16, [400, 380] * 10, [1] * 20, [0, 20], [352], q_scale=40.0)
    c.shared().check(peaked=True)


def test_without_offsets_or_lse_and_on_another_stream():
    c = Shared(73, "bf16", 8, 2, 128, 16, [390, 405, 333], [1, 1, 1], [0, 3], [320]).shared()
    want, lse = c.out.clone(), c.lse.clone()
    c.out.fill_(1.0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c.shared(stream=s, offs=False)
    s.synchronize()
    assert torch.equal(c.out, want) and torch.equal(c.lse, lse)
    c.out.fill_(1.0)
    c.shared(lse=False)
    assert torch.equal(c.out, want)


@pytest.mark.parametrize("n", [3, 20])
@pytest.mark.parametrize("groups,told,max_group", [
    ([0, "n"], [-1], None), ([0, "n+1"], [90], None), ([-1, "n"], [90], None), ([2, 1, 2], [90, 90], None),
    ([0, "n", 1], [90, 90], None), ([0, "n"], [90], 1)])
def test_bad_groups_are_flagged_and_not_shared(n, groups, told, max_group):
    lens = [100 + i for i in range(n)]
    c = Shared(74, "bf16", 8, 2, 64, 16, lens, [1] * n, [0, n], [96])
    real = [{"n": n, "n+1": n + 1}.get(g, g) for g in groups]
    c.d["groups"] = torch.tensor(real, dtype=torch.int32, device="cuda")
    c.d["prefix"] = torch.tensor(told, dtype=torch.int32, device="cuda")
    c.G = len(told)
    c.max_group = n if max_group is None else max_group
    size = B.kv_attention_shared_workspace_size(c.cfg, n, c.T, 1, c.G, c.max_group)
    c.sws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    c.shared()
    assert c.status() == (5, B.DEV_BAD_SEGMENT)
    c.check()


@pytest.mark.parametrize("n", [3, 20])
def test_bad_requests_and_pages(n):
    """A request with bad offsets ends the sharing of its group; a bad page of a
    prefix is left out for all."""
    lens, qs = [100 + i for i in range(n)], [2] * n
    c = Shared(75, "bf16", 8, 2, 64, 16, lens, qs, [0, n], [96])
    offs = c.offs.copy()
    offs[n] = c.T + 5                                     # the last request leaves [0, T]
    c.d["offs"].copy_(torch.from_numpy(offs))
    c.shared()
    assert c.status() == (5, B.DEV_BAD_SEGMENT)
    c.check(only=range(n - 1))
    assert (c.out[int(c.offs[n - 1]):] == 3).all()
    c.d["offs"].copy_(torch.from_numpy(c.offs))
    page = int(c.table[0, 1])
    table = np.where(c.table == page, 9999, c.table)
    c.d["table"].copy_(torch.from_numpy(table))
    c.shared()
    assert c.status() == (5, B.DEV_BAD_PAGE)
    want, lse = c.out.clone(), c.lse.clone()
    c.run()                                               # the same keys left out
    assert B.moe_get_status(c.ws) == (5, B.DEV_BAD_PAGE)
    assert torch.isfinite(want.float()).all()
    # two ways of the same sums: a rounding of bf16 each
    assert ((want.float() - c.out.float()).abs() <= 2.0 ** -7 * c.out.float().abs() + 2.0 ** -10).all()
    assert ((lse - c.lse).abs() <= 2.0 ** -15 * (1 + lse.abs())).all()


def test_windows_many_rows_and_few_pages_are_the_unshared_attention():
    for kw, q in ((dict(window=50), 1), (dict(), 33), (dict(wide=False), 1)):
        c = Shared(76, "bf16", 8, 2, 128, 16, [300, 290], [q, q], [0, 2], [250], **kw)
        assert c.sws.numel() >= c.ws.numel()
        c.shared()
        assert c.status() == (0, 0)
        got = c.out.clone(), c.lse.clone()
        c.run()
        assert torch.equal(c.out, got[0]) and torch.equal(c.lse, got[1])
    c = Shared(77, "f32", 8, 2, 128, 16, [300, 290], [1, 1], [0], [])     # no groups
    c.shared()
    assert c.status() == (0, 0)
    c.check()


def test_not_a_number_stays_with_its_row():
    c = Shared(78, "bf16", 8, 2, 128, 16, [400] * 18, [1] * 18, [0, 18], [384])
    want = c.shared().out.clone()
    c.q[3, 2, 7] = float("nan")
    c.shared()
    keep = torch.ones(18, 8, dtype=torch.bool, device="cuda")
    keep[3, 2] = False
    assert torch.equal(c.out[keep], want[keep]) and torch.isnan(c.out[3, 2].float()).all()


@pytest.mark.parametrize("dtype,n", [("bf16", 4), ("bf16", 24), ("f32", 4)])
def test_in_a_graph_whose_lengths_and_groups_change(dtype, n):
    """A captured call follows the device's lengths, prefixes and groups; two graphs
    on one workspace, one after the other, do not disturb each other."""
    lens = [260 + i for i in range(n)]
    c = Shared(79, dtype, 8, 2, 128, 16, lens, [1] * n, [0, n], [256], max_group=n)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.shared()
        graphs = []
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=side):
                c.shared()
    torch.cuda.synchronize()
    for cut, prefix in ((0, 256), (0, 0), (70, 160), (200, 64)):
        c.lens = [m - cut for m in lens]
        c.d["lens"].copy_(torch.tensor(c.lens, dtype=torch.int32))
        c.d["prefix"].fill_(prefix)
        for g in graphs:
            c.out.fill_(1.0)
            g.replay()
            torch.cuda.synchronize()
            k, v = c.k, c.v
            c.k, c.v = [x[:m] for x, m in zip(k, c.lens)], [x[:m] for x, m in zip(v, c.lens)]
            c.check()
            c.k, c.v = k, v


def test_more_requests_than_a_block_has_threads():
    n = 1100
    c = Shared(80, "bf16", 4, 1, 64, 16, [70 + i % 7 for i in range(n)], [1] * n,
               list(range(0, n, 2)) + [n], [64] * (n // 2)).shared()
    assert c.status() == (0, 0)
    c.check(only=range(0, n, 37))
    c = Shared(81, "bf16", 4, 1, 64, 16, [70 + i % 7 for i in range(n)], [1] * n, [0, n], [64]).shared()
    assert c.status() == (0, 0)
    c.check(only=range(0, n, 37))
