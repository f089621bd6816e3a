"""Cases of the operators that a serving loop needs around the cache and the
blocks of a layer: norms with gate and residual, pages of the cache that several
requests share, and attention for requests that share a prefix.

``run`` computes a case either in plain torch operations (``own`` false) or by
the library's entry points (``own`` true), on the same inputs.

The cache is ``[pages, kv_heads, page_size * head_dim * 9 / 8]`` bytes. One
(page, kv head) block holds the keys' codes ``[page_size, head_dim / 2]``, the
keys' scales ``[page_size, head_dim / 16]``, then the values' codes and scales.
A code is a 4-bit float (e2m1), two to a byte, the lower channel in the low
half. A scale is an 8-bit float (e4m3) for 16 neighbouring channels.

A pool of pages is ``table [rows, max_pages]``, ``held [rows]`` (entries of each
row in use) and ``refs [pages]`` (rows that hold each page, 0 is free).
"""
import math
import random

import torch

own = False

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GROUP = 16
NEG = float("-inf")


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of 64 requests: a block's output joins the residual, the next block's norm
        dict(name="norm_step", op="norm", kind="rms", dtype="bf16", residual="bf16", tokens=64,
             hidden=2048, post=False, gate="none", scale=1.0),
        # a prompt chunk, normed on both sides of the block, a gate per channel, fp32 residual
        dict(name="norm_prompt", op="norm", kind="rms", dtype="bf16", residual="f32", tokens=8192,
             hidden=4096, post=True, gate="channel", scale=0.5),
        # fp32 layers with means and biases, a sigmoid gate per token, an odd count of tokens
        dict(name="norm_layer_f32", op="norm", kind="layer", dtype="f32", residual="f32",
             tokens=4097, hidden=5120, post=False, gate="token", scale=1.0),
        # a step of 64 rows in a small pool: some end, their rows are forked anew, all get a token's room
        dict(name="share_step", op="share", rows=64, pages=4096, page=16, low=1, high=900, forks=8,
             tokens=1, caches=4, kv_heads=8, dim=128),
        # 512 rows of a large pool, long prompts forked, drafts of 7 tokens
        dict(name="share_many", op="share", rows=512, pages=262144, page=16, low=100, high=16000,
             forks=192, tokens=7, caches=2, kv_heads=2, dim=64),
        # a few pages of every layer of a small model, to another cache
        dict(name="copy_step", op="copy", pages=512, moved=5, page=16, caches=24, kv_heads=8, dim=128),
        # a long prompt's pages in every layer
        dict(name="copy_prompt", op="copy", pages=1536, moved=509, page=64, caches=32, kv_heads=8,
             dim=128),
        # a pool with two fifths of its pages free, scattered
        dict(name="compact", op="compact", rows=96, pages=4096, page=32, caches=16, kv_heads=8,
             dim=128, free=0.4),
        # four samples of a short prompt: latency
        dict(name="attend_one", op="attend", dtype="bf16", groups=1, seqs=4, heads=16, kv_heads=2,
             dim=128, page=16, prefix=1000, least=1000, own=64, queries=1, spread=1),
        # a decode step of 64 samples of one long prompt
        dict(name="attend_step", op="attend", dtype="bf16", groups=1, seqs=64, heads=32, kv_heads=8,
             dim=128, page=64, prefix=32768, least=32768, own=1024, queries=1, spread=2),
        # fp32 layers: five prompts of different lengths, drafts of 3 tokens
        dict(name="attend_groups_f32", op="attend", dtype="f32", groups=5, seqs=4, heads=24,
             kv_heads=4, dim=64, page=32, prefix=4099, least=200, own=300, queries=3, spread=3),
        # three long documents, 48 requests on each, drafts of 2 tokens
        dict(name="attend_documents", op="attend", dtype="bf16", groups=3, seqs=48, heads=32,
             kv_heads=8, dim=128, page=64, prefix=65535, least=20000, own=2048, queries=2, spread=4),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "share", "copy", "compact", "attend", "attend", "attend", "attend"])
    if op == "norm":
        hidden = rng.choice([_log(rng, 64, 8192), 8 * _log(rng, 16, 1024), 128 * rng.randint(8, 64)])
        return dict(op=op, kind=rng.choice(["rms", "rms", "layer"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), residual=rng.choice(["bf16", "f32"]),
                    tokens=_log(rng, 1, min(16384, 8192 * 4096 // hidden)), hidden=hidden,
                    post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token", "full"]),
                    scale=rng.choice([1.0, 0.22, 0.5]))
    kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    size = kv * page * dim * 9 // 8
    if op == "share":
        rows = _log(rng, 2, 512)
        high = _log(rng, 20, 16000)
        pages = rows * (-(-high // page) + 4) + _log(rng, 16, 100000)
        while pages * size > 1 << 32:
            rows, high = max(2, rows // 2), max(20, high // 2)
            pages = rows * (-(-high // page) + 4) + 16
        return dict(op=op, rows=rows, pages=pages, page=page, low=rng.randint(1, 20), high=high,
                    forks=rng.randint(1, max(1, rows // 2)), tokens=rng.choice([1, 1, 2, 5, 40]),
                    caches=rng.randint(1, max(1, min(16, (1 << 32) // (pages * size)))), kv_heads=kv,
                    dim=dim)
    if op == "copy":
        caches = _log(rng, 1, 64)
        moved = _log(rng, 1, max(1, min(4000, (1 << 30) // (size * caches))))
        return dict(op=op, pages=2 * moved + rng.randint(1, 50), moved=moved, page=page, caches=caches,
                    kv_heads=kv, dim=dim)
    if op == "compact":
        caches = _log(rng, 1, 32)
        pages = _log(rng, 20, max(21, min(65536, (1 << 31) // (size * caches))))
        return dict(op=op, rows=_log(rng, 2, 300), pages=pages, page=page, caches=caches, kv_heads=kv,
                    dim=dim, free=rng.choice([0.05, 0.3, 0.5, 0.8]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if kv * group > 64:
        group = 64 // kv
    groups, seqs = rng.choice([1, 1, 2, 3, 6]), _log(rng, 2, 64)
    queries = rng.choice([1, 1, 1, 2, 4, 9])
    prefix = _log(rng, 64, 65536)
    own_tokens = max(queries, _log(rng, 1, 2048))
    while (groups * seqs * queries * kv * group * dim * (prefix + own_tokens) > 48 * 3 * 2 * 32 * 128 * 40000
           or groups * prefix * kv * dim > 3 * 65536 * 8 * 128):
        if prefix > own_tokens or seqs == 2:
            prefix = max(1, prefix // 2)
            own_tokens = max(queries, own_tokens // 2 if prefix < own_tokens else own_tokens)
        else:
            seqs = max(2, seqs // 2)
    return dict(op=op, dtype=dtype, groups=groups, seqs=seqs, heads=kv * group, kv_heads=kv, dim=dim,
                page=page, prefix=max(prefix, 1), least=max(1, prefix // rng.choice([1, 3])),
                own=own_tokens, queries=queries, spread=rng.randint(1, 1 << 30))


def _requests(case):
    """Prefix of each group, and the own tokens and query tokens of its requests."""
    rng = random.Random(case["spread"])
    prefix, own_tokens, qs = [], [], []
    for g in range(case["groups"]):
        prefix.append(case["prefix"] if g == 0 else _log(rng, case["least"], case["prefix"]))
        n = case["seqs"] if g == 0 else rng.randint((case["seqs"] + 1) // 2, case["seqs"])
        q = [case["queries"] if i == 0 else rng.randint((case["queries"] + 1) // 2, case["queries"])
             for i in range(n)]
        own_tokens.append([max(q[i], case["own"] if i == 0 else _log(rng, 1, case["own"]))
                           for i in range(n)])
        qs.append(q)
    return prefix, own_tokens, qs


def _lengths(case):
    """Tokens of each row of a pool, from the case alone."""
    rng = random.Random(case["rows"] * 7919 + case["pages"])
    return [_log(rng, case["low"], case["high"]) for _ in range(case["rows"])]


def _page_bytes(case):
    return case["kv_heads"] * case["page"] * case["dim"] * 9 // 8


def work(case):
    op = case["op"]
    if op == "norm":
        n, t = case["tokens"] * case["hidden"], case["tokens"]
        eb, rb = (2 if case["dtype"] == "bf16" else 4), (2 if case["residual"] == "bf16" else 4)
        gate = {"none": 0, "channel": case["hidden"], "token": t, "full": n}[case["gate"]]
        vectors = (1 + case["post"]) * (2 if case["kind"] == "layer" else 1) * case["hidden"]
        return dict(bytes=n * (2 * eb + 2 * rb) + gate * eb + 4 * vectors,
                    flops=n * (8 if case["post"] else 5))
    if op == "share":
        ps, lens, forks = case["page"], _lengths(case), case["forks"]
        ended, new = lens[-forks:], lens[:case["rows"] - forks]
        entries = sum(-(-n // ps) for n in ended)
        taken = [new[i % len(new)] if new else 0 for i in range(forks)]
        entries += 2 * sum(-(-n // ps) for n in taken)
        copies = sum(n % ps != 0 for n in taken)
        return dict(bytes=4 * (case["pages"] + 2 * entries + 6 * case["rows"])
                    + 2 * copies * case["caches"] * _page_bytes(case), flops=case["pages"])
    if op == "copy":
        return dict(bytes=2 * case["moved"] * case["caches"] * _page_bytes(case) + 8 * case["moved"],
                    flops=case["moved"])
    if op == "compact":
        p, f = case["pages"], case["free"]
        moves = int(p * (1 - f) * f)       # free pages below the count of used ones, in the mean
        return dict(bytes=2 * moves * case["caches"] * _page_bytes(case) + 12 * p, flops=p)
    d, kv, h = case["dim"], case["kv_heads"], case["heads"]
    eb = 2 if case["dtype"] == "bf16" else 4
    keys, pairs, tq, pages = 0, 0, 0, 0
    for p, owns, qs in zip(*_requests(case)):
        keys += p + sum(owns)
        for o, q in zip(owns, qs):
            pairs += q * (p + o - q) + q * (q + 1) // 2
            tq += q
            pages += -(-(p + o) // case["page"])
    return dict(bytes=2 * kv * (d * 9 // 16) * keys + tq * h * (2 * eb * d + 4) + 4 * pages,
                flops=4 * d * h * pairs)


# ------------------------------------------------------------------ inputs
def _quantise(x):
    """Codes and scales of fp32 rows [..., D]: groups of 16 channels share the
    e4m3 value nearest to their largest magnitude over 6."""
    g = x.unflatten(-1, (-1, GROUP))
    s = (g.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    y = torch.where(sf > 0, g.abs() / sf, torch.zeros((), device=x.device))
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5)
            + (y >= 3.5) + (y > 5.0)).to(torch.uint8)
    code = (code | ((g < 0) & (code > 0)).to(torch.uint8) * 8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _parts(cache, page, dim):
    """Views of the keys' codes and scales and of the values' in the cache: [pages, kv_heads, page, n]."""
    sizes = (page * dim // 2, page * dim // 16, page * dim // 2, page * dim // 16)
    out, at = [], 0
    for n in sizes:
        out.append(cache[..., at:at + n].unflatten(-1, (page, n // page)))
        at += n
    return out


def _fill(cache, page, dim, gen):
    """Keys (some channels far larger than others) and values of a filled cache."""
    kc, ks, vc, vs = _parts(cache, page, dim)
    loud = torch.exp(0.6 * torch.randn(cache.shape[1], 1, dim, generator=gen, device=cache.device))
    step = max(1, (1 << 27) // (cache.shape[1] * page * dim))
    for i in range(0, cache.shape[0], step):
        n = min(step, cache.shape[0] - i)
        shape = (n, cache.shape[1], page, dim)
        k = torch.randn(shape, generator=gen, device=cache.device) * loud
        kc[i:i + n], ks[i:i + n] = _quantise(k.bfloat16().float())
        v = torch.randn(shape, generator=gen, device=cache.device)
        vc[i:i + n], vs[i:i + n] = _quantise(v.bfloat16().float())


def _caches(case, pages, gen):
    """A cache per layer, of any bytes: these operators do not look into a page."""
    shape = (pages, case["kv_heads"], case["page"] * case["dim"] * 9 // 8)
    return [torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)
            for _ in range(case["caches"])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case, plan=None)
    return {"norm": _prepare_norm, "share": _prepare_share, "copy": _prepare_copy,
            "compact": _prepare_compact, "attend": _prepare_attend}[case["op"]](s, case, gen)


def _prepare_norm(s, case, gen):
    t, h, dt, rt = case["tokens"], case["hidden"], TYPES[case["dtype"]], TYPES[case["residual"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    loud = torch.exp(0.7 * randn(h))
    s["y"] = (randn(t, h) * loud).to(dt)
    s["x"] = (2.0 * randn(t, h) * loud + (0.5 if case["kind"] == "layer" else 0.0)).to(rt)
    for name in ("post", "pre"):
        here = name == "pre" or case["post"]
        s[name + "_w"] = 1.0 + 0.2 * randn(h) if here else None
        s[name + "_b"] = 0.1 * randn(h) if here and case["kind"] == "layer" else None
    s["gate"] = {"none": lambda: None, "channel": lambda: randn(h).to(dt),
                 "token": lambda: randn(t, 1).to(dt), "full": lambda: randn(t, h).to(dt)}[case["gate"]]()
    s["x_out"] = torch.empty(t, h, dtype=rt, device="cuda")
    s["h"] = torch.empty(t, h, dtype=dt, device="cuda")
    return s


def _prepare_share(s, case, gen):
    """Rows of their own pages. The last `forks` of them end, and are then forked
    from the first ones in turn."""
    ps, rows, pages, forks = case["page"], case["rows"], case["pages"], case["forks"]
    lens = _lengths(case)
    counts = [-(-n // ps) for n in lens]
    width = -(-(case["high"] + case["tokens"]) // ps) + 1
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    count = torch.tensor(counts, device="cuda")
    first = count.cumsum(0) - count
    col = torch.arange(width, device="cuda")
    table = torch.where(col < count[:, None], order[(first[:, None] + col).clamp(max=pages - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[order[:sum(counts)].long()] = 1
    # one buffer, so that a pass starts from the same pool again with one copy
    # (the page a copy goes to is free at the start of each pass, so the caches need none)
    s["first"] = torch.cat([table.flatten(), count.int(), refs])
    s["buffer"] = torch.empty_like(s["first"])
    table, held, refs = s["buffer"].split([rows * width, rows, pages])
    s["table"], s["held"], s["refs"] = table.view(rows, width), held, refs
    s["caches"] = _caches(case, pages, gen)
    left = rows - forks
    child = torch.arange(left, rows, device="cuda", dtype=torch.int32)
    parent = (torch.arange(forks, device="cuda") % left).int()
    lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["ended"], s["child"], s["parent"] = child, child, parent
    s["shared"] = lens[parent.long()].contiguous()
    s["start"] = torch.cat([lens[:left], s["shared"]])
    s["end"] = s["start"] + case["tokens"]
    return s


def _prepare_copy(s, case, gen):
    n, pages = case["moved"], case["pages"]
    s["from"] = _caches(case, pages, gen)
    s["to"] = [torch.zeros_like(c) for c in s["from"]]
    s["src"] = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)[:n].contiguous()
    s["dst"] = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)[:n].contiguous()
    return s


def _prepare_compact(s, case, gen):
    """Rows share out the pages in use, every fourth row holds the first pages of the row before as well."""
    rows, pages = case["rows"], case["pages"]
    used = max(1, int(round(pages * (1 - case["free"]))))
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)[:used]
    count = torch.full((rows,), used // rows, device="cuda") + (torch.arange(rows, device="cuda") < used % rows)
    first = count.cumsum(0) - count
    width = int(used // rows) * 2 + 3
    col = torch.arange(width, device="cuda")
    both = (torch.arange(rows, device="cuda") % 4 == 3)
    shared = torch.where(both, torch.roll(count, 1) // 2, torch.zeros_like(count))
    begin = torch.roll(first, 1)
    index = torch.where(col < shared[:, None], begin[:, None] + col,
                        first[:, None] + col - shared[:, None]).clamp(0, used - 1)
    held = count + shared
    live = col < held[:, None]
    table = torch.where(live, order[index], torch.full((), -1, dtype=torch.int32, device="cuda"))
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs.scatter_add_(0, table.clamp(min=0).flatten().long(), live.flatten().int())
    # (moved pages stay readable in their old places, so the caches need no fresh start)
    s["first"] = torch.cat([table.flatten(), held.int(), refs])
    s["buffer"] = torch.empty_like(s["first"])
    table, held, refs = s["buffer"].split([rows * width, rows, pages])
    s["table"], s["held"], s["refs"] = table.view(rows, width), held, refs
    s["used"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["caches"] = _caches(case, pages, gen)
    return s


def _prepare_attend(s, case, gen):
    page, kv, d, h = case["page"], case["kv_heads"], case["dim"], case["heads"]
    prefix, owns, qs = _requests(case)
    # full pages of a prefix are shared; the page that it ends in is each request's own copy
    pages = sum(p // page for p in prefix) + sum(-(-(p + o) // page) - p // page
                                                for p, row in zip(prefix, owns) for o in row) + 3
    s["cache"] = torch.empty(pages, kv, page * d * 9 // 8, dtype=torch.uint8, device="cuda")
    _fill(s["cache"], page, d, gen)
    order = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)
    seqs = sum(len(row) for row in owns)
    width = max(-(-(p + max(row)) // page) for p, row in zip(prefix, owns))
    s["table"] = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
    parts = _parts(s["cache"], page, d)
    at, b, lens, counts, offsets = 0, 0, [], [], [0]
    for p, row, q in zip(prefix, owns, qs):
        full, rest = p // page, p % page
        common = order[at:at + full]
        at += full
        for i, o in enumerate(row):
            n = -(-(p + o) // page) - full
            s["table"][b, :full] = common
            s["table"][b, full:full + n] = order[at:at + n]
            if rest and i > 0:
                for x in parts:
                    x[order[at], :, :rest] = x[head, :, :rest]
            elif rest:
                head = order[at]
            at += n
            b += 1
            lens.append(p + o)
            counts.append(q[i])
        offsets.append(b)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    total = [0]
    for c in counts:
        total.append(total[-1] + c)
    s["q_offsets"], s["seq_lens"] = ints(total), ints(lens)
    s["group_offsets"], s["prefix_lens"] = ints(offsets), ints(prefix)
    s["prefix"], s["lens"], s["counts"], s["groups"] = prefix, lens, counts, offsets
    s["max_q"] = max(counts)
    s["max_group"] = max(sum(q) for q in qs)
    q = 1.5 * torch.randn(total[-1], h + 2 * kv, d, generator=gen, device="cuda")
    s["q"] = q.to(TYPES[case["dtype"]])[:, :h]           # the fused projection's rows
    s["out"] = torch.empty(total[-1], h, d, dtype=s["q"].dtype, device="cuda")
    s["lse"] = torch.empty(total[-1], h, device="cuda")
    return s


# ------------------------------------------------------------------ passes
def run(s):
    op = s["case"]["op"]
    if op in ("share", "compact"):
        s["buffer"].copy_(s["first"])
    if own:
        return {"norm": _own_norm, "share": _own_share, "copy": _own_copy, "compact": _own_compact,
                "attend": _own_attend}[op](s)
    return {"norm": _plain_norm, "share": _plain_share, "copy": _plain_copy,
            "compact": _plain_compact, "attend": _plain_attend}[op](s)


def _plan(s):
    """The library's handles, which a user's program makes once and keeps."""
    if s["plan"] is not None:
        return s["plan"]
    from expert_moe_layer_gb300 import binding as B
    c = s["case"]
    p = dict(lib=B)
    if c["op"] == "norm":
        p["cfg"] = B.make_norm_config(c["hidden"], kind=c["kind"], act_dtype=c["dtype"],
                                      residual_dtype=c["residual"], post_norm=c["post"],
                                      residual_scale=c["scale"],
                                      gate="sigmoid" if c["gate"] == "token" else "linear")
        s["plan"] = p
        return p
    p["cfg"] = B.make_attn_config(c.get("heads", c["kv_heads"]), c["kv_heads"], c["dim"], c["page"],
                                  act_dtype=c.get("dtype", "bf16"))
    if c["op"] == "copy":
        p["from"], p["to"] = B.make_kv_caches(p["cfg"], s["from"]), B.make_kv_caches(p["cfg"], s["to"])
    elif c["op"] == "attend":
        n = B.kv_attention_shared_workspace_size(p["cfg"], len(s["lens"]), s["q"].shape[0], s["max_q"],
                                                 len(s["prefix"]), s["max_group"])
        p["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    else:
        p["pool"] = B.make_kv_pool(p["cfg"], s["table"], s["held"], s["refs"], s["caches"])
        n = B.kv_pool_workspace_size(p["cfg"], p["pool"], c["rows"])
        p["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    s["plan"] = p
    return p


def _own_norm(s):
    p = _plan(s)
    p["lib"].moe_norm(p["cfg"], s["case"]["tokens"], s["y"], s["x"], s["post_w"], s["post_b"], s["gate"],
                      s["pre_w"], s["pre_b"], s["x_out"], s["h"])
    return dict(x=s["x_out"], h=s["h"])


def _own_share(s):
    p, n = _plan(s), s["case"]["forks"]
    B, cfg, pool, ws = p["lib"], p["cfg"], p["pool"], p["ws"]
    B.moe_kv_release(cfg, pool, n, s["ended"], None, ws)
    B.moe_kv_fork(cfg, pool, n, s["parent"], s["child"], s["shared"], ws)
    B.moe_kv_reserve(cfg, pool, s["case"]["rows"], None, s["start"], s["end"], ws)
    return dict(table=s["table"], held=s["held"], refs=s["refs"], caches=s["caches"])


def _own_copy(s):
    p = _plan(s)
    p["lib"].moe_kv_copy_pages(p["cfg"], p["from"], p["to"], s["case"]["moved"], s["src"], s["dst"])
    return s["to"]


def _own_compact(s):
    p = _plan(s)
    p["lib"].moe_kv_compact(p["cfg"], p["pool"], s["used"], p["ws"])
    return dict(table=s["table"], held=s["held"], refs=s["refs"], used=s["used"], caches=s["caches"])


def _own_attend(s):
    p = _plan(s)
    p["lib"].moe_kv_attention_shared(p["cfg"], len(s["lens"]), s["q"].shape[0], s["max_q"],
                                     len(s["prefix"]), s["max_group"], s["q"], s["q_offsets"],
                                     s["seq_lens"], s["table"], s["group_offsets"], s["prefix_lens"],
                                     s["cache"], s["out"], s["lse"], p["ws"])
    return dict(out=s["out"], lse=s["lse"])


def _normed(x, w, b, layer):
    if layer:
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    return x if b is None else x + b


def _plain_norm(s):
    c = s["case"]
    layer = c["kind"] == "layer"
    u = s["y"].float()
    if c["post"]:
        u = _normed(u, s["post_w"], s["post_b"], layer)
    if s["gate"] is not None:
        g = s["gate"].float()
        u = u * (1.0 / (1.0 + (-g).exp()) if c["gate"] == "token" else g)
    r = s["x"].float() + c["scale"] * u
    return dict(x=r.to(s["x"].dtype), h=_normed(r, s["pre_w"], s["pre_b"], layer).to(s["y"].dtype))


def _add_refs(refs, entries, live, by):
    """refs[entries] += by where live."""
    refs.scatter_add_(0, torch.where(live, entries, torch.zeros_like(entries)).flatten().long(),
                      live.flatten().int() * by)


def _plain_share(s):
    c = s["case"]
    ps, table, held, refs = c["page"], s["table"], s["held"], s["refs"]
    col = torch.arange(table.shape[1], device="cuda")
    # rows that ended give their pages back
    r = s["ended"].long()
    live = col < held[r][:, None]
    _add_refs(refs, table[r], live, -1)
    table[r] = torch.where(live, torch.full_like(table[r], -1), table[r])
    held[r] = 0
    # forks hold their parents' pages
    n = (s["shared"] + ps - 1) // ps
    live = col < n[:, None]
    entries = table[s["parent"].long()]
    _add_refs(refs, entries, live, 1)
    ch = s["child"].long()
    table[ch] = torch.where(live, entries, table[ch])
    held[ch] = n
    # room for the next tokens: pages past the last one, and those that others hold too
    start, end = s["start"], s["end"]
    need = ((end + ps - 1) // ps)[:, None]
    lo = (start // ps)[:, None]
    old = (col < held[:, None]) & (col >= lo) & (col < need)
    old &= refs[table.clamp(min=0).long()] > 1
    new = (col >= held[:, None]) & (col < need)
    fresh = old | new
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True).int()     # lowest ids first
    rank = fresh.flatten().cumsum(0).view(fresh.shape) - 1
    page = torch.where(fresh, free[rank.clamp(0, free.shape[0] - 1)], table)
    # the page in which a row goes on, where others hold it too, with what it has
    cut = (start % ps != 0) & old.gather(1, lo.long().clamp(max=table.shape[1] - 1))[:, 0]
    at = lo.long().clamp(max=table.shape[1] - 1)
    src, dst = table.gather(1, at)[:, 0].long(), page.gather(1, at)[:, 0].long()
    src = torch.where(cut, src, table[0, 0].long())      # a page onto itself where nothing is copied
    dst = torch.where(cut, dst, table[0, 0].long())
    for x in s["caches"]:
        x[dst] = x[src]
    _add_refs(refs, table, old, -1)
    refs.scatter_add_(0, page.clamp(min=0).flatten().long(), fresh.flatten().int())
    table.copy_(page)
    held.copy_(torch.maximum(held, need[:, 0]))
    return dict(table=table, held=held, refs=refs, caches=s["caches"])


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for x, y in zip(s["from"], s["to"]):
        y[dst] = x[src]
    return s["to"]


def _plain_compact(s):
    table, held, refs = s["table"], s["held"], s["refs"]
    pages = refs.shape[0]
    live = refs > 0
    used = live.sum()
    ids = torch.arange(pages, device="cuda")
    high, low = live & (ids >= used), ~live & (ids < used)
    # the k-th used page past the count of used ones goes to the k-th free page before it
    src, dst = high.nonzero()[:, 0], low.nonzero()[:, 0]
    for x in s["caches"]:
        x[dst] = x[src]
    to = ids.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    mine = torch.arange(table.shape[1], device="cuda") < held[:, None]
    table.copy_(torch.where(mine, to[table.clamp(min=0).long()].int(), table))
    s["used"][0] = used
    return dict(table=table, held=held, refs=refs, used=s["used"], caches=s["caches"])


def _values(codes, scales):
    """fp32 values of code bytes [..., D/2] and scale bytes [..., D/16]."""
    one = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    b = torch.arange(256, device=codes.device)
    lut = torch.stack([one[b & 15], one[b >> 4]], dim=1)
    x = lut[codes.to(torch.int32)].flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _plain_attend(s):
    """Each group's prefix in one product for all of its rows, then each request's own tokens."""
    c = s["case"]
    kv, d, h, page = c["kv_heads"], c["dim"], c["heads"], c["page"]
    parts = _parts(s["cache"], page, d)
    out, lse = torch.empty_like(s["out"]), torch.empty_like(s["lse"])
    at = 0
    for g, p in enumerate(s["prefix"]):
        b0, b1 = s["groups"][g], s["groups"][g + 1]
        t = torch.arange(p, device="cuda")
        id0 = s["table"][b0, t // page].long()
        rows = [x[id0, :, t % page].transpose(0, 1) for x in parts]           # [kv, P, n]
        k0, v0 = _values(rows[0], rows[1]), _values(rows[2], rows[3])
        counts, lens = s["counts"][b0:b1], s["lens"][b0:b1]
        m, most = max(counts), max(lens) - p
        n = sum(counts)
        q = s["q"][at:at + n].float().unflatten(1, (kv, h // kv))
        scale = d ** -0.5
        x0 = torch.einsum("tkgd,knd->ktgn", q, k0) * scale                    # [kv, t, g, P]
        # own tokens, padded to the longest request of the group
        t = p + torch.arange(most, device="cuda")
        seq = torch.arange(b0, b1, device="cuda")
        ids = s["table"][seq[:, None], (t // page).clamp(max=s["table"].shape[1] - 1)].long()
        own_rows = [x[ids, :, (t % page).expand_as(ids)].transpose(1, 2) for x in parts]  # [b, kv, o, n]
        k1, v1 = _values(own_rows[0], own_rows[1]), _values(own_rows[2], own_rows[3])
        off = s["q_offsets"].long()[b0:b1 + 1] - at
        row = torch.arange(n, device="cuda")
        b = torch.searchsorted(off[1:], row, right=True)
        j = row - off[b]
        padded = torch.zeros(b1 - b0, m, kv, h // kv, d, device="cuda")
        padded[b, j] = q
        x1 = torch.einsum("bmkgd,bkod->bmkgo", padded, k1) * scale
        last = s["seq_lens"].long()[b0:b1] - (off[1:] - off[:-1])
        seen = t <= (last[:, None] + torch.arange(m, device="cuda"))[..., None]
        x1.masked_fill_(~seen[:, :, None, None], NEG)
        x1 = x1[b, j].transpose(0, 1)                                          # [kv, t, g, o]
        top = torch.maximum(x0.amax(-1, keepdim=True), x1.amax(-1, keepdim=True))
        x0.sub_(top).exp_()
        x1 = (x1 - top).exp()
        total = x0.sum(-1, keepdim=True) + x1.sum(-1, keepdim=True)
        o = torch.einsum("ktgn,knd->ktgd", x0, v0)
        pad1 = torch.zeros(b1 - b0, m, kv, h // kv, most, device="cuda")
        pad1[b, j] = x1.transpose(0, 1)
        o = o + torch.einsum("bmkgo,bkod->bmkgd", pad1, v1)[b, j].transpose(0, 1)
        o = o / total
        out[at:at + n] = o.transpose(0, 1).flatten(1, 2).to(out.dtype)
        lse[at:at + n] = (top + total.log())[..., 0].transpose(0, 1).flatten(1, 2)
        at += n
    return dict(out=out, lse=lse)


# ------------------------------------------------------- the same in 64 bits
def _exact_norm(case, s):
    def normed(x, w, b):
        if case["kind"] == "layer":
            var, mean = torch.var_mean(x, dim=-1, correction=0, keepdim=True)
            x = x - mean
        else:
            var = (x * x).sum(-1, keepdim=True) / x.shape[-1]
        x = x / torch.sqrt(var + 1e-6) * w.double()
        return x if b is None else x + b.double()

    u = s["y"].double()
    if case["post"]:
        u = normed(u, s["post_w"], s["post_b"])
    if case["gate"] == "token":
        u = u / (1.0 + torch.exp(-s["gate"].double()))
    elif case["gate"] != "none":
        u = u * s["gate"].double()
    r = s["x"].double() + case["scale"] * u
    return dict(x=r, h=normed(r, s["pre_w"], s["pre_b"]))


def exact(case, seed):
    if case["op"] not in ("norm", "attend"):
        return None                                    # copies and whole numbers
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    kv, d, h, page = case["kv_heads"], case["dim"], case["heads"], case["page"]
    g = h // kv
    level = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, NEG, dtype=torch.float64, device="cuda")

    def rows(codes, scales):
        n = codes.reshape(-1, d // 2)
        n = torch.stack([n & 15, n >> 4], -1).flatten(-2).int()
        x = level[n & 7] * (1 - 2 * (n >> 3)).double()
        return x * scales.reshape(-1, d // 16).view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, 1)

    at = 0
    for b, (n, q) in enumerate(zip(s["lens"], s["counts"])):
        ids = s["table"][b, :-(-n // page)].long()
        for j in range(kv):
            kc, ks, vc, vs = _parts(s["cache"][ids, j:j + 1], page, d)
            k, v = rows(kc[:, 0], ks[:, 0])[:n], rows(vc[:, 0], vs[:, 0])[:n]
            x = s["q"][at:at + q, j * g:(j + 1) * g].double()
            x = torch.einsum("mgd,nd->mgn", x, k) / math.sqrt(d)
            hide = torch.arange(n, device="cuda") > n - q + torch.arange(q, device="cuda")[:, None]
            x = x.masked_fill(hide[:, None], NEG)
            w = torch.logsumexp(x, -1)
            lse[at:at + q, j * g:(j + 1) * g] = w
            out[at:at + q, j * g:(j + 1) * g] = torch.einsum("mgn,nd->mgd", (x - w[..., None]).exp(), v)
        at += q
    return dict(out=out, lse=lse)
