"""Cases of the attention operators beside the MoE layer: rotary positions,
the append of rotated keys and of values to a paged 4-bit cache, and attention
over that cache.

``run`` computes a case either in plain torch operations (``own`` false) or by
the library's entry points (``own`` true), on the same inputs.

The cache is ``[pages, kv_heads, page_size * head_dim * 9 / 8]`` bytes. One
(page, kv head) block holds the keys' codes ``[page_size, head_dim / 2]``, the
keys' scales ``[page_size, head_dim / 16]``, then the values' codes and scales.
A code is a 4-bit float (e2m1), two to a byte, the lower channel in the low
half. A scale is an 8-bit float (e4m3) for 16 neighbouring channels.
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
        # one decode step of a batch of 64 requests: queries in the fused projection's rows
        dict(name="rope_step", op="rope", dtype="bf16", tokens=64, heads=32, dim=128, rotary=128,
             layout="half", positions=32768, inverse=False),
        # a prompt's queries, half of each head rotated, neighbouring channels paired
        dict(name="rope_prompt", op="rope", dtype="bf16", tokens=8192, heads=40, dim=128,
             rotary=64, layout="interleaved", positions=16384, inverse=False),
        # turning rotated fp32 rows back (the gradient's direction), an odd count of them
        dict(name="rope_back", op="rope", dtype="f32", tokens=4097, heads=16, dim=256, rotary=256,
             layout="half", positions=8192, inverse=True),
        # the cosines and sines of one step's tokens, for requests far beyond any table
        dict(name="table_step", op="table", rotary=64, tokens=64, positions=1 << 20,
             scaling="none", base=1e4, factor=1.0, original=2048),
        # the rows of 131072 cached tokens, with the per-dimension ramp of a long-context model
        dict(name="table_long", op="table", rotary=128, tokens=131072, positions=1 << 20,
             scaling="yarn", base=1e6, factor=16.0, original=8192),
        # the new token of each of 64 requests into the cache
        dict(name="append_step", op="append", dtype="bf16", tokens=64, heads=32, kv_heads=8,
             dim=128, rotary=128, layout="half", positions=32768, page=64),
        # a prompt chunk of 8192 tokens into the cache
        dict(name="append_prompt", op="append", dtype="bf16", tokens=8192, heads=40, kv_heads=8,
             dim=128, rotary=64, layout="interleaved", positions=16384, page=16),
        # one request's single token over a short context: latency
        dict(name="attend_one", op="attend", dtype="bf16", seqs=1, heads=16, kv_heads=2, dim=128,
             page=16, low=1000, high=1000, queries=1, window=0, spread=0),
        # a decode step of 64 requests of very different lengths
        dict(name="attend_step", op="attend", dtype="bf16", seqs=64, heads=32, kv_heads=8,
             dim=128, page=64, low=1, high=16384, queries=1, window=0, spread=1),
        # a decode step of 8 requests over long documents
        dict(name="attend_long", op="attend", dtype="bf16", seqs=8, heads=32, kv_heads=8,
             dim=128, page=64, low=131071, high=131071, queries=1, window=0, spread=0),
        # fp32 layers: a few tokens per request (drafts to be checked), sliding window
        dict(name="attend_draft_f32", op="attend", dtype="f32", seqs=21, heads=24, kv_heads=4,
             dim=64, page=32, low=17, high=4096, queries=5, window=1000, spread=2),
        # prompt chunks of four requests, each after a context of its own
        dict(name="attend_prompt", op="attend", dtype="bf16", seqs=4, heads=32, kv_heads=8,
             dim=128, page=64, low=2048, high=16384, queries=2048, window=0, spread=3),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "table", "append", "append", "attend", "attend", "attend", "attend"])
    if op == "table":
        r = 2 * rng.randint(16, 64)
        return dict(op=op, rotary=r, tokens=_log(rng, 16, 131072),
                    positions=_log(rng, 1 << 13, 1 << 23),
                    scaling=rng.choice(["none", "linear", "ntk", "parts", "yarn"]),
                    base=rng.choice([1e4, 5e5, 1e6]), factor=rng.choice([2.0, 8.0, 16.0]),
                    original=rng.choice([2048, 4096, 8192]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    if kv * group > 64:
        group = 64 // kv
    heads = kv * group
    layout = rng.choice(["half", "interleaved"])
    rotary = rng.choice([dim, dim // 2, dim - 2 * rng.randint(1, dim // 4)])
    if op == "rope":
        most = 8192 * 40 * 128 // (heads * dim)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, min(8192, most)), heads=heads, dim=dim,
                    rotary=rotary, layout=layout, positions=_log(rng, 8192, 32768),
                    inverse=rng.random() < 0.3)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        most = 8192 * 40 * 128 // ((heads + 2 * kv) * dim)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, min(8192, most)), heads=heads,
                    kv_heads=kv, dim=dim, rotary=rotary, layout=layout,
                    positions=_log(rng, 8192, 32768), page=page)
    window = rng.choice([0, 0, 0, _log(rng, 64, 4096)])
    spread = rng.randint(1, 1 << 30)
    if rng.random() < 0.6:  # a decode step, a few tokens at most
        seqs = _log(rng, 1, 128)
        most = min(131072, 64 * 8192 * 8 * 128 // (seqs * kv * dim))
        high = _log(rng, 16, max(17, most))
        queries = rng.choice([1, 1, 1, 2, 4])
    else:
        seqs = rng.randint(1, 8)
        queries = _log(rng, 16, 4096 // seqs)
        high = queries + _log(rng, 1, 8192)
        if dtype == "f32":
            queries = min(queries, 256)
        while 4 * dim * heads * seqs * queries * high > 6e11:
            queries //= 2
    return dict(op=op, dtype=dtype, seqs=seqs, heads=heads, kv_heads=kv, dim=dim, page=page,
                low=max(1, high // rng.choice([1, 2, 16])), high=high, queries=queries,
                window=window, spread=spread)


def _lengths(case):
    """Tokens in the cache and query tokens of each request."""
    rng = random.Random(case["spread"])
    lens, qs = [], []
    for i in range(case["seqs"]):
        n = case["high"] if i == 0 else _log(rng, case["low"], case["high"])
        q = case["queries"] if i == 0 or case["queries"] == 1 else \
            rng.randint((case["queries"] + 1) // 2, case["queries"])
        lens.append(n)
        qs.append(min(q, n))
    return lens, qs


def _visible(n, q, window):
    """(query, key) pairs of a request: query i sees the keys up to its own."""
    if not window:
        return q * (n - q) + q * (q + 1) // 2
    first, last = n - q + 1, n
    short = max(0, min(last, window) - first + 1)
    return short * (2 * first + short - 1) // 2 + (q - short) * window


def work(case):
    op = case["op"]
    if op == "table":
        n = case["tokens"] * case["rotary"]
        return dict(bytes=4 * n + 4 * case["tokens"], flops=2 * n)
    eb = 2 if case["dtype"] == "bf16" else 4
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        t = case["tokens"]
        return dict(bytes=2 * eb * n + 4 * t + 4 * min(t, case["positions"]) * case["rotary"],
                    flops=3 * t * case["heads"] * case["rotary"])
    d, kv, h = case["dim"], case["kv_heads"], case["heads"]
    row = d * 9 // 16
    if op == "append":
        t = case["tokens"]
        moved = eb * d * (2 * h + 2 * kv) + 2 * kv * row       # q in and out, k and v in, rows out
        back = 2 * kv * (row + eb * d)                        # the appended rows read back
        return dict(bytes=t * (moved + back + 4 + 16) + 4 * min(t, case["positions"]) * case["rotary"],
                    flops=t * (3 * (h + kv) * case["rotary"] + 6 * kv * d))
    lens, qs = _lengths(case)
    keys, pairs = 0, 0
    for n, q in zip(lens, qs):
        w = case["window"]
        keys += min(n, q + w - 1) if w else n
        pairs += _visible(n, q, w)
    tq = sum(qs)
    return dict(bytes=2 * kv * row * keys + tq * h * (2 * eb * d + 4) + 4 * sum(-(-n // case["page"]) for n in lens),
                flops=4 * d * h * pairs)


# ------------------------------------------------------------------ inputs
def _frequencies(rotary, base, scaling, factor, original):
    """Radians per position of each pair, and the factor on the cosines and sines."""
    i = torch.arange(0, rotary, 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    f = base ** (-i / rotary)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "parts":       # by wavelength, between 1 and 4 of them in the original context
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    if scaling == "yarn":        # a ramp over the dimensions, from 32 turns down to 1
        def at(turns):
            return rotary * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rotary - 1)
        if low == high:
            high += 0.001
        ramp = ((torch.arange(rotary // 2, dtype=torch.float64) - low) / (high - low)).clamp(0, 1)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _table(positions, rotary, base, scaling, factor, original):
    f, m = _frequencies(rotary, base, scaling, factor, original)
    a = positions.double()[:, None] * f.to(positions.device)
    return torch.cat([a.cos() * m, a.sin() * m], dim=1).float()


def _quantise(x):
    """Codes and scales of fp32 rows [..., D]: groups of 16 channels share the
    e4m3 value nearest to their largest magnitude over 6."""
    x = torch.where(x != x, torch.zeros((), device=x.device), x)
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


def _values(codes, scales):
    """fp32 values of code bytes [..., D/2] and scale bytes [..., D/16]."""
    one = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device=codes.device)
    b = torch.arange(256, device=codes.device)
    lut = torch.stack([one[b & 15], one[b >> 4]], dim=1)
    x = lut[codes.to(torch.int32)].flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


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


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = dict(case=case)
    op = case["op"]
    if op == "table":
        s["positions"] = torch.randint(0, case["positions"], (case["tokens"],), generator=gen,
                                       device=dev, dtype=torch.int32)
        s["out"] = torch.empty(case["tokens"], case["rotary"], device=dev)
        _config(s, dict(rotary_dim=case["rotary"], rope_positions=case["tokens"],
                        head_dim=-(-case["rotary"] // 64) * 64, num_heads=1, num_kv_heads=1))
        return s
    dt, d, h = TYPES[case["dtype"]], case["dim"], case["heads"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if op in ("rope", "append"):
        t, kv = case["tokens"], case.get("kv_heads", 8)
        s["table"] = _table(torch.arange(case["positions"], device=dev), case["rotary"], 1e4, "none",
                            1.0, 1)
        at = torch.arange(t, device=dev)
        if t <= 256:      # a step: one token of each request, anywhere
            s["positions"] = torch.randint(0, case["positions"], (t,), generator=gen, device=dev,
                                           dtype=torch.int32)
        else:             # a prompt chunk: consecutive tokens
            first = seed % max(1, case["positions"] - t)
            s["positions"] = ((first + at) % case["positions"]).int()
        rows = randn(t, h + 2 * kv, d).to(dt)     # the fused projection's rows
        s["q"] = rows[:, :h]
        s["q_out"] = torch.empty(t, h, d, dtype=dt, device=dev)
        if op == "append":
            s["k"], s["v"] = rows[:, h:h + kv], rows[:, h + kv:]
            page = case["page"]
            pages = 2 * -(-t // page) + 1
            s["cache"] = torch.zeros(pages, kv, page * d * 9 // 8, dtype=torch.uint8, device=dev)
            if t <= 256:
                s["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:t]
            else:
                order = torch.randperm(pages, generator=gen, device=dev)
                s["slots"] = order[at // page] * page + at % page
            s["k_out"] = torch.empty(t, kv, d, dtype=dt, device=dev)
            s["v_out"] = torch.empty(t, kv, d, dtype=dt, device=dev)
        _config(s, dict(num_heads=h, num_kv_heads=kv, head_dim=d, page_size=case.get("page", 16),
                        act_dtype=case["dtype"], rotary_dim=case["rotary"],
                        rope_layout=case["layout"], rope_positions=case["positions"]))
        return s
    lens, qs = _lengths(case)
    page, kv = case["page"], case["kv_heads"]
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 3
    s["cache"] = torch.empty(pages, kv, page * d * 9 // 8, dtype=torch.uint8, device=dev)
    _fill(s["cache"], page, d, gen)
    order = torch.randperm(pages, generator=gen, device=dev, dtype=torch.int32)
    s["page_table"] = torch.zeros(len(lens), max(counts), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(counts):
        s["page_table"][i, :n] = order[at:at + n]
        at += n
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    offs = [0]
    for q in qs:
        offs.append(offs[-1] + q)
    s["q_offsets"] = torch.tensor(offs, dtype=torch.int32, device=dev)
    s["max_len"], s["max_q"] = max(lens), max(qs)
    s["q"] = (1.5 * randn(offs[-1], h + 2 * kv, d)).to(dt)[:, :h]
    s["out"] = torch.empty(offs[-1], h, d, dtype=dt, device=dev)
    s["lse"] = torch.empty(offs[-1], h, device=dev)
    _config(s, dict(num_heads=h, num_kv_heads=kv, head_dim=d, page_size=page,
                    act_dtype=case["dtype"], window=case["window"]))
    return s


def _config(s, fields):
    """What a user of the library keeps beside the tensors; made at the first own pass."""
    s["fields"] = fields
    s["plan"] = None


# ------------------------------------------------------------------ passes
def run(s):
    if own:
        return _own(s)
    return {"table": _plain_table, "rope": _plain_rope, "append": _plain_append,
            "attend": _plain_attend}[s["case"]["op"]](s)


def _own(s):
    case = s["case"]
    op = case["op"]
    if s["plan"] is None:
        from expert_moe_layer_gb300 import binding as B
        cfg = B.make_attn_config(**s["fields"])
        p = dict(cfg=cfg, lib=B)
        if op == "table":
            p["scaling"] = B.make_rope_scaling(case["base"], case["scaling"], case["factor"],
                                               case["original"])
        if op == "attend":
            n = B.kv_attention_workspace_size(cfg, case["seqs"], s["q"].shape[0], s["max_q"])
            p["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        s["plan"] = p
    p = s["plan"]
    cfg, B = p["cfg"], p["lib"]
    if op == "table":
        B.moe_rope_table(cfg, case["tokens"], s["positions"], p["scaling"], s["out"])
        return s["out"]
    if op == "rope":
        B.moe_rope(cfg, case["tokens"], s["q"], s["positions"], s["table"], s["q_out"],
                   inverse=case["inverse"])
        return s["q_out"]
    if op == "append":
        t = case["tokens"]
        B.moe_kv_append(cfg, t, s["q"], s["k"], s["v"], s["positions"], s["slots"], s["table"],
                        s["q_out"], s["cache"])
        B.moe_kv_read(cfg, t, s["slots"], s["cache"], s["k_out"], s["v_out"])
        return dict(q=s["q_out"], k=s["k_out"], v=s["v_out"])
    B.moe_kv_attention(cfg, case["seqs"], s["q"].shape[0], s["max_q"], s["q"], s["q_offsets"],
                       s["seq_lens"], s["page_table"], s["cache"], s["out"], s["lse"], p["ws"])
    return dict(out=s["out"], lse=s["lse"])


def _plain_table(s):
    c = s["case"]
    return _table(s["positions"], c["rotary"], c["base"], c["scaling"], c["factor"], c["original"])


def _rotate(x, positions, table, rotary, layout, inverse=False):
    """fp32 rows [T, heads, D] with their first `rotary` channels turned."""
    cs = table[positions.long()][:, None]
    cos, sin = cs[..., :rotary // 2], cs[..., rotary // 2:]
    if inverse:
        sin = -sin
    r = x[..., :rotary]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else r.chunk(2, dim=-1)
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if layout == "interleaved" else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rotary:]], -1)


def _plain_rope(s):
    c = s["case"]
    return _rotate(s["q"].float(), s["positions"], s["table"], c["rotary"], c["layout"],
                   c["inverse"]).to(s["q"].dtype)


def _plain_append(s):
    c = s["case"]
    dt = s["q"].dtype
    q = _rotate(s["q"].float(), s["positions"], s["table"], c["rotary"], c["layout"]).to(dt)
    k = _rotate(s["k"].float(), s["positions"], s["table"], c["rotary"], c["layout"]).to(dt)
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    kc, ks, vc, vs = _parts(s["cache"], c["page"], c["dim"])
    kc[page, :, at], ks[page, :, at] = _quantise(k.float())
    vc[page, :, at], vs[page, :, at] = _quantise(s["v"].float())
    return dict(q=q, k=_values(kc[page, :, at], ks[page, :, at]).to(dt),
                v=_values(vc[page, :, at], vs[page, :, at]).to(dt))


def _plain_attend(s):
    c = s["case"]
    kv, d, h = c["kv_heads"], c["dim"], c["heads"]
    g = h // kv
    kc, ks, vc, vs = (p[s["page_table"].long()].transpose(2, 3).flatten(1, 2)
                      for p in _parts(s["cache"], c["page"], d))       # [B, tokens, kv, n]
    n = kc.shape[1]
    k, v = _values(kc, ks).transpose(1, 2), _values(vc, vs).transpose(1, 2)   # [B, kv, tokens, D]
    off, b, m = s["q_offsets"].long(), c["seqs"], s["max_q"]
    tq = s["q"].shape[0]
    row = (off[:-1, None] + torch.arange(m, device=off.device)).clamp(max=tq - 1)
    q = s["q"].float()[row].unflatten(2, (kv, g)).permute(0, 2, 3, 1, 4)      # [B, kv, g, m, D]
    x = (q.reshape(b, kv, g * m, d) @ k.transpose(2, 3)).unflatten(2, (g, m)) * (d ** -0.5)
    lens = s["seq_lens"].long()
    last = (lens - (off[1:] - off[:-1]))[:, None] + torch.arange(m, device=off.device)
    key = torch.arange(n, device=off.device)
    seen = key <= last[..., None]
    if c["window"]:
        seen &= key > last[..., None] - c["window"]
    seen &= key < lens[:, None, None]
    x.masked_fill_(~seen[:, None, None], NEG)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ v).unflatten(2, (g, m)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    t = torch.arange(tq, device=off.device)
    seq = torch.searchsorted(off[1:], t, right=True)
    at = t - off[seq]
    out = o.permute(0, 3, 1, 2, 4)[seq, at].flatten(1, 2)                     # [T, heads, D]
    return dict(out=out.to(s["q"].dtype), lse=lse.permute(0, 3, 1, 2)[seq, at].flatten(1, 2))


# ------------------------------------------------------- the same in 64 bits
def _turn64(x, s, inverse=False):
    c = s["case"]
    r = c["rotary"]
    i = torch.arange(r // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if c["layout"] == "interleaved" else (i, i + r // 2)
    cs = s["table"].double()[s["positions"].long()][:, None]
    z = torch.complex(x[..., a].double(), x[..., b].double())
    w = torch.complex(cs[..., :r // 2], cs[..., r // 2:])
    z = z * (w.conj() if inverse else w)
    out = x.double().clone()
    out[..., a], out[..., b] = z.real, z.imag
    return out


def _nearest64(x, steps):
    """The nearest of `steps` (ascending, the even ones by index at ties) to each value."""
    mids = (steps[1:] + steps[:-1]) / 2
    low, high = torch.bucketize(x, mids), torch.bucketize(x, mids, right=True)
    return steps[torch.where(low % 2 == 0, low, high)]


def _stored64(x):
    """What 4-bit storage makes of 64-bit rows: nearest scale, nearest level, ties to even."""
    scales8 = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    level = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    g = x.unflatten(-1, (-1, GROUP))
    scale = _nearest64(g.abs().amax(-1, keepdim=True) / 6, scales8)
    y = torch.where(scale > 0, g.abs() / scale, torch.zeros_like(g))
    return (_nearest64(y, level) * scale * g.sign()).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        f, m = _frequencies(case["rotary"], case["base"], case["scaling"], case["factor"],
                            case["original"])
        a = torch.outer(s["positions"].double(), f.cuda())
        z = torch.polar(torch.full_like(a, m), a)
        return torch.cat([z.real, z.imag], 1)
    if op == "rope":
        return _turn64(s["q"], s, case["inverse"])
    if op == "append":
        dt = s["q"].dtype
        return dict(q=_turn64(s["q"], s), k=_stored64(_turn64(s["k"], s).to(dt).double()),
                    v=_stored64(s["v"].double()))
    kv, d, h, page = case["kv_heads"], case["dim"], case["heads"], case["page"]
    g = h // kv
    level = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    lens, qs = _lengths(case)
    out = torch.zeros(sum(qs), h, d, dtype=torch.float64, device="cuda")
    lse = torch.full((sum(qs), h), NEG, dtype=torch.float64, device="cuda")

    def rows(codes, scales):
        n = codes.reshape(-1, d // 2)
        n = torch.stack([n & 15, n >> 4], -1).flatten(-2).int()
        x = level[n & 7] * (1 - 2 * (n >> 3)).double()
        return x * scales.reshape(-1, d // 16).view(torch.float8_e4m3fn).double().repeat_interleave(GROUP, 1)

    at = 0
    for b, (n, q) in enumerate(zip(lens, qs)):
        ids = s["page_table"][b, :-(-n // page)].long()
        for j in range(kv):
            kc, ks, vc, vs = _parts(s["cache"][ids, j:j + 1], page, d)
            k, v = rows(kc[:, 0], ks[:, 0])[:n], rows(vc[:, 0], vs[:, 0])[:n]
            for i in range(0, q, 512):
                m = min(512, q - i)
                x = s["q"][at + i:at + i + m, j * g:(j + 1) * g].double()
                x = torch.einsum("mgd,nd->mgn", x, k) / math.sqrt(d)
                pos = n - q + i + torch.arange(m, device="cuda")[:, None]
                key = torch.arange(n, device="cuda")
                hide = key > pos
                if case["window"]:
                    hide |= key <= pos - case["window"]
                x = x.masked_fill(hide[:, None], NEG)
                w = torch.logsumexp(x, -1)
                lse[at + i:at + i + m, j * g:(j + 1) * g] = w
                x = (x - w[..., None]).exp()
                out[at + i:at + i + m, j * g:(j + 1) * g] = torch.einsum("mgn,nd->mgd", x, v)
        at += q
    return dict(out=out, lse=lse)
