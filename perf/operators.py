"""What is measured of windowed attention and of the 4-bit key/value cache.

Four operators, each in its plain form (elementary torch operations in float32) and
through this library's public calls (``own``):

- "window_fwd"  attention in which a query sees the last ``window`` keys and the first
                ``sinks`` ones: (O, LSE) of a prompt in layout order;
- "window_bwd"  its gradients (dQ, dK, dV) from dO, with the forward's O and LSE;
- "cache"       keys and values of new tokens quantised into a paged 4-bit cache, then
                read back from it as the values it stands for;
- "attend"      attention of a few new tokens per sequence over that cache: (O, LSE).

The cache's bytes are those of include/ra.h: blocks of 16 tokens, each with the key
codes, the key parameters, the value codes and the value parameters.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a short prompt on three shards with ragged tiles: latency
        dict(name="window_fwd_900_striped", op="window_fwd", batch=1, seq=900, heads_q=4, heads_kv=2, d=128, shards=3,
             layout="striped", window=100, sinks=4, dtype="bf16"),
        # the library's float32 path at the toy sizes of its tests
        dict(name="window_fwd_f32_96", op="window_fwd", batch=2, seq=96, heads_q=4, heads_kv=4, d=32, shards=4,
             layout="zigzag", window=17, sinks=2, dtype="f32"),
        # the 32k causal workload (32 query heads, 8 key/value heads, 8 shards) under a 4096-token window
        dict(name="window_fwd_32k_zigzag", op="window_fwd", batch=1, seq=32768, heads_q=32, heads_kv=8, d=128, shards=8,
             layout="zigzag", window=4096, sinks=4, dtype="bf16"),
        # the 131k workload under a short window, where a query tile meets few key tiles
        dict(name="window_fwd_131k_contiguous", op="window_fwd", batch=1, seq=131072, heads_q=32, heads_kv=8, d=128,
             shards=32, layout="contiguous", window=1024, sinks=64, dtype="bf16"),
        # training steps' gradients: short and ragged; float32; the 32k workload
        dict(name="window_bwd_900_contiguous", op="window_bwd", batch=1, seq=900, heads_q=4, heads_kv=2, d=128, shards=3,
             layout="contiguous", window=100, sinks=4, dtype="bf16"),
        dict(name="window_bwd_f32_96", op="window_bwd", batch=2, seq=96, heads_q=4, heads_kv=2, d=32, shards=4,
             layout="zigzag", window=17, sinks=2, dtype="f32"),
        dict(name="window_bwd_32k_zigzag", op="window_bwd", batch=1, seq=32768, heads_q=32, heads_kv=8, d=128, shards=8,
             layout="zigzag", window=4096, sinks=4, dtype="bf16"),
        # one decoding step's tokens of 64 sequences; a whole 32k prompt
        dict(name="cache_token_x64", op="cache", batch=64, rows=1, heads_kv=8, d=128, page_rows=64, start=32767,
             ragged=False, dtype="bf16"),
        dict(name="cache_prompt_32k", op="cache", batch=1, rows=32768, heads_kv=8, d=128, page_rows=64, start=0,
             ragged=False, dtype="bf16"),
        # a few drafted tokens on short float32 sequences; a decoding step of 32 sequences of up to 32k tokens under a
        # window; one long sequence without
        dict(name="attend_300_f32", op="attend", batch=2, rows=3, length=300, heads_q=8, heads_kv=2, d=64, page_rows=16,
             window=0, sinks=0, dtype="f32"),
        dict(name="attend_32k_x32_window", op="attend", batch=32, rows=1, length=32768, heads_q=32, heads_kv=8, d=128,
             page_rows=64, window=8192, sinks=4, dtype="bf16"),
        dict(name="attend_1m", op="attend", batch=1, rows=1, length=1048576, heads_q=32, heads_kv=8, d=128, page_rows=64,
             window=0, sinks=0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window_fwd", "window_bwd", "cache", "attend"])
    heads_kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    if op.startswith("window"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        shards = rng.choice([1, 2, 3, 4, 8])
        layout = rng.choice(["contiguous", "striped", "zigzag"])
        if dtype == "f32":
            seq, d = _log_int(rng, 8, 400), rng.choice([8, 13, 32, 64, 128])
            heads_kv, group = min(heads_kv, 4), min(group, 2)
        else:
            seq, d = _log_int(rng, 8, 32768), 128
        unit = shards * (2 if layout == "zigzag" else 1)
        seq = max(1, seq // unit) * unit
        return dict(op=op, batch=rng.choice([1, 1, 2]) if seq <= 8192 else 1, seq=seq, heads_q=heads_kv * group,
                    heads_kv=heads_kv, d=d, shards=shards, layout=layout,
                    window=min(_log_int(rng, 1, 4096), seq), sinks=rng.choice([0, 1, 4, 4, 64, 200]), dtype=dtype)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d, page_rows = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 112, 256])
    if op == "cache":
        batch, rows = rng.choice([1, 2, 5, 16, 64]), _log_int(rng, 1, 32768)
        rows = max(1, min(rows, 32768 * 4 // (batch * heads_kv) // (2 if dtype == "f32" else 1)))
        return dict(op=op, batch=batch, rows=rows, heads_kv=heads_kv, d=d, page_rows=page_rows,
                    start=rng.randrange(0, 2000), ragged=rng.random() < 0.5, dtype=dtype)
    batch, length = rng.choice([1, 2, 5, 16, 64]), _log_int(rng, 1, 300000)
    length = max(1, min(length, 8388608 // (batch * heads_kv)))
    windowed = rng.random() < 0.5
    return dict(op=op, batch=batch, rows=rng.choice([1, 1, 1, 2, 5, 16]), length=length, heads_q=heads_kv * group,
                heads_kv=heads_kv, d=d, page_rows=page_rows, window=_log_int(rng, 1, 20000) if windowed else 0,
                sinks=rng.choice([0, 4, 100]) if windowed else 0, dtype=dtype)


# ------------------------------------------------------------------ inputs --
def _rng(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _kv_rows(g, *shape):
    """Rows as projections leave them: per channel an offset and a size of its own, a few channels large."""
    d = shape[-1]
    size = torch.exp(0.5 * _randn(g, d))
    return _randn(g, *shape).mul_(size).add_(0.5 * _randn(g, d))


def positions(layout, seq, shards):
    """Natural position of every layout-ordered row."""
    j = torch.arange(seq, device=DEV)
    n = seq // shards
    p, i = j // n, j % n
    if layout == "contiguous":
        return j
    if layout == "striped":
        return i * shards + p
    c = n // 2
    return torch.where(i < c, p * c + i, (2 * shards - 1 - p) * c + i - c)


def _lengths(case, g):
    """Sequence lengths: the first is the longest, the others between an eighth of it and all of it."""
    b, top = case["batch"], case["length"]
    low = max(1, top // 8)
    n = low + (torch.rand(b, generator=g, device=DEV) * (top - low + 1)).long()
    n = n.clamp(max=top)
    n[0] = top
    return n


def _pages(batch, rows, page_rows, g):
    """A page table whose pages lie scattered over a pool a little larger than needed."""
    width = -(-rows // page_rows)
    pool = batch * width + 3
    order = torch.randperm(pool, generator=g, device=DEV)[:batch * width]
    return order.reshape(batch, width).to(torch.int32).contiguous(), pool


def prepare(case, seed):
    g = _rng(seed)
    dt = TYPES[case["dtype"]]
    st = dict(case=case)
    if case["op"].startswith("window"):
        b, s, hq, hk, d = (case[x] for x in ("batch", "seq", "heads_q", "heads_kv", "d"))
        st["q"] = _randn(g, b, hq, s, d).to(dt)
        st["k"], st["v"] = (_randn(g, b, hk, s, d).to(dt) for _ in range(2))
        st["pos"] = positions(case["layout"], s, case["shards"])
        st["row_of"] = torch.argsort(st["pos"])
        if case["op"] == "window_bwd":
            o, lse = _plain_window_fwd(st)
            st["o"], st["lse"] = o, lse
            st["dout"] = _randn(g, b, hq, s, d).to(dt)
        if own:
            import context_ring_attention_gb300 as ra
            st["plan"] = ra.ra_plan_window(b, s, hq, hk, d, case["shards"], case["window"], case["sinks"],
                                           layout=case["layout"], dtype=case["dtype"])
        return st
    b, t, hk, d, pr = (case[x] for x in ("batch", "rows", "heads_kv", "d", "page_rows"))
    if case["op"] == "cache":
        st["k"], st["v"] = (_kv_rows(g, b, hk, t, d).to(dt) for _ in range(2))
        st["table"], pool = _pages(b, case["start"] + t, pr, g)
        st["first"] = torch.full((b,), case["start"], dtype=torch.int32, device=DEV)
        if case["ragged"]:  # the padded rows of a batch of prompts stay out of the cache
            st["count"] = (torch.rand(b, generator=g, device=DEV) * (t + 1)).long().clamp(max=t).to(torch.int32)
        else:
            st["count"] = torch.full((b,), t, dtype=torch.int32, device=DEV)
        st["cache"] = torch.zeros(pool * hk * pr * d * 5 // 4, dtype=torch.uint8, device=DEV)
        heads_q, window, sinks = hk, 0, 0
    else:
        lengths = _lengths(case, g)
        st["lengths"] = lengths.tolist()  # a serving loop knows them on the host as well
        st["length"] = lengths.to(torch.int32)
        st["table"], pool = _pages(b, case["length"], pr, g)
        st["cache"] = _random_cache(pool, hk, pr, d, g)
        st["q"] = _randn(g, b, case["heads_q"], t, d).to(dt)
        heads_q, window, sinks = case["heads_q"], case["window"], case["sinks"]
    st["pool"] = pool
    if own:
        import context_ring_attention_gb300 as ra
        st["plan"] = ra.ra_kv4_plan(pool, pr, heads_q, hk, d, dtype=case["dtype"], window=window, sinks=sinks)
    return st


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import context_ring_attention_gb300 as ra
        plan = state["plan"]
        if op == "window_fwd":
            return ra.ra_fwd(plan, state["q"], state["k"], state["v"])
        if op == "window_bwd":
            return ra.ra_bwd(plan, state["q"], state["k"], state["v"], state["o"], state["lse"], state["dout"])
        if op == "cache":
            ra.ra_kv4_write(plan, state["cache"], state["k"], state["v"], state["table"], state["first"], state["count"])
            return ra.ra_kv4_read(plan, state["cache"], state["table"], state["first"], case["rows"], state["count"])
        return ra.ra_kv4_attend(plan, state["cache"], state["q"], state["table"], state["length"])
    return {"window_fwd": _plain_window_fwd, "window_bwd": _plain_window_bwd, "cache": _plain_cache,
            "attend": _plain_attend}[op](state)


def _window_pairs(rows, window, sinks):
    """Visible (query, key) pairs of queries at positions 0..rows-1."""
    w = min(window, rows) if window else rows
    pairs = w * (w + 1) // 2 + (rows - w) * w
    # sinks outside the window: query i has min(sinks, i - w + 1) of them
    far = rows - w
    few = min(sinks, far)
    return pairs + few * (few + 1) // 2 + (far - few) * sinks if window else pairs


def work(case):
    d, e = case["d"], 2 if case["dtype"] == "bf16" else 4
    if case["op"].startswith("window"):
        rq = case["batch"] * case["heads_q"] * case["seq"]
        rk = case["batch"] * case["heads_kv"] * case["seq"]
        pairs = case["batch"] * case["heads_q"] * _window_pairs(case["seq"], case["window"], case["sinks"])
        if case["op"] == "window_fwd":
            return {"bytes": (2 * rq + 2 * rk) * d * e + 4 * rq, "flops": 4 * d * pairs}
        return {"bytes": (4 * rq + 4 * rk) * d * e + 4 * rq, "flops": 10 * d * pairs}
    if case["op"] == "cache":
        rows = case["batch"] * case["heads_kv"] * case["rows"] * (0.5 if case["ragged"] else 1)
        return {"bytes": int(rows * (4 * d * e + d * 5 // 4)), "flops": int(rows * d * 8)}
    # lengths lie between an eighth of the longest and the longest
    top, t = case["length"], case["rows"]
    mean = top if case["batch"] == 1 else (top + (case["batch"] - 1) * 0.5625 * top) / case["batch"]
    seen = min(mean, case["window"] + t + case["sinks"]) if case["window"] else mean
    keys = case["batch"] * seen
    rq = case["batch"] * case["heads_q"] * t
    return {"bytes": int(keys * case["heads_kv"] * d * 5 // 4 + rq * (2 * d * e + 4)),
            "flops": int(4 * d * keys * case["heads_q"] * t)}


# ------------------------------------------------- plain form: the window --
def _band(case, i0, i1):
    """Keys that some query of positions [i0, i1) sees: [0, a) and [lo, i1), and which of them each sees."""
    w, sinks = case["window"], case["sinks"]
    lo = max(0, i0 - w + 1)
    a = min(sinks, lo)
    j = torch.cat([torch.arange(a, device=DEV), torch.arange(lo, i1, device=DEV)])
    i = torch.arange(i0, i1, device=DEV)[:, None]
    return a, lo, (j <= i) & ((j > i - w) | (j < sinks))


def _cut(x, a, lo, i1):
    return torch.cat([x[:, :, :a], x[:, :, lo:i1]], 2) if a else x[:, :, lo:i1]


def _chunk(case):
    n = case["window"] + 1024
    per_row = case["batch"] * case["heads_q"] * n
    return max(64, min(1024, (1 << 29) // per_row))


def _plain_window_fwd(st):
    case = st["case"]
    b, s, hq, hk, d = (case[x] for x in ("batch", "seq", "heads_q", "heads_kv", "d"))
    q, k, v = (st[x].index_select(2, st["row_of"]).float() for x in ("q", "k", "v"))
    g = hq // hk
    o = torch.empty((b, hq, s, d), device=DEV)
    lse = torch.empty((b, hq, s), device=DEV)
    c = _chunk(case)
    for i0 in range(0, s, c):
        i1 = min(s, i0 + c)
        a, lo, seen = _band(case, i0, i1)
        kk, vv = _cut(k, a, lo, i1), _cut(v, a, lo, i1)
        qq = q[:, :, i0:i1].reshape(b, hk, g * (i1 - i0), d)
        x = (qq @ kk.transpose(-1, -2)).mul_(1 / math.sqrt(d)).view(b, hk, g, i1 - i0, -1)
        x.masked_fill_(~seen, -math.inf)
        m = x.amax(-1, keepdim=True)
        x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        y = (x.view(b, hk, g * (i1 - i0), -1) @ vv).view(b, hk, g, i1 - i0, d) / l
        o[:, :, i0:i1] = y.reshape(b, hq, i1 - i0, d)
        lse[:, :, i0:i1] = (m + l.log()).reshape(b, hq, i1 - i0)
    return o.index_select(2, st["pos"]).to(st["q"].dtype), lse.index_select(2, st["pos"])


def _plain_window_bwd(st):
    case = st["case"]
    b, s, hq, hk, d = (case[x] for x in ("batch", "seq", "heads_q", "heads_kv", "d"))
    q, k, v, o, do, lse = (st[x].index_select(2, st["row_of"]).float() for x in ("q", "k", "v", "o", "dout", "lse"))
    g, scale = hq // hk, 1 / math.sqrt(d)
    delta = (o * do).sum(-1)
    dq, dk, dv = torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    c = _chunk(case)
    for i0 in range(0, s, c):
        i1 = min(s, i0 + c)
        a, lo, seen = _band(case, i0, i1)
        kk, vv = _cut(k, a, lo, i1), _cut(v, a, lo, i1)
        flat = lambda x: x[:, :, i0:i1].reshape(b, hk, g * (i1 - i0), -1)
        col = lambda x: flat(x.unsqueeze(-1))
        qq, dd = flat(q), flat(do)
        p = (qq @ kk.transpose(-1, -2)).mul_(scale).sub_(col(lse)).exp_()
        p.view(b, hk, g, i1 - i0, -1).masked_fill_(~seen, 0.0)
        ds = (dd @ vv.transpose(-1, -2)).sub_(col(delta)).mul_(p)
        dq[:, :, i0:i1] = (ds @ kk).mul_(scale).reshape(b, hq, i1 - i0, d)
        for grad, part in ((dk, (ds.transpose(-1, -2) @ qq).mul_(scale)), (dv, p.transpose(-1, -2) @ dd)):
            if a:
                grad[:, :, :a] += part[:, :, :a]
            grad[:, :, lo:i1] += part[:, :, a:]
    return tuple(x.index_select(2, st["pos"]).to(st["q"].dtype) for x in (dq, dk, dv))


# -------------------------------------------------- plain form: the cache --
def _quantise(x):
    """Codes 0..15 and (scale, low) of every 32 channels, as float32 values that bf16 holds."""
    g = x.float().unflatten(-1, (-1, 32))
    low = g.amin(-1).bfloat16().float()
    scale = ((g.amax(-1) - low) / 15).bfloat16().float()
    bad = ~(torch.isfinite(g).all(-1) & torch.isfinite(scale))
    scale = torch.where(bad | (scale < 2.0 ** -100), torch.zeros_like(scale), scale)
    low = torch.where(bad, torch.full_like(low, math.nan), low)
    # in 64 bits: a value next to the border of two codes has to fall on its own side
    t = (g.double() - low.double()[..., None]) / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[..., None]
    codes = (t + 0.5).floor().clamp(0, 15)
    codes = torch.where((scale > 0)[..., None], codes, torch.zeros_like(codes))
    return codes.to(torch.uint8), scale, low


def _nibbles_to_bytes(n):
    n = n.unflatten(-1, (-1, 2))
    return n[..., 0] | (n[..., 1] << 4)


def _bytes_to_nibbles(x):
    return torch.stack([x & 15, x >> 4], -1).flatten(-2)


def _parts(cache, pool, heads, page_rows, d):
    """Views [page, head, block, row, byte] of the key codes, key parameters, value codes, value parameters."""
    blocks = cache.view(pool, heads, page_rows // 16, 20 * d)
    cut = (0, 8 * d, 10 * d, 18 * d, 20 * d)
    return [blocks[..., cut[n]:cut[n + 1]].unflatten(-1, (16, -1)) for n in range(4)]


def _row_bytes(x, key):
    """One row's code bytes and parameter bytes."""
    codes, scale, low = _quantise(x)
    unit = 8 if key else 4
    n = codes.unflatten(-1, (-1, unit)).transpose(-3, -2).flatten(-3)
    par = torch.stack([scale, low], -1).bfloat16().flatten(-2).contiguous().view(torch.uint8)
    return _nibbles_to_bytes(n), par


def _row_values(code_bytes, par_bytes, key):
    d = code_bytes.shape[-1] * 2
    unit = 8 if key else 4
    n = _bytes_to_nibbles(code_bytes).unflatten(-1, (32 // unit, d // 32, unit)).transpose(-3, -2).flatten(-2)
    par = par_bytes.contiguous().view(torch.bfloat16).float().unflatten(-1, (-1, 2))
    return (n.float() * par[..., 0:1] + par[..., 1:2]).flatten(-2)


def _random_cache(pool, heads, page_rows, d, g):
    """A cache full of quantised rows, page by page."""
    cache = torch.empty(pool * heads * page_rows * d * 5 // 4, dtype=torch.uint8, device=DEV)
    parts = _parts(cache, pool, heads, page_rows, d)
    blocks = page_rows // 16
    step = max(1, (1 << 25) // (heads * page_rows * d))
    for p0 in range(0, pool, step):
        p1 = min(pool, p0 + step)
        for n, key in ((0, True), (2, False)):
            codes, par = _row_bytes(_kv_rows(g, p1 - p0, heads, blocks, 16, d), key)
            parts[n][p0:p1] = codes
            parts[n + 1][p0:p1] = par
    return cache


def _places(table, at, page_rows):
    """page, block and row of the block for positions `at` [batch, rows] of every sequence."""
    page = table.long().gather(1, at // page_rows)
    return page, at % page_rows // 16, at % 16


def _plain_cache(st):
    case = st["case"]
    b, t, hk, d, pr = (case[x] for x in ("batch", "rows", "heads_kv", "d", "page_rows"))
    parts = _parts(st["cache"], st["pool"], hk, pr, d)
    row = torch.arange(t, device=DEV)
    at = st["first"].long()[:, None] + row
    page, block, line = (x[:, None, :] for x in _places(st["table"], at, pr))
    head = torch.arange(hk, device=DEV)[None, :, None]
    live = (row < st["count"].long()[:, None])[:, None, :, None]
    out = []
    for n, (x, key) in enumerate(((st["k"], True), (st["v"], False))):
        codes, par = _row_bytes(x, key)
        place = (page, head, block, line)
        parts[2 * n][place] = torch.where(live, codes, parts[2 * n][place])
        parts[2 * n + 1][place] = torch.where(live, par, parts[2 * n + 1][place])
        y = _row_values(parts[2 * n][place], parts[2 * n + 1][place], key)
        out.append(torch.where(live, y, torch.zeros_like(y)).to(x.dtype))
    return tuple(out)


def _visible_rows(case, length):
    """Positions that some of the new tokens of a sequence of this length sees."""
    t, w = case["rows"], case["window"]
    lo = max(0, length - t - w + 1) if w else 0
    a = min(case["sinks"], lo)
    return torch.cat([torch.arange(a, device=DEV), torch.arange(lo, length, device=DEV)])


def _plain_attend(st):
    case = st["case"]
    b, t, hq, hk, d, pr = (case[x] for x in ("batch", "rows", "heads_q", "heads_kv", "d", "page_rows"))
    parts = _parts(st["cache"], st["pool"], hk, pr, d)
    g = hq // hk
    o = torch.empty((b, hq, t, d), device=DEV)
    lse = torch.empty((b, hq, t), device=DEV)
    for n, length in enumerate(st["lengths"]):
        j = _visible_rows(case, length)
        i = torch.arange(length - t, length, device=DEV)[:, None]
        seen = j <= i
        if case["window"]:
            seen = seen & ((j > i - case["window"]) | (j < case["sinks"]))
        page, block, line = (x[0][None, :] for x in _places(st["table"][n:n + 1], j[None], pr))
        head = torch.arange(hk, device=DEV)[:, None]
        k = _row_values(parts[0][page, head, block, line], parts[1][page, head, block, line], True)
        v = _row_values(parts[2][page, head, block, line], parts[3][page, head, block, line], False)
        x = (st["q"][n].float().view(hk, g * t, d) @ k.transpose(-1, -2)).div_(math.sqrt(d)).view(hk, g, t, -1)
        x.masked_fill_(~seen, -math.inf)
        m = x.amax(-1, keepdim=True)
        # a token before the sequence's first position sees nothing: O = 0, LSE = -inf
        x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
        l = x.sum(-1, keepdim=True)
        y = (x.view(hk, g * t, -1) @ v).view(hk, g, t, d) / torch.where(l > 0, l, torch.ones_like(l))
        o[n] = y.reshape(hq, t, d)
        lse[n] = (m + l.log()).reshape(hq, t)
    return o.to(st["q"].dtype), lse


# ---------------------------------------------------------------- in 64 bits --
def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    return {"window_fwd": _exact_window, "window_bwd": _exact_window_bwd, "cache": _exact_cache,
            "attend": _exact_attend}[case["op"]](st)


def _exact_blocks(st, rows):
    """For every (batch, head): blocks of layout rows, the layout rows that any of them sees, and which each sees."""
    case, pos = st["case"], st["pos"]
    order = torch.argsort(pos)
    for r0 in range(0, case["seq"], rows):
        mine = order[r0:r0 + rows]
        gap = pos[mine][:, None] - pos[None, :]
        vis = (gap >= 0) & ((gap < case["window"]) | (pos[None, :] < case["sinks"]))
        cols = vis.any(0).nonzero()[:, 0]
        yield mine, cols, vis[:, cols]


def _exact_window(st):
    case = st["case"]
    b, s, hq, hk, d = (case[x] for x in ("batch", "seq", "heads_q", "heads_kv", "d"))
    o = torch.zeros((b, hq, s, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((b, hq, s), dtype=torch.float64, device=DEV)
    for mine, cols, vis in _exact_blocks(st, 512):
        for h in range(hq):
            q = st["q"][:, h, mine].double()
            k, v = (st[x][:, h // (hq // hk), cols].double() for x in ("k", "v"))
            x = torch.einsum("bid,bjd->bij", q, k) / math.sqrt(d)
            x = torch.where(vis, x, torch.full_like(x, -math.inf))
            top = torch.logsumexp(x, -1)
            o[:, h, mine] = torch.einsum("bij,bjd->bid", torch.exp(x - top[..., None]), v)
            lse[:, h, mine] = top
    return o, lse


def _exact_window_bwd(st):
    case = st["case"]
    hq, hk, d = case["heads_q"], case["heads_kv"], case["d"]
    dq, dk, dv = (torch.zeros_like(st[x], dtype=torch.float64) for x in ("q", "k", "v"))
    for mine, cols, vis in _exact_blocks(st, 512):
        for h in range(hq):
            n = h // (hq // hk)
            q, do, o = (st[x][:, h, mine].double() for x in ("q", "dout", "o"))
            k, v = st["k"][:, n, cols].double(), st["v"][:, n, cols].double()
            x = torch.einsum("bid,bjd->bij", q, k) / math.sqrt(d) - st["lse"][:, h, mine].double()[..., None]
            p = torch.where(vis, torch.exp(x), torch.zeros_like(x))
            slope = torch.einsum("bid,bjd->bij", do, v) - (do * o).sum(-1, keepdim=True)
            ds = p * slope / math.sqrt(d)
            dq[:, h, mine] = torch.einsum("bij,bjd->bid", ds, k)
            dk[:, n].index_add_(1, cols, torch.einsum("bij,bid->bjd", ds, q))
            dv[:, n].index_add_(1, cols, torch.einsum("bij,bid->bjd", p, do))
    return dq, dk, dv


def _exact_cache(st):
    """The values that the quantised rows stand for.  The two parameters are bf16 numbers by definition: the minimum
    rounded, and a fifteenth of the range (a float32 difference and quotient) rounded."""
    live = torch.arange(st["case"]["rows"], device=DEV) < st["count"][:, None]
    out = []
    for x in (st["k"], st["v"]):
        y = torch.zeros_like(x, dtype=torch.float64)
        for c in range(0, x.shape[-1], 32):
            part = x[..., c:c + 32].double()
            low = part.min(-1, keepdim=True).values.float().bfloat16().double()
            span = (part.max(-1, keepdim=True).values - low).float().double()
            step = (span / 15).float().bfloat16().double()
            step = torch.where(step < 2.0 ** -100, torch.zeros_like(step), step)
            code = torch.zeros_like(part)
            for n in range(15):  # one code further at every border that the value reaches
                code += (part - low >= (n + 0.5) * step) & (step > 0)
            y[..., c:c + 32] = low + step * code
        out.append(torch.where(live[:, None, :, None], y, torch.zeros_like(y)))
    return tuple(out)


def _exact_attend(st):
    case = st["case"]
    b, t, hq, hk, d, pr = (case[x] for x in ("batch", "rows", "heads_q", "heads_kv", "d", "page_rows"))
    raw = st["cache"].view(-1, 20 * d)  # one block of 16 tokens a row
    ch = torch.arange(d, device=DEV)
    # the byte and the shift of every channel's code, from the definition of the format
    k_nib = (ch % 32 // 8 * (d // 32) + ch // 32) * 8 + ch % 8
    v_nib = (ch % 32 // 4 * (d // 32) + ch // 32) * 4 + ch % 4
    o = torch.zeros((b, hq, t, d), dtype=torch.float64, device=DEV)
    lse = torch.full((b, hq, t), -math.inf, dtype=torch.float64, device=DEV)
    for n in range(b):
        length = st["lengths"][n]
        at = torch.arange(length - t, length, device=DEV)[:, None]
        j = torch.arange(length, device=DEV)[None]
        vis = j <= at
        if case["window"]:
            vis = vis & ((at - j < case["window"]) | (j < case["sinks"]))
        cols = vis.any(0).nonzero()[:, 0]
        vis = vis[:, cols]
        page = st["table"][n, cols // pr].long()
        for h in range(hk):
            block = (page * hk + h) * (pr // 16) + cols % pr // 16
            line = (cols % 16)[:, None]
            row = block[:, None]

            def values(base, nib):
                code = (raw[row, base + line * (d // 2) + nib // 2] >> (nib % 2 * 4)) & 15
                par = raw[row, base + 8 * d + line * (d // 8) + torch.arange(d // 8, device=DEV)]
                par = par.contiguous().view(torch.bfloat16).double().repeat_interleave(32, -1)
                step = par.view(len(cols), d // 32, 2, 32)[:, :, 0].reshape(len(cols), d)
                low = par.view(len(cols), d // 32, 2, 32)[:, :, 1].reshape(len(cols), d)
                return code.double() * step + low

            k, v = values(0, k_nib), values(10 * d, v_nib)
            for i in range(h * (hq // hk), (h + 1) * (hq // hk)):
                x = st["q"][n, i].double() @ k.T / math.sqrt(d)
                x = torch.where(vis, x, torch.full_like(x, -math.inf))
                top = torch.logsumexp(x, -1, keepdim=True)
                p = torch.where(vis, torch.exp(x - top), torch.zeros_like(x))
                o[n, i] = p @ v
                lse[n, i] = top[:, 0]
    return o, lse
