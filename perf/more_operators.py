"""What is measured of rotary positions and of the paged key/value cache: appending, attention of chunks, eviction.

Five operators, each in its plain form (elementary torch operations in float32, angles in
float64) and through this library's public calls (``own``):

- "rope"    queries and keys [B, H, S, d] in layout order rotated by their positions (or, "bwd",
            the gradients with respect to them rotated back);
- "append"  new tokens of a packed batch: queries and keys rotated, keys and values into the
            pages of their sequences;
- "attend"  attention of a chunk of new tokens per sequence over the paged cache: (O, LSE);
- "weigh"   the attention weight that every cached key received from such a chunk, added to
            what it received before;
- "evict"   the heaviest keys of every sequence and head kept, moved together into other pages.

A packed batch lays the sequences' tokens one after the other: q [tokens, heads, d], sequence b
has rows offset[b] to offset[b + 1] - 1, and length[b] counts its tokens in the cache, those
among them.  The cache is [pages, 2, heads_kv, page_rows, d]: a page's keys, then its values.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the 32k prompt (32 query heads, 8 key/value heads, 8 shards): queries and keys as the projections leave
        # them, rotated into the ring's tensors, with positions scaled for a context longer than the trained one
        dict(name="rope_32k_zigzag", op="rope", direction="fwd", batch=1, seq=32768, heads_q=32, heads_kv=8, d=128, rot=128,
             interleaved=False, scaling="bands", layout="zigzag", shards=8, strided=True, dtype="bf16"),
        # a short training step's gradients on three shards, part of the head, float32: latency
        dict(name="rope_bwd_900_f32", op="rope", direction="bwd", batch=2, seq=900, heads_q=4, heads_kv=2, d=64, rot=48,
             interleaved=True, scaling="ramp", layout="striped", shards=3, strided=False, dtype="f32"),
        # one decoding step's tokens of 64 sequences; a prompt's first chunk
        dict(name="append_token_x64", op="append", batch=64, rows=1, shape="even", length=600, heads_q=32, heads_kv=8, d=128,
             rot=128, interleaved=False, scaling="bands", page_rows=64, dtype="bf16"),
        dict(name="append_chunk_8k", op="append", batch=1, rows=8192, shape="even", length=9000, heads_q=32, heads_kv=8, d=128,
             rot=128, interleaved=False, scaling="none", page_rows=64, dtype="bf16"),
        # a few drafted tokens on short float32 sequences: latency
        dict(name="attend_300_f32", op="attend", batch=3, rows=5, shape="ragged", length=300, heads_q=8, heads_kv=2, d=64,
             page_rows=16, window=0, sinks=0, dtype="f32"),
        # a prompt's last chunk over the 32k before it
        dict(name="attend_chunk_2k_over_32k", op="attend", batch=1, rows=2048, shape="even", length=32768, heads_q=32,
             heads_kv=8, d=128, page_rows=64, window=0, sinks=0, dtype="bf16"),
        # a serving step: one prompt's chunk among the single tokens of 31 other sequences, under a window
        dict(name="attend_mixed_x32", op="attend", batch=32, rows=512, shape="one", length=16384, heads_q=32, heads_kv=8,
             d=128, page_rows=128, window=8192, sinks=4, dtype="bf16"),
        # a decoding step of 16 sequences of 4k to 32k tokens
        dict(name="attend_token_x16", op="attend", batch=16, rows=1, shape="even", length=32768, heads_q=32, heads_kv=8,
             d=128, page_rows=64, window=0, sinks=0, dtype="bf16"),
        # the weights of a decoding step, and of a prompt's chunk
        dict(name="weigh_token_x16", op="weigh", batch=16, rows=1, shape="even", length=8192, heads_q=32, heads_kv=8, d=128,
             page_rows=64, window=0, sinks=0, dtype="bf16"),
        dict(name="weigh_chunk_1k_over_32k", op="weigh", batch=1, rows=1000, shape="even", length=32768, heads_q=32,
             heads_kv=8, d=128, page_rows=64, window=0, sinks=0, dtype="bf16"),
        # 16 sequences back to a budget of 4096 after 256 tokens; a long prompt cut to a quarter
        dict(name="evict_x16_4k", op="evict", batch=16, length=4352, keep=4096, first=4, recent=512, heads_kv=8, d=128,
             page_rows=64, dtype="bf16"),
        dict(name="evict_33k_to_8k", op="evict", batch=1, length=33001, keep=8192, first=4, recent=1024, heads_kv=8, d=128,
             page_rows=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "weigh", "evict"])
    heads_kv = rng.choice([1, 2, 4, 8])
    heads_q = heads_kv * rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    turn = dict(interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "bands", "ramp"]))
    if op == "rope":
        d = rng.choice([24, 64, 80, 128, 128])
        shards, layout = rng.choice([1, 2, 3, 4, 8]), rng.choice(["contiguous", "striped", "zigzag"])
        unit = shards * (2 if layout == "zigzag" else 1)
        batch = rng.choice([1, 1, 2, 5])
        seq = min(_log_int(rng, 1, 32768), 32768 * 20 // (batch * (heads_q + heads_kv)))
        return dict(op=op, direction=rng.choice(["fwd", "bwd"]), batch=batch, seq=max(1, seq // unit) * unit, heads_q=heads_q,
                    heads_kv=heads_kv, d=d, rot=rng.choice([d, d, d // 2, d // 4 * 2 - 2]), **turn, layout=layout,
                    shards=shards, strided=rng.random() < 0.5, dtype=dtype)
    d, page_rows, batch = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 112, 256]), rng.choice([1, 2, 5, 16, 64])
    if op == "append":
        rows = min(_log_int(rng, 1, 8192), 8192 * 20 // (batch * (heads_q + 2 * heads_kv)))
        return dict(op=op, batch=batch, rows=max(1, rows), shape=rng.choice(["even", "ragged"]),
                    length=max(1, rows) + rng.randrange(0, 500), heads_q=heads_q, heads_kv=heads_kv, d=d,
                    rot=rng.choice([d, d // 2]), **turn, page_rows=page_rows, dtype=dtype)
    if op == "evict":
        length = min(_log_int(rng, 16, 60000), (1 << (17 if dtype == "f32" else 18)) // (batch * heads_kv))
        keep = max(1, int(length * rng.uniform(0.1, 1.1)))
        first = min(rng.choice([0, 1, 4, 64]), keep)
        return dict(op=op, batch=batch, length=length, keep=keep, first=first,
                    recent=min(keep - first, int(keep * rng.choice([0.0, 0.1, 0.5, 1.0]))), heads_kv=heads_kv, d=d,
                    page_rows=page_rows, dtype=dtype)
    rows = _log_int(rng, 1, 2048)
    pairs = (1 << 27 if dtype == "f32" else 1 << 30) // heads_q
    length = max(1, min(_log_int(rng, 1, 65536), (1 << (20 if dtype == "f32" else 21)) // (batch * heads_kv)))
    rows = max(1, min(rows, length, pairs // length))
    windowed = rng.random() < 0.4
    return dict(op=op, batch=batch, rows=rows, shape=rng.choice(["even", "ragged", "one"]) if rows * length * batch <= pairs else "one",
                length=length, heads_q=heads_q, heads_kv=heads_kv, d=d, page_rows=page_rows,
                window=_log_int(rng, 1, 20000) if windowed else 0, sinks=rng.choice([0, 4, 100]) if windowed else 0,
                dtype=dtype)


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


def _scaling(case):
    """Positions are stretched by 8 for a context beyond the 8192 tokens that the frequencies were trained on."""
    name = case["scaling"]
    if name in ("none",):
        return dict(base=10000.0, scaling=name)
    if name in ("linear", "base"):
        return dict(base=10000.0, scaling=name, factor=8.0)
    if name == "bands":
        return dict(base=500000.0, scaling=name, factor=8.0, original=8192, low=1.0, high=4.0)
    return dict(base=10000.0, scaling=name, factor=8.0, original=8192, low=1.0, high=32.0, amplitude=1.2079441541679836)


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


def _batch(case, g):
    """Counts of new tokens and lengths per sequence.  The first sequence has `rows` new tokens and the full length,
    the others between an eighth of it and all of it, and as many new tokens ("even"), up to as many ("ragged", the
    same counts for every seed) or one."""
    b, rows, top = case["batch"], case["rows"], case["length"]
    low = max(1, top // 8)
    length = (low + (torch.rand(b, generator=g, device=DEV) * (top - low + 1)).long()).clamp(max=top)
    count = {"even": torch.full((b,), rows, device=DEV), "one": torch.ones(b, dtype=torch.long, device=DEV),
             "ragged": 1 + 7919 * torch.arange(1, b + 1, device=DEV) % rows}[case["shape"]]
    length[0], count[0] = top, rows
    return count, torch.maximum(length, count)


def _pages(batch, rows, page_rows, g, more=0):
    """A page table whose pages lie scattered over a pool a little larger than needed; `more` rows of further pages."""
    width, extra = -(-rows // page_rows), -(-more // page_rows)
    pool = batch * (width + extra) + 3
    order = torch.randperm(pool, generator=g, device=DEV)[:batch * (width + extra)].to(torch.int32)
    return order[:batch * width].reshape(batch, width).contiguous(), order[batch * width:].reshape(batch, extra).contiguous(), pool


def _full_cache(pool, heads, page_rows, d, dt, g):
    cache = torch.empty((pool, 2, heads, page_rows, d), dtype=dt, device=DEV)
    step = max(1, (1 << 26) // (2 * heads * page_rows * d))
    for p0 in range(0, pool, step):
        part = cache[p0:p0 + step]
        part.copy_(_kv_rows(g, *part.shape))
    return cache


def prepare(case, seed):
    g = _rng(seed)
    dt, op, d = TYPES[case["dtype"]], case["op"], case["d"]
    st = dict(case=case)
    if own:
        import context_ring_attention_gb300 as ra
    if op == "rope":
        b, s = case["batch"], case["seq"]
        for name, heads in (("q", case["heads_q"]), ("k", case["heads_kv"])):
            x = _randn(g, b, s, heads, d).to(dt).transpose(1, 2)
            # a prompt comes in the projections' order and its gradients go back into it
            there = case["strided"] and case["direction"] == "bwd"
            st[name] = x if case["strided"] and not there else x.contiguous()
            st[name + "_out"] = torch.empty((b, s, heads, d), dtype=dt, device=DEV).transpose(1, 2) if there else None
        if own:
            st["rope"] = ra.ra_rope_plan(d, case["rot"], interleaved=case["interleaved"], dtype=case["dtype"], **_scaling(case))
        return st
    hk, pr = case["heads_kv"], case["page_rows"]
    if op == "evict":
        b, top = case["batch"], case["length"]
        low = max(1, top - top // 8)
        n = (low + (torch.rand(b, generator=g, device=DEV) * (top - low + 1)).long()).clamp(max=top)
        n[0] = top
        st["lengths"], st["length"] = n.tolist(), n.to(torch.int32)
        st["table"], st["new_table"], st["pool"] = _pages(b, top, pr, g, more=min(case["keep"], top))
        st["cache"] = _full_cache(st["pool"], hk, pr, d, dt, g)
        width = st["table"].shape[1] * pr
        # a few keys hold most of the weight; some never got any
        w = torch.exp(2.0 * _randn(g, b, hk, width))
        st["weight"] = torch.where(torch.rand((b, hk, width), generator=g, device=DEV) < 0.1, torch.zeros_like(w), w)
        st["weight_out"] = torch.zeros_like(st["weight"])
        heads_q, window, sinks = hk, 0, 0
    else:
        count, length = _batch(case, g)
        st["counts"], st["lengths"] = count.tolist(), length.tolist()  # a serving loop knows them on the host as well
        st["length"] = length.to(torch.int32)
        st["offset"] = torch.cat([torch.zeros_like(count[:1]), count.cumsum(0)]).to(torch.int32)
        tokens, heads_q = sum(st["counts"]), case["heads_q"]
        st["table"], _, st["pool"] = _pages(case["batch"], case["length"], pr, g)
        if op == "append":
            # one projection's output: a token's queries, keys and values side by side
            x = _kv_rows(g, tokens, heads_q + 2 * hk, d).to(dt)
            st["q"], st["k"], st["v"] = x.split([heads_q, hk, hk], 1)
            st["cache"] = torch.zeros((st["pool"], 2, hk, pr, d), dtype=dt, device=DEV)
            window, sinks = 0, 0
        else:
            st["cache"] = _full_cache(st["pool"], hk, pr, d, dt, g)
            st["q"] = _randn(g, tokens, heads_q, d).to(dt)
            window, sinks = case["window"], case["sinks"]
        if op == "weigh":
            st["lse"] = _plain_attend(st, lse_only=True)
            width = st["table"].shape[1] * pr
            st["weight"] = torch.exp(2.0 * _randn(g, case["batch"], hk, width))
            st["weight_out"] = torch.zeros_like(st["weight"])
    if own:
        st["plan"] = ra.ra_paged_plan(st["pool"], pr, heads_q, hk, d, dtype=case["dtype"], window=window, sinks=sinks)
        if op == "append":
            st["rope"] = ra.ra_rope_plan(d, case["rot"], interleaved=case["interleaved"], dtype=case["dtype"], **_scaling(case))
    return st


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "weigh": _plain_weigh,
                "evict": _plain_evict}[op](state)
    import context_ring_attention_gb300 as ra
    if op == "rope":
        call = ra.ra_rope if case["direction"] == "fwd" else ra.ra_rope_bwd
        return call(state["rope"], state["q"], state["k"], layout=case["layout"], n_shards=case["shards"],
                    q_out=state["q_out"], k_out=state["k_out"])
    plan, cache, table, length = state["plan"], state["cache"], state["table"], state["length"]
    if op == "append":
        return ra.ra_paged_append(plan, cache, state["k"], state["v"], table, state["offset"], length, rope=state["rope"],
                                  q=state["q"]), cache
    if op == "attend":
        return ra.ra_paged_attend(plan, cache, state["q"], table, state["offset"], length)
    if op == "weigh":
        return ra.ra_paged_weigh(plan, cache, state["q"], state["lse"], table, state["offset"], length,
                                 state["weight_out"], weight_in=state["weight"])
    kept, new_length = ra.ra_paged_evict(plan, cache, table, length, state["weight"], case["keep"], first=case["first"],
                                         recent=case["recent"], new_table=state["new_table"], weight_out=state["weight_out"])
    return kept, new_length, state["weight_out"], cache


def _pairs(case):
    """Expected visible (query, key) pairs and visible keys of a batch, over one head."""
    top, w, sinks = case["length"], case["window"], case["sinks"]
    mean = 0.5625 * top
    pairs = keys = 0.0
    for n in range(case["batch"]):
        length = top if n == 0 else mean
        rows = case["rows"] if n == 0 or case["shape"] == "even" else (case["rows"] + 1) / 2 if case["shape"] == "ragged" else 1
        length = max(length, rows)
        seen = length - (rows - 1) / 2
        pairs += rows * (min(seen, w + sinks) if w else seen)
        keys += min(length, w + rows - 1 + sinks) if w else length
    return pairs, keys


def _tokens(case):
    rows, b = case["rows"], case["batch"]
    return rows + (b - 1) * {"even": rows, "ragged": (rows + 1) / 2, "one": 1}[case["shape"]]


def work(case):
    d, e, hk = case["d"], 2 if case["dtype"] == "bf16" else 4, case["heads_kv"]
    if case["op"] == "rope":
        rows = case["batch"] * case["seq"] * (case["heads_q"] + hk)
        return {"bytes": 2 * rows * d * e, "flops": 3 * rows * case["rot"]}
    if case["op"] == "append":
        rows = _tokens(case) * (case["heads_q"] + 2 * hk)
        return {"bytes": int(2 * rows * d * e), "flops": int(3 * _tokens(case) * (case["heads_q"] + hk) * case["rot"])}
    if case["op"] == "evict":
        top = case["length"]
        n = top + (case["batch"] - 1) * 0.9375 * top
        kept = min(case["keep"], top) * case["batch"]
        # the weights of all slots; the kept rows, their weights and indices
        return {"bytes": int(hk * (4 * n + kept * (4 * d * e + 8))), "flops": int(hk * n)}
    pairs, keys = _pairs(case)
    rows = _tokens(case) * case["heads_q"]
    if case["op"] == "attend":
        return {"bytes": int(2 * keys * hk * d * e + rows * (2 * d * e + 4)), "flops": int(4 * d * pairs * case["heads_q"])}
    n = case["length"] * (1 + 0.5625 * (case["batch"] - 1))
    return {"bytes": int(keys * hk * d * e + rows * (d * e + 4) + 8 * n * hk), "flops": int(2 * d * pairs * case["heads_q"])}


# --------------------------------------------------- plain form: positions --
def _angles(case, pos):
    """Cosine and sine [..., rot / 2] of the positions' angles, in float64 and then rounded."""
    rot, s = case["rot"], _scaling(case)
    j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    base, factor = s["base"], s.get("factor", 1.0)
    if s["scaling"] == "base":
        base = base * factor ** (rot / (rot - 2)) if rot > 2 else base
    theta = base ** (-2.0 * j / rot)
    if s["scaling"] == "linear":
        theta = theta / factor
    elif s["scaling"] == "bands":
        turns = s["original"] * theta / (2 * math.pi)
        own_part = ((turns - s["low"]) / (s["high"] - s["low"])).clamp(0, 1)
        theta = own_part * theta + (1 - own_part) * theta / factor
    elif s["scaling"] == "ramp":
        index = lambda t: rot * math.log(s["original"] / (2 * math.pi * t)) / (2 * math.log(base))
        lo, hi = max(math.floor(index(s["high"])), 0), min(math.ceil(index(s["low"])), rot - 1)
        part = ((j - lo) / (hi - lo if hi != lo else 0.001)).clamp(0, 1)
        theta = (1 - part) * theta + part * theta / factor
    a = pos.double()[..., None] * theta
    amp = s.get("amplitude", 1.0)
    return (a.cos() * amp).float(), (a.sin() * amp).float()


def _rotate(case, x, cos, sin):
    """x [..., d] rotated by angles that broadcast against [..., rot / 2], in float32."""
    rot = case["rot"]
    x = x.float()
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(st):
    case = st["case"]
    cos, sin = _angles(case, positions(case["layout"], case["seq"], case["shards"]))
    if case["direction"] == "bwd":
        sin = -sin
    return tuple(_rotate(case, st[x], cos, sin).to(st[x].dtype) for x in ("q", "k"))


def _slots(st):
    """Sequence and slot of every new token."""
    seq = torch.repeat_interleave(torch.arange(len(st["counts"]), device=DEV), torch.tensor(st["counts"], device=DEV))
    row = torch.arange(len(seq), device=DEV) - st["offset"].long()[seq]
    count = st["offset"][1:] - st["offset"][:-1]
    return seq, (st["length"] - count).long()[seq] + row


def _plain_append(st):
    case = st["case"]
    pr = case["page_rows"]
    seq, slot = _slots(st)
    cos, sin = (x[:, None] for x in _angles(case, slot))
    page = st["table"][seq, slot // pr].long()
    dt = st["cache"].dtype
    st["cache"][page, 0, :, slot % pr] = _rotate(case, st["k"], cos, sin).to(dt)
    st["cache"][page, 1, :, slot % pr] = st["v"]
    return _rotate(case, st["q"], cos, sin).to(dt), st["cache"]


# --------------------------------------------------- plain form: attention --
def _cached(st, n, j, which, dtype):
    """Rows j of sequence n: [heads_kv, len(j), d]."""
    pr = st["case"]["page_rows"]
    return st["cache"][st["table"][n, j // pr].long(), which, :, j % pr].transpose(0, 1).to(dtype)


def _row_blocks(case, count, keys):
    step = max(1, (1 << 28) // (case["heads_q"] * max(1, keys)))
    return [(i, min(count, i + step)) for i in range(0, count, step)]


def _seen_keys(case, lo_slot, hi_slot):
    """Slots that some token of the slots [lo_slot, hi_slot) sees, and which of them each sees."""
    w, sinks = case["window"], case["sinks"]
    lo = max(0, lo_slot - w + 1) if w else 0
    j = torch.cat([torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, hi_slot, device=DEV)])
    i = torch.arange(lo_slot, hi_slot, device=DEV)[:, None]
    return j, (j <= i) & ((j > i - w) | (j < sinks)) if w else j <= i


def _plain_attend(st, lse_only=False):
    case = st["case"]
    hq, hk, d = case["heads_q"], case["heads_kv"], case["d"]
    g = hq // hk
    tokens = st["q"].shape[0]
    o = torch.empty((tokens, hq, d), device=DEV)
    lse = torch.empty((tokens, hq), device=DEV)
    at = 0
    for n, (count, length) in enumerate(zip(st["counts"], st["lengths"])):
        for i0, i1 in _row_blocks(case, count, length):
            t = i1 - i0
            j, seen = _seen_keys(case, length - count + i0, length - count + i1)
            q = st["q"][at + i0:at + i1].float().view(t, hk, g, d).permute(1, 2, 0, 3).reshape(hk, g * t, d)
            x = (q @ _cached(st, n, j, 0, torch.float32).transpose(-1, -2)).div_(math.sqrt(d)).view(hk, g, t, -1)
            x.masked_fill_(~seen, -math.inf)
            m = x.amax(-1, keepdim=True)
            x.sub_(m).exp_()
            l = x.sum(-1, keepdim=True)
            lse[at + i0:at + i1] = (m + l.log())[..., 0].permute(2, 0, 1).reshape(t, hq)
            if not lse_only:
                y = (x.view(hk, g * t, -1) @ _cached(st, n, j, 1, torch.float32)).view(hk, g, t, d) / l
                o[at + i0:at + i1] = y.permute(2, 0, 1, 3).reshape(t, hq, d)
        at += count
    return lse if lse_only else (o.to(st["q"].dtype), lse)


def _plain_weigh(st):
    case = st["case"]
    hq, hk, d = case["heads_q"], case["heads_kv"], case["d"]
    g, at = hq // hk, 0
    for n, (count, length) in enumerate(zip(st["counts"], st["lengths"])):
        total = torch.zeros((hk, length), device=DEV)
        for i0, i1 in _row_blocks(case, count, length):
            t = i1 - i0
            j, seen = _seen_keys(case, length - count + i0, length - count + i1)
            q = st["q"][at + i0:at + i1].float().view(t, hk, g, d).permute(1, 2, 0, 3).reshape(hk, g * t, d)
            x = (q @ _cached(st, n, j, 0, torch.float32).transpose(-1, -2)).div_(math.sqrt(d)).view(hk, g, t, -1)
            x.sub_(st["lse"][at + i0:at + i1].view(t, hk, g).permute(1, 2, 0)[..., None]).exp_()
            total.index_add_(1, j, x.masked_fill_(~seen, 0.0).sum((1, 2)))
        # the call's own tokens had no weight before
        total[:, :length - count] += st["weight"][n, :, :length - count]
        st["weight_out"][n, :, :length] = total
        at += count
    return st["weight_out"]


# ---------------------------------------------------- plain form: eviction --
def _plain_evict(st):
    case = st["case"]
    hk, pr, keep, first, recent = (case[x] for x in ("heads_kv", "page_rows", "keep", "first", "recent"))
    b = case["batch"]
    kept = torch.full((b, hk, keep), -1, dtype=torch.int32, device=DEV)
    head = torch.arange(hk, device=DEV)[:, None]
    rows = []
    for n, length in enumerate(st["lengths"]):
        if length <= keep:
            slots = torch.arange(length, device=DEV).expand(hk, length)
        else:
            w = st["weight"][n, :, :length].clone()
            w[:, :first] = math.inf
            w[:, length - recent:] = math.inf
            order = torch.sort(w, dim=-1, descending=True, stable=True).indices  # ties: the lowest slot first
            slots = order[:, :keep].sort(-1).values
        m = slots.shape[1]
        kept[n, :, :m] = slots
        rows.append((n, m, slots, st["cache"][st["table"][n][slots // pr].long(), :, head, slots % pr]))
    for n, m, slots, x in rows:
        to = torch.arange(m, device=DEV)
        st["cache"][st["new_table"][n, to // pr].long(), :, head, to % pr] = x
        st["weight_out"][n, :, :m] = st["weight"][n].gather(1, slots)
    new_length = torch.minimum(st["length"], torch.full_like(st["length"], keep))
    return kept, new_length, st["weight_out"], st["cache"]


# ---------------------------------------------------------------- in 64 bits --
def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    st = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend, "weigh": _exact_weigh,
            "evict": _exact_evict}[case["op"]](st)


def _turn(case, x, pos, sign=1.0):
    """Pairs of channels as complex numbers, times amplitude * e^(i angle); pos broadcasts against x[..., 0]."""
    rot, s = case["rot"], _scaling(case)
    factor, half = s.get("factor", 1.0), rot // 2
    speed = []
    for j in range(half):
        base = s["base"]
        if s["scaling"] == "base" and rot > 2:
            base *= factor ** (rot / (rot - 2))
        f = math.exp(-2 * j / rot * math.log(base))
        if s["scaling"] == "linear":
            f /= factor
        if s["scaling"] == "bands":
            r = min(1.0, max(0.0, (s["original"] * f / math.tau - s["low"]) / (s["high"] - s["low"])))
            f = f / factor + r * (f - f / factor)
        if s["scaling"] == "ramp":
            place = [rot / 2 * math.log(s["original"] / (math.tau * t)) / math.log(base) for t in (s["high"], s["low"])]
            lo, hi = max(0, math.floor(place[0])), min(rot - 1, math.ceil(place[1]))
            r = min(1.0, max(0.0, (j - lo) / (hi - lo if hi > lo else 0.001)))
            f = f + r * (f / factor - f)
        speed.append(f)
    angle = pos.double().unsqueeze(-1) * torch.tensor(speed, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.full_like(angle, s.get("amplitude", 1.0)), sign * angle)
    y = x.double().clone()
    one, two = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
    z = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * turn
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_rope(st):
    case = st["case"]
    pos = positions(case["layout"], case["seq"], case["shards"])
    sign = 1.0 if case["direction"] == "fwd" else -1.0
    out = []
    for x in (st["q"], st["k"]):
        y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        for h in range(x.shape[1]):
            y[:, h] = _turn(case, x[:, h], pos, sign)
        out.append(y)
    return tuple(out)


def _exact_append(st):
    case = st["case"]
    pr, cache = case["page_rows"], st["cache"].double()
    q = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for n, (count, length) in enumerate(zip(st["counts"], st["lengths"])):
        slot = torch.arange(length - count, length, device=DEV)
        rows = slice(at, at + count)
        q[rows] = _turn(case, st["q"][rows], slot[:, None])
        k, v = _turn(case, st["k"][rows], slot[:, None]), st["v"][rows].double()
        for p in range((length - count) // pr, -(-length // pr)):  # page by page
            here = (slot // pr == p).nonzero()[:, 0]
            page = int(st["table"][n, p])
            cache[page, 0].index_copy_(1, slot[here] - p * pr, k[here].transpose(0, 1))
            cache[page, 1].index_copy_(1, slot[here] - p * pr, v[here].transpose(0, 1))
        at += count
    return q, cache


def _exact_scores(st, n, at, h, rows, which_keys):
    """float64 scores of tokens `rows` of sequence n and query head h against every slot up to the last one seen,
    -inf where a token does not see the slot, and the slots' rows of the cache."""
    case = st["case"]
    hk, pr, d = case["heads_kv"], case["page_rows"], case["d"]
    count, length = st["counts"][n], st["lengths"][n]
    mine = torch.arange(length - count, length, device=DEV)[rows][:, None]
    slot = torch.arange(int(mine.max()) + 1, device=DEV)
    gone = mine - slot[None]  # how far back
    vis = gone >= 0
    if case["window"]:
        vis &= (gone < case["window"]) | (slot[None] < case["sinks"])
    pages = st["table"][n, :-(-len(slot) // pr)].long()
    keys, values = (st["cache"][pages, which, h // (case["heads_q"] // hk)].reshape(-1, d)[:len(slot)].double()
                    if which in which_keys else None for which in (0, 1))
    q = st["q"][at:at + count][rows, h].double()
    x = torch.einsum("id,jd->ij", q, keys) * d ** -0.5
    return torch.where(vis, x, torch.full_like(x, -math.inf)), vis, values


def _exact_attend(st):
    case = st["case"]
    hq, d = case["heads_q"], case["d"]
    o = torch.zeros((st["q"].shape[0], hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((st["q"].shape[0], hq), dtype=torch.float64, device=DEV)
    at = 0
    for n, count in enumerate(st["counts"]):
        for r0 in range(0, count, 1024):
            rows = slice(r0, min(count, r0 + 1024))
            for h in range(hq):
                x, vis, v = _exact_scores(st, n, at, h, rows, (0, 1))
                top = torch.logsumexp(x, -1)
                out = slice(at + rows.start, at + rows.stop)
                o[out, h] = torch.exp(x - top[:, None]) @ v
                lse[out, h] = top
        at += count
    return o, lse


def _exact_weigh(st):
    case = st["case"]
    hq, hk = case["heads_q"], case["heads_kv"]
    out = torch.zeros(st["weight"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for n, (count, length) in enumerate(zip(st["counts"], st["lengths"])):
        old = length - count
        out[n, :, :old] = st["weight"][n, :, :old].double()
        for r0 in range(0, count, 1024):
            rows = slice(r0, min(count, r0 + 1024))
            for h in range(hq):
                x, vis, _ = _exact_scores(st, n, at, h, rows, (0,))
                p = torch.exp(x - st["lse"][at:at + count][rows, h].double()[:, None])
                out[n, h // (hq // hk), :p.shape[1]] += torch.where(vis, p, torch.zeros_like(p)).sum(0)
        at += count
    return out


def _exact_evict(st):
    """Slot by slot from the definition: a slot stays when it is protected or fewer than the free places are taken by
    heavier slots and by lower slots of the same weight."""
    case = st["case"]
    b, hk, pr, keep, first, recent = (case[x] for x in ("batch", "heads_kv", "page_rows", "keep", "first", "recent"))
    kept = torch.full((b, hk, keep), -1, dtype=torch.int32, device=DEV)
    weight_out, cache = st["weight_out"].double(), st["cache"].double()
    new_length = torch.tensor([min(n, keep) for n in st["lengths"]], dtype=torch.int32, device=DEV)
    for n, length in enumerate(st["lengths"]):
        slot = torch.arange(length, device=DEV)
        for h in range(hk):
            stay = slot
            if length > keep:
                w = st["weight"][n, h, :length].double()
                free = (slot >= first) & (slot < length - recent)
                places = keep - first - recent
                levels = torch.unique(w[free])
                lo, hi = 0, len(levels)  # the largest level that at least `places` free slots reach
                while lo < hi:
                    mid = (lo + hi) // 2
                    if int((free & (w >= levels[mid])).sum()) >= places:
                        lo = mid + 1
                    else:
                        hi = mid
                take = ~free
                if places:
                    border = levels[lo - 1]
                    above, equal = free & (w > border), free & (w == border)
                    take = take | above | (equal & (equal.cumsum(0) <= places - int(above.sum())))
                stay = take.nonzero()[:, 0]
            kept[n, h, :len(stay)] = stay
            weight_out[n, h, :len(stay)] = st["weight"][n, h, stay].double()
            to = torch.arange(len(stay), device=DEV)
            rows = st["cache"][st["table"][n, stay // pr].long(), :, h, stay % pr].double()
            cache[st["new_table"][n, to // pr].long(), :, h, to % pr] = rows
    return kept, new_length, weight_out, cache
