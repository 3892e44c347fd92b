"""The operators of a bounded KV cache, for measurement: attention with a sliding window and first tokens that stay
visible (a decode step, and chunks of a prompt, over the paged cache), the decode step that also accumulates each cached
token's attention weight, and the eviction that keeps the tokens of largest accumulated weight.

Each operator has a plain form (elementary torch operations in fp32, rounded once) and the call that a user makes of
this package, chosen by ``own``.  Shapes are those of one attention layer: the 32/8 and 64/8 head layouts of the
decode workloads, head_dim 64 and 128, blocks of 16 and 32 tokens, f16, bf16 and fp8-e4m3 caches.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------------ cases
def _case(name, op, seqs, lo, hi, hq, hkv, d, bs, q, kv, **more):
    c = {"op": op, "seqs": seqs, "len_min": lo, "len_max": hi, "q_heads": hq, "kv_heads": hkv, "head_dim": d,
         "block": bs, "q_dtype": q, "kv_dtype": kv, **more}
    return {"name": name, **c} if name else c


def listed():
    return [
        # one user far into a long chat, the first tokens and the last 4096 visible: latency counts
        _case("window decode 1 seq", "decode_window", 1, 31999, 31999, 32, 8, 128, 16, "bf16", "bf16", window=4096, sinks=4),
        # a full serving batch of 64/8 heads, contexts from a few hundred to 16k tokens
        _case("window decode 64 seqs", "decode_window", 64, 300, 16000, 64, 8, 128, 32, "bf16", "bf16", window=4096, sinks=4),
        # head_dim 64 with an fp8 cache, an odd window and number of first tokens, some contexts shorter than the window
        _case("window decode fp8 d64", "decode_window", 33, 1, 5000, 32, 8, 64, 16, "bf16", "fp8", window=1000, sinks=5),
        # one 512-token chunk of a long prompt after 4096 tokens of context
        _case("window chunk 512", "prefill_window", 1, 512, 512, 32, 8, 128, 16, "bf16", "bf16", start=4096, window=1024, sinks=4),
        # a batch of whole-prompt chunks, 2048 tokens each: bound by the tensor cores
        _case("window chunks 8x2048", "prefill_window", 8, 2048, 2048, 64, 8, 128, 16, "bf16", "bf16", start=2048, window=1024, sinks=4),
        # ragged chunks over an fp8 cache, the shortest of one token
        _case("window chunks fp8 ragged", "prefill_window", 5, 1, 701, 32, 8, 128, 32, "bf16", "fp8", start=1500, window=400, sinks=17),
        # decode steps that accumulate attention weight: one user
        _case("weights decode 1 seq", "decode_weights", 1, 8191, 8191, 32, 8, 128, 16, "bf16", "bf16"),
        # a serving batch of 64/8 heads
        _case("weights decode 64 seqs", "decode_weights", 64, 100, 8192, 64, 8, 128, 32, "bf16", "bf16"),
        # small f16 batch, head_dim 64, odd lengths
        _case("weights decode f16 d64", "decode_weights", 9, 1, 2047, 16, 8, 64, 16, "f16", "f16"),
        # after one long prompt: 8192 cached tokens down to 2048
        _case("evict 8192 to 2048", "evict", 1, 8192, 8192, 32, 8, 128, 16, "bf16", "bf16", budget=2048, sinks=4, recent=256, again=False),
        # a batch of prompts halved
        _case("evict 64 seqs to half", "evict", 64, 3000, 4096, 64, 8, 128, 32, "bf16", "bf16", budget=1777, sinks=4, recent=128, again=False),
        # steady state of a decode loop: every 16 tokens the cache goes back to its budget
        _case("evict steady state", "evict", 32, 1040, 1040, 32, 8, 64, 16, "f16", "f16", budget=1024, sinks=4, recent=256, again=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    op = rng.choice(["decode_window", "prefill_window", "decode_weights", "evict"])
    while True:
        hq, hkv = rng.choice([(32, 8), (64, 8), (16, 8), (40, 8), (8, 8), (24, 2)])
        d, bs = rng.choice([64, 128]), rng.choice([16, 32])
        q = rng.choice(["bf16", "f16"])
        kv = rng.choice([q, q, "fp8"])
        if op == "prefill_window":
            hi = _log(rng, 1, 2048)
            c = _case("", op, rng.randint(1, 8), rng.randint(1, hi), hi, hq, hkv, d, bs, q, kv, start=rng.choice([0, _log(rng, 1, 16000)]),
                      window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 33, 100]))
        elif op == "decode_window":
            hi = _log(rng, 1, 32000)
            c = _case("", op, _log(rng, 1, 64), rng.randint(1, hi), hi, hq, hkv, d, bs, q, kv, window=_log(rng, 1, 8192),
                      sinks=rng.choice([0, 1, 4, 33, 100]))
        elif op == "decode_weights":
            hi = _log(rng, 1, 16000)
            c = _case("", op, _log(rng, 1, 64), rng.randint(1, hi), hi, hq, hkv, d, bs, q, kv)
        else:
            sinks, recent = rng.choice([0, 4, 33]), rng.choice([1, 64, 200])
            budget = sinks + recent + _log(rng, 1, 4000)
            again = rng.random() < 0.5
            hi = budget + _log(rng, 1, 64 if again else 8000)
            c = _case("", op, _log(rng, 1, 64), hi if again else rng.randint(1, hi), hi, hq, hkv, d, bs, q, q, budget=budget,
                      sinks=sinks, recent=recent, again=again)
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def _lens(c):
    """The case's lengths: evenly spread over its range, in an order that is neither rising nor falling."""
    n, lo, hi = c["seqs"], c["len_min"], c["len_max"]
    if n == 1:
        return [hi]
    step = next(s for s in range(max(1, int(0.618 * n)), 2 * n) if math.gcd(s, n) == 1)
    return [lo + (hi - lo) * ((i * step + n - 1) % n) // (n - 1) for i in range(n)]


def _visible(n, window, sinks):
    """Tokens that the last of n sees."""
    return min(n, window) + min(sinks, max(0, n - window))


def work(c):
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    eb = 1 if c["kv_dtype"] == "fp8" else 2
    row = 2 * hkv * d * eb                        # K and V of one token
    lens = _lens(c)
    if c["op"] == "decode_window":
        seen = sum(_visible(n, c["window"], c["sinks"]) for n in lens)
        return {"bytes": seen * row + 4 * hq * d * len(lens), "flops": 4 * hq * d * seen}
    if c["op"] == "decode_weights":
        seen = sum(lens)
        return {"bytes": seen * (row + 8 * hkv) + 4 * hq * d * len(lens), "flops": (4 * hq * d + 2 * hq) * seen}
    if c["op"] == "prefill_window":
        w, s, pairs, keys = c["window"], c["sinks"], 0, 0
        for n in lens:
            pairs += sum(_visible(c["start"] + r + 1, w, s) for r in range(n))
            low = max(0, c["start"] + 1 - w)
            keys += c["start"] + n - low + min(s, low)
        return {"bytes": keys * row + 4 * hq * d * sum(lens), "flops": 4 * hq * d * pairs}
    b, s, r = c["budget"], c["sinks"], c["recent"]
    total = 0.0
    for n in lens:
        kept = min(n, b)
        moved = 0.0
        if n > b:                                 # the last ones, and their share of the others behind the budget
            late = min(r, n - b)
            moved = late + (n - b - late) * (b - s - r) / max(1, n - s - r)
        # weights and earlier positions read, both written for the kept, the moved rows read and written
        total += hkv * (4 * n + 4 * (b if c["again"] else 0) + 8 * kept) + 2 * moved * row
    return {"bytes": total, "flops": sum(lens) * hkv}


# ------------------------------------------------------------------------------------------------ inputs
def _pool(g, c, blocks):
    shape = (blocks, c["kv_heads"], c["block"], c["head_dim"])
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    if c["kv_dtype"] == "fp8":                     # codes of N(0, 1) values over a scale that puts 5.0 at the largest code
        return (x.float() * (448.0 / 5.0)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), 5.0 / 448.0
    return x.to(TYPES[c["kv_dtype"]]), 1.0


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, bs, hkv, hq, d, n = c["op"], c["block"], c["kv_heads"], c["q_heads"], c["head_dim"], c["seqs"]
    lens = _lens(c)
    start = c.get("start", 0)
    ctx = torch.tensor([start + m for m in lens] if op == "prefill_window" else lens)
    # blocks that hold a token which is seen get a place in the pool, in random order; the entries of the others, given
    # back long ago, and those behind the end are -1
    most = int(ctx.max())
    first = torch.arange(-(-most // bs)) * bs
    need = first[None] < ctx[:, None]
    if "window" in c:
        low = (start + 1 if op == "prefill_window" else ctx[:, None]) - c["window"]
        need &= (first[None] < c["sinks"]) | (first[None] + bs > low)
    tables = torch.full(need.shape, -1, dtype=torch.int32)
    blocks = int(need.sum())
    pool = blocks + blocks // 4 + 8
    order = torch.randperm(pool, generator=g, device=DEV).cpu()
    tables[need] = order[:blocks].to(torch.int32)
    k, ks = _pool(g, c, pool)
    v, vs = _pool(g, c, pool)
    rows = sum(lens) if op == "prefill_window" else n
    q = (1.5 * torch.randn((rows, hq, d), generator=g, device=DEV)).to(TYPES[c["q_dtype"]])
    st = {"case": c, "k": k, "v": v, "k_scale": ks, "v_scale": vs, "q": q, "out": torch.empty_like(q), "scale": d ** -0.5,
          "tables": tables.to(DEV), "lens": ctx.to(DEV, torch.int32), "max_len": most}
    if op == "prefill_window":
        cu = torch.zeros(n + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        st |= {"cu": cu.to(DEV), "start": torch.full((n,), start, dtype=torch.int32, device=DEV), "max_q": max(lens)}
    if op in ("decode_weights", "evict"):
        # a few tokens with most of the weight, many with next to none, some with exactly none
        w = torch.exp(2.0 * torch.randn((n, hkv, most), generator=g, device=DEV) - 4.0)
        w *= torch.rand((n, hkv, most), generator=g, device=DEV) > 0.1
        w[:, :, :4] += 5.0
        st["weights"] = w
    if op == "evict":
        del st["q"], st["out"]
        b, s = c["budget"], c["sinks"]
        seen, old = ctx.clone(), torch.zeros_like(ctx)
        pos = torch.full((n, hkv, most), -7, dtype=torch.int32, device=DEV)
        if c["again"]:
            # kept by earlier evictions: the first tokens, then some of those up to where the untouched ones begin
            seen, old = ctx + 5 * b, torch.full_like(ctx, b)
            gap = 6.0
            at = torch.arange(b, device=DEV, dtype=torch.float64)
            jitter = torch.rand((n, hkv, b), generator=g, device=DEV, dtype=torch.float64)
            pos[:, :, :b] = torch.where(at < s, at, s + torch.floor((at - s + jitter) * gap * (b - s / gap) / b)).to(torch.int32)
        st |= {"seen": seen.to(DEV, torch.int32), "old": old.to(DEV, torch.int32), "positions": pos,
               "new_weights": torch.zeros_like(w), "new_positions": torch.zeros_like(pos), "new_lens": torch.zeros_like(st["lens"])}
    if own:
        import paged_kv_cache_writes_gb300 as pa

        st["cache"] = pa.kv_cache_desc(k, ks, vs)
        size = 0
        if op == "decode_window":
            size = pa.pa_decode_window_workspace_bytes(n, hq, hkv, d, bs, most, c["window"], c["sinks"])
        elif op == "decode_weights":
            size = pa.pa_decode_weights_workspace_bytes(n, hq, hkv, d, most)
        elif op == "evict":
            size = pa.pa_evict_workspace_bytes(n, hkv, most, c["budget"])
        st["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------------------------ the passes
def run(st):
    c = st["case"]
    if own:
        return _own(st, c)
    return {"decode_window": _decode_window, "prefill_window": _prefill_window, "decode_weights": _decode_weights,
            "evict": _evict}[c["op"]](st, c)


def _own(st, c):
    import paged_kv_cache_writes_gb300 as pa

    if c["op"] == "decode_window":
        pa.pa_decode_window(st["q"], st["k"], st["v"], st["cache"], st["tables"], st["lens"], st["max_len"], c["window"],
                            c["sinks"], st["scale"], st["out"], st["workspace"])
        return st["out"]
    if c["op"] == "prefill_window":
        pa.pa_prefill_chunk_window(st["q"], st["cu"], st["start"], st["max_q"], st["k"], st["v"], st["cache"], st["tables"],
                                   st["lens"], st["max_len"], c["window"], c["sinks"], st["scale"], st["out"])
        return st["out"]
    if c["op"] == "decode_weights":
        pa.pa_decode_weights(st["q"], st["k"], st["v"], st["cache"], st["tables"], st["lens"], st["max_len"], st["scale"],
                             st["out"], st["weights"], workspace=st["workspace"])
        return st["out"], st["weights"]
    pa.pa_evict(st["k"], st["v"], st["cache"], st["tables"], st["lens"], st["max_len"], st["seen"], st["old"], c["budget"],
                c["sinks"], c["recent"], st["weights"], st["positions"], st["new_weights"], st["new_positions"], st["new_lens"],
                workspace=st["workspace"])
    return st["k"], st["v"], st["new_weights"], st["new_positions"], st["new_lens"]


def _rows(pool, scale, st, at):
    """Cache rows at token positions `at` [sequences, tokens] as fp32 [sequences, kv_heads, tokens, head_dim]."""
    bs = st["case"]["block"]
    at = at.clamp(0, st["max_len"] - 1)
    block = st["tables"].long().gather(1, at // bs).clamp(min=0)
    x = pool[block, :, at % bs]
    if pool.dtype == torch.uint8:
        x = x.view(torch.float8_e4m3fn).float() * scale
    return x.float().transpose(1, 2)


def _attend(q, k, v, mask, scale):
    """softmax(scale q k^T) v over the keys in `mask`: q [n, h, g * rows, d], k and v [n, h, keys, d], in fp32."""
    s = (q @ k.transpose(-1, -2)) * scale
    s.masked_fill_(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, 1.0, total), p, total


def _decode_window(st, c):
    n, hq, d = st["q"].shape
    hkv, w, s = c["kv_heads"], c["window"], c["sinks"]
    end = st["lens"].long()[:, None]
    first = torch.arange(s, device=DEV)[None]
    last = end - w + torch.arange(w, device=DEV)[None]
    at = torch.cat([first.expand(n, s), last], 1)
    mask = torch.cat([first < end - w, last >= 0], 1)
    q = st["q"].float().view(n, hkv, hq // hkv, d)
    o, _, _ = _attend(q, _rows(st["k"], st["k_scale"], st, at), _rows(st["v"], st["v_scale"], st, at), mask[:, None, None], st["scale"])
    return o.reshape(n, hq, d).to(st["q"].dtype)


def _prefill_window(st, c):
    total, hq, d = st["q"].shape
    n, m, hkv, w, s = c["seqs"], st["max_q"], c["kv_heads"], c["window"], c["sinks"]
    g = hq // hkv
    cu, start = st["cu"].long(), st["start"].long()
    row = torch.arange(total, device=DEV)
    chunk = torch.searchsorted(cu[1:], row, right=True)
    r = row - cu[chunk]
    q = torch.zeros((n, m, hkv, g, d), device=DEV)
    q[chunk, r] = st["q"].float().view(total, hkv, g, d)
    # keys that some row may see: the first ones, and from the first row's window on
    first = torch.arange(s, device=DEV)[None].expand(n, s)
    low = start[:, None] + 1 - w
    late = low + torch.arange(w - 1 + m, device=DEV)[None]
    at = torch.cat([first, late], 1)
    here = (start[:, None] + torch.arange(m, device=DEV)[None])[:, :, None]
    near = (late[:, None] <= here) & (late[:, None] > here - w) & (late[:, None] >= 0)
    mask = torch.cat([(first[:, None] <= here - w), near], 2)
    q = q.permute(0, 2, 3, 1, 4).reshape(n, hkv, g * m, d)
    full = mask[:, None, None].expand(n, 1, g, m, mask.shape[2]).reshape(n, 1, g * m, mask.shape[2])
    o, _, _ = _attend(q, _rows(st["k"], st["k_scale"], st, at), _rows(st["v"], st["v_scale"], st, at), full, st["scale"])
    o = o.view(n, hkv, g, m, d).permute(0, 3, 1, 2, 4)
    return o[chunk, r].reshape(total, hq, d).to(st["q"].dtype)


def _decode_weights(st, c):
    n, hq, d = st["q"].shape
    hkv = c["kv_heads"]
    end = st["lens"].long()[:, None]
    at = torch.arange(st["max_len"], device=DEV)[None].expand(n, -1)
    here = at < end
    q = st["q"].float().view(n, hkv, hq // hkv, d)
    o, p, total = _attend(q, _rows(st["k"], st["k_scale"], st, at), _rows(st["v"], st["v_scale"], st, at), here[:, None, None], st["scale"])
    w = (p / total).sum(2)
    old = st["weights"]
    old.copy_(torch.where(here[:, None], torch.where((at < end - 1)[:, None], old, 0.0) + w, old))
    return o.reshape(n, hq, d).to(st["q"].dtype), old


def _evict(st, c):
    b, bs = c["budget"], c["block"]
    w, n, hkv, most = st["weights"], c["seqs"], c["kv_heads"], st["max_len"]
    end, seen = st["lens"].long()[:, None, None], st["seen"].long()[:, None, None]
    slot = torch.arange(most, device=DEV)
    pos = torch.where(slot < st["old"][:, None, None], st["positions"].long(), seen - end + slot)
    safe = (pos < c["sinks"]) | (pos >= seen - c["recent"])
    rank = torch.where(safe, math.inf, w)
    rank = torch.where(slot < end, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(safe).scatter_(-1, order[..., :b], True) & (slot < end)
    hole, mover = ~kept & (slot < torch.minimum(end, torch.tensor(b, device=DEV))), kept & (slot >= b)
    big = most + b
    holes = torch.sort(torch.where(hole, slot, big)).values[..., :b]
    movers = torch.sort(torch.where(mover, slot, big)).values[..., :b]
    m = holes.shape[-1]
    src = torch.arange(m + 1, device=DEV).expand(n, hkv, m + 1).clone()
    src = src.scatter_(-1, holes.clamp(max=m), movers)[..., :m]
    to = torch.arange(m, device=DEV)
    live = (to < torch.minimum(end, torch.tensor(b, device=DEV))).expand(n, hkv, m)
    src = torch.where(live, src, 0)
    new_w, new_p = st["new_weights"], st["new_positions"]
    new_w[..., :m] = torch.where(live, w.gather(-1, src), new_w[..., :m])
    new_p[..., :m] = torch.where(live, pos.gather(-1, src).to(torch.int32), new_p[..., :m])
    move = live & (src != to)
    i, h, j = move.nonzero(as_tuple=True)
    a = src[i, h, j]
    tables = st["tables"].long()
    st["k"][tables[i, j // bs], h, j % bs] = st["k"][tables[i, a // bs], h, a % bs]
    st["v"][tables[i, j // bs], h, j % bs] = st["v"][tables[i, a // bs], h, a % bs]
    st["new_lens"].copy_(torch.clamp(st["lens"], max=b))
    return st["k"], st["v"], new_w, new_p, st["new_lens"]


# ------------------------------------------------------------------------------------------------ in 64 bits
def _sequence(st, pool, scale, i, end):
    """Sequence i's first `end` cache rows [kv_heads, end, head_dim] in 64 bits; rows of blocks it no longer has are zero."""
    c = st["case"]
    ids = st["tables"][i, : -(-end // c["block"])].long()
    x = pool[ids.clamp(min=0)]
    x = x.view(torch.float8_e4m3fn).to(torch.float64) * scale if pool.dtype == torch.uint8 else x.to(torch.float64)
    x = torch.where((ids >= 0)[:, None, None, None], x, 0.0)
    return x.permute(1, 0, 2, 3).reshape(c["kv_heads"], -1, c["head_dim"])[:, :end]


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "evict":
        return _exact_evict(st, c)
    hkv, g, d = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    q = st["q"].to(torch.float64)
    out = torch.zeros_like(q)
    new = st["weights"].to(torch.float64) if c["op"] == "decode_weights" else None
    at = 0
    for i, n in enumerate(_lens(c)):
        rows = n if c["op"] == "prefill_window" else 1
        end = int(st["lens"][i])
        k, v = _sequence(st, st["k"], st["k_scale"], i, end), _sequence(st, st["v"], st["v_scale"], i, end)
        key, here = torch.arange(end, device=DEV)[None], (end - rows + torch.arange(rows, device=DEV))[:, None]
        seen = key <= here
        if "window" in c:
            seen = seen & ((key < c["sinks"]) | (here - key < c["window"]))
        for h in range(hkv):
            for x in range(h * g, (h + 1) * g):
                s = torch.einsum("rd,kd->rk", q[at:at + rows, x], k[h]) * st["scale"]
                p = torch.softmax(torch.where(seen, s, -math.inf), -1)
                out[at:at + rows, x] = torch.einsum("rk,kd->rd", p, v[h])
                if new is not None:
                    if x == h * g:
                        new[i, h, end - 1] = 0.0
                    new[i, h, :end] += p[0]
        at += rows
    return out if new is None else (out, new)


def _exact_evict(st, c):
    b, bs = c["budget"], c["block"]
    k, v = st["k"].clone(), st["v"].clone()
    w, pos, new_w, new_p = (st[x].cpu() for x in ("weights", "positions", "new_weights", "new_positions"))
    new_w = new_w.to(torch.float64)
    lens, seen, old, tables = (st[x].tolist() for x in ("lens", "seen", "old", "tables"))
    to, come = [], []
    for i in range(c["seqs"]):
        n = lens[i]
        for h in range(c["kv_heads"]):
            p = torch.cat([pos[i, h, : old[i]], torch.arange(seen[i] - n + old[i], seen[i], dtype=torch.int32)])[:n]
            slots = torch.arange(n)
            if n > b:
                safe = (p < c["sinks"]) | (p >= seen[i] - c["recent"])
                others = slots[~safe]
                best = others[torch.argsort(-w[i, h, others].to(torch.float64), stable=True)[: b - int(safe.sum())]]
                kept = torch.zeros(n, dtype=torch.bool)
                kept[slots[safe]] = True
                kept[best] = True
                gone, late = slots[:b][~kept[:b]], slots[b:][kept[b:]]
                slots = slots[:b].clone()
                slots[gone] = late
                for x, y in zip(gone.tolist(), late.tolist()):
                    to.append((tables[i][x // bs], h, x % bs))
                    come.append((tables[i][y // bs], h, y % bs))
            new_w[i, h, : len(slots)] = w[i, h, slots].to(torch.float64)
            new_p[i, h, : len(slots)] = p[slots]
    if to:
        t, f = torch.tensor(to, device=DEV).T, torch.tensor(come, device=DEV).T
        k[t[0], t[1], t[2]] = st["k"][f[0], f[1], f[2]]
        v[t[0], t[1], t[2]] = st["v"][f[0], f[1], f[2]]
    return k.to(torch.float64), v.to(torch.float64), new_w.to(DEV), new_p.to(DEV), torch.clamp(st["lens"], max=b)
