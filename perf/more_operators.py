"""The operators of a cache in 8 bits with a scale for each block and KV head, for measurement: the append that rotates
queries and keys by their positions and stores keys and values (in a 16-bit or fp8 cache too), and the attention that reads
such a cache, one token per sequence or chunks of a prompt.

Each operator has a plain form (elementary torch operations in fp32, rounded once) and the call that a user makes of
this package, chosen by ``own``.  Shapes are those of one attention layer: the 32/8 and 64/8 head layouts of the decode
workloads, head_dim 64 and 128, blocks of 16 and 32 tokens.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
LEAST, MOST = -64, 32                             # exponents of the scales that an append chooses


# ------------------------------------------------------------------------------------------------ cases
def _case(name, op, seqs, lo, hi, start, hq, hkv, d, bs, q, **more):
    """`seqs` sequences with lo..hi new tokens each after start tokens, or, decoding, lo..hi tokens in all."""
    c = {"op": op, "seqs": seqs, "len_min": lo, "len_max": hi, "start": start, "q_heads": hq, "kv_heads": hkv, "head_dim": d,
         "block": bs, "q_dtype": q, **more}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a decode step's new tokens, one per sequence, into a bf16 cache: latency counts
        _case("append 64 decodes", "append", 64, 1, 1, 31000, 32, 8, 128, 16, "bf16", kv="bf16", rope=128, pairs=False),
        # four prompt chunks of 2048 tokens at once into a bf16 cache
        _case("append 4x2048", "append", 4, 2048, 2048, 2048, 64, 8, 128, 16, "bf16", kv="bf16", rope=128, pairs=False),
        # ragged chunks into an fp8 cache with one scale, half of the elements rotated, as neighbouring pairs
        _case("append fp8 ragged", "append", 7, 1, 701, 1501, 32, 8, 64, 32, "f16", kv="fp8", rope=32, pairs=True),
        # the decode step's new tokens into blocks that hold some already, whose scale may have to grow
        _case("append scaled 64 decodes", "append", 64, 1, 1, 8001, 64, 8, 128, 32, "bf16", kv="scaled", rope=128, pairs=False),
        # prompt chunks that begin and end inside a block
        _case("append scaled 4x2048", "append", 4, 2048, 2048, 2043, 64, 8, 128, 32, "bf16", kv="scaled", rope=128, pairs=False),
        # ragged chunks beside single tokens
        _case("append scaled ragged", "append", 9, 1, 333, 777, 16, 8, 64, 16, "f16", kv="scaled", rope=64, pairs=True),
        # one user far into a long chat
        _case("decode 1 seq", "decode", 1, 31999, 31999, 0, 32, 8, 128, 16, "bf16"),
        # a full serving batch, contexts from a few hundred to 16k tokens
        _case("decode 64 seqs", "decode", 64, 300, 16000, 0, 64, 8, 128, 32, "bf16"),
        # head_dim 64, f16 queries, an uneven group, odd lengths from one token on
        _case("decode f16 d64", "decode", 33, 1, 5000, 0, 40, 8, 64, 16, "f16"),
        # one 512-token chunk of a long prompt after 4096 tokens
        _case("chunk 512", "prefill", 1, 512, 512, 4096, 32, 8, 128, 16, "bf16"),
        # four chunks of 2048 tokens: bound by the tensor cores
        _case("chunks 4x2048", "prefill", 4, 2048, 2048, 2048, 64, 8, 128, 32, "bf16"),
        # ragged chunks, the shortest of one token
        _case("chunks ragged d64", "prefill", 5, 1, 701, 1500, 32, 8, 64, 16, "f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        b, f = most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    op = rng.choice(["append", "append", "decode", "prefill"])
    while True:
        hq, hkv = rng.choice([(32, 8), (64, 8), (16, 8), (40, 8), (8, 8), (24, 2)])
        d, bs, q = rng.choice([64, 128]), rng.choice([16, 32]), rng.choice(["bf16", "f16"])
        hi = _log(rng, 1, 2048)
        if op == "append":
            one = rng.random() < 0.4               # a decode step
            c = _case("", op, _log(rng, 1, 256) if one else rng.randint(1, 9), 1 if one else rng.randint(1, hi), 1 if one else hi,
                      rng.choice([0, _log(rng, 1, 30000)]), hq, hkv, d, bs, q, kv=rng.choice([q, "fp8", "scaled", "scaled"]),
                      rope=rng.choice([d, d, d // 2, 16]), pairs=rng.random() < 0.4)
        elif op == "decode":
            hi = _log(rng, 1, 32000)
            c = _case("", op, _log(rng, 1, 64), rng.randint(1, hi), hi, 0, hq, hkv, d, bs, q)
        else:
            c = _case("", op, rng.randint(1, 8), rng.randint(1, hi), hi, rng.choice([0, _log(rng, 1, 8000)]), hq, hkv, d, bs, q)
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


def work(c):
    hq, hkv, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block"]
    lens, start = _lens(c), c["start"]
    tokens = sum(lens)
    row = 2 * hkv * d                              # codes of K and V of one token
    scales = 8 * hkv                               # of one block
    if c["op"] == "append":
        eb = 2 if c["kv"] in TYPES else 1
        blocks = sum((start + n - 1) // bs - start // bs + 1 for n in lens)
        # q read and written, k and v read, rows of the table, slots and positions, what is stored
        return {"bytes": tokens * (4 * hq * d + 2 * row + 4 * c["rope"] + 12 + eb * row) + (scales * blocks if c["kv"] == "scaled" else 0),
                "flops": 3 * tokens * (hq + hkv) * c["rope"]}
    if c["op"] == "decode":
        return {"bytes": tokens * row + sum(-(-n // bs) for n in lens) * scales + 4 * hq * d * len(lens), "flops": 4 * hq * d * tokens}
    keys = sum(start + n for n in lens)
    pairs = sum(n * start + n * (n + 1) // 2 for n in lens)
    return {"bytes": keys * row + sum(-(-(start + n) // bs) for n in lens) * scales + 4 * hq * d * tokens, "flops": 4 * hq * d * pairs}


# ------------------------------------------------------------------------------------------------ inputs
def _power(amax):
    """The smallest power of two 2^e, LEAST <= e <= MOST, with amax <= 448 * 2^e (or the largest)."""
    m, e = torch.frexp(amax)                       # 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - torch.where(m <= 0.875, 9, 8), LEAST).clamp(LEAST, MOST)
    return torch.ldexp(torch.ones_like(amax), e)


def _scaled_pool(g, c, blocks):
    """Codes and scales of tokens whose magnitudes differ from block to block and head to head."""
    shape = (blocks, c["kv_heads"], c["block"], c["head_dim"])
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
    x *= torch.exp(0.5 * torch.randn(shape[:2] + (1, 1), generator=g, device=DEV)).to(x.dtype)
    scale = _power(x.abs().amax((2, 3)).float())
    return (x * (1 / scale)[..., None, None].to(x.dtype)).to(E4M3).view(torch.uint8), scale


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, bs, hkv, hq, d, n = c["op"], c["block"], c["kv_heads"], c["q_heads"], c["head_dim"], c["seqs"]
    lens, start = _lens(c), c["start"]
    ctx = torch.tensor([start + m for m in lens])
    most = int(ctx.max())
    # every block's place in the pool, in random order (an append's: of the blocks that it touches); entries behind a
    # sequence's end are -1
    first = torch.arange(-(-most // bs)) * bs
    need = first[None] < ctx[:, None]
    if op == "append":
        need &= first[None] + bs > start
    tables = torch.full(need.shape, -1, dtype=torch.int32)
    blocks = int(need.sum())
    pool = blocks + blocks // 4 + 8
    tables[need] = torch.randperm(pool, generator=g, device=DEV).cpu()[:blocks].to(torch.int32)
    rows = n if op == "decode" else sum(lens)
    kind = c.get("kv", "scaled")
    k_scales = v_scales = None
    if kind == "scaled":
        k, k_scales = _scaled_pool(g, c, pool)
        v, v_scales = _scaled_pool(g, c, pool)
    else:
        k, v = (torch.randn((pool, hkv, bs, d), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        k, v = (x.to(TYPES[kind]) if kind in TYPES else (x * 64).to(E4M3).view(torch.uint8) for x in (k, v))
    st = {"case": c, "k": k, "v": v, "k_scales": k_scales, "v_scales": v_scales, "tables": tables.to(DEV),
          "lens": ctx.to(DEV, torch.int32), "max_len": most}
    ty = TYPES[c["q_dtype"]]
    if op == "append":
        # queries, keys and values side by side, as a projection leaves them; tokens of different magnitude
        x = torch.randn((rows, hq + 2 * hkv, d), generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn((rows, hq + 2 * hkv, 1), generator=g, device=DEV))
        qkv = x.to(ty)
        pos = torch.cat([torch.arange(start, start + m) for m in lens])
        seq = torch.repeat_interleave(torch.arange(n), torch.tensor(lens))
        slots = tables[seq, pos // bs].long() * bs + pos % bs
        inv = 10000.0 ** (-torch.arange(c["rope"] // 2, dtype=torch.float64) * 2 / c["rope"])
        angle = torch.arange(most, dtype=torch.float64)[:, None] * inv
        st |= {"q": qkv[:, :hq], "k_new": qkv[:, hq:hq + hkv], "v_new": qkv[:, hq + hkv:], "slots": slots.to(DEV),
               "positions": pos.to(DEV, torch.int32), "table": torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV),
               "q_out": torch.empty((rows, hq, d), dtype=ty, device=DEV), "scale": 6.0 / 448.0 if kind == "fp8" else 1.0}
    else:
        st["q"] = (1.5 * torch.randn((rows, hq, d), generator=g, device=DEV)).to(ty)
        st |= {"out": torch.empty_like(st["q"]), "scale": d ** -0.5}
    if op == "prefill":
        cu = torch.zeros(n + 1, dtype=torch.int32)
        cu[1:] = torch.cumsum(torch.tensor(lens), 0)
        st |= {"cu": cu.to(DEV), "start": torch.full((n,), start, dtype=torch.int32, device=DEV), "max_q": max(lens)}
    if own:
        import paged_kv_cache_writes_gb300 as pa

        st["cache"] = pa.kv_cache_desc(k, *((st["scale"], st["scale"]) if kind == "fp8" else ()))
        if op == "decode":
            size = pa.pa_decode_scaled_workspace_bytes(n, hq, hkv, d, most)
            st["workspace"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------------------------------------ the passes
def run(st):
    c = st["case"]
    if own:
        return _own(st, c)
    return {"append": _append, "decode": _decode, "prefill": _prefill}[c["op"]](st, c)


def _stored(st, c):
    """What an append leaves: the queries, the pools (codes by their values) and their scales."""
    k, v = st["k"], st["v"]
    if c["kv"] not in TYPES:
        k, v = k.view(E4M3), v.view(E4M3)
    return (st["q_out"], k, v) + ((st["k_scales"], st["v_scales"]) if c["kv"] == "scaled" else ())


def _own(st, c):
    import paged_kv_cache_writes_gb300 as pa

    if c["op"] == "append":
        pa.pa_rope_and_cache(st["q"], st["k_new"], st["v_new"], st["positions"], st["table"], st["slots"], st["k"], st["v"],
                             st["cache"], st["q_out"], interleaved=c["pairs"], k_scales=st["k_scales"], v_scales=st["v_scales"])
        return _stored(st, c)
    if c["op"] == "decode":
        pa.pa_decode_scaled(st["q"], st["k"], st["v"], st["cache"], st["k_scales"], st["v_scales"], st["tables"], st["lens"],
                            st["max_len"], st["scale"], st["out"], st["workspace"])
        return st["out"]
    pa.pa_prefill_chunk_scaled(st["q"], st["cu"], st["start"], st["max_q"], st["k"], st["v"], st["cache"], st["k_scales"],
                               st["v_scales"], st["tables"], st["lens"], st["max_len"], st["scale"], st["out"])
    return st["out"]


def _rotate(x, cos, sin, pairs):
    """x [tokens, heads, head_dim], its first elements rotated by cos and sin [tokens, rope / 2]."""
    r = 2 * cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., : r // 2], x[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _code(x):
    return x.clamp(-448, 448).to(E4M3)


def _append(st, c):
    bs, r = c["block"], c["rope"]
    row = st["table"][st["positions"].long()]
    cos, sin = row[:, : r // 2], row[:, r // 2:]
    st["q_out"].copy_(_rotate(st["q"].float(), cos, sin, c["pairs"]))
    block, off = st["slots"] // bs, st["slots"] % bs
    for pool, scales, x in ((st["k"], st["k_scales"], _rotate(st["k_new"].float(), cos, sin, c["pairs"])),
                            (st["v"], st["v_scales"], st["v_new"].float())):
        if c["kv"] in TYPES:
            pool[block, :, off] = x.to(pool.dtype)
        elif c["kv"] == "fp8":
            pool[block, :, off] = _code(x / st["scale"]).view(torch.uint8)
        else:
            # of every block its largest new element and its first new slot
            amax = torch.zeros_like(scales).index_reduce_(0, block, x.abs().amax(-1), "amax")[block]
            held = torch.full((len(scales),), float(bs), device=DEV).index_reduce_(0, block, off.float(), "amin")[block]
            old = scales[block]
            new = torch.where((held[:, None] > 0) & (amax <= 448 * old), old, _power(amax))
            # what the block holds already, by its new scale (each of a block's tokens writes the same)
            codes = pool[block].view(E4M3).float()
            moved = _code(codes * (old / new)[..., None, None])
            keep = torch.arange(bs, device=DEV) < held[:, None]
            pool[block] = torch.where(keep[:, None, :, None], moved.view(torch.uint8), pool[block])
            pool[block, :, off] = _code(x / new[..., None]).view(torch.uint8)
            scales[block] = new
    return _stored(st, c)


def _rows(pool, scales, st):
    """The cached rows of every sequence in fp32 [sequences, kv_heads, tokens, head_dim]."""
    block = st["tables"].long().clamp(min=0)
    x = pool[block].view(E4M3).float() * scales[block][..., None, None]
    n, b, h, s, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, b * s, d)[:, :, : st["max_len"]]


def _attend(q, k, v, mask, scale):
    """softmax(scale q k^T) v over the keys in `mask`: q [n, h, rows, d], k and v [n, h, keys, d], in fp32."""
    s = (q @ k.transpose(-1, -2)) * scale
    s.masked_fill_(~mask, -math.inf)
    s -= s.amax(-1, keepdim=True)
    p = s.exp_()
    return (p @ v) / p.sum(-1, keepdim=True)


def _decode(st, c):
    n, hq, d = st["q"].shape
    seen = torch.arange(st["max_len"], device=DEV) < st["lens"][:, None, None, None]
    q = st["q"].float().view(n, c["kv_heads"], -1, d)
    o = _attend(q, _rows(st["k"], st["k_scales"], st), _rows(st["v"], st["v_scales"], st), seen, st["scale"])
    return o.reshape(n, hq, d).to(st["q"].dtype)


def _prefill(st, c):
    total, hq, d = st["q"].shape
    n, m, hkv = c["seqs"], st["max_q"], c["kv_heads"]
    g = hq // hkv
    cu = st["cu"].long()
    row = torch.arange(total, device=DEV)
    chunk = torch.searchsorted(cu[1:], row, right=True)
    r = row - cu[chunk]
    q = torch.zeros((n, m, hkv, g, d), device=DEV)
    q[chunk, r] = st["q"].float().view(total, hkv, g, d)
    seen = torch.arange(st["max_len"], device=DEV) <= c["start"] + torch.arange(m, device=DEV)[:, None]
    o = _attend(q.permute(0, 2, 3, 1, 4).reshape(n, hkv, g * m, d), _rows(st["k"], st["k_scales"], st),
                _rows(st["v"], st["v_scales"], st), seen.repeat(g, 1), st["scale"])
    o = o.view(n, hkv, g, m, d).permute(0, 3, 1, 2, 4)
    return o[chunk, r].reshape(total, hq, d).to(st["q"].dtype)


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(c, seed):
    st = prepare(c, seed)
    return _exact_append(st, c) if c["op"] == "append" else _exact_attention(st, c)


def _exact_append(st, c):
    bs, r, pairs = c["block"], c["rope"], c["pairs"]
    angle = st["table"].double()[st["positions"].long()]

    def turn(x):
        z = x.double().clone()
        i = torch.arange(r // 2, device=DEV)
        at, to = (2 * i, 2 * i + 1) if pairs else (i, i + r // 2)
        w = torch.complex(angle[:, : r // 2], angle[:, r // 2:])[:, None]
        y = torch.complex(z[..., at], z[..., to]) * w
        z[..., at], z[..., to] = y.real, y.imag
        return z

    found = [turn(st["q"])]
    scales = []
    powers = torch.tensor([2.0 ** e for e in range(LEAST, MOST + 1)], dtype=torch.float64, device=DEV)
    slots = st["slots"].tolist()
    for pool, old, x in ((st["k"], st["k_scales"], turn(st["k_new"])), (st["v"], st["v_scales"], st["v_new"].double())):
        if c["kv"] in TYPES:
            out = pool.double()
        else:
            out = pool.view(E4M3).double()
        if c["kv"] != "scaled":
            y = x if c["kv"] in TYPES else _code(x / float(torch.tensor(st["scale"]).float())).double()
            for h in range(c["kv_heads"]):
                out[st["slots"] // bs, h, st["slots"] % bs] = y[:, h]
        else:
            new = old.double()
            of = {}
            for t, s in enumerate(slots):
                of.setdefault(s // bs, []).append(t)
            for b, ts in of.items():
                offs = [slots[t] % bs for t in ts]
                y, held = x[ts], min(offs)
                want = powers[torch.searchsorted(448 * powers[:-1], y.abs().amax((0, 2)))]
                was = new[b].clone()
                new[b] = want if held == 0 else torch.where(y.abs().amax((0, 2)) <= 448 * was, was, want)
                out[b, :, :held] = _code(out[b, :, :held] * (was / new[b])[:, None, None]).double()
                out[b][:, offs] = _code(y / new[b][None, :, None]).double().transpose(0, 1)
            scales.append(new)
        found.append(out)
    return tuple(found + scales)


def _exact_attention(st, c):
    hkv, g, bs = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["block"]
    q = st["q"].double()
    out = torch.zeros_like(q)
    at = 0
    for i, n in enumerate(_lens(c)):
        rows, end = (1 if c["op"] == "decode" else n), int(st["lens"][i])
        ids = st["tables"][i, : -(-end // bs)].long()
        seen = torch.arange(end, device=DEV)[None] <= (end - rows + torch.arange(rows, device=DEV))[:, None]
        for h in range(hkv):
            k, v = ((pool[ids, h].view(E4M3).double() * s[ids, h].double()[:, None, None]).reshape(-1, c["head_dim"])[:end]
                    for pool, s in ((st["k"], st["k_scales"]), (st["v"], st["v_scales"])))
            for x in range(h * g, (h + 1) * g):
                p = torch.softmax(torch.where(seen, (q[at:at + rows, x] @ k.T) * st["scale"], -math.inf), -1)
                out[at:at + rows, x] = p @ v
        at += rows
    return out
