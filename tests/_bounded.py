"""Plain 64-bit forms of the bounded-cache operators (sliding window with first tokens that stay visible, accumulated
attention weights, eviction) and the error bounds their kernels are held to.

Bounds, per output element, from how the kernels compute (u = 2^-24):
* scores: products of the stored values are exact; a row of head_dim products is summed 16 or 32 at a time into an fp32
  accumulator, so a score is off by at most e = scale * 24 * 2^-23 * sum |q||k| (at most 8 partial sums and, within
  one, 16 terms aligned to the largest).  With an fp8 cache the query's two or three e4m3 terms leave up to 2^-21 of
  its largest element: + scale * 2^-21 * max |q| * sum |k|.  In log2 units t is rounded to fp32 twice and 2^t is
  within 2^-22: + 4 u |s| + 2^-22 in the exponent.
* a softmax weight a is then off by at most (2 e + 2^-21) a, and sum a V by that times A = sum a |V|.
* P in the second product: bf16 caches hi + lo, within 2^-15 (decode) or 2^-16 (prefill), or for a prefill's bf16 output
  rounded to nearest, 2^-8, numerator and denominator: 2^-7 A; f16 P rounded to nearest,
  2^-11, numerator and denominator: 2^-10 A, and below 2^-14 to 2^-25: n 2^-25 max |V|; an fp8 decode holds 256 p to
  2^-8 of itself + 2^-14: 2^-8 A + n 2^-22 max |V|.  fp32 sums of n terms: 2^-24 (16 + n / 16) A.
* the stored output: half a step of its type."""
import math

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Cache:
    """A paged cache of random K and V for given lengths, on the CPU; `pools` gives the device copies.  Blocks that no
    sequence uses, and the tail of each last block, hold NaN; block-table entries behind the end are far out of range."""

    def __init__(self, lens, hkv, d, bs, kv, seed, scales=(0.011, 0.013), per_head=False, far=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.d, self.bs, self.kv, self.far = list(lens), hkv, d, bs, kv, far
        nblk = [-(-n // bs) for n in lens]
        self.num_blocks = sum(nblk) + 5
        order = torch.randperm(self.num_blocks, generator=g)
        self.tables = torch.full((len(lens), max(1, max(nblk, default=1)) + 2), 1 << 30, dtype=torch.int32)
        at = 0
        for i, n in enumerate(nblk):
            self.tables[i, :n] = order[at:at + n].to(torch.int32)
            at += n
        shape = (self.num_blocks, hkv, bs, d)
        self.k_scale, self.v_scale = (scales if kv == "fp8" else (1.0, 1.0))
        self.head_scales = None
        if kv == "fp8":
            if per_head:
                self.head_scales = [s * (1.0 + 0.25 * torch.arange(hkv, dtype=torch.float32)) for s in scales]
            self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8) for _ in range(2))
        else:
            self.k, self.v = (torch.full(shape, math.nan, dtype=DT[kv]) for _ in range(2))
        for i, n in enumerate(lens):
            p = torch.arange(n)
            b, o = self.tables[i].long()[p // bs], p % bs
            for pool in (self.k, self.v):
                x = torch.randn((n, hkv, d), generator=g)
                if kv == "fp8":
                    pool[b, :, o] = (x * 80).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                else:
                    pool[b, :, o] = x.to(DT[kv])

    def rows(self, which, i, n):
        """K or V of sequence i's first n tokens [hkv, n, d] in 64 bits."""
        pool = self.k if which == "k" else self.v
        p = torch.arange(n)
        x = pool[self.tables[i].long()[p // self.bs], :, p % self.bs].transpose(0, 1)
        if self.kv == "fp8":
            x = x.contiguous().view(torch.float8_e4m3fn).double()
            s = self.k_scale if which == "k" else self.v_scale
            if self.head_scales is not None:
                return x * self.head_scales[0 if which == "k" else 1].double()[:, None, None]
            return x * float(np.float32(s))
        return x.double()

    def poison(self, i, dead):
        """Tokens `dead` (bool [n]) of sequence i hold NaN and infinity; blocks of dead tokens alone leave the table."""
        n, bs = len(dead), self.bs
        p = torch.arange(n)[dead]
        b, o = self.tables[i].long()[p // bs], p % bs
        for pool, bad in ((self.k, math.inf), (self.v, math.nan)):
            if self.kv == "fp8":
                pool[b, :, o] = 0x7F   # e4m3 has no infinity
            else:
                pool[b, :, o] = bad
        for j in range(-(-n // bs)):
            if bool(dead[j * bs:(j + 1) * bs].all()):
                self.tables[i, j] = -1

    def device(self, pa):
        """(k, v, tables, descriptor) on the GPU; far: at the end of pools whose byte offsets pass 32 bits."""
        k, v, tables = self.k.cuda(), self.v.cuda(), self.tables
        if self.far:
            first = (5 << 30) // (k[0].numel() * k.element_size())
            pools = [torch.empty((first + self.num_blocks, *k.shape[1:]), dtype=k.dtype, device="cuda") for _ in range(2)]
            pools[0][first:], pools[1][first:] = k, v
            k, v = pools
            tables = torch.where((tables >= 0) & (tables < self.num_blocks), tables + first, tables)
        self.dev_scales = None if self.head_scales is None else [s.cuda() for s in self.head_scales]
        desc = pa.kv_cache_desc(k, self.k_scale, self.v_scale, *(self.dev_scales or (None, None)))
        return k, v, tables.cuda(), desc


def visible(t, n, window, sinks):
    """Which of n tokens the query at position t sees."""
    p = torch.arange(n)
    return (p <= t) & ((p < sinks) | (p > t - window))


def attend(q, k, v, seen, scale, kv, out, prefill=False, p_terms=2):
    """q [r, hq, d] (the stored values), k and v [hkv, n, d] in 64 bits, seen [r, n].  Returns (out [r, hq, d],
    bound on |kernel - out|, weights [r, hq, n], relative bound of the weights [r, hq])."""
    r, hq, d = q.shape
    hkv, n = k.shape[:2]
    g = hq // hkv
    x = q.double().view(r, hkv, g, d)
    k0 = torch.where(seen.any(0)[None, :, None], k, 0.0)
    v0 = torch.where(seen.any(0)[None, :, None], v, 0.0)
    s = torch.einsum("rhgd,hnd->rhgn", x, k0) * scale
    e = torch.einsum("rhgd,hnd->rhgn", x.abs(), k0.abs()) * abs(scale) * 24 * 2.0 ** -23
    if kv == "fp8":
        e = e + abs(scale) * 2.0 ** -21 * x.abs().amax(-1, keepdim=True) * k0.abs().sum(-1)[None, :, None, :]
    e = e + 4 * 2.0 ** -24 * s.abs() + 2.0 ** -22
    m = seen[:, None, None, :]
    e = torch.where(m, e, 0.0).amax(-1)
    s = torch.where(m, s, -math.inf)
    a = torch.where(m.any(-1, keepdim=True), torch.softmax(s, -1), 0.0)
    a = torch.nan_to_num(a)
    o = torch.einsum("rhgn,hnd->rhgd", a, v0)
    big = torch.einsum("rhgn,hnd->rhgd", a, v0.abs())
    count = seen.sum(-1).double()[:, None, None, None]
    vmax = v0.abs().amax() if n else torch.tensor(0.0)
    rel = (2 * e + 2.0 ** -21)[..., None] + 2.0 ** -24 * (16 + count / 16)
    if kv == "bf16":
        rel, low = rel + (2.0 ** -15 if not prefill else 2.0 ** -7 if out == "bf16" else 2.0 ** -16), 0.0
    elif kv == "f16" or prefill:
        rel, low = rel + 2.0 ** -10, count * 2.0 ** -25 * vmax
    elif p_terms == 3:   # 256 p in three e4m3 terms: within 2^-12 of it, or 2^-18 where it is small
        rel, low = rel + 2.0 ** -12, count * 2.0 ** -26 * vmax
    else:
        rel, low = rel + 2.0 ** -8, count * 2.0 ** -22 * vmax
    bound = rel * big + low
    bound = bound + HALF_STEP[out] * (o.abs() + bound) + (2.0 ** -25 if out == "f16" else 1e-38)
    return o.reshape(r, hq, d), bound.reshape(r, hq, d), a.reshape(r, hq, n), (2 * e + 2.0 ** -20).reshape(r, hq)


def check(got, want, bound, what=""):
    g = got.double().cpu()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    worst = ((g - want).abs() / bound).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: error is {worst:.3g} of its bound"
    return worst


def evict(weights, positions, n, seen, old, budget, sinks, recent):
    """The plain eviction of one (sequence, KV head): the slot whose token ends up in each of min(n, budget) slots, and
    every slot's position.  weights, positions: 1-D."""
    pos = [int(positions[s]) if s < old else seen - n + s for s in range(n)]
    if n <= budget:
        return list(range(n)), pos
    safe = [pos[s] < sinks or pos[s] >= seen - recent for s in range(n)]

    def rank(s):   # protected first, then by weight; NaN below everything; ties to the lowest slot
        w = float(weights[s])
        return (0, 0.0, s) if safe[s] else (1, -w, s) if w == w else (2, 0.0, s)

    kept = set(sorted(range(n), key=rank)[:budget])
    holes = [s for s in range(budget) if s not in kept]
    movers = [s for s in range(budget, n) if s in kept]
    src = list(range(budget))
    for h, m in zip(holes, movers):
        src[h] = m
    return src, pos
