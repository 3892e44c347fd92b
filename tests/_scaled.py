"""Plain 64-bit (and bit-exact) forms of the block-scaled cache: the append that rotates, quantises and raises scales, and
the attention over codes with a scale per block and KV head, with the error bounds the kernels are held to.

The append's arithmetic is fixed to the bit: products and sums of the rotation are rounded to fp32 one by one, a scale
is a power of two found by comparing, code * old / new and x / scale are exact or IEEE divisions in fp32, and e4m3 is
rounded to nearest even.  So codes, scales and 16-bit rows are compared for equality.

Bounds of the attention, per output element (u = 2^-24; scores and their bound e as in tests/_bounded.py, K being code
times scale):
* chunks with bf16 queries and output take a query row, its largest element at 2^e in [128, 256), as hi + lo, e4m3 both:
  exact where the element's last bit, 2^-7 of its power of two, is e4m3's smallest step 2^-9 or more, else off by half of
  that step, 2^-10: 2^-17 of the largest element, in the place of 2^-21.
* the exponent of a weight is t = s + log2 vs - max: log2 vs is within 2 ulp of its value and t is rounded, so e grows
  by 2^-21 (1 + |log2 vs|); the same factor meets numerator and sum.
* the second product takes w = p vs in f16, rounded once for a 16-bit output, 2^-11 of it or 2^-25 where it is small (it is
  at least 1 at the row's largest); for an fp32 output hi + lo, 2^-22 or 2^-25.  The small-value terms are of the row's
  largest w: n of them times the largest code.
* the sum is that of the unrounded p, in fp32 over n terms: 2^-24 (16 + n / 16).
* the stored output: half a step of its type."""
import math

import numpy as np
import torch

from _bounded import DT, HALF_STEP

E4M3 = torch.float8_e4m3fn


def e4m3_values():
    """The 128 values of codes 0..127 (code 127: NaN)."""
    v = []
    for c in range(128):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    v[127] = math.nan
    return np.array(v)


_V = e4m3_values()
_MID = (_V[:126] + _V[1:127]) / 2           # between code i and i + 1


def encode(x):
    """e4m3 codes of fp32 values: nearest, ties to the even code, saturating; NaN to 127."""
    x = np.asarray(x, np.float64)
    a = np.abs(np.where(np.isnan(x), 0.0, x))
    lo = np.searchsorted(_MID, a, "left")       # the number of midpoints below a
    tie = (lo < 126) & (a == _MID[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    code = np.where(np.isnan(x), 127, code).astype(np.uint8)
    return code | ((np.signbit(x) & ~np.isnan(x)).astype(np.uint8) << 7)


def decode(c):
    c = np.asarray(c)
    v = _V[c & 127]
    return np.where(c & 128, -v, v)


def power_for(amax):
    e = -64
    while e < 32 and amax > 448.0 * 2.0 ** e:
        e += 1
    return np.float32(2.0 ** e)


def rotate(x, table, positions, interleaved):
    """x fp32 [T, H, D] rotated as the kernel rotates, products and sums rounded to fp32."""
    y = x.astype(np.float32).copy()
    r = table.shape[1]
    c, s = (table[positions][:, None, i * (r // 2):(i + 1) * (r // 2)].astype(np.float32) for i in (0, 1))
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    a, b = y[..., ia].copy(), y[..., ib].copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., ia] = a * c - b * s
        y[..., ib] = b * c + a * s
    return y


def append(x, slots, codes, scales, bs):
    """Store rows x fp32 [T, H, D] (already rotated) at `slots` into codes uint8 [blocks, H, bs, D] and scales fp32
    [blocks, H], in place."""
    blocks = {}
    for t, s in enumerate(slots):
        if s >= 0:
            blocks.setdefault(int(s) // bs, []).append((t, int(s) % bs))
    for b, toks in blocks.items():
        ts, offs = [t for t, _ in toks], [o for _, o in toks]
        held = min(offs)
        for h in range(x.shape[1]):
            y = x[ts, h]
            fin = np.abs(y[np.isfinite(y)])
            amax = np.float32(fin.max()) if fin.size else np.float32(0)
            old = scales[b, h]
            if held > 0 and not 2.0 ** -64 <= old <= 2.0 ** 32:
                continue
            new = power_for(float(amax))
            if held > 0 and amax <= np.float32(448) * old:
                new = old
            elif held > 0:
                codes[b, h, :held] = encode((decode(codes[b, h, :held]) * (float(old) / float(new))).astype(np.float32))
            with np.errstate(over="ignore"):
                codes[b, h, offs] = encode(y / new)
            scales[b, h] = new


def table(n, r, base=10000.0):
    """cos_sin of positions 0..n-1: fp32 [n, r]."""
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(r // 2) / r)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class ScaledCache:
    """A block-scaled cache of random codes and scales for given lengths, on the CPU.  Blocks that no sequence uses and the
    tail of each last block hold NaN codes, unused blocks NaN scales; table entries behind the end are far out of range.
    spread: standard deviation of log2 of the scales; powers: whether they are powers of two."""

    def __init__(self, lens, hkv, d, bs, seed, spread=1.5, powers=True, far=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.d, self.bs, self.far = list(lens), hkv, d, bs, far
        nblk = [-(-n // bs) for n in lens]
        self.num_blocks = sum(nblk) + 5
        order = torch.randperm(self.num_blocks, generator=g)
        self.tables = torch.full((len(lens), max(1, max(nblk, default=1)) + 2), 1 << 30, dtype=torch.int32)
        shape = (self.num_blocks, hkv, bs, d)
        self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8) for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:2], math.nan) for _ in range(2))
        at = 0
        for i, n in enumerate(nblk):
            ids = order[at:at + n]
            self.tables[i, :n] = ids.to(torch.int32)
            at += n
            for s in (self.ks, self.vs):
                e = -6.5 + spread * torch.randn((n, hkv), generator=g)
                s[ids] = torch.exp2(e.round() if powers else e).float()
            p = torch.arange(lens[i])
            b, o = self.tables[i].long()[p // bs], p % bs
            for pool in (self.k, self.v):
                x = torch.randn((lens[i], hkv, d), generator=g)
                pool[b, :, o] = (x * 90).clamp(-448, 448).to(E4M3).view(torch.uint8)

    def rows(self, which, i, n):
        """(codes' values [hkv, n, d], scales [hkv, n]) of sequence i's first n tokens in 64 bits."""
        pool, sc = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        p = torch.arange(n)
        b = self.tables[i].long()[p // self.bs]
        x = pool[b, :, p % self.bs].transpose(0, 1).contiguous()
        return x.view(E4M3).double(), sc[b].T.double()

    def device(self, pa):
        """(k, v, tables, descriptor, k scales, v scales) on the GPU; far: byte offsets past 32 bits."""
        k, v, ks, vs, tables = self.k.cuda(), self.v.cuda(), self.ks.cuda(), self.vs.cuda(), self.tables
        if self.far:
            first = (5 << 30) // k[0].numel()
            shape = (first + self.num_blocks, *k.shape[1:])
            pools = [torch.empty(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
            sc = [torch.full(shape[:2], math.nan, device="cuda") for _ in range(2)]
            pools[0][first:], pools[1][first:], sc[0][first:], sc[1][first:] = k, v, ks, vs
            (k, v), (ks, vs) = pools, sc
            tables = torch.where((tables >= 0) & (tables < self.num_blocks), tables + first, tables)
        return k, v, tables.cuda(), pa.kv_cache_desc(k), ks, vs


def attend(q, k, v, seen, scale, out, chunk):
    """q [r, hq, d]; k, v: (codes [hkv, n, d], scales [hkv, n]) in 64 bits; seen [r, n].  (out, bound) [r, hq, d]."""
    (kc, ks), (vc, vs) = k, v
    r, hq, d = q.shape
    hkv, n = kc.shape[:2]
    x = q.double().view(r, hkv, hq // hkv, d)
    kk = kc * ks[..., None]
    s = torch.einsum("rhgd,hnd->rhgn", x, kk) * scale
    e = torch.einsum("rhgd,hnd->rhgn", x.abs(), kk.abs()) * abs(scale) * 24 * 2.0 ** -23
    terms = 2.0 ** -17 if chunk and out == "bf16" else 2.0 ** -21
    e = e + abs(scale) * terms * x.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)[None, :, None, :]
    lv = torch.log2(vs)[None, :, None, :]
    e = e + 4 * 2.0 ** -24 * s.abs() + 2.0 ** -22 + 2.0 ** -21 * (1 + lv.abs())
    m = seen[:, None, None, :]
    e = torch.where(m, e, 0.0).amax(-1) if n else torch.zeros(s.shape[:-1], dtype=torch.float64)
    s = torch.where(m, s, -math.inf)
    a = torch.nan_to_num(torch.softmax(s, -1))
    w = a * vs[None, :, None, :]
    o = torch.einsum("rhgn,hnd->rhgd", w, vc)
    big = torch.einsum("rhgn,hnd->rhgd", w, vc.abs())
    count = seen.sum(-1).double()[:, None, None, None]
    rel = (2 * e + 2.0 ** -20)[..., None] + 2.0 ** -24 * (16 + count / 16)
    rel, low = rel + (2.0 ** -22 if out == "f32" else 2.0 ** -11), 2.0 ** -25
    top = (w.amax(-1, keepdim=True) if n else 0.0) * 448.0
    b = rel * big + low * count * top
    b = b + HALF_STEP[out] * (o.abs() + b) + (2.0 ** -25 if out == "f16" else 1e-38)
    return o.reshape(r, hq, d), b.reshape(r, hq, d)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_decode(pa, c, q, scale, out="f32", stream=None):
    k, v, tables, desc, ks, vs = c.device(pa)
    n, hq, d = q.shape
    most = max(c.lens, default=0)
    size = pa.pa_decode_scaled_workspace_bytes(n, hq, c.hkv, d, most)
    assert size > 0
    ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    o = torch.full(q.shape, math.nan, dtype=DT[out], device="cuda")
    q, lens = q.cuda(), i32(c.lens)
    torch.cuda.synchronize()                       # (the call may go to another stream)
    pa.pa_decode_scaled(q, k, v, desc, ks, vs, tables, lens, most, scale, o, ws, stream=stream)
    assert pa.pa_get_device_error(stream) == 0
    return o


def run_chunks(pa, c, q, rows, scale, out="f32", stream=None):
    """rows[i]: the chunk's tokens, the last of sequence i's."""
    k, v, tables, desc, ks, vs = c.device(pa)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    start = [n - r for n, r in zip(c.lens, rows)]
    o = torch.full(q.shape, math.nan, dtype=DT[out], device="cuda")
    q, cu_dev, start, lens = q.cuda(), i32(cu), i32(start), i32(c.lens)
    torch.cuda.synchronize()                       # (the call may go to another stream)
    pa.pa_prefill_chunk_scaled(q, cu_dev, start, max(rows), k, v, desc, ks, vs, tables, lens, max(c.lens),
                               scale, o, stream=stream)
    assert pa.pa_get_device_error(stream) == 0
    return o, cu


def causal(n, rows):
    """seen [rows, n] of a chunk of the last `rows` of n tokens."""
    return torch.arange(n)[None] <= (n - rows + torch.arange(rows))[:, None]
