"""Every type of output of the bounded-cache attention calls, within bounds that follow from how many bits each holds P in:
a term of P that is dropped, doubled or put into the wrong rows is far outside them.  And the same call twice gives the
same bits.

The scores' part of the bounds is that of tests/_bounded.py; the second product's is here.  A = sum a |V| over the visible
tokens, n their number:
* 16-bit caches, decode: P = hi + lo.  bf16: both truncated, within 2^-15 of p.  f16: both rounded to nearest, within
  2^-22 of p, or 2^-25 where that is below f16's smallest step (2^-24).  The sum is that of the unrounded P.
* fp8 caches, decode: 256 p in e4m3 terms, each within 2^-4 of what is left, and the next one 16 times as fine: two terms
  hold it to 2^-8, or 2^-14 (half of the second's smallest step, 2^-9 / 16 / 2) where it is small, three to 2^-12, or 2^-18.
  A bf16 output takes two, any other three.
* chunks: a 16-bit output takes P rounded to nearest, the sum being that of the rounded P: numerator and denominator are
  each off by 2^-8 (bf16 cache) or 2^-11 (f16 and fp8 caches, whose operands are f16) at most, and by 2^-25 a key below
  f16's normal range.  P is at most 2^8 there (the running maximum may lag by that factor) and p of the row's largest
  score at least 1, so that 2^-25 a key is at most n 2^-25 max |V| of the output.  An fp32 output takes P as hi + lo:
  within 2^-16 of p for a bf16 cache (rounded), 2^-22 or 2^-25 for the others, the sum unrounded."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import Cache, DT, HALF_STEP, attend, check, visible

pytestmark = pytest.mark.gpu

LENS = [1, 15, 16, 33, 127, 130, 511, 700, 1537]
TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")]


def bound_of(q, k, v, seen, scale, kv, out, chunk):
    """(the 64-bit result, the bound of an output of type `out`)."""
    o, _, a, rel_w = attend(q, k, v, seen, scale, kv, "f32")
    r, hq, d = o.shape
    hkv, n = k.shape[:2]
    v0 = torch.where(seen.any(0)[None, :, None], v, 0.0)
    big = torch.einsum("rhgn,hnd->rhgd", a.view(r, hkv, hq // hkv, n), v0.abs()).reshape(r, hq, d)
    count, vmax = seen.sum(-1).double()[:, None, None], v0.abs().amax()
    # rel_w = 2 e + 2^-20 of tests/_bounded.py; fp32 sums of n terms
    rel = rel_w[..., None] + 2.0 ** -24 * (16 + count / 16)
    if chunk and out != "f32":
        rel, low = (rel + 2.0 ** -7, 0.0) if kv == "bf16" else (rel + 2.0 ** -10, 2.0 ** -25)
    elif kv == "bf16":
        rel, low = rel + (2.0 ** -16 if chunk else 2.0 ** -15), 0.0
    elif kv == "f16" or chunk:
        rel, low = rel + 2.0 ** -22, 2.0 ** -25
    elif out == "bf16":
        rel, low = rel + 2.0 ** -8, 2.0 ** -22
    else:
        rel, low = rel + 2.0 ** -12, 2.0 ** -26
    b = rel * big + low * count * vmax
    return o, b + HALF_STEP[out] * (o.abs() + b) + (2.0 ** -25 if out == "f16" else 1e-38)


def outputs(qt):
    return [qt, "f32"]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_decode(c, q, call, out, window, sinks, scale):
    k, v, tables, desc = c.device(pa)
    n, hq, d = q.shape
    most = max(c.lens)
    got = []
    for fill in (0x5A, 0xFF):                              # twice, over different leftovers in the workspace
        o = torch.full(q.shape, float("nan"), dtype=DT[out], device="cuda")
        if call == "window":
            size = pa.pa_decode_window_workspace_bytes(n, hq, c.hkv, d, c.bs, most, window, sinks)
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            pa.pa_decode_window(q.cuda(), k, v, desc, tables, i32(c.lens), most, window, sinks, scale, o, ws)
            got.append([o])
        else:
            size = pa.pa_decode_weights_workspace_bytes(n, hq, c.hkv, d, most)
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            w = torch.zeros((n, c.hkv, most), device="cuda")
            pa.pa_decode_weights(q.cuda(), k, v, desc, tables, i32(c.lens), most, scale, o, w, workspace=ws)
            got.append([o, w])
        assert pa.pa_get_device_error() == 0
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.uint8).cpu(), y.view(torch.uint8).cpu())
    return got[0][0]


def decode_case(lens, hq, hkv, d, bs, qt, kv, out, call, window=2 ** 31 - 1, sinks=0, seed=0, **kw):
    c = Cache(lens, hkv, d, bs, kv, seed, **kw)
    q = (1.5 * torch.randn((len(lens), hq, d), generator=torch.Generator().manual_seed(seed + 1))).to(DT[qt])
    want = []
    for i, n in enumerate(lens):
        seen = visible(n - 1, n, window, sinks)
        want.append(bound_of(q[i:i + 1], c.rows("k", i, n), c.rows("v", i, n), seen[None], d ** -0.5, kv, out, False))
        c.poison(i, ~seen)
    o = run_decode(c, q, call, out, window, sinks, d ** -0.5)
    for i, n in enumerate(lens):
        check(o[i:i + 1], *want[i], f"sequence {i} of {n} tokens")


@pytest.mark.parametrize("call", ["window", "weights"])
@pytest.mark.parametrize("qt,kv,out", [(q, k, o) for q, k in TYPES for o in outputs(q)])
@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 4, 64, 16), (16, 2, 64, 32), (24, 2, 64, 16), (8, 2, 128, 16), (16, 2, 128, 32),
                                         (26, 2, 128, 16)])
def test_decode_outputs(call, qt, kv, out, hq, hkv, d, bs):
    bounds = (90, 5) if call == "window" else (2 ** 31 - 1, 0)
    decode_case(LENS, hq, hkv, d, bs, qt, kv, out, call, *bounds, seed=hq + d)


@pytest.mark.parametrize("call", ["window", "weights"])
@pytest.mark.parametrize("qt,kv,out", [(q, k, o) for q, k in TYPES for o in outputs(q)])
def test_decode_outputs_of_large_batches(call, qt, kv, out):
    """The launch with a plan kernel, whose CTAs merge split rows among themselves."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 1400, (150,), generator=g).tolist()
    decode_case(lens, 8, 2, 64, 16, qt, kv, out, call, *((700, 9) if call == "window" else ()), seed=4)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_decode_outputs_with_scales_per_head(out):
    decode_case(LENS, 8, 4, 128, 16, "bf16", "fp8", out, "window", 64, 4, seed=5, per_head=True)


def chunk_case(chunks, hq, hkv, d, bs, qt, kv, out, window, sinks, seed=0, scale=None, shape=None, **kw):
    lens = [s + r for s, r in chunks]
    c = Cache(lens, hkv, d, bs, kv, seed, **kw)
    total = sum(r for _, r in chunks)
    q = 1.5 * torch.randn((total, hq, d), generator=torch.Generator().manual_seed(seed + 1))
    if shape:
        shape(c, q)
    q = q.to(DT[qt])
    scale = d ** -0.5 if scale is None else scale
    want, cu = [], [0]
    for i, (s, r) in enumerate(chunks):
        n = s + r
        seen = torch.stack([visible(s + x, n, window, sinks) for x in range(r)])
        want.append(bound_of(q[cu[-1]:cu[-1] + r], c.rows("k", i, n), c.rows("v", i, n), seen, scale, kv, out, True))
        c.poison(i, ~seen.any(0))
        cu.append(cu[-1] + r)
    k, v, tables, desc = c.device(pa)
    got = []
    for _ in range(2):
        o = torch.full((total, hq, d), float("nan"), dtype=DT[out], device="cuda")
        pa.pa_prefill_chunk_window(q.cuda(), i32(cu), i32([s for s, _ in chunks]), max(r for _, r in chunks), k, v, desc, tables,
                                   i32(lens), max(lens), window, sinks, scale, o)
        assert pa.pa_get_device_error() == 0
        got.append(o)
    assert torch.equal(got[0].view(torch.uint8).cpu(), got[1].view(torch.uint8).cpu())
    for i, (s, r) in enumerate(chunks):
        check(got[0][cu[i]:cu[i] + r], *want[i], f"chunk {i}: {r} rows at {s}")


CHUNKS = [(0, 1), (0, 77), (300, 130), (1000, 1), (517, 40)]


@pytest.mark.parametrize("qt,kv,out", [(q, k, o) for q, k in TYPES for o in outputs(q)])
@pytest.mark.parametrize("hq,hkv,d,bs", [(2, 2, 64, 16), (16, 2, 64, 32), (10, 2, 128, 16), (32, 2, 128, 32)])
def test_chunk_outputs(qt, kv, out, hq, hkv, d, bs):
    chunk_case(CHUNKS, hq, hkv, d, bs, qt, kv, out, 90, 5, seed=hq + d)


@pytest.mark.parametrize("qt,kv,out", [(q, k, o) for q, k in TYPES for o in outputs(q)])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_outputs_with_two_ctas_per_sm(qt, kv, out, d):
    chunk_case([(200, 330), (0, 401), (37, 250)], 32, 8, d, 16, qt, kv, out, 250, 9, seed=d)


@pytest.mark.parametrize("qt,out", [(q, o) for q in ("bf16", "f16") for o in outputs(q)])
@pytest.mark.parametrize("rise", [20.0, 24.0, 60.0])
def test_chunk_outputs_with_rising_scores(qt, out, rise):
    """Scores that rise along the keys by `rise` in log2 units, so that the running maximum lags behind a row's scores (P
    is then as large as 2^8) and is brought up to date in between."""
    n, d = 370, 128
    base = torch.randn((1, d), generator=torch.Generator().manual_seed(41))
    ramp = rise * 0.6931 * d ** 0.5 * (torch.arange(n) / n)[:, None] / float((base * base).sum())

    def shape(c, q):
        q += base - 0.9 * q                                # every query close to `base`
        p = torch.arange(n)
        c.k[c.tables[0].long()[p // 16], 0, p % 16] = (ramp * base).to(c.k.dtype)

    chunk_case([(300, 70)], 4, 1, d, 16, qt, qt, out, 100000, 0, seed=31, shape=shape)
