"""The attention over a block-scaled cache where V's scales lie far apart: blocks of large values ("loud") have zero codes in
the even elements, so that there the tokens of small values alone decide the output, and must not be lost beside the others.

Bound of those elements, from the definition's own terms (no term of the loud blocks): as in tests/_scaled.py, but
* a weight is within 2^-11 of itself for a 16-bit output; for an fp32 one within 2^-22, or 2^-17 in a key tile one of
  whose scales is under 2^-8 of the largest of the tiles so far;
* in other tiles a weight times its scale is held to 2^-25 where the row's largest so far is 2^7 or more: 2^-32 of that one,
  whose scale is at most 2^8 times the token's, so 2^-24 of the row's largest weight, times the token's own scale."""
import math

import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import DT, HALF_STEP
from _scaled import ScaledCache, causal, run_chunks, run_decode

pytestmark = pytest.mark.gpu

OUT = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


def loud(c, where, small, large):
    """V's scales 2^small, and 2^large in the loud blocks, whose even elements are 0."""
    for i, n in enumerate(c.lens):
        b = c.tables[i, :-(-n // c.bs)].long()
        at = torch.arange(len(b))
        big = {"first": at == 0, "last": at == len(b) - 1, "some": at % 3 == 1, "most": at % 4 != 2}[where]
        c.vs[b] = torch.where(big, 2.0 ** large, 2.0 ** small)[:, None].expand(-1, c.hkv).float()
        for x in b[big]:
            c.v[x, :, :, ::2] = torch.where(c.v[x, :, :, ::2] == 0x7F, c.v[x, :, :, ::2], 0)   # (rows behind the end stay NaN)


def attend(q, k, v, seen, scale, out, chunk):
    """(out, bound) [r, hq, d] in 64 bits."""
    (kc, ks), (vc, vs) = k, v
    r, hq, d = q.shape
    hkv, n = kc.shape[:2]
    x = q.double().view(r, hkv, hq // hkv, d)
    kk = kc * ks[..., None]
    s = torch.einsum("rhgd,hnd->rhgn", x, kk) * scale
    e = torch.einsum("rhgd,hnd->rhgn", x.abs(), kk.abs()) * abs(scale) * 24 * 2.0 ** -23
    terms = 2.0 ** -17 if chunk and out == "bf16" else 2.0 ** -21
    e = e + abs(scale) * terms * x.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)[None, :, None, :]
    e = e + 4 * 2.0 ** -24 * s.abs() + 2.0 ** -22 + 2.0 ** -21 * (1 + torch.log2(vs).abs())[None, :, None, :]
    m = seen[:, None, None, :]
    e = torch.where(m, e, 0.0).amax(-1)
    a = torch.softmax(torch.where(m, s, -math.inf), -1)
    vv = vc * vs[..., None]
    o = torch.einsum("rhgn,hnd->rhgd", a, vv)
    big = torch.einsum("rhgn,hnd->rhgd", a, vv.abs())
    floor = 2.0 ** -24 * a.amax(-1)[..., None] * torch.einsum("rhgn,hnd->rhgd", m.double().expand(a.shape), vv.abs())
    held = 2.0 ** -11 if out != "f32" else 2.0 ** -22 if vs.max() <= 256 * vs.min() else 2.0 ** -17
    rel = (2 * e + 2.0 ** -20)[..., None] + 2.0 ** -24 * (16 + n / 16) + held
    b = rel * big + floor
    b = b + HALF_STEP[out] * (o.abs() + b) + (2.0 ** -25 if out == "f16" else 1e-38)
    return o.reshape(r, hq, d), b.reshape(r, hq, d)


def quiet(got, want, bound, what):
    g, w, b = got.double().cpu()[..., ::2], want[..., ::2], bound[..., ::2]
    assert torch.isfinite(g).all(), what
    worst = ((g - w).abs() / b).max().item()
    assert worst <= 1.0, f"{what}: error is {worst:.3g} of its bound"


def run(case, lens, rows, hq, hkv, d, bs, qt, out, where, small, large, seed):
    c = ScaledCache(lens, hkv, d, bs, seed, spread=0.5)
    loud(c, where, small, large)
    if case == "decode":
        rows = [1] * len(lens)
    q = (1.5 * torch.randn((sum(rows), hq, d), generator=torch.Generator().manual_seed(seed + 1))).to(DT[qt])
    scale = d ** -0.5
    if case == "decode":
        o, cu = run_decode(pa, c, q, scale, out), list(range(len(lens) + 1))
    else:
        o, cu = run_chunks(pa, c, q, rows, scale, out)
    for i, (n, r) in enumerate(zip(lens, rows)):
        want, bound = attend(q[cu[i]:cu[i + 1]], c.rows("k", i, n), c.rows("v", i, n), causal(n, r), scale, out, case == "chunk")
        quiet(o[cu[i]:cu[i + 1]], want, bound, f"sequence {i}: {r} of {n} tokens")


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("qt,out", OUT)
@pytest.mark.parametrize("where", ["first", "last", "some", "most"])
@pytest.mark.parametrize("ratio", [7, 8, 9, 14, 20, 26, 36])
def test_quiet_tokens_beside_loud_ones(case, qt, out, where, ratio):
    run(case, [40, 300, 1111], [40, 100, 150], 8, 2, 128, 16, qt, out, where, -6, ratio - 6, seed=ratio)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("qt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("where", ["first", "some"])
@pytest.mark.parametrize("bs", [16, 32])
def test_the_whole_range_of_scales(case, qt, out, where, bs):
    run(case, [33, 700], [33, 130], 8, 2, 64, bs, qt, out, where, -64, 32, seed=5)


@pytest.mark.parametrize("qt,out", OUT)
@pytest.mark.parametrize("d", [64, 128])
def test_decode_of_many_tiles_per_warp(qt, out, d):
    """Enough rows for a warp to take loud tiles and quiet ones in turn."""
    g = torch.Generator().manual_seed(d)
    lens = torch.randint(1500, 2500, (40,), generator=g).tolist()
    for where in ("some", "most", "first"):
        run("decode", lens, None, 16, 4, d, 32, qt, out, where, -10, 20, seed=d)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("where", ["first", "last", "some"])
def test_far_into_a_context(case, where):
    for qt, out in OUT:
        run(case, [6001, 4300], [130, 20], 8, 2, 128, 16, qt, out, where, -8, 10, seed=3)
        run(case, [9000], [64], 8, 1, 64, 16, qt, out, where, -8, 14, seed=4)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(32, 2, 64, 16), (17, 1, 64, 32), (32, 2, 128, 32), (20, 2, 128, 16), (5, 5, 64, 16)])
def test_heads(case, hq, hkv, d, bs):
    """Every kernel's form of the heads, and (chunks) two query tiles per CTA and one."""
    for qt, out in OUT:
        run(case, [50, 901], [50, 30], hq, hkv, d, bs, qt, out, "some", -8, 12, seed=hq + d)
    if case == "chunk":
        for qt, out in OUT:
            run(case, [1100, 700], [700, 700], 32, 4, d, bs, qt, out, "some", -8, 12, seed=hq + d)
