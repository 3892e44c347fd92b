"""pa_decode_scaled and pa_prefill_chunk_scaled against the 64-bit form, within bounds derived from their arithmetic
(tests/_scaled.py).  Tails of blocks and unused blocks hold NaN codes, unused blocks NaN scales."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import DT, check
from _scaled import ScaledCache, attend, causal, run_chunks, run_decode

pytestmark = pytest.mark.gpu

LENS = [1, 15, 16, 33, 127, 128, 130, 511, 513, 700, 1537]
OUT = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


def queries(n, hq, d, qt, seed):
    return (1.5 * torch.randn((n, hq, d), generator=torch.Generator().manual_seed(seed))).to(DT[qt])


def decode_case(lens, hq, hkv, d, bs, qt, out, seed=0, scale=None, change=None, **kw):
    c = ScaledCache(lens, hkv, d, bs, seed, **kw)
    if change:
        change(c)
    q = queries(len(lens), hq, d, qt, seed + 1)
    scale = d ** -0.5 if scale is None else scale
    o = run_decode(pa, c, q, scale, out)
    for i, n in enumerate(lens):
        want, bound = attend(q[i:i + 1], c.rows("k", i, n), c.rows("v", i, n), causal(n, 1), scale, out, False)
        check(o[i:i + 1], want, bound, f"sequence {i} of {n} tokens")


def chunk_case(lens, rows, hq, hkv, d, bs, qt, out, seed=0, scale=None, change=None, **kw):
    c = ScaledCache(lens, hkv, d, bs, seed, **kw)
    if change:
        change(c)
    q = queries(sum(rows), hq, d, qt, seed + 1)
    scale = d ** -0.5 if scale is None else scale
    o, cu = run_chunks(pa, c, q, rows, scale, out)
    for i, (n, r) in enumerate(zip(lens, rows)):
        want, bound = attend(q[cu[i]:cu[i + 1]], c.rows("k", i, n), c.rows("v", i, n), causal(n, r), scale, out, True)
        check(o[cu[i]:cu[i + 1]], want, bound, f"chunk {i}: {r} of {n} tokens")


HEADS = [(4, 4, 64, 16), (16, 2, 64, 32), (32, 2, 64, 16), (17, 1, 64, 16), (5, 5, 128, 16), (10, 2, 128, 32), (16, 2, 128, 32),
         (32, 2, 128, 16), (40, 2, 128, 16), (19, 1, 128, 32)]


@pytest.mark.parametrize("qt,out", OUT)
@pytest.mark.parametrize("hq,hkv,d,bs", HEADS)
def test_decode_heads_and_types(hq, hkv, d, bs, qt, out):
    decode_case(LENS, hq, hkv, d, bs, qt, out, seed=hq + d)


@pytest.mark.parametrize("n", [1, 2, 3, 7, 64, 300, 1100, 2500])
def test_decode_numbers_of_rows(n):
    """From rows cut into many pieces to many rows in one piece, past the rows a CTA has at hand at a time."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 6000 // n + 40, (n,), generator=g).tolist()
    decode_case(lens, 4, 2, 64, 16, "bf16", "f32", seed=n)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_one_long_row_and_empty_rows(d):
    decode_case([9001], 8, 2, d, 32, "bf16", "bf16", seed=d)
    decode_case([0, 5, 0, 600], 8, 2, d, 16, "bf16", "f32", seed=d + 1)


def test_decode_many_rows():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(1, 900, (160,), generator=g).tolist()
    decode_case(lens, 8, 2, 128, 16, "bf16", "bf16", seed=9)


@pytest.mark.parametrize("qt,out", OUT)
@pytest.mark.parametrize("hq,hkv,d,bs", HEADS)
def test_chunk_heads_and_types(hq, hkv, d, bs, qt, out):
    chunk_case([1, 40, 129, 300], [1, 33, 129, 100], hq, hkv, d, bs, qt, out, seed=hq + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qt,out", OUT)
def test_chunks_two_ctas_per_sm(d, qt, out):
    chunk_case([900, 701, 640], [900, 300, 640], 32, 4, d, 16, qt, out, seed=d)


@pytest.mark.parametrize("qt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_chunks_of_many_key_tiles(qt, out):
    """Scales come by groups of key tiles: sequences that end in every part of a group, two query tiles per CTA."""
    chunk_case([2600, 1025, 1600, 1100], [500, 300, 200, 300], 32, 4, 64, 16, qt, out, seed=21)


def test_chunk_far_into_a_context():
    chunk_case([6000], [130], 8, 2, 128, 32, "bf16", "f32", seed=3)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("scale", [0.0, -0.09, 0.7])
def test_softmax_scales(case, scale):
    if case == "decode":
        decode_case(LENS, 8, 2, 128, 16, "bf16", "f32", seed=4, scale=scale)
    else:
        chunk_case([300, 77], [200, 77], 8, 2, 128, 16, "bf16", "f32", seed=4, scale=scale)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("spread,powers", [(0.0, True), (6.0, True), (4.0, False)])
def test_spread_of_scales(case, spread, powers):
    for qt, out in OUT:
        if case == "decode":
            decode_case(LENS, 8, 2, 128, 16, qt, out, seed=6, spread=spread, powers=powers)
        else:
            chunk_case([300, 77, 500], [200, 77, 30], 8, 2, 64, 16, qt, out, seed=6, spread=spread, powers=powers)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("small,large", [(-64, 0), (-30, 0), (-64, 32), (0, 32)])
def test_heavy_tokens_with_small_values(case, small, large):
    """The tokens that hold most of the softmax have the smallest values: their weight must not be lost from the sum,
    where their weight times V's scale is far below the others'."""
    def change(c):
        for i, n in enumerate(c.lens):
            nb = -(-n // c.bs)
            b = c.tables[i, :nb].long()
            heavy = torch.arange(nb) % 3 == 0
            c.vs[b] = torch.where(heavy, 2.0 ** small, 2.0 ** large)[:, None].expand(-1, c.hkv).float()
            c.ks[b] = torch.where(heavy, 2.0 ** -5, 2.0 ** -9)[:, None].expand(-1, c.hkv).float()
    if case == "decode":
        decode_case([40, 300, 1537], 8, 2, 128, 16, "bf16", "f32", seed=7, change=change)
    else:
        chunk_case([40, 300, 1000], [40, 100, 200], 8, 2, 128, 16, "bf16", "f32", seed=7, change=change)


@pytest.mark.parametrize("case", ["decode", "chunk"])
def test_far_blocks(case):
    if case == "decode":
        decode_case([700, 33], 64, 8, 128, 32, "bf16", "bf16", seed=8, far=True)
    else:
        chunk_case([700, 33], [100, 33], 64, 8, 128, 32, "bf16", "bf16", seed=8, far=True)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("bad", [0.0, -1.0, float("nan"), float("inf"), 2.0 ** 33, 2.0 ** -65])
def test_bad_scales_are_reported(case, bad):
    c = ScaledCache([100, 300], 2, 128, 16, 11)
    c.vs[int(c.tables[1, 7]), 1] = bad
    k, v, tables, desc, ks, vs = c.device(pa)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    if case == "decode":
        q = queries(2, 8, 128, "bf16", 12)
        o = torch.empty_like(q, device="cuda")
        ws = torch.empty(pa.pa_decode_scaled_workspace_bytes(2, 8, 2, 128, 300), dtype=torch.uint8, device="cuda")
        pa.pa_decode_scaled(q.cuda(), k, v, desc, ks, vs, tables, lens, 300, 0.1, o, ws)
        rows = [(0, 1)]
    else:
        q = queries(120, 8, 128, "bf16", 12)
        o = torch.empty_like(q, device="cuda")
        cu, start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 20, 120], [80, 200]))
        pa.pa_prefill_chunk_scaled(q.cuda(), cu, start, 100, k, v, desc, ks, vs, tables, lens, 300, 0.1, o)
        rows = [(0, 20)]
    assert pa.pa_get_device_error() == 4
    for a, b in rows:                                  # the other sequence is served
        want, bound = attend(q[a:b], c.rows("k", 0, 100), c.rows("v", 0, 100), causal(100, b - a), 0.1, "bf16", case == "chunk")
        check(o[a:b], want, bound, "the other sequence")


@pytest.mark.parametrize("case", ["decode", "chunk"])
def test_same_bits_twice_and_on_a_stream(case):
    c = ScaledCache([700, 1, 64, 350], 2, 128, 16, 13)
    s = torch.cuda.Stream()
    if case == "decode":
        q = queries(4, 16, 128, "bf16", 14)
        a, b = run_decode(pa, c, q, 0.1, "bf16"), run_decode(pa, c, q, 0.1, "bf16")
        torch.cuda.synchronize()
        d = run_decode(pa, c, q, 0.1, "bf16", stream=s)
    else:
        q = queries(400, 16, 128, "bf16", 14)
        rows = [300, 1, 64, 35]
        a, b = run_chunks(pa, c, q, rows, 0.1, "bf16")[0], run_chunks(pa, c, q, rows, 0.1, "bf16")[0]
        torch.cuda.synchronize()
        d = run_chunks(pa, c, q, rows, 0.1, "bf16", stream=s)[0]
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and torch.equal(a.view(torch.uint8), d.view(torch.uint8))


@pytest.mark.parametrize("hq,hkv", [(128, 1), (64, 1), (66, 2)])
def test_wide_groups(hq, hkv):
    """Groups of more query heads than a share has."""
    for d, bs in ((64, 32), (128, 16)):
        decode_case([1, 300, 40], hq, hkv, d, bs, "bf16", "f32", seed=hq + d)
        chunk_case([1, 300, 40], [1, 20, 40], hq, hkv, d, bs, "f16", "f16", seed=hq + d)


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("bad", [-1, 1 << 29])
def test_bad_blocks_are_reported(case, bad):
    """A block id out of range where a token is: an error, nothing read there, the other sequences served."""
    c = ScaledCache([100, 300, 70], 2, 128, 16, 15)
    c.tables[1, 7] = bad
    k, v, tables, desc, ks, vs = c.device(pa)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    if case == "decode":
        q = queries(3, 8, 128, "bf16", 16)
        o = torch.empty_like(q, device="cuda")
        ws = torch.empty(pa.pa_decode_scaled_workspace_bytes(3, 8, 2, 128, 300), dtype=torch.uint8, device="cuda")
        pa.pa_decode_scaled(q.cuda(), k, v, desc, ks, vs, tables, lens, 300, 0.1, o, ws)
        rows = [(0, 0, 1), (2, 2, 3)]
    else:
        q = queries(140, 8, 128, "bf16", 16)
        o = torch.empty_like(q, device="cuda")
        cu, start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 20, 120, 140], [80, 200, 50]))
        pa.pa_prefill_chunk_scaled(q.cuda(), cu, start, 100, k, v, desc, ks, vs, tables, lens, 300, 0.1, o)
        rows = [(0, 0, 20), (2, 120, 140)]
    assert pa.pa_get_device_error() == 4
    for i, a, b in rows:
        n = c.lens[i]
        want, bound = attend(q[a:b], c.rows("k", i, n), c.rows("v", i, n), causal(n, b - a), 0.1, "bf16", case == "chunk")
        check(o[a:b], want, bound, f"sequence {i}")


@pytest.mark.parametrize("length", [-3, 301, 1 << 30])
def test_bad_lengths_are_reported(length):
    """A decode length below 0 or beyond max_seq_len: an error, cut to what is there, the other sequences served."""
    c = ScaledCache([100, 300, 70], 2, 128, 16, 17)
    k, v, tables, desc, ks, vs = c.device(pa)
    lens = torch.tensor([100, length, 70], dtype=torch.int32, device="cuda")
    q = queries(3, 8, 128, "bf16", 18)
    o = torch.empty_like(q, device="cuda")
    ws = torch.empty(pa.pa_decode_scaled_workspace_bytes(3, 8, 2, 128, 300), dtype=torch.uint8, device="cuda")
    pa.pa_decode_scaled(q.cuda(), k, v, desc, ks, vs, tables, lens, 300, 0.1, o, ws)
    assert pa.pa_get_device_error() == 4
    for i, n in ((0, 100), (1, 0 if length < 0 else 300), (2, 70)):
        want, bound = attend(q[i:i + 1], c.rows("k", i, n), c.rows("v", i, n), causal(n, 1), 0.1, "bf16", False)
        check(o[i:i + 1], want, bound, f"sequence {i}")


def test_calls_without_rows():
    c = ScaledCache([20], 2, 128, 16, 19)
    k, v, tables, desc, ks, vs = c.device(pa)
    none = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    some = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_decode_scaled(none, k, v, desc, ks, vs, tables[:0], some[:0], 0, 0.1, none)
    pa.pa_prefill_chunk_scaled(none, some, some[:0], 0, k, v, desc, ks, vs, tables[:0], some[:0], 0, 0.1, none)
    row = torch.full((1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = row.clone()                                  # (a chunk without rows; the row behind it is no chunk's)
    pa.pa_prefill_chunk_scaled(row, torch.cat([some, some]), some, 5, k, v, desc, ks, vs, tables, some, 20, 0.1, out)
    assert torch.equal(out, row)
    x = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    pa.pa_rope_and_cache(None, x, x, None, None, torch.empty(0, dtype=torch.int64, device="cuda"), k, v, desc, k_scales=ks, v_scales=vs)
    pa.pa_copy_blocks_scaled(k, v, desc, ks, vs, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert pa.pa_get_device_error() == 0
