"""Sliding-window attention with first tokens that stay visible, on the GPU: pa_decode_window and
pa_prefill_chunk_window against the 64-bit form over the visible tokens, within bounds derived from their arithmetic
(tests/_bounded.py).  Tokens that are not visible hold NaN and infinity, and the block-table entries of blocks without a
visible token are -1."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import Cache, DT, attend, check, visible

pytestmark = pytest.mark.gpu

LENS = [1, 15, 16, 33, 127, 128, 130, 511, 513, 700, 1537]


def decode(c, q, window, sinks, scale, out="f32", ps=0, stream=None):
    k, v, tables, desc = c.device(pa)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    most = max(c.lens, default=0)
    n, hq, d = q.shape
    size = pa.pa_decode_window_workspace_bytes(n, hq, c.hkv, d, c.bs, most, window, sinks, ps)
    assert size > 0
    ws = torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda")
    o = torch.full(q.shape, float("nan"), dtype=DT[out], device="cuda")
    pa.pa_decode_window(q.cuda(), k, v, desc, tables, lens, most, window, sinks, scale, o, ws, ps, stream=stream)
    assert pa.pa_get_device_error() == 0
    return o


def decode_case(lens, hq, hkv, d, bs, qt, kv, window, sinks, seed=0, out="f32", ps=0, scale=None, **kw):
    c = Cache(lens, hkv, d, bs, kv, seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    q = (1.5 * torch.randn((len(lens), hq, d), generator=g)).to(DT[qt])
    scale = d ** -0.5 if scale is None else scale
    want = []
    for i, n in enumerate(lens):
        seen = visible(n - 1, n, window, sinks)
        want.append(attend(q[i:i + 1], c.rows("k", i, n), c.rows("v", i, n), seen[None], scale, kv, out, p_terms=3 if qt == "f16" else 2))
        c.poison(i, ~seen)
    o = decode(c, q, window, sinks, scale, out, ps)
    for i in range(len(lens)):
        check(o[i:i + 1], want[i][0], want[i][1], f"sequence {i} of {lens[i]} tokens")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 16), (100, 17), (128, 0), (1000, 33), (100000, 5)])
@pytest.mark.parametrize("bs", [16, 32])
def test_decode_windows(window, sinks, bs):
    decode_case(LENS, 8, 2, 128, bs, "bf16", "bf16", window, sinks, seed=window + bs)


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 4, 64, 16), (16, 2, 64, 32), (32, 2, 64, 16), (17, 1, 64, 16), (5, 5, 128, 16),
                                         (10, 2, 128, 32), (32, 2, 128, 16), (40, 2, 128, 16), (19, 1, 128, 32)])
def test_decode_heads_and_types(qt, kv, hq, hkv, d, bs):
    decode_case(LENS, hq, hkv, d, bs, qt, kv, 90, 5, seed=hq + d)


@pytest.mark.parametrize("ps", [32, 64, 96, 512, 1024])
def test_decode_partitions_inside_the_cut(ps):
    # partitions of 32 tokens can lie entirely between the last first token and the window's start
    for sinks, window in ((0, 1), (1, 70), (17, 17), (31, 33), (33, 300)):
        decode_case([64, 95, 400, 777], 8, 2, 128, 32, "bf16", "bf16", window, sinks, seed=ps + sinks, ps=ps)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_decode_output_types_and_negative_scale(out):
    decode_case(LENS, 8, 2, 128, 16, "bf16", "bf16", 64, 4, seed=3, out=out, scale=-0.05)


def test_decode_per_head_scales():
    decode_case(LENS, 8, 4, 128, 16, "bf16", "fp8", 64, 4, seed=5, per_head=True)


def test_decode_empty_sequences():
    c = Cache([0, 40, 0], 2, 128, 16, "bf16", 1)
    q = torch.randn((3, 8, 128), generator=torch.Generator().manual_seed(2)).bfloat16()
    o = decode(c, q, 10, 2, 0.1)
    assert (o[0] == 0).all() and (o[2] == 0).all() and (o[1] != 0).any()


def test_decode_without_a_cut_agrees_with_pa_decode():
    # the two cut rows into partitions of their own: each is within its bound of the exact result
    c = Cache(LENS, 2, 128, 16, "bf16", 7)
    q = torch.randn((len(LENS), 16, 128), generator=torch.Generator().manual_seed(8)).bfloat16().cuda()
    o = decode(c, q.cpu(), 2 ** 31 - 1, 0, 0.09)
    k, v, tables, desc = c.device(pa)
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.pa_decode_workspace_bytes(len(LENS), 16, 2, 128, max(LENS)), dtype=torch.uint8, device="cuda")
    ref = torch.empty((len(LENS), 16, 128), dtype=torch.float32, device="cuda")
    pa.pa_decode(q, k, v, desc, tables, lens, max(LENS), 0.09, ref, ws)
    for i, n in enumerate(LENS):
        _, bound, _, _ = attend(q[i:i + 1].cpu(), c.rows("k", i, n), c.rows("v", i, n), torch.ones((1, n), dtype=bool), 0.09, "bf16", "f32")
        assert ((o[i:i + 1].double() - ref[i:i + 1].double()).abs().cpu() <= 2 * bound).all()


def test_decode_batches_past_the_direct_launch():
    # more rows than a scheduler warp deals itself, and more units than fit: the plan kernel's path
    g = torch.Generator().manual_seed(1)
    decode_case(torch.randint(0, 90, (140,), generator=g).clamp(min=1).tolist(), 4, 2, 64, 16, "bf16", "bf16", 33, 3, seed=8)
    decode_case([3000, 5, 2900, 700] * 8, 16, 8, 64, 16, "bf16", "bf16", 2500, 9, seed=9)


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("bf16", "fp8")])
def test_blocks_past_32_bit_offsets(qt, kv):
    decode_case([40, 700], 8, 2, 128, 16, qt, kv, 90, 5, seed=11, far=True)
    chunk_case([(300, 130), (0, 77)], 8, 2, 128, 16, qt, kv, 90, 5, seed=12, far=True)


def test_decode_bad_metadata_is_reported():
    c = Cache([100, 50], 2, 128, 16, "bf16", 9)
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    c.tables[1, 3] = c.num_blocks          # block of the last tokens
    k, v, tables, desc = c.device(pa)
    lens = torch.tensor([100, 50], dtype=torch.int32, device="cuda")
    o = torch.zeros((2, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(pa.pa_decode_window_workspace_bytes(2, 4, 2, 128, 16, 100, 20, 0), dtype=torch.uint8, device="cuda")
    pa.pa_decode_window(q.cuda(), k, v, desc, tables, lens, 100, 20, 0, 0.1, o, ws)
    assert pa.pa_get_device_error() == 4
    lens[0] = -3
    tables[1, 3] = 0
    pa.pa_decode_window(q.cuda(), k, v, desc, tables, lens, 100, 20, 0, 0.1, o, ws)
    assert pa.pa_get_device_error() == 4
    assert pa.pa_get_device_error() == 0


def chunk_case(chunks, hq, hkv, d, bs, qt, kv, window, sinks, seed=0, out="f32", scale=None, **kw):
    """chunks: (start, rows) pairs."""
    lens = [s + r for s, r in chunks]
    c = Cache(lens, hkv, d, bs, kv, seed, **kw)
    total = sum(r for _, r in chunks)
    g = torch.Generator().manual_seed(seed + 1)
    q = (1.5 * torch.randn((total, hq, d), generator=g)).to(DT[qt])
    scale = d ** -0.5 if scale is None else scale
    want, cu = [], [0]
    for i, (s, r) in enumerate(chunks):
        n = s + r
        seen = torch.stack([visible(s + x, n, window, sinks) for x in range(r)]) if r else torch.zeros((0, n), dtype=bool)
        if r:
            want.append(attend(q[cu[-1]:cu[-1] + r], c.rows("k", i, n), c.rows("v", i, n), seen, scale, kv, out, prefill=True))
        else:
            want.append(None)
        c.poison(i, ~seen.any(0))
        cu.append(cu[-1] + r)
    k, v, tables, desc = c.device(pa)
    o = torch.full((total + 3, hq, d), 7.0, dtype=DT[out], device="cuda")
    pa.pa_prefill_chunk_window(q.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                               torch.tensor([s for s, _ in chunks], dtype=torch.int32, device="cuda"),
                               max(r for _, r in chunks), k, v, desc, tables,
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens), window, sinks, scale, o[:total])
    assert pa.pa_get_device_error() == 0
    for i, (s, r) in enumerate(chunks):
        if r:
            check(o[cu[i]:cu[i] + r], want[i][0], want[i][1], f"chunk {i}: {r} rows at {s}")
    assert (o[total:] == 7.0).all()          # rows behind the last chunk


CHUNKS = [(0, 1), (0, 77), (300, 130), (1000, 1), (517, 40), (64, 0)]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 16), (100, 17), (128, 0), (400, 33), (100000, 5)])
@pytest.mark.parametrize("bs", [16, 32])
def test_chunk_windows(window, sinks, bs):
    chunk_case(CHUNKS, 8, 2, 128, bs, "bf16", "bf16", window, sinks, seed=window + bs)


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("hq,hkv,d,bs", [(2, 2, 64, 16), (16, 2, 64, 32), (9, 1, 64, 16), (5, 5, 128, 32), (10, 2, 128, 16),
                                         (32, 2, 128, 16), (130, 1, 64, 32)])
def test_chunk_heads_and_types(qt, kv, hq, hkv, d, bs):
    chunk_case(CHUNKS, hq, hkv, d, bs, qt, kv, 90, 5, seed=hq + d)


@pytest.mark.parametrize("qt,kv,d", [("bf16", "bf16", 128), ("f16", "f16", 64), ("bf16", "fp8", 128), ("f16", "fp8", 64)])
def test_chunk_two_tiles_per_cta(qt, kv, d):
    # enough rows that every SM has a CTA of two Q tiles
    chunk_case([(200, 900), (0, 1000), (37, 513)], 32, 8, d, 16, qt, kv, 250, 9, seed=d)


@pytest.mark.parametrize("qt,kv,out", [("bf16", "bf16", "f32"), ("bf16", "bf16", "bf16"), ("f16", "f16", "f32"), ("bf16", "fp8", "f32")])
@pytest.mark.parametrize("d,hkv", [(128, 2), (128, 8), (64, 8)])
def test_chunk_last_tiles_of_every_length(qt, kv, out, d, hkv):
    # the last tile's keys: 1 to 128, with few CTAs and with two per SM; what an earlier launch left behind them is no score
    ends = [1, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 79, 80, 96, 97, 111, 112, 113, 127, 128, 129, 144, 161]
    chunk_case([(max(0, n - 9), min(n, 9)) for n in ends], 2 * hkv, hkv, d, 16, qt, kv, 100, 3, seed=d + hkv, out=out)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_chunk_output_types_and_negative_scale(out):
    chunk_case(CHUNKS, 8, 2, 128, 16, "bf16", "bf16", 64, 4, seed=3, out=out, scale=-0.05)


def test_chunk_of_scale_zero_takes_the_mean():
    chunk_case(CHUNKS, 8, 2, 128, 16, "bf16", "bf16", 64, 4, seed=6, scale=0.0)
    chunk_case(CHUNKS, 8, 2, 64, 32, "bf16", "fp8", 64, 4, seed=7, scale=0.0)


def test_chunk_per_head_scales():
    chunk_case(CHUNKS, 8, 4, 128, 16, "bf16", "fp8", 64, 4, seed=5, per_head=True)


def test_chunk_of_one_row_agrees_with_decode():
    n, window, sinks = 700, 120, 7
    c = Cache([n], 2, 128, 16, "bf16", 21)
    q = torch.randn((1, 8, 128), generator=torch.Generator().manual_seed(22)).bfloat16()
    a = decode(c, q, window, sinks, 0.09)
    k, v, tables, desc = c.device(pa)
    o = torch.empty((1, 8, 128), dtype=torch.float32, device="cuda")
    pa.pa_prefill_chunk_window(q.cuda(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                               torch.tensor([n - 1], dtype=torch.int32, device="cuda"), 1, k, v, desc, tables,
                               torch.tensor([n], dtype=torch.int32, device="cuda"), n, window, sinks, 0.09, o)
    _, bound, _, _ = attend(q, c.rows("k", 0, n), c.rows("v", 0, n), visible(n - 1, n, window, sinks)[None], 0.09, "bf16", "f32")
    assert ((a.double() - o.double()).abs().cpu() <= 2 * bound).all()
