"""pa_decode_weights on the GPU: the attention output and the accumulated attention weights against the 64-bit form,
within derived bounds (tests/_bounded.py); a running weight adds one fp32 rounding (and the decay's)."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import Cache, DT, attend, check

pytestmark = pytest.mark.gpu

LENS = [1, 15, 16, 33, 127, 128, 130, 511, 513, 700, 1537]


def weights_case(lens, hq, hkv, d, bs, qt, kv, seed=0, out="f32", ps=0, decay=1.0, fresh=None, rows=None, pad=0, **kw):
    c = Cache(lens, hkv, d, bs, kv, seed, **kw)
    g = torch.Generator().manual_seed(seed + 1)
    n, most = len(lens), max(lens)
    q = (1.5 * torch.randn((n, hq, d), generator=g)).to(DT[qt])
    held = max(rows) + 2 if rows else n
    old = torch.rand((held, hkv, most + pad), generator=g) * 3
    # what stands for tokens without a running weight is never read
    start = [m - 1 for m in lens] if fresh is None else fresh
    at = list(range(n)) if rows is None else rows
    for i, m in enumerate(lens):
        old[at[i], :, max(0, start[i]):m] = float("nan")
    k, v, tables, desc = c.device(pa)
    w = old.cuda()
    o = torch.full(q.shape, float("nan"), dtype=DT[out], device="cuda")
    size = pa.pa_decode_weights_workspace_bytes(n, hq, hkv, d, most, ps)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pa.pa_decode_weights(q.cuda(), k, v, desc, tables, i32(lens), most, d ** -0.5, o, w, i32(rows), i32(fresh), decay, ws, ps)
    assert pa.pa_get_device_error() == 0
    left = torch.ones(old.shape, dtype=bool)
    for i, m in enumerate(lens):
        if m == 0:
            assert (o[i] == 0).all()
            continue
        ref, bound, a, rel = attend(q[i:i + 1], c.rows("k", i, m), c.rows("v", i, m), torch.ones((1, m), dtype=bool), d ** -0.5, kv, out,
                                     p_terms=3 if qt == "f16" else 2)
        check(o[i:i + 1], ref, bound, f"output of sequence {i}")
        a, rel = a[0].view(hkv, hq // hkv, m), rel[0].view(hkv, hq // hkv, 1)
        before = torch.where(torch.arange(m) < start[i], old[at[i], :, :m].double() * decay, 0.0)
        want = before + a.sum(1)
        tol = (a * rel).sum(1) + 2.0 ** -24 * (hq // hkv + 2) * (want.abs() + before.abs()) + 1e-38
        check(w[at[i], :, :m], want, tol, f"weights of sequence {i} of {m} tokens")
        left[at[i], :, :m] = False
    assert torch.equal(w.cpu()[left].view(torch.int32), old[left].view(torch.int32))   # everything else untouched


@pytest.mark.parametrize("qt,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "fp8"), ("f16", "fp8")])
@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 4, 64, 16), (16, 2, 64, 32), (32, 2, 64, 16), (17, 1, 64, 16), (5, 5, 128, 16),
                                         (10, 2, 128, 32), (32, 2, 128, 16), (40, 2, 128, 16), (19, 1, 128, 32)])
def test_heads_and_types(qt, kv, hq, hkv, d, bs):
    weights_case(LENS, hq, hkv, d, bs, qt, kv, seed=hq + d)


@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("ps", [0, 32, 96])
def test_decay_and_partitions(decay, ps):
    weights_case(LENS, 8, 2, 128, 16, "bf16", "bf16", seed=ps, ps=ps, decay=decay)


def test_no_decayed_weight_is_read():
    """decay 0: whatever stands for the running weights (NaN, infinities) leaves nothing behind."""
    c = Cache([700, 33], 2, 128, 16, "bf16", 14)
    k, v, tables, desc = c.device(pa)
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    lens = torch.tensor([700, 33], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([650, 33], dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(2, 8, 2, 128, 700), dtype=torch.uint8, device="cuda")
    got = []
    for stale in (0.0, float("nan"), float("inf")):
        w = torch.full((2, 2, 700), stale, device="cuda")
        pa.pa_decode_weights(q, k, v, desc, tables, lens, 700, 0.09, torch.empty_like(q), w, None, fresh, 0.0, ws)
        got.append([w[0].cpu(), w[1, :, :33].cpu()])
    assert pa.pa_get_device_error() == 0
    for g in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(g, got[0]))


def test_fresh_tokens():
    weights_case([40, 700, 130, 5], 8, 2, 128, 16, "bf16", "bf16", seed=3, fresh=[0, 300, 130, 4])


def test_named_rows_and_padded_strides():
    weights_case([40, 700, 0, 5], 8, 2, 128, 32, "bf16", "bf16", seed=4, rows=[5, 0, 3, 1], pad=13)


def test_per_head_scales():
    weights_case(LENS, 8, 4, 128, 16, "bf16", "fp8", seed=5, per_head=True)


def test_long_sequence():
    weights_case([9001], 16, 2, 128, 16, "bf16", "bf16", seed=6, out="bf16")


def test_batches_past_the_direct_launch():
    g = torch.Generator().manual_seed(1)
    weights_case(torch.randint(0, 90, (140,), generator=g).tolist(), 4, 2, 64, 16, "bf16", "bf16", seed=8)
    weights_case([3000, 5, 2900, 700] * 8, 16, 8, 64, 16, "f16", "f16", seed=9)


def test_blocks_past_32_bit_offsets():
    weights_case([40, 700], 8, 2, 128, 16, "bf16", "bf16", seed=11, far=True)


def test_shared_blocks():
    """Two sequences over the same blocks each have weights of their own."""
    c = Cache([300], 2, 128, 16, "bf16", 8)
    k, v, tables, desc = c.device(pa)
    tables = tables.repeat(2, 1).contiguous()
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(1)).bfloat16()
    lens = torch.tensor([300, 211], dtype=torch.int32, device="cuda")
    w = torch.zeros((2, 2, 300), device="cuda")
    o = torch.empty((2, 8, 128), dtype=torch.float32, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(2, 8, 2, 128, 300), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        pa.pa_decode_weights(q.cuda(), k, v, desc, tables, lens, 300, 0.09, o, w, workspace=ws)
    assert pa.pa_get_device_error() == 0
    for i, n in enumerate((300, 211)):
        _, _, a, rel = attend(q[i:i + 1], c.rows("k", 0, n), c.rows("v", 0, n), torch.ones((1, n), dtype=bool), 0.09, "bf16", "f32")
        a, rel = a[0].view(2, 4, n), rel[0].view(2, 4, 1)
        times = torch.where(torch.arange(n) < n - 1, 2.0, 1.0)      # the last token's running weight starts anew
        check(w[i, :, :n], times * a.sum(1), times * (a * rel).sum(1) + 1e-6 * a.sum(1) + 1e-38, f"sequence {i}")
        assert (w[i, :, n:] == 0).all()


def test_bad_rows_are_reported_and_skipped():
    c = Cache([50, 60], 2, 64, 16, "f16", 9)
    k, v, tables, desc = c.device(pa)
    q = torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda")
    w = torch.full((2, 2, 60), 3.0, device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(2, 4, 2, 64, 60), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([50, 60], dtype=torch.int32, device="cuda")
    rows = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    pa.pa_decode_weights(q, k, v, desc, tables, lens, 60, 0.1, torch.empty_like(q), w, rows, None, 1.0, ws)
    assert pa.pa_get_device_error() == 4
    assert (w[1] == 3.0).all() and (w[0] != 3.0).all()
