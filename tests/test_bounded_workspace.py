"""Workspace sizes of the bounded-cache decodes: one that is large enough for a batch is large enough for every smaller one, of
fewer sequences, shorter ones or a smaller window, as a serving loop keeps one workspace for all its steps."""
import itertools

import pytest

import paged_kv_cache_writes_gb300 as pa

SEQS = [0, 1, 2, 3, 5, 9, 10, 18, 19, 20, 37, 38, 39, 75, 76, 77, 128, 129, 300]
LENS = [0, 1, 63, 64, 65, 512, 513, 1000, 1024, 1216, 1217, 4864, 4865, 9728, 9729, 40000]
HEADS = [(1, 1, 128), (8, 2, 128), (32, 8, 128), (40, 2, 128), (128, 4, 64), (64, 64, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("ps", [0, 32, 96, 512, 1024])
def test_decode_weights_workspace_grows(hq, hkv, d, ps):
    size = {(n, m): pa.pa_decode_weights_workspace_bytes(n, hq, hkv, d, m, ps) for n, m in itertools.product(SEQS, LENS)}
    for i, j in itertools.product(range(len(SEQS)), range(len(LENS))):
        here = size[SEQS[i], LENS[j]]
        assert here > 0 or SEQS[i] == 0
        assert i == 0 or here >= size[SEQS[i - 1], LENS[j]], (SEQS[i], LENS[j])
        assert j == 0 or here >= size[SEQS[i], LENS[j - 1]], (SEQS[i], LENS[j])


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("bs", [16, 32])
def test_decode_window_workspace_grows(hq, hkv, d, bs):
    windows, sinks = [1, 16, 100, 1000, 1025, 4096, 100000, 2 ** 31 - 1], [0, 1, 33, 1000]
    for n, m in itertools.product(SEQS, LENS):
        at = [[pa.pa_decode_window_workspace_bytes(n, hq, hkv, d, bs, m, w, s) for s in sinks] for w in windows]
        for i, row in enumerate(at):
            assert row == sorted(row), (n, m, windows[i])
            assert i == 0 or all(x >= y for x, y in zip(row, at[i - 1])), (n, m, windows[i])
    for w, s in itertools.product((100, 5000), (0, 33)):
        for m in LENS:
            row = [pa.pa_decode_window_workspace_bytes(n, hq, hkv, d, bs, m, w, s) for n in SEQS]
            assert row == sorted(row), (m, w, s)
        for n in SEQS:
            row = [pa.pa_decode_window_workspace_bytes(n, hq, hkv, d, bs, m, w, s) for m in LENS]
            assert row == sorted(row), (n, w, s)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2)])
def test_sizes_near_the_limits_of_a_partition(hq, hkv):
    """Every number of sequences and every length around the places where rows are cut differently."""
    sizes = [pa.pa_decode_weights_workspace_bytes(n, hq, hkv, 128, 1300) for n in range(0, 160)]
    assert sizes == sorted(sizes)
    for n in (1, 2, 7, 76 // hkv):
        sizes = [pa.pa_decode_weights_workspace_bytes(n, hq, hkv, 128, m) for m in range(0, 3000)]
        assert sizes == sorted(sizes)
        sizes = [pa.pa_decode_window_workspace_bytes(n, hq, hkv, 128, 16, m, 1500, 4) for m in range(0, 3000)]
        assert sizes == sorted(sizes)


@pytest.mark.gpu
def test_one_workspace_for_every_batch():
    """A loop whose batch and contexts shrink, on one workspace sized for its largest step."""
    import torch
    from _bounded import Cache, attend, check, visible

    lens = [1200 - 13 * i for i in range(40)]
    c = Cache(lens, 1, 128, 16, "bf16", 3)
    k, v, tables, desc = c.device(pa)
    q = torch.randn((40, 4, 128), generator=torch.Generator().manual_seed(4)).bfloat16()
    size = pa.pa_decode_window_workspace_bytes(40, 4, 1, 128, 16, 1200, 1000, 4)
    size_w = pa.pa_decode_weights_workspace_bytes(40, 4, 1, 128, 1200)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    ws_w = torch.empty(size_w, dtype=torch.uint8, device="cuda")
    for n, cut in ((40, 0), (38, 0), (37, 300), (19, 0), (18, 600), (9, 100), (3, 0), (2, 500), (1, 0), (1, 1100)):
        now = [m - cut for m in lens[:n]]
        now = [max(1, m) for m in now]
        sl = torch.tensor(now, dtype=torch.int32, device="cuda")
        o = torch.empty((n, 4, 128), device="cuda")
        ow, w = torch.empty_like(o), torch.zeros((n, 1, max(now)), device="cuda")
        pa.pa_decode_window(q[:n].cuda(), k, v, desc, tables[:n].contiguous(), sl, max(now), 1000, 4, 0.09, o, ws)
        pa.pa_decode_weights(q[:n].cuda(), k, v, desc, tables[:n].contiguous(), sl, max(now), 0.09, ow, w, workspace=ws_w)
        assert pa.pa_get_device_error() == 0
        for i in (0, n // 2, n - 1):
            m = now[i]
            for got, window in ((o, 1000), (ow, m)):
                ref, bound, _, _ = attend(q[i:i + 1], c.rows("k", i, m), c.rows("v", i, m), visible(m - 1, m, window, 4)[None], 0.09,
                                          "bf16", "f32")
                check(got[i:i + 1], ref, bound, f"{n} sequences, row {i}")
