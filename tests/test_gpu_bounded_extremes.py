"""The bounded-cache calls where their bounds are far from what a batch holds, and in batches of very many sequences."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import Cache, attend, check, evict, visible

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.int16).cpu()


@pytest.mark.parametrize("n,most", [(3, 200000), (3, 1 << 20), (40, 100000), (200, 30000)])
def test_decodes_under_a_bound_far_above_the_lengths(n, most):
    """max_seq_len promises many partitions a row (with few sequences, and past the direct launch); the lengths need few."""
    lens = [1 + (37 * i) % 700 for i in range(n)]
    c = Cache(lens, 2, 64, 16, "bf16", n)
    k, v, tables, desc = c.device(pa)
    q = torch.randn((n, 6, 64), generator=torch.Generator().manual_seed(n)).bfloat16()
    o, ow = (torch.full((n, 6, 64), float("nan"), device="cuda") for _ in range(2))
    w = torch.full((n, 2, most), 7.0, device="cuda")
    ws = torch.full((pa.pa_decode_window_workspace_bytes(n, 6, 2, 64, 16, most, 90000, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    pa.pa_decode_window(q.cuda(), k, v, desc, tables, i32(lens), most, 90000, 4, 0.125, o, ws)
    ws = torch.full((pa.pa_decode_weights_workspace_bytes(n, 6, 2, 64, most),), 0xFF, dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(q.cuda(), k, v, desc, tables, i32(lens), most, 0.125, ow, w, None, i32([0] * n), 1.0, ws)
    assert pa.pa_get_device_error() == 0
    for i, m in enumerate(lens):
        ref, bound, a, rel = attend(q[i:i + 1], c.rows("k", i, m), c.rows("v", i, m), torch.ones((1, m), dtype=bool), 0.125, "bf16", "f32")
        check(o[i:i + 1], ref, bound, f"window, sequence {i}")
        check(ow[i:i + 1], ref, bound, f"weights, sequence {i}")
        a, rel = a[0].view(2, 3, m), rel[0].view(2, 3, 1)
        check(w[i, :, :m], a.sum(1), (a * rel).sum(1) + 2.0 ** -24 * 5 * a.sum(1) + 1e-38, f"weights of sequence {i}")
        assert (w[i, :, m:] == 7.0).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("max_q", [41, 130, 5000])
def test_chunks_under_a_bound_far_above_their_rows(kv, max_q):
    chunks = [(0, 1), (300, 41), (17, 30), (64, 0), (900, 7)]
    lens = [s + r for s, r in chunks]
    c = Cache(lens, 2, 128, 16, kv, 5)
    k, v, tables, desc = c.device(pa)
    total = sum(r for _, r in chunks)
    q = torch.randn((total, 8, 128), generator=torch.Generator().manual_seed(6)).bfloat16()
    cu = [0]
    for _, r in chunks:
        cu.append(cu[-1] + r)
    o = torch.full((total + 9, 8, 128), 7.0, device="cuda")
    pa.pa_prefill_chunk_window(q.cuda(), i32(cu), i32([s for s, _ in chunks]), max_q, k, v, desc, tables, i32(lens), 100000, 90, 5, 0.1,
                               o[:total])
    assert pa.pa_get_device_error() == 0
    assert (o[total:] == 7.0).all()
    for i, (s, r) in enumerate(chunks):
        if r:
            seen = torch.stack([visible(s + x, s + r, 90, 5) for x in range(r)])
            ref, bound, _, _ = attend(q[cu[i]:cu[i + 1]], c.rows("k", i, s + r), c.rows("v", i, s + r), seen, 0.1, kv, "f32", prefill=True)
            check(o[cu[i]:cu[i + 1]], ref, bound, f"chunk {i}")


def test_very_many_sequences():
    """70,000 sequences of up to 40 tokens: decodes and an eviction, the rows named in reverse; a sample checked in full, the rest
    for what they have to leave alone."""
    n, most, bs, budget = 70000, 40, 16, 20
    g = torch.Generator().manual_seed(9)
    lens = torch.randint(0, most + 1, (n,), generator=g)
    lens[:3], lens[-2:] = torch.tensor([0, 1, 40]), torch.tensor([40, 0])
    k = torch.randn((3 * n, 1, bs, 64), generator=g).bfloat16()
    v = torch.randn((3 * n, 1, bs, 64), generator=g).bfloat16()
    tables = torch.randperm(3 * n, generator=g).view(n, 3).to(torch.int32)
    q = torch.randn((n, 2, 64), generator=g).bfloat16()
    rows = torch.arange(n - 1, -1, -1, dtype=torch.int32)
    dk, dv, dt, dl, dr = k.cuda(), v.cuda(), tables.cuda(), lens.to(torch.int32).cuda(), rows.cuda()
    desc = pa.kv_cache_desc(dk)
    o, ow = (torch.empty((n, 2, 64), device="cuda") for _ in range(2))
    w = torch.full((n, 1, most), 7.0, device="cuda")
    ws = torch.empty(pa.pa_decode_window_workspace_bytes(n, 2, 1, 64, bs, most, 10, 2), dtype=torch.uint8, device="cuda")
    pa.pa_decode_window(q.cuda(), dk, dv, desc, dt, dl, most, 10, 2, 0.125, o, ws)
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(n, 2, 1, 64, most), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(q.cuda(), dk, dv, desc, dt, dl, most, 0.125, ow, w, dr, torch.zeros_like(dl), 1.0, ws)
    assert pa.pa_get_device_error() == 0
    assert (o[lens == 0] == 0).all() and (ow[lens == 0] == 0).all()
    cw = w.cpu()
    sample = [0, 1, 2, 3, 77, 32767, 32768, 65535, 65536, n - 2, n - 1]

    def cached(pool, i):
        return pool[tables[i].long(), 0].view(1, -1, 64)[:, :lens[i]].double()

    for i in sample:
        m = int(lens[i])
        if m:
            for got, window, sinks in ((o, 10, 2), (ow, most, 0)):
                ref, bound, a, rel = attend(q[i:i + 1], cached(k, i), cached(v, i), visible(m - 1, m, window, sinks)[None], 0.125, "bf16", "f32")
                check(got[i:i + 1], ref, bound, f"sequence {i}")
            check(w[n - 1 - i, :, :m], a.sum(1), (a * rel[..., None]).sum(1) + 2.0 ** -24 * 4 * a.sum(1) + 1e-38, f"weights of sequence {i}")
    slot = torch.arange(most)
    behind = slot[None] >= lens.flip(0)[:, None]            # row r holds sequence n - 1 - r
    assert (cw[:, 0][behind] == 7.0).all()
    total = torch.where(behind, 0.0, cw[:, 0].double()).sum(-1)
    assert ((total - 2.0 * (lens.flip(0) > 0)).abs() < 1e-4).all()

    p, nl = torch.zeros(w.shape, dtype=torch.int32, device="cuda"), torch.full_like(dl, -5)
    nw, np_ = torch.full_like(w, 3.0), torch.full_like(p, 3)
    ws = torch.empty(pa.pa_evict_workspace_bytes(n, 1, most, budget), dtype=torch.uint8, device="cuda")
    pa.pa_evict(dk, dv, desc, dt, dl, most, dl, torch.zeros_like(dl), budget, 2, 5, w, p, nw, np_, nl, dr, ws)
    assert pa.pa_get_device_error() == 0
    assert torch.equal(nl.cpu().long(), lens.clamp(max=budget))
    kept = slot[None] < lens.flip(0).clamp(max=budget)[:, None]
    assert (nw.cpu()[:, 0][~kept] == 3.0).all() and (np_.cpu()[:, 0][~kept] == 3).all()
    gk, gv = dk.cpu(), dv.cpu()
    for i in sample:
        m, r = int(lens[i]), n - 1 - i
        src, pos = evict(cw[r, 0], p.cpu()[r, 0], m, m, 0, budget, 2, 5)
        for j, s in enumerate(src):
            assert nw[r, 0, j].item() == cw[r, 0, s].item() and np_[r, 0, j].item() == pos[s]
            for got, was in ((gk, k), (gv, v)):
                assert torch.equal(got[tables[i, j // bs], 0, j % bs], was[tables[i, s // bs], 0, s % bs])
    # slots behind the budget, and sequences within it, keep their rows
    small = (lens <= budget).nonzero().flatten()
    t = tables[small].long().flatten()
    assert torch.equal(bits(gk[t]), bits(k[t])) and torch.equal(bits(gv[t]), bits(v[t]))
    late = tables[:, 2].long()                             # slots 32 to 47: beyond the budget of every sequence
    assert torch.equal(bits(gk[late]), bits(k[late])) and torch.equal(bits(gv[late]), bits(v[late]))
