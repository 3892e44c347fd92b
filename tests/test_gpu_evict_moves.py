"""pa_evict's moves on the GPU: done by the selection's launch and by a launch of their own (more moves than the first one
does itself), and those whose block ids are out of range: such a destination keeps its own token, weight and position."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import Cache, evict

pytestmark = pytest.mark.gpu


def bits(t):
    t = t.contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def moves_case(lens, hkv, d, bs, kv, budget, sinks, recent, seed, most=None, bad=(), alias=False, again=False):
    """bad: (sequence, block-table index, id) triples, ids that the kernel's own check refuses."""
    c = Cache(lens, hkv, d, bs, kv, seed)
    c.k, c.v = (x if kv == "fp8" else torch.nan_to_num(x) for x in (c.k, c.v))
    good = c.tables.clone()
    for i, j, b in bad:
        c.tables[i, j] = b
    n, most = len(lens), most or max(lens)
    old = [min(m, budget) if again else 0 for m in lens]
    seen = [m + 3 * budget if again else m for m in lens]
    g = torch.Generator().manual_seed(seed + 1)
    w = torch.rand((n, hkv, most), generator=g)
    p = torch.full(w.shape, -9, dtype=torch.int32)
    for i in range(n):
        for h in range(hkv):
            p[i, h, :old[i]] = torch.randperm(seen[i] - lens[i] + old[i], generator=g)[:old[i]].to(torch.int32)
    k, v, tables, desc = c.device(pa)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dw, dp = w.cuda(), p.cuda()
    nw, np_ = (dw, dp) if alias else (torch.full_like(dw, 7.0), torch.full_like(dp, 7))
    nl = i32([-5] * n)
    ws = torch.full((pa.pa_evict_workspace_bytes(n, hkv, most, budget),), 0xFF, dtype=torch.uint8, device="cuda")
    pa.pa_evict(k, v, desc, tables, i32(lens), most, i32(seen), i32(old), budget, sinks, recent, dw, dp, nw, np_, nl, workspace=ws)
    error = pa.pa_get_device_error()
    want_k, want_v = c.k.clone(), c.v.clone()
    want_w, want_p = (w.clone(), p.clone()) if alias else (torch.full_like(w, 7.0), torch.full_like(p, 7))
    refused = 0
    for i, m in enumerate(lens):
        ids, real = c.tables[i].long(), good[i].long()
        for h in range(hkv):
            src, pos = evict(w[i, h].tolist(), p[i, h].tolist(), m, seen[i], old[i], budget, sinks, recent)
            src, pos = torch.tensor(src), torch.tensor(pos, dtype=torch.int32)
            to = torch.arange(len(src))
            inside = lambda s: (ids[s // bs] >= 0) & (ids[s // bs] < c.num_blocks)  # noqa: E731
            stay = (src != to) & ~(inside(src) & inside(to))
            refused += int(stay.sum())
            src = torch.where(stay, to, src)
            want_w[i, h, :len(src)], want_p[i, h, :len(src)] = w[i, h, src], pos[src]
            to, src = to[src != to], src[src != to]
            want_k[real[to // bs], h, to % bs] = c.k[real[src // bs], h, src % bs]
            want_v[real[to // bs], h, to % bs] = c.v[real[src // bs], h, src % bs]
    assert (refused > 0) == bool(bad) and error == (4 if bad else 0)
    assert nl.tolist() == [min(m, budget) for m in lens]
    assert torch.equal(np_.cpu(), want_p)
    assert torch.equal(bits(nw), bits(want_w))
    assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v))


# of the first sequence: a destination's block, a source's, both of a move; ids just behind the pool, below 0, far out
BAD = [[(0, 1, "behind")], [(0, 9, -1)], [(0, 0, -1), (0, 10, 2 ** 31 - 1)], [(0, 8, -2 ** 31), (1, 2, "behind")]]


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("bad", BAD)
def test_refused_moves_leave_their_slots(bad, alias, again):
    lens = [200, 180, 90]
    blocks = sum(-(-n // 16) for n in lens) + 5
    bad = [(i, j, blocks if b == "behind" else b) for i, j, b in bad]
    moves_case(lens, 2, 64, 16, "bf16", 100, 4, 20, 21, bad=bad, alias=alias, again=again)


def many(seqs):
    return [2100 - 17 * i for i in range(seqs)]


@pytest.mark.parametrize("kv,d,alias,again", [("bf16", 128, False, False), ("fp8", 64, True, True), ("f16", 64, True, False)])
def test_moves_in_a_launch_of_their_own(kv, d, alias, again):
    # 60 x 4 heads of 1000 moves at most: more than 196,608
    moves_case(many(60), 4, d, 32, kv, 1000, 4, 50, d, most=4000, alias=alias, again=again)


@pytest.mark.parametrize("alias", [False, True])
def test_refused_moves_in_a_launch_of_their_own(alias):
    lens = many(60)
    blocks = sum(-(-n // 32) for n in lens) + 5
    moves_case(lens, 4, 64, 32, "bf16", 1000, 4, 50, 5, most=4000, alias=alias,
               bad=[(0, 3, blocks), (7, 60, -1), (59, 0, -7), (59, 32, 1 << 30)])


@pytest.mark.parametrize("most", [100, 300000, 400000])
def test_refused_moves_of_every_cluster_form(most):
    # one CTA a head and a list in shared memory; eight CTAs, keys in shared memory; keys read again
    moves_case([100], 1, 64, 16, "bf16", 60, 4, 10, most, most=most, bad=[(0, 1, -1), (0, 5, 1 << 20)])
