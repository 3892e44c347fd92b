"""pa_evict on the GPU: which tokens stay, where they go, and what happens to everything else, bit for bit against the
plain form (tests/_bounded.py)."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import Cache, evict

pytestmark = pytest.mark.gpu


def bits(t):
    t = t.contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def evict_case(lens, hkv, d, bs, kv, budget, sinks, recent, seed=0, seen=None, old=None, rows=None, pad=0, alias=False,
               weights=None, most=None):
    c = Cache(lens, hkv, d, bs, kv, seed)
    c.k, c.v = (x if kv == "fp8" else torch.nan_to_num(x) for x in (c.k, c.v))
    g = torch.Generator().manual_seed(seed + 1)
    n = len(lens)
    most = most or max(max(lens), 1)
    seen, old = seen or list(lens), old or [0] * n
    at = rows or list(range(n))
    held = max(at) + 2
    w = torch.rand((held, hkv, most + pad), generator=g) if weights is None else weights
    p = torch.full(w.shape, -9, dtype=torch.int32)
    for i in range(n):
        for h in range(hkv):   # distinct earlier positions, in any order
            p[at[i], h, :old[i]] = torch.randperm(max(1, seen[i] - lens[i] + old[i]), generator=g)[:old[i]].to(torch.int32)
    k, v, tables, desc = c.device(pa)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    dw, dp, dl = w.cuda(), p.cuda(), i32(lens)
    nw, np_ = (dw, dp) if alias else (torch.full_like(dw, 7.0), torch.full_like(dp, 7))
    nl = i32([-5] * n)
    ws = torch.full((pa.pa_evict_workspace_bytes(n, hkv, most, budget),), 0xFF, dtype=torch.uint8, device="cuda")
    pa.pa_evict(k, v, desc, tables, dl, most, i32(seen), i32(old), budget, sinks, recent, dw, dp, nw, np_, nl,
                None if rows is None else i32(rows), ws)
    assert pa.pa_get_device_error() == 0
    want_k, want_v = c.k.clone(), c.v.clone()
    want_w, want_p = (w.clone(), p.clone()) if alias else (torch.full_like(w, 7.0), torch.full_like(p, 7))
    for i, m in enumerate(lens):
        t = c.tables[i].tolist()
        for h in range(hkv):
            src, pos = evict(w[at[i], h], p[at[i], h], m, seen[i], old[i], budget, sinks, recent)
            for j, s in enumerate(src):
                want_w[at[i], h, j], want_p[at[i], h, j] = w[at[i], h, s], pos[s]
                if s != j:
                    want_k[t[j // bs], h, j % bs] = c.k[t[s // bs], h, s % bs]
                    want_v[t[j // bs], h, j % bs] = c.v[t[s // bs], h, s % bs]
    assert nl.tolist() == [min(m, budget) for m in lens]
    assert torch.equal(np_.cpu(), want_p)
    assert torch.equal(bits(nw), bits(want_w))
    assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v))


@pytest.mark.parametrize("kv", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("d,bs", [(64, 16), (128, 16), (128, 32)])
def test_types(kv, d, bs):
    evict_case([1, 20, 64, 65, 200, 333], 3, d, bs, kv, 64, 4, 10, seed=d + bs)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (7, 3, 4), (50, 0, 0), (50, 20, 30), (1000, 4, 4)])
def test_budgets(budget, sinks, recent):
    evict_case([1, 2, 49, 50, 51, 400], 2, 64, 16, "f16", budget, sinks, recent, seed=budget)


def test_again_after_an_eviction():
    evict_case([120, 101, 140, 100], 2, 64, 16, "bf16", 100, 4, 30, seen=[500, 101, 900, 777], old=[100, 0, 100, 100], seed=4)


def test_in_place_metadata():
    evict_case([120, 101, 140, 30], 2, 64, 16, "bf16", 100, 4, 30, seen=[500, 101, 900, 30], old=[100, 0, 100, 0], alias=True, seed=5)


def test_named_rows_and_padded_strides():
    evict_case([120, 101, 140], 2, 64, 32, "bf16", 90, 4, 30, rows=[4, 0, 2], pad=11, seed=6)


def test_empty_sequences():
    evict_case([0, 100, 0], 2, 64, 16, "bf16", 50, 4, 30, seed=7)


@pytest.mark.parametrize("kind", ["equal", "zeros", "special"])
def test_ties_and_special_weights(kind):
    lens = [300, 1500]
    w = torch.full((3, 2, 1500), 0.25)
    if kind == "zeros":
        w = torch.where(torch.rand(w.shape, generator=torch.Generator().manual_seed(1)) < 0.5, 0.0, -0.0)
    elif kind == "special":
        g = torch.Generator().manual_seed(2)
        pick = torch.randint(0, 8, w.shape, generator=g)
        values = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -3.0, 3.4e38])
        w = values[pick]
    evict_case(lens, 2, 64, 16, "f16", 128, 4, 20, weights=w, seed=8)


@pytest.mark.parametrize("n,budget", [(1024, 1023), (1025, 1024), (4096, 2048), (5000, 4999), (9000, 31), (20011, 10007)])
def test_lengths(n, budget):
    evict_case([n], 1, 64, 16, "bf16", budget, 4, 16, seed=n)


@pytest.mark.parametrize("most", [600, 20000, 400000, 1 << 20])
def test_cluster_sizes(most):
    # the bound on the lengths decides how many CTAs share a head and whether the keys fit in shared memory
    evict_case([600, 333, 100], 2, 64, 16, "bf16", 150, 4, 30, most=most, seed=most, weights=torch.randint(0, 40, (4, 2, most)) / 8)


@pytest.mark.parametrize("kv,d", [("bf16", 128), ("fp8", 64)])
def test_many_moves(kv, d):
    # more moves than one launch does: 24 x 4 heads of up to 2100 slots to 1000
    evict_case([2100 - 37 * i for i in range(24)], 4, d, 32, kv, 1000, 4, 50, most=4000, seed=d)


@pytest.mark.parametrize("seqs,most", [(8, 30000), (40, 12000)])
def test_few_moves_under_a_large_bound(seqs, most):
    # the bound promises many moves (and, with few sequences, a cluster per head), the lengths make few
    evict_case([300 + i for i in range(seqs)], 2, 64, 16, "f16", 290, 4, 20, most=most, seed=seqs)


def test_a_bound_above_every_length():
    evict_case([120, 101], 2, 64, 16, "bf16", 90, 4, 30, most=5000, seed=9)


def test_blocks_past_32_bit_offsets():
    c = Cache([200], 2, 128, 16, "bf16", 12, far=True)
    k, v, tables, desc = c.device(pa)
    t, far = tables[0].long().cpu(), k.shape[0] - c.num_blocks
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    w = torch.rand((1, 2, 200), generator=torch.Generator().manual_seed(3))
    p = torch.zeros((1, 2, 200), dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.pa_evict_workspace_bytes(1, 2, 200, 90), dtype=torch.uint8, device="cuda")
    pa.pa_evict(k, v, desc, tables, i32([200]), 200, i32([200]), i32([0]), 90, 4, 10, w.cuda(), p, w.cuda(), p.clone(),
                i32([0]), workspace=ws)
    assert pa.pa_get_device_error() == 0
    for h in range(2):
        src, _ = evict(w[0, h], p[0, h], 200, 200, 0, 90, 4, 10)
        for j, s in enumerate(src):
            assert torch.equal(bits(k[t[j // 16], h, j % 16]), bits(c.k[t[s // 16] - far, h, s % 16]))
            assert torch.equal(bits(v[t[j // 16], h, j % 16]), bits(c.v[t[s // 16] - far, h, s % 16]))


def test_more_protected_tokens_than_the_budget():
    # positions that cannot be: every token says it is among the first; the lowest slots stay
    c = Cache([100], 1, 64, 16, "bf16", 13)
    k, v, tables, desc = c.device(pa)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    w, p = torch.rand((1, 1, 100), device="cuda"), torch.zeros((1, 1, 100), dtype=torch.int32, device="cuda")
    nw, np_, nl = torch.zeros_like(w), torch.full_like(p, 7), i32([0])
    ws = torch.empty(pa.pa_evict_workspace_bytes(1, 1, 100, 50), dtype=torch.uint8, device="cuda")
    pa.pa_evict(k, v, desc, tables, i32([100]), 100, i32([500]), i32([100]), 50, 4, 0, w, p, nw, np_, nl, workspace=ws)
    assert pa.pa_get_device_error() == 0
    assert torch.equal(nw[0, 0, :50], w[0, 0, :50]) and (np_[0, 0, :50] == 0).all() and (np_[0, 0, 50:] == 7).all()


def test_bad_metadata_is_reported_and_skipped():
    c = Cache([100, 100, 100, 100], 2, 64, 16, "bf16", 11)
    k, v, tables, desc = c.device(pa)
    before_k = bits(k)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    w = torch.rand((4, 2, 100), device="cuda")
    p = torch.zeros((4, 2, 100), dtype=torch.int32, device="cuda")
    ws = torch.empty(pa.pa_evict_workspace_bytes(4, 2, 100, 50), dtype=torch.uint8, device="cuda")
    for lens, rows in (([101, 0, 0, 0], None), ([-1, 0, 0, 0], None), ([100, 0, 0, 0], [4, 0, 1, 2]), ([100, 0, 0, 0], [-1, 0, 1, 2])):
        nl = i32([9] * 4)
        pa.pa_evict(k, v, desc, tables, i32(lens), 100, i32([200] * 4), i32([0] * 4), 50, 0, 0, w, p, w, p, nl,
                    None if rows is None else i32(rows), ws)
        assert pa.pa_get_device_error() == 4
        assert torch.equal(bits(k), before_k) and nl.tolist() == lens
    tables[0, :3] = c.num_blocks           # destinations out of range: reported, those rows stay
    pa.pa_evict(k, v, desc, tables, i32([100, 0, 0, 0]), 100, i32([100] * 4), i32([0] * 4), 50, 0, 0, w, p, w, p, i32([0] * 4), None, ws)
    assert pa.pa_get_device_error() == 4


def test_two_sequences_of_one_weights_row():
    """Not a meaningful call (the rows have to be distinct): whatever stays, every access is in range, and nothing else changes."""
    for n, most in ((700, 700), (900, 400000)):      # keys in shared memory, and read again in every phase
        c = Cache([n, n, n], 1, 64, 16, "fp8", 15)
        k, v, tables, desc = c.device(pa)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        w = torch.rand((3, 1, most), device="cuda")
        p = torch.zeros((3, 1, most), dtype=torch.int32, device="cuda")
        before, nl = w.clone(), i32([0] * 3)
        ws = torch.empty(pa.pa_evict_workspace_bytes(3, 1, most, 300), dtype=torch.uint8, device="cuda")
        pa.pa_evict(k, v, desc, tables, i32([n, n, 100]), most, i32([n, n, 100]), i32([0] * 3), 300, 4, 10, w, p, w, p, nl,
                    i32([1, 1, 0]), ws)
        assert pa.pa_get_device_error() in (0, 4)
        assert nl.tolist() == [300, 300, 100]
        assert torch.equal(w[0], before[0]) and torch.equal(w[2], before[2])
        third = c.tables[2, :-(-n // 16)].long()      # its blocks (the entries behind them are out of range), on the CPU
        assert torch.equal(k.cpu()[third], c.k[third]) and torch.equal(v.cpu()[third], c.v[third])
