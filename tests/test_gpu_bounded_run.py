"""The bounded-cache calls together, as a serving loop uses them: the block manager's tables and slots, cache writes, the
decodes and chunks, and what bounds the cache (release_window; unshare, copy, evict, truncate), step by step against a
64-bit model that keeps every token.  Then the calls on other streams and in captured graphs."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import attend, check, evict, visible

pytestmark = pytest.mark.gpu

HKV, HQ, D, BS = 2, 8, 128, 16
SCALE = 0.08


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    """A block manager over a pool of NaN, with the device tensors of a few sequences."""

    def __init__(self, blocks, seed):
        self.g = torch.Generator().manual_seed(seed)
        self.bm = pa.BlockManager(blocks, BS, shuffle_seed=seed)
        self.k = torch.full((blocks, HKV, BS, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.desc = pa.kv_cache_desc(self.k)

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g).bfloat16()

    def copy(self, pairs):
        if len(pairs):
            pa.pa_copy_blocks(self.k, self.v, self.desc, torch.from_numpy(pairs).cuda())

    def write(self, seq, k, v):
        """Append tokens k, v [n, HKV, D] to a sequence."""
        slots, pairs = self.bm.append(seq, len(k))
        self.copy(pairs)
        pa.pa_reshape_and_cache(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), self.k, self.v, self.desc)

    def tables(self, seqs, width=64):
        t = torch.full((len(seqs), width), -1, dtype=torch.int32)
        for i, s in enumerate(seqs):
            b, _ = self.bm.block_table(s)
            t[i, :len(b)] = torch.from_numpy(b)
        return t.cuda()


def test_sliding_window_loop():
    """Two prompts in chunks, then decode steps; blocks that the window has left go back to the pool at once."""
    window, sinks = 70, 5
    lp = Loop(40, 3)                                  # both sequences without a window would need 52 blocks
    seqs = [lp.bm.new_sequence(), lp.bm.new_sequence()]
    hist = [[torch.zeros((0, HKV, D)), torch.zeros((0, HKV, D))] for _ in seqs]

    def add(i, n):
        k, v = lp.rand(n, HKV, D), lp.rand(n, HKV, D)
        lp.write(seqs[i], k, v)
        hist[i] = [torch.cat([a, b.float()]) for a, b in zip(hist[i], (k, v))]

    def want(i, q, t0):
        n = len(hist[i][0])
        seen = torch.stack([visible(t0 + r, n, window, sinks) for r in range(len(q))])
        k, v = (x.double().transpose(0, 1) for x in hist[i])
        return attend(q, k, v, seen, SCALE, "bf16", "f32", prefill=len(q) > 1)

    for step in range(4):                             # chunks of 80 and 100 tokens
        sizes = (80, 100)
        starts = [len(h[0]) for h in hist]
        for i, n in enumerate(sizes):
            add(i, n)
        q = [lp.rand(n, HQ, D) for n in sizes]
        out = torch.empty((sum(sizes), HQ, D), device="cuda")
        lens = [len(h[0]) for h in hist]
        pa.pa_prefill_chunk_window(torch.cat(q).cuda(), i32([0, sizes[0], sum(sizes)]), i32(starts), max(sizes), lp.k, lp.v, lp.desc,
                                   lp.tables(seqs), i32(lens), max(lens), window, sinks, SCALE, out)
        assert pa.pa_get_device_error() == 0
        for i, at in enumerate((0, sizes[0])):
            ref, bound, _, _ = want(i, q[i], starts[i])
            check(out[at:at + sizes[i]], ref, bound, f"chunk {step} of sequence {i}")
            lp.bm.release_window(seqs[i], window, sinks)
    for step in range(40):
        for i in range(2):
            add(i, 1)
        q = lp.rand(2, HQ, D)
        lens = [len(h[0]) for h in hist]
        out = torch.empty((2, HQ, D), device="cuda")
        ws = torch.empty(pa.pa_decode_window_workspace_bytes(2, HQ, HKV, D, BS, max(lens), window, sinks), dtype=torch.uint8, device="cuda")
        pa.pa_decode_window(q.cuda(), lp.k, lp.v, lp.desc, lp.tables(seqs), i32(lens), max(lens), window, sinks, SCALE, out, ws)
        assert pa.pa_get_device_error() == 0
        for i in range(2):
            ref, bound, _, _ = want(i, q[i:i + 1], lens[i] - 1)
            check(out[i:i + 1], ref, bound, f"step {step} of sequence {i}")
            lp.bm.release_window(seqs[i], window, sinks)
    assert lp.bm.stats().used_blocks <= 2 * (1 + -(-(window + BS - 1) // BS))


def test_eviction_loop_with_a_fork():
    """A prompt, a branch of it, decode steps that accumulate weights, evictions back to a budget: the cache of each
    (sequence, KV head) against a model that holds the kept tokens' rows, weights and positions."""
    budget, sinks, recent, stride = 100, 4, 20, 160
    lp = Loop(48, 7)
    a = lp.bm.new_sequence()
    k, v = lp.rand(90, HKV, D), lp.rand(90, HKV, D)
    lp.write(a, k, v)
    b = lp.bm.fork(a)
    seqs = [a, b]
    # model: per sequence and head, lists of (k, v, weight, position); total tokens seen; slots before which order is lost
    model = [[[[k[t, h].double(), v[t, h].double(), 0.0, t] for t in range(90)] for h in range(HKV)] for _ in seqs]
    seen, old, fresh = [90, 90], [0, 0], [0, 0]
    weights = torch.full((2, HKV, stride), float("nan"), device="cuda")
    positions = torch.zeros((2, HKV, stride), dtype=torch.int32, device="cuda")
    evictions = 0
    for step in range(60):
        for i, s in enumerate(seqs):
            if step % 3 or i == 0:                    # the branch runs slower
                kn, vn = lp.rand(1, HKV, D), lp.rand(1, HKV, D)
                lp.write(s, kn, vn)
                for h in range(HKV):
                    model[i][h].append([kn[0, h].double(), vn[0, h].double(), 0.0, seen[i]])
                seen[i] += 1
        lens = [len(m[0]) for m in model]
        q = (2 * torch.randn((2, HQ, D), generator=lp.g)).bfloat16()
        out = torch.empty((2, HQ, D), device="cuda")
        ws = torch.empty(pa.pa_decode_weights_workspace_bytes(2, HQ, HKV, D, max(lens)), dtype=torch.uint8, device="cuda")
        pa.pa_decode_weights(q.cuda(), lp.k, lp.v, lp.desc, lp.tables(seqs), i32(lens), max(lens), SCALE, out, weights,
                             fresh_from=i32([f if f < n else n for f, n in zip(fresh, lens)]), decay=0.9, workspace=ws)
        assert pa.pa_get_device_error() == 0
        for i in range(2):
            n = lens[i]
            kk = torch.stack([torch.stack([e[0] for e in model[i][h]]) for h in range(HKV)])
            vv = torch.stack([torch.stack([e[1] for e in model[i][h]]) for h in range(HKV)])
            ref, bound, w, rel = attend(q[i:i + 1], kk, vv, torch.ones((1, n), dtype=bool), SCALE, "bf16", "f32")
            check(out[i:i + 1], ref, bound, f"step {step} of sequence {i}")
            got = weights[i, :, :n].double().cpu()
            for h in range(HKV):
                a_h, rel_h = w[0, h * 4:(h + 1) * 4], rel[0, h * 4:(h + 1) * 4, None]
                old_w = torch.tensor([e[2] for e in model[i][h]], dtype=torch.float64)
                want = torch.where(torch.arange(n) < fresh[i], 0.9 * old_w, 0.0) + a_h.sum(0)
                # the model goes on from the kernel's weights: each step is checked by itself
                check(got[h], want, (a_h * rel_h).sum(0) + 2.0 ** -22 * want + 1e-38, f"weights of sequence {i}, head {h}, step {step}")
                for e, x in zip(model[i][h], got[h].tolist()):
                    e[2] = x
            fresh[i] = n
        if max(lens) >= budget + 12:
            evictions += 1
            for s, n in zip(seqs, lens):
                lp.copy(lp.bm.unshare(s, min(n, budget)))
            new = i32([0, 0])
            ws = torch.empty(pa.pa_evict_workspace_bytes(2, HKV, max(lens), budget), dtype=torch.uint8, device="cuda")
            pa.pa_evict(lp.k, lp.v, lp.desc, lp.tables(seqs), i32(lens), max(lens), i32(seen), i32(old), budget, sinks, recent, weights,
                        positions, weights, positions, new, workspace=ws)
            assert pa.pa_get_device_error() == 0
            for i, s in enumerate(seqs):
                n = min(lens[i], budget)
                for h in range(HKV):
                    m = model[i][h]
                    src, pos = evict([e[2] for e in m], [e[3] for e in m], lens[i], seen[i], lens[i], budget, sinks, recent)
                    assert pos == [e[3] for e in m]
                    model[i][h] = [m[x] for x in src]
                    assert positions[i, h, :n].tolist() == [e[3] for e in model[i][h]]
                assert new[i].item() == n
                lp.bm.truncate(s, n)
                old[i] = fresh[i] = n
    assert evictions >= 3
    assert lp.bm.stats().shared_blocks <= 1


def decode_inputs(seed, lens=(300, 77, 512)):
    g = torch.Generator().manual_seed(seed)
    blocks = sum(-(-n // BS) for n in lens) + 3
    t = torch.zeros((len(lens), 40), dtype=torch.int32)
    order, at = torch.randperm(blocks, generator=g), 0
    for i, n in enumerate(lens):
        m = -(-n // BS)
        t[i, :m] = order[at:at + m].to(torch.int32)
        at += m
    k, v = (torch.randn((blocks, HKV, BS, D), generator=g).bfloat16().cuda() for _ in range(2))
    return k, v, t.cuda(), i32(list(lens)), torch.randn((len(lens), HQ, D), generator=g).bfloat16().cuda()


def calls(k, v, t, lens, q, ws, outs):
    """The decodes and a chunk over one set of inputs, into outs = [window, weights' out, weights, chunk]."""
    d = pa.kv_cache_desc(k)
    pa.pa_decode_window(q, k, v, d, t, lens, 512, 100, 4, SCALE, outs[0], ws)
    pa.pa_decode_weights(q, k, v, d, t, lens, 512, SCALE, outs[1], outs[2], fresh_from=torch.zeros_like(lens), workspace=ws)
    pa.pa_prefill_chunk_window(q, torch.arange(4, dtype=torch.int32, device="cuda"), lens - 1, 1, k, v, d, t, lens, 512, 100, 4,
                               SCALE, outs[3])


def fresh_outs(q):
    return [torch.zeros_like(q), torch.zeros_like(q), torch.zeros((3, HKV, 512), device="cuda"), torch.zeros_like(q)]


def workspace():
    n = max(pa.pa_decode_window_workspace_bytes(3, HQ, HKV, D, BS, 512, 100, 4), pa.pa_decode_weights_workspace_bytes(3, HQ, HKV, D, 512))
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def test_another_stream_and_captured_graphs_that_share_a_workspace():
    x, y = decode_inputs(1), decode_inputs(2)
    ws = workspace()
    want = []
    for z in (x, y):
        outs = fresh_outs(z[4])
        calls(*z, ws, outs)
        want.append(outs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [fresh_outs(z[4]) for z in (x, y)]
    with torch.cuda.stream(s):
        calls(*x, ws, got[0])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[0], want[0]))
    # two graphs over the same workspace, replayed in turn on one stream
    graphs = []
    for z, outs in zip((x, y), got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            calls(*z, ws, outs)
        graphs.append(g)
    for _ in range(3):
        for outs in got:
            for o in outs:
                o.zero_()
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_calls_at_once_with_workspaces_of_their_own():
    x, y = decode_inputs(3), decode_inputs(4)
    want = []
    for z in (x, y):
        outs = fresh_outs(z[4])
        calls(*z, workspace(), outs)
        want.append(outs)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [workspace() for _ in range(2)]
    got = [fresh_outs(z[4]) for z in (x, y)]
    torch.cuda.synchronize()
    for _ in range(10):
        for z, s, ws, outs in zip((x, y), streams, spaces, got):
            with torch.cuda.stream(s):
                calls(*z, ws, outs)
    torch.cuda.synchronize()
    assert pa.pa_get_device_error() == 0
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_a_captured_eviction_replays_on_new_weights():
    k, v, t, lens, _ = decode_inputs(5)
    d = pa.kv_cache_desc(k)
    w, p = torch.rand((3, HKV, 512), device="cuda"), torch.zeros((3, HKV, 512), dtype=torch.int32, device="cuda")
    nw, np_, nl, zero = torch.zeros_like(w), torch.zeros_like(p), torch.zeros_like(lens), torch.zeros_like(lens)
    ws = torch.empty(pa.pa_evict_workspace_bytes(3, HKV, 512, 200), dtype=torch.uint8, device="cuda")
    k0, v0 = k.clone(), v.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pa.pa_evict(k, v, d, t, lens, 512, lens, zero, 200, 4, 30, w, p, nw, np_, nl, workspace=ws)
    for seed in (1, 2):
        k.copy_(k0)
        v.copy_(v0)
        w.copy_(torch.rand(w.shape, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        assert nl.tolist() == [200, 77, 200]
        for i, n in enumerate((300, 77, 512)):
            for h in range(HKV):
                src, pos = evict(w[i, h].tolist(), p[i, h].tolist(), n, n, 0, 200, 4, 30)
                assert np_[i, h, :len(src)].tolist() == [pos[j] for j in src]
                rows = torch.arange(len(src), device="cuda")
                at = torch.tensor(src, device="cuda")
                for pool, before in ((k, k0), (v, v0)):
                    assert torch.equal(pool[t[i].long()[rows // BS], h, rows % BS], before[t[i].long()[at // BS], h, at % BS])
