"""The calls of a block-scaled cache together, as a serving loop uses them: the block manager's slots and tables, prompts
appended and attended in chunks, decode steps, a fork whose shared block is copied before it is written, a truncation;
codes and scales bit for bit and outputs within their bounds at every step.  Then captured graphs and streams."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import DT, check
from _scaled import append, attend, causal, decode, i32, rotate, table

pytestmark = pytest.mark.gpu

HQ, HKV, SCALE, MAX_POS = 8, 2, 0.09, 2000


class Loop:
    def __init__(self, d, bs, qt, out, blocks, seed, max_seqs):
        self.g = torch.Generator().manual_seed(seed)
        self.d, self.bs, self.qt, self.out = d, bs, qt, out
        self.bm = pa.BlockManager(blocks, bs, shuffle_seed=seed)
        shape = (blocks, HKV, bs, d)
        self.codes = [np.full(shape, 0x7F, np.uint8) for _ in range(2)]
        self.scales = [np.full(shape[:2], np.nan, np.float32) for _ in range(2)]
        self.k, self.v = (torch.from_numpy(c).cuda() for c in self.codes)
        self.ks, self.vs = (torch.from_numpy(s).cuda() for s in self.scales)
        self.desc = pa.kv_cache_desc(self.k)
        self.table = table(MAX_POS, d // 2)
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.ws = torch.empty(pa.pa_decode_scaled_workspace_bytes(max_seqs, HQ, HKV, d, MAX_POS), dtype=torch.uint8, device="cuda")

    def copy(self, pairs):
        if len(pairs):
            pa.pa_copy_blocks_scaled(self.k, self.v, self.desc, self.ks, self.vs, torch.from_numpy(pairs).cuda())
            for a, b in pairs:
                for x in (*self.codes, *self.scales):
                    x[b] = x[a]

    def step(self, seqs, counts, louder=1.0):
        """Append counts[i] tokens to seqs[i]; attend them: as a decode if all counts are 1, else as chunks."""
        starts = [self.bm.block_table(s)[1] for s in seqs]
        slots = []
        for s, n in zip(seqs, counts):
            at, pairs = self.bm.append(s, n)
            self.copy(pairs)
            slots.append(at)
        slots, T = np.concatenate(slots), sum(counts)
        x = (louder * torch.randn((T, HQ + 2 * HKV, self.d), generator=self.g)).to(DT[self.qt])
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(starts, counts)]).astype(np.int32)
        dev = x.cuda()
        q = torch.empty((T, HQ, self.d), dtype=x.dtype, device="cuda")
        pa.pa_rope_and_cache(dev[:, :HQ], dev[:, HQ:HQ + HKV], dev[:, HQ + HKV:], torch.from_numpy(pos).cuda(), self.table_dev,
                             torch.from_numpy(slots).cuda(), self.k, self.v, self.desc, q, k_scales=self.ks, v_scales=self.vs)
        f = x.float().numpy()
        turned = rotate(f[:, :HQ + HKV], self.table, pos, False)
        append(turned[:, HQ:], slots, self.codes[0], self.scales[0], self.bs)
        append(f[:, HQ + HKV:], slots, self.codes[1], self.scales[1], self.bs)
        q_want = torch.from_numpy(turned[:, :HQ]).to(x.dtype)

        lens = [a + n for a, n in zip(starts, counts)]
        tables = torch.full((len(seqs), -(-max(lens) // self.bs)), -1, dtype=torch.int32)
        for i, s in enumerate(seqs):
            b, _ = self.bm.block_table(s)
            tables[i, :len(b)] = torch.from_numpy(b)
        o = torch.full((T, HQ, self.d), math.nan, dtype=DT[self.out], device="cuda")
        args = (self.k, self.v, self.desc, self.ks, self.vs, tables.cuda(), i32(lens), max(lens), SCALE, o)
        chunk = max(counts) > 1
        if chunk:
            pa.pa_prefill_chunk_scaled(q, i32(np.concatenate([[0], np.cumsum(counts)]).tolist()), i32(starts), max(counts), *args)
        else:
            pa.pa_decode_scaled(q, *args, self.ws)
        assert pa.pa_get_device_error() == 0
        assert torch.equal(q.cpu(), q_want)
        for got, want in ((self.k, self.codes[0]), (self.v, self.codes[1])):
            assert np.array_equal(got.cpu().numpy(), want)
        for got, want in ((self.ks, self.scales[0]), (self.vs, self.scales[1])):
            assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)
        at = 0
        for i, (s, n, length) in enumerate(zip(seqs, counts, lens)):
            p = np.arange(length)
            b, r = self.bm.block_table(s)[0][p // self.bs], p % self.bs
            k, v = ((torch.from_numpy(decode(c[b, :, r])).transpose(0, 1), torch.from_numpy(x[b]).T.double())
                    for c, x in zip(self.codes, self.scales))
            want, bound = attend(q_want[at:at + n], k, v, causal(length, n), SCALE, self.out, chunk)
            check(o[at:at + n], want, bound, f"sequence {i}: {n} of {length} tokens")
            at += n


@pytest.mark.parametrize("d,bs,qt,out", [(128, 16, "bf16", "bf16"), (128, 32, "f16", "f32"), (64, 16, "f16", "f16"), (64, 32, "bf16", "f32")])
def test_serving_loop(d, bs, qt, out):
    lp = Loop(d, bs, qt, out, 120, d + bs, 8)
    a, b = lp.bm.new_sequence(), lp.bm.new_sequence()
    lp.step([a, b], [130, 37])
    lp.step([a, b], [65, 1])
    lp.step([b, a], [300, 2])
    for _ in range(3):
        lp.step([a, b], [1, 1])
    c = lp.bm.fork(a)                                     # its last block is shared: copied before either writes to it
    lp.step([a, b, c], [1, 1, 1], louder=5.0)             # (the blocks' scales grow)
    lp.step([c, a], [1, 1])
    e = lp.bm.fork(c)
    lp.step([e, c, b, a], [9, 40, 1, 3], louder=0.1)
    lp.bm.truncate(b, lp.bm.block_table(b)[1] - 5)        # codes behind the end stay; new ones overwrite them
    for louder in (1.0, 20.0, 1.0):
        lp.step([a, b, c, e], [1, 1, 1, 1], louder)
    lp.bm.free(a)
    f = lp.bm.new_sequence()                              # its blocks held other sequences' codes and scales
    lp.step([f, b], [200, 1])
    lp.step([f, b, c, e], [1, 1, 1, 1])


class Decodes:
    """A decode step (append, attention) of n sequences over static tensors, to be captured; and the same, called."""

    def __init__(self, n, seed, d=128, bs=16, most=600):
        g = torch.Generator().manual_seed(seed)
        self.n, self.most, self.d, width = n, most, d, -(-most // bs)
        self.k, self.v = (torch.full((n * width, HKV, bs, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full((n * width, HKV), math.nan, device="cuda") for _ in range(2))
        self.desc = pa.kv_cache_desc(self.k)
        self.tables_host = torch.randperm(n * width, generator=g).view(n, width).to(torch.int32)
        self.tables, self.bs = self.tables_host.cuda(), bs
        self.table = torch.from_numpy(table(most, d)).cuda()
        self.ws = torch.empty(pa.pa_decode_scaled_workspace_bytes(n, HQ, HKV, d, most), dtype=torch.uint8, device="cuda")
        self.lens = torch.randint(0, most - 20, (n,), generator=g)
        tokens = [(i, p) for i in range(n) for p in range(int(self.lens[i]))]
        x = torch.randn((len(tokens), 2 * HKV, d), generator=g).bfloat16().cuda()
        if tokens:
            pa.pa_rope_and_cache(None, x[:, :HKV], x[:, HKV:], None, None, self.slots(tokens), self.k, self.v, self.desc,
                                 k_scales=self.ks, v_scales=self.vs)
        self.x = torch.zeros((n, HQ + 2 * HKV, d), dtype=torch.bfloat16, device="cuda")
        self.pos, self.len_dev = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))
        self.slot = torch.full((n,), -1, dtype=torch.int64, device="cuda")
        self.q = torch.zeros((n, HQ, d), dtype=torch.bfloat16, device="cuda")
        self.o = torch.zeros((n, HQ, d), device="cuda")
        torch.cuda.synchronize()

    def slots(self, tokens):
        return torch.tensor([int(self.tables_host[i, p // self.bs]) * self.bs + p % self.bs for i, p in tokens],
                            dtype=torch.int64, device="cuda")

    def feed(self, seed, padded=()):
        """The next step's inputs; a padded sequence has no token (position and slot -1) and length 0."""
        g = torch.Generator().manual_seed(seed)
        live = [i for i in range(self.n) if i not in padded]
        pos, slot, lens = torch.full((self.n,), -1), torch.full((self.n,), -1), torch.zeros(self.n, dtype=torch.int64)
        pos[live], lens[live] = self.lens[live], self.lens[live] + 1
        slot[live] = self.slots([(i, int(self.lens[i])) for i in live]).cpu()
        self.lens[live] += 1
        self.x.copy_(torch.randn(self.x.shape, generator=g).bfloat16())
        self.pos.copy_(pos), self.slot.copy_(slot), self.len_dev.copy_(lens)

    def call(self, stream=None):
        x = self.x
        pa.pa_rope_and_cache(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.pos, self.table, self.slot, self.k, self.v,
                             self.desc, self.q, k_scales=self.ks, v_scales=self.vs, stream=stream)
        pa.pa_decode_scaled(self.q, self.k, self.v, self.desc, self.ks, self.vs, self.tables, self.len_dev, self.most, SCALE,
                            self.o, self.ws, stream=stream)

    def state(self):
        return [t.clone() for t in (self.k, self.v, self.ks.view(torch.int32), self.vs.view(torch.int32), self.q, self.o)]


@pytest.mark.parametrize("n", [1, 7, 70])
def test_captured_steps(n):
    """Replays with other lengths, slots and padded rows give the bits of the calls."""
    a, b = Decodes(n, 4), Decodes(n, 4)
    b.call()                                              # (all padding: changes nothing but q and out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.call()
    for step in range(18):
        padded = () if step % 3 else range(0, n, 4)
        for s in (a, b):
            s.feed(step, padded)
        a.call()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.state(), b.state()):
            assert torch.equal(x, y), step
    assert pa.pa_get_device_error() == 0


def test_two_graphs_at_once():
    """Two captured loops, each with its own workspace, replayed on two streams at once."""
    runs = [Decodes(40, 5), Decodes(9, 6)]
    alone = [Decodes(40, 5), Decodes(9, 6)]
    for s in runs + alone:
        s.feed(1)
    graphs = []
    for s in runs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.call()
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    for s in alone:
        for _ in range(20):
            s.call()
    torch.cuda.synchronize()
    for s, t in zip(runs, alone):
        for x, y in zip(s.state(), t.state()):
            assert torch.equal(x, y)
    assert pa.pa_get_device_error() == 0


def test_one_workspace_for_calls_in_turn():
    """Batches of other sizes use one workspace one after another on a stream."""
    runs = [Decodes(n, 10 + n) for n in (3, 50, 1, 20)]
    big = max((s.ws for s in runs), key=torch.numel)
    st = torch.cuda.Stream()
    for s in runs:
        s.feed(2)
    torch.cuda.synchronize()
    for s in runs:
        s.call()
    want = [s.o.clone() for s in runs]
    torch.cuda.synchronize()
    for s in runs:
        s.ws = big
        s.o.fill_(math.nan)
    torch.cuda.synchronize()
    for _ in range(3):
        for s in runs:
            s.call(stream=st)                             # (the tokens are in the cache: stored again, the same)
    torch.cuda.synchronize()
    for s, w in zip(runs, want):
        assert torch.equal(s.o, w)
    assert pa.pa_get_device_error(st) == 0
