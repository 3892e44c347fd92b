"""pa_rope_and_cache into a block-scaled cache, and pa_copy_blocks_scaled: codes and scales bit for bit against the plain
form, step after step on the same cache, with the rest of the pools untouched."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import DT
from _scaled import append, rotate, table

pytestmark = pytest.mark.gpu


class Pools:
    """Pools of random codes and NaN scales, and the model's copies of them; sequences are appended block by block."""

    def __init__(self, hkv, d, bs, dt, blocks, seed, r, hq=0, interleaved=False, far=False):
        self.g = np.random.default_rng(seed)
        self.hkv, self.d, self.bs, self.dt, self.hq, self.inter = hkv, d, bs, dt, hq, interleaved
        self.table = table(3000, r) if r else None
        self.first = (5 << 30) // (hkv * bs * d) if far else 0      # byte offsets past 32 bits
        shape = (self.first + blocks, hkv, bs, d)
        self.codes = [self.g.integers(0, 256, (blocks, hkv, bs, d)).astype(np.uint8) for _ in range(2)]
        self.scales = [np.full((blocks, hkv), np.nan, np.float32) for _ in range(2)]
        self.k, self.v = (torch.empty(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:2], math.nan, device="cuda") for _ in range(2))
        self.k[self.first:], self.v[self.first:] = (torch.from_numpy(c).cuda() for c in self.codes)
        self.free = list(self.g.permutation(blocks))
        self.seqs = {}
        self.desc = pa.kv_cache_desc(self.k)

    def put_scales(self):
        for t, s in ((self.ks, self.scales[0]), (self.vs, self.scales[1])):
            t[self.first:] = torch.from_numpy(s).cuda()

    def slots(self, seq, n):
        """Slots of n more tokens of a sequence."""
        blocks, length = self.seqs.setdefault(seq, ([], 0))
        out = []
        for p in range(length, length + n):
            if p // self.bs == len(blocks):
                blocks.append(int(self.free.pop()))
            out.append(blocks[p // self.bs] * self.bs + p % self.bs)
        self.seqs[seq] = (blocks, length + n)
        return out

    def rows(self, T, size=1.0):
        x = self.g.standard_normal((T, self.hq + 2 * self.hkv, self.d)) * np.exp(0.7 * self.g.standard_normal((T, self.hq + 2 * self.hkv, 1)))
        return torch.from_numpy((x * size).astype(np.float32)).to(DT[self.dt])

    def step(self, x, slots, pos=None, err=0, stream=None):
        """Append rows x [T, hq + 2 hkv, d] at `slots`, here and in the model, and compare everything."""
        T = len(x)
        slots = np.asarray(slots, np.int64)
        pos = (self.g.integers(0, 3000, T) if pos is None else np.asarray(pos)).astype(np.int32)
        dev = x.cuda()
        q, k, v = dev[:, :self.hq], dev[:, self.hq:self.hq + self.hkv], dev[:, self.hq + self.hkv:]
        out = torch.full((T, self.hq, self.d), 7.0, dtype=x.dtype, device="cuda") if self.hq else None
        rot = self.table is not None
        off = np.where(slots >= 0, slots + self.first * self.bs, slots)
        pa.pa_rope_and_cache(q if self.hq else None, k, v, torch.from_numpy(pos).cuda() if rot else None,
                             torch.from_numpy(self.table).cuda() if rot else None, torch.from_numpy(off).cuda(), self.k, self.v, self.desc,
                             out, interleaved=self.inter, k_scales=self.ks, v_scales=self.vs, stream=stream)
        assert pa.pa_get_device_error() == err
        f = x.float().numpy()
        live = (pos >= 0) & (pos < 3000) if rot else np.ones(T, bool)
        p = np.clip(pos, 0, 2999)
        kk, vv = f[:, self.hq:self.hq + self.hkv], f[:, self.hq + self.hkv:]
        if rot:
            kk = rotate(kk, self.table, p, self.inter)
        here = np.where(live & (slots < len(self.codes[0]) * self.bs), slots, -1)
        for y, c, s in ((kk, self.codes[0], self.scales[0]), (vv, self.codes[1], self.scales[1])):
            append(y, here, c, s, self.bs)
        if self.hq:
            want = torch.full((T, self.hq, self.d), 7.0, dtype=x.dtype)
            want[live] = torch.from_numpy(rotate(f[:, :self.hq], self.table, p, self.inter))[live].to(x.dtype)
            assert torch.equal(out.cpu(), want)
        self.same()

    def same(self):
        for got, want in ((self.ks, self.scales[0]), (self.vs, self.scales[1])):
            assert np.array_equal(got[self.first:].cpu().numpy().view(np.uint32) & 0x7FFFFFFF,
                                  want.view(np.uint32) & 0x7FFFFFFF), "scales"
        for got, want in ((self.k, self.codes[0]), (self.v, self.codes[1])):
            assert np.array_equal(got[self.first:].cpu().numpy(), want), "codes"


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("d,bs", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("r,interleaved", [(64, False), (48, True), (0, False)])
def test_prompts_then_decodes(dt, d, bs, r, interleaved):
    """Ragged prompts, then single tokens that grow blocks and their scales, then mixed steps."""
    p = Pools(2, d, bs, dt, 60, seed=d + bs + r, r=r, hq=4 if r else 0, interleaved=interleaved)

    def step(sizes, size=1.0):
        slots = sum((p.slots(i, n) for i, n in enumerate(sizes)), [])
        p.step(p.rows(len(slots), size), slots)

    step([1, 15, 16, 17, 70, 33, 100])
    for k in range(12):
        step([1] * 7, size=1.5 ** (k % 7))           # larger and larger: scales grow, twice
    step([1, 40, 1, 0, 5, 1, 31])
    step([31, 1, 2, 3, 0, 47, 9], size=0.01)         # small ones keep the block's scale


@pytest.mark.parametrize("T", [1, 5, 31, 33, 257, 1500])
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_sizes(T, hkv):
    """From a token to enough of them for windows of 32 (every window size of the launcher)."""
    p = Pools(hkv, 128, 32, "bf16", T // 32 + 40, seed=T, r=128, hq=hkv)
    n = T // 3
    for sizes in ((T - 2 * n, n, n), (7, 0, 45)):
        slots = sum((p.slots(i, m) for i, m in enumerate(sizes)), [])
        p.step(p.rows(len(slots)), slots)


def test_many_single_tokens():
    p = Pools(8, 64, 16, "f16", 1100, seed=1, r=64)
    for _ in range(3):
        p.step(p.rows(1000), sum((p.slots(i, 1) for i in range(1000)), []))


def test_padding_and_holes():
    """Padding tokens between a block's tokens, tokens that are not stored, slots left out and slots out of order."""
    p = Pools(2, 128, 16, "bf16", 30, seed=2, r=128, hq=2)
    slots = np.array(p.slots(0, 40) + p.slots(1, 30))
    pos = p.g.integers(0, 3000, 70)
    pos[[3, 4, 20, 41, 69]] = -1
    slots[[0, 33, 50]] = -1
    # slot 0 of the first block is not stored: what the block then seems to hold has no scale, which is reported
    p.step(p.rows(70), slots, pos, err=4)
    slots = np.array(p.slots(4, 40) + p.slots(5, 30))
    slots[[5, 33, 50]] = -1
    p.step(p.rows(70), slots, pos)
    a = p.slots(2, 16)
    p.step(p.rows(16), a[::-1])
    b = p.slots(3, 16)
    p.step(p.rows(2), b[:2])
    p.step(p.rows(6), [b[2], -1, b[7], -1, -1, b[5]])


def test_positions_and_slots_out_of_range():
    p = Pools(2, 64, 16, "bf16", 20, seed=3, r=64, hq=2)
    slots = np.array(p.slots(0, 50))
    slots[[5, 20]] = 20 * 16, 1 << 50
    pos = p.g.integers(0, 3000, 50)
    p.step(p.rows(50), slots, pos, err=4)
    pos[[2, 30]] = 3000, 2 ** 31 - 1
    slots = np.array(p.slots(1, 50))
    p.step(p.rows(50), slots, pos, err=4)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_extremes(dt):
    """Zeros, infinities, NaN, the largest values and the smallest ones."""
    p = Pools(1, 64, 16, dt, 30, seed=4, r=0)
    big, tiny = (3.3e38, 1e-38) if dt == "bf16" else (65504.0, 6e-8)
    for values in ([0.0] * 5, [1.0, math.inf, -math.inf], [1.0, math.nan, -2.0], [math.nan] * 3, [math.inf], [big, -big, 1.0], [tiny, 0.0],
                   [448.0], [449.0], [447.0, 0.3], [1.75 * 2.0 ** -10], [1.8 * 2.0 ** -10]):
        x = torch.zeros((3, 2, 64))
        x.view(-1)[:len(values)] = torch.tensor(values)
        x[2, 1, -len(values):] = torch.tensor(values)
        seq = len(p.seqs)
        p.step(x.to(DT[dt]), p.slots(seq, 3))
        p.step(p.rows(2), p.slots(seq, 2))            # more tokens behind them
        p.step(torch.zeros((1, 2, 64), dtype=DT[dt]), p.slots(seq, 1))


def test_scales_of_other_makers():
    """Blocks that hold tokens under scales that are no powers of two, and scales out of range (reported, nothing stored)."""
    p = Pools(2, 128, 32, "bf16", 12, seed=5, r=128)
    slots = p.slots(0, 20) + p.slots(1, 20) + p.slots(2, 20)
    for s in p.scales:
        for i in range(3):
            s[p.seqs[i][0][0]] = (0.0123, 3.3) if i < 2 else (2.0 ** -64, 2.0 ** 32)
    p.put_scales()
    for size in (0.1, 30.0, 3000.0):
        slots = sum((p.slots(i, 3) for i in range(3)), [])
        p.step(p.rows(9, size), slots)
    for bad in (0.0, -1.0, math.nan, math.inf, 2.0 ** 33, 2.0 ** -65):
        p.scales[0][p.seqs[0][0][0], 1] = bad
        p.put_scales()
        p.step(p.rows(2), p.slots(0, 1) + p.slots(1, 1), err=4)
        p.seqs[0] = (p.seqs[0][0], p.seqs[0][1] - 1)


def test_blocks_past_32_bits():
    p = Pools(8, 128, 32, "bf16", 30, seed=6, r=128, far=True)
    p.step(p.rows(300), p.slots(0, 150) + p.slots(1, 150))
    p.step(p.rows(2, 4.0), p.slots(0, 1) + p.slots(1, 1))


def test_copy_blocks():
    p = Pools(3, 64, 16, "bf16", 30, seed=7, r=64)
    p.step(p.rows(100), p.slots(0, 100))
    src, dst = p.seqs[0][0][:4], [int(p.free.pop()) for _ in range(4)]
    pairs = torch.tensor(list(zip(src, dst)), dtype=torch.int32)
    pa.pa_copy_blocks_scaled(p.k, p.v, p.desc, p.ks, p.vs, pairs.cuda())
    assert pa.pa_get_device_error() == 0
    for c, s in zip(p.codes, p.scales):
        c[dst], s[dst] = c[src], s[src]
    p.same()
    bad = torch.tensor([[src[0], 30], [-1, dst[0]], [src[3], dst[0]]], dtype=torch.int32)   # the good pair is still copied
    pa.pa_copy_blocks_scaled(p.k, p.v, p.desc, p.ks, p.vs, bad.cuda())
    assert pa.pa_get_device_error() == 4
    for c, s in zip(p.codes, p.scales):
        c[dst[0]], s[dst[0]] = c[src[3]], s[src[3]]
    p.same()
