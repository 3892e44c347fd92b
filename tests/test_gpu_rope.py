"""pa_rope_and_cache into 16-bit caches and fp8 caches with fixed scales: bit for bit against the plain form (its
arithmetic is fixed), and the rotation against 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import DT
from _scaled import decode, encode, rotate, table

pytestmark = pytest.mark.gpu


class Step:
    """T tokens with random positions and slots, as views into one QKV tensor; `pad`: some tokens padding, some not stored."""

    def __init__(self, T, hq, hkv, d, bs, dt, r, seed, pad=False, extra=0, pool="same"):
        g = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.bs, self.dt = hq, hkv, d, bs, dt
        x = torch.from_numpy(g.standard_normal((T, hq + 2 * hkv + extra, d)).astype(np.float32)).to(DT[dt])
        self.qkv = x
        self.blocks = -(-T // bs) + 9
        self.slots = g.permutation(self.blocks * bs)[:T].astype(np.int64)
        self.npos = 5000
        self.pos = g.integers(0, self.npos, T).astype(np.int32)
        self.pos[:1] = self.npos - 1
        self.table = table(self.npos, r) if r else None
        if pad:
            self.pos[1::5] = -1
            self.slots[1::5] = 1 << 60           # of padding tokens nothing is read
            self.slots[2::5] = -1
        kind = dt if pool == "same" else pool
        shape = (self.blocks, hkv, bs, d)
        self.k0, self.v0 = (torch.from_numpy(g.integers(0, 255, shape).astype(np.uint8)) if kind == "fp8" else
                            torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(DT[dt]) for _ in range(2))
        self.fp8 = kind == "fp8"

    def parts(self, x):
        return x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:self.hq + 2 * self.hkv]

    def run(self, interleaved, in_place=False, no_q=False, scales=(0.03, 0.05), stream=None):
        q, k, v = self.parts(self.qkv.cuda())
        kc, vc = self.k0.cuda(), self.v0.cuda()
        self.desc = pa.kv_cache_desc(kc, *(scales if self.fp8 else ()))
        out = None
        if no_q:
            q = None
        elif in_place:
            q = out = q.contiguous()
        else:
            out = torch.full((len(k), self.hq, self.d), 7.0, dtype=q.dtype, device="cuda")
        pos = None if self.table is None else torch.from_numpy(self.pos).cuda()
        tab = None if self.table is None else torch.from_numpy(self.table).cuda()
        pa.pa_rope_and_cache(q, k, v, pos, tab, torch.from_numpy(self.slots).cuda(), kc, vc, self.desc, out,
                             interleaved=interleaved, stream=stream)
        err = pa.pa_get_device_error()
        return out, kc, vc, err

    def want(self, interleaved, q_start, scales=(0.03, 0.05)):
        """(q_out over q_start, k pool, v pool)"""
        q, k, v = (p.float().numpy() for p in self.parts(self.qkv))
        live = self.pos >= 0 if self.table is not None else np.ones(len(k), bool)
        if self.table is not None:
            p = np.maximum(self.pos, 0)
            q, k = rotate(q, self.table, p, interleaved), rotate(k, self.table, p, interleaved)
        out = q_start.clone()
        out[live] = torch.from_numpy(q)[live].to(q_start.dtype)
        kc, vc = self.k0.clone(), self.v0.clone()
        for t in np.nonzero(live & (self.slots >= 0) & (self.slots < self.blocks * self.bs))[0]:
            b, o = divmod(int(self.slots[t]), self.bs)
            for pool, x, s in ((kc, k, scales[0]), (vc, v, scales[1])):
                pool[b, :, o] = torch.from_numpy(encode(x[t] / np.float32(s))) if self.fp8 else torch.from_numpy(x[t]).to(pool.dtype)
        return out, kc, vc

    def check(self, interleaved, **kw):
        out, kc, vc, err = self.run(interleaved, **kw)
        assert err == 0
        start = torch.full((len(self.qkv), self.hq, self.d), 7.0, dtype=self.qkv.dtype)
        if kw.get("in_place"):
            start = self.parts(self.qkv)[0].clone()
        wq, wk, wv = self.want(interleaved, start)
        if out is not None:
            assert torch.equal(out.cpu(), wq)
        assert torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("pool", ["same", "fp8"])
@pytest.mark.parametrize("d,r", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_and_rotations(dt, pool, d, r, interleaved):
    Step(37, 8, 2, d, 16, dt, r, seed=d + r, pad=True, pool=pool).check(interleaved)


@pytest.mark.parametrize("T", [1, 2, 65, 700])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (17, 1), (64, 8), (128, 2)])
def test_tokens_and_heads(T, hq, hkv):
    Step(T, hq, hkv, 128, 32, "bf16", 128, seed=T + hq).check(False)


def test_many_heads():
    Step(3, 700, 100, 64, 16, "f16", 64, seed=2).check(True)


def test_in_place_and_gaps_between_tokens():
    Step(33, 8, 2, 128, 16, "bf16", 128, seed=3, extra=3).check(False)
    Step(33, 8, 2, 128, 16, "bf16", 96, seed=4, pad=True).check(False, in_place=True)
    Step(33, 8, 2, 64, 16, "f16", 64, seed=5).check(True, in_place=True)


@pytest.mark.parametrize("pool", ["same", "fp8"])
def test_without_queries_or_rotation(pool):
    Step(50, 4, 2, 128, 16, "bf16", 64, seed=6, pool=pool).check(False, no_q=True)
    s = Step(50, 4, 2, 128, 16, "bf16", 0, seed=7, pool=pool)      # stored as pa_reshape_and_cache stores them
    s.slots[3::7] = -1
    s.check(False, no_q=True)
    _, kc, vc, _ = s.run(False, no_q=True)
    k2, v2 = s.k0.cuda(), s.v0.cuda()
    _, k, v = s.parts(s.qkv.cuda())
    pa.pa_reshape_and_cache(k, v, torch.from_numpy(s.slots).cuda(), k2, v2, s.desc)
    assert torch.equal(kc, k2) and torch.equal(vc, v2)


def test_rotation_against_64_bits():
    # products and sum rounded to fp32: off by 2^-24 (|a c| + |b s| + |y|); then half a step of bf16
    s = Step(200, 4, 2, 128, 16, "bf16", 128, seed=8)
    out, _, _, err = s.run(False)
    assert err == 0
    x, t = s.parts(s.qkv)[0].double(), torch.from_numpy(s.table).double()[s.pos][:, None]
    c, n, a, b = t[..., :64], t[..., 64:], x[..., :64], x[..., 64:]
    y = torch.cat([a * c - b * n, b * c + a * n], -1)
    size = torch.cat([(a * c).abs() + (b * n).abs(), (b * c).abs() + (a * n).abs()], -1)
    off = 2.0 ** -24 * (size + y.abs())
    assert ((out.cpu().double() - y).abs() <= off + 2.0 ** -8 * (y.abs() + off) + 1e-38).all()


def test_pages_out_of_range():
    """A position past the table, a slot past the pool: reported, skipped, the other tokens served."""
    s = Step(40, 4, 2, 128, 16, "bf16", 128, seed=9)
    s.slots[7] = s.blocks * 16
    out, kc, vc, err = s.run(False)
    assert err == 4
    wq, wk, wv = s.want(False, torch.full((40, 4, 128), 7.0, dtype=torch.bfloat16))
    assert torch.equal(out.cpu(), wq) and torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)
    s.slots[7] = 3
    s.pos[9], s.pos[10] = s.npos, 2 ** 31 - 1
    out, kc, vc, err = s.run(False)
    assert err == 4
    s.pos[9] = s.pos[10] = -1
    wq, wk, wv = s.want(False, torch.full((40, 4, 128), 7.0, dtype=torch.bfloat16))
    assert torch.equal(out.cpu(), wq) and torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)


def test_per_head_scales():
    s = Step(30, 4, 2, 64, 16, "bf16", 64, seed=10, pool="fp8")
    hs = [torch.tensor([0.02, 0.07], device="cuda"), torch.tensor([0.5, 0.01], device="cuda")]
    q, k, v = s.parts(s.qkv.cuda())
    kc, vc = s.k0.cuda(), s.v0.cuda()
    pa.pa_rope_and_cache(None, k, v, torch.from_numpy(s.pos).cuda(), torch.from_numpy(s.table).cuda(),
                         torch.from_numpy(s.slots).cuda(), kc, vc, pa.kv_cache_desc(kc, 1.0, 1.0, *hs))
    assert pa.pa_get_device_error() == 0
    _, kk, vv = (p.float().numpy() for p in s.parts(s.qkv))
    kk = rotate(kk, s.table, s.pos, False)
    b, o = s.slots // 16, s.slots % 16
    for pool, x, h in ((kc, kk, hs[0]), (vc, vv, hs[1])):
        got = pool.cpu().numpy()[b, :, o]
        assert np.array_equal(got, encode(x / h.cpu().numpy()[None, :, None]))
        assert np.isfinite(decode(got)).all()


def test_binding_refusals():
    s = Step(8, 4, 2, 128, 16, "bf16", 128, seed=11)
    q, k, v = s.parts(s.qkv.cuda())
    kc, vc = s.k0.cuda(), s.v0.cuda()
    pos, tab, slots = torch.from_numpy(s.pos).cuda(), torch.from_numpy(s.table).cuda(), torch.from_numpy(s.slots).cuda()
    d = pa.kv_cache_desc(kc)
    out = torch.empty((8, 4, 128), dtype=torch.bfloat16, device="cuda")

    def call(**kw):
        a = {**dict(q=q, k=k, v=v, positions=pos, cos_sin=tab, slot_mapping=slots, k_cache=kc, v_cache=vc, cache=d, q_out=out), **kw}
        pa.pa_rope_and_cache(**a)

    call()
    for kw in (dict(q_out=None), dict(q_out=out[:, :2]), dict(k=k[:, :1]), dict(v=v.half()), dict(v=v[:4]), dict(positions=pos[:4]),
               dict(positions=pos.long()), dict(positions=None), dict(cos_sin=None), dict(cos_sin=tab.double()),
               dict(slot_mapping=slots.int()), dict(slot_mapping=slots[:4]), dict(k=k.cpu()), dict(q=q.transpose(1, 2)),
               dict(q=q.float()), dict(k_cache=kc[:1]), dict(k_scales=torch.ones(2, 2, device="cuda")), dict(v=v.contiguous())):
        with pytest.raises((ValueError, TypeError, pa.PaError)):
            call(**kw)

    with pytest.raises(pa.PaError):
        call(cos_sin=torch.from_numpy(table(50, 24)).cuda())       # rope_dim 24
    assert pa.pa_get_device_error() == 0


def test_one_head_of_any_stride():
    """A single head's stride between heads says nothing: rows as a transposed view gives them."""
    s = Step(9, 1, 1, 64, 16, "bf16", 64, seed=12)
    q, k, v = s.parts(s.qkv.cuda())
    pos, tab, slots = torch.from_numpy(s.pos).cuda(), torch.from_numpy(s.table).cuda(), torch.from_numpy(s.slots).cuda()
    got = []
    for change in (lambda x: x, lambda x: x.contiguous().view(1, 9, 64).transpose(0, 1)):
        kc, vc = s.k0.cuda(), s.v0.cuda()
        out = torch.empty((9, 1, 64), dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_and_cache(change(q), change(k), change(v), pos, tab, slots, kc, vc, pa.kv_cache_desc(kc), out)
        got.append((kc, vc, out))
    assert change(k).stride(1) != 64
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert pa.pa_get_device_error() == 0
