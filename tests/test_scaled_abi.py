"""The append that rotates and the block-scaled calls without a GPU: refusals through the C ABI before anything is
launched, workspace sizes, the binding's checks, and the test model's own e4m3 codes."""
import ctypes

import numpy as np
import pytest
import torch

from _scaled import decode, encode, power_for

FAKE = 0x100000   # never dereferenced on these paths
FAR = 0x10000000


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_writes_gb300 import build_lib
    build_lib.build()
    import paged_kv_cache_writes_gb300 as pa
    return pa


def desc(pa, **kw):
    d = dict(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, kv_dtype=pa.PA_FP8_E4M3, k_scale=1.0, v_scale=1.0)
    return pa.PaKvCache(**{**d, **kw})


def rope(pa, d, **kw):
    a = dict(q=FAR, q_stride=4096, q_out=2 * FAR, hq=32, k=3 * FAR, v=4 * FAR, dt=1, T=4, stride=1024, pos=FAKE, table=FAKE, np=100,
             r=128, inter=0, slots=FAKE, kc=5 * FAR, vc=6 * FAR, ks=7 * FAR, vs=8 * FAR)
    a.update(kw)
    return pa.lib().pa_rope_and_cache(a["q"], a["q_stride"], a["q_out"], a["hq"], a["k"], a["v"], a["dt"], a["T"], a["stride"],
                                      a["pos"], a["table"], a["np"], a["r"], a["inter"], a["slots"], a["kc"], a["vc"],
                                      None if d is None else ctypes.byref(d), a["ks"], a["vs"], None)


@pytest.mark.parametrize("kw,desc_kw,want", [
    (dict(T=0), {}, 0),
    (dict(T=-1), {}, 1),
    (dict(hq=-1), {}, 1),
    (dict(r=-16), {}, 1),
    (dict(r=24), {}, 2),
    (dict(r=144), {}, 2),
    (dict(r=128), dict(head_dim=64), 2),
    (dict(r=0), {}, 1),                               # queries without a rotation
    (dict(np=0), {}, 1),
    (dict(dt=2), {}, 2),
    (dict(dt=3), {}, 2),
    (dict(stride=1016), {}, 1),
    (dict(stride=1028), {}, 1),
    (dict(q_stride=4088), {}, 1),
    (dict(q_stride=4100), {}, 1),
    (dict(k=None), {}, 1), (dict(v=None), {}, 1), (dict(slots=None), {}, 1), (dict(kc=None), {}, 1), (dict(vc=None), {}, 1),
    (dict(q=None), {}, 1), (dict(q_out=None), {}, 1), (dict(pos=None), {}, 1), (dict(table=None), {}, 1),
    (dict(k=FAKE + 8), {}, 1), (dict(q=FAKE + 8), {}, 1), (dict(q_out=FAKE + 8), {}, 1), (dict(slots=FAKE + 4), {}, 1),
    (dict(pos=FAKE + 2), {}, 1), (dict(table=FAKE + 4), {}, 1), (dict(kc=FAKE + 8), {}, 1),
    (dict(ks=None), {}, 1), (dict(vs=None), {}, 1), (dict(ks=7 * FAR + 2), {}, 1),
    (dict(vs=7 * FAR), {}, 1), (dict(vs=7 * FAR + 4), {}, 1),          # one array for both
    (dict(), dict(k_head_scales=FAKE, v_head_scales=FAKE), 1),
    (dict(), dict(kv_dtype=1), 2),                    # block scales of a 16-bit cache
    (dict(), dict(block_size=8), 2), (dict(), dict(head_dim=96), 2), (dict(), dict(num_blocks=0), 1),
    (dict(ks=None, vs=None, dt=0), dict(kv_dtype=1), 2),                # f16 tokens, bf16 cache
    (dict(ks=None, vs=None), dict(k_scale=0.0), 1),   # used there, and not by a block-scaled cache:
    (dict(T=0), dict(k_scale=0.0, v_scale=float("nan")), 0),
    # q_out over what is read or written elsewhere
    (dict(q_out=FAR + 16), {}, 1), (dict(q_out=FAR, q_stride=4104), {}, 1), (dict(q_out=FAR - 32), {}, 1),
    (dict(q_out=3 * FAR), {}, 1), (dict(q_out=4 * FAR + 6 * 1024), {}, 1), (dict(q_out=5 * FAR + 1024), {}, 1),
    (dict(q_out=6 * FAR - 16), {}, 1),
])
def test_rope_refusals(pa, kw, desc_kw, want):
    assert rope(pa, desc(pa, **desc_kw), **kw) == want


def test_no_descriptor(pa):
    assert rope(pa, None) == 1
    assert pa.lib().pa_copy_blocks_scaled(FAKE, FAKE, None, FAKE, FAR, FAKE, 1, None) == 1


@pytest.mark.parametrize("kw,want", [
    (dict(n=0), 0), (dict(n=-1), 1), (dict(pairs=None), 1), (dict(pairs=FAKE + 4), 1), (dict(k=None), 1), (dict(v=FAKE + 8), 1),
    (dict(ks=None), 1), (dict(vs=None), 1), (dict(ks=None, n=0), 1), (dict(vs=7 * FAR), 1)])
def test_copy_refusals(pa, kw, want):
    a = {**dict(k=5 * FAR, v=6 * FAR, ks=7 * FAR, vs=8 * FAR, pairs=FAKE, n=3), **kw}
    d = desc(pa)
    assert pa.lib().pa_copy_blocks_scaled(a["k"], a["v"], ctypes.byref(d), a["ks"], a["vs"], a["pairs"], a["n"], None) == want


ATTENTION = [
    (dict(n=0), {}, 0), (dict(n=-1), {}, 1), (dict(hq=30), {}, 1), (dict(q=None), {}, 1), (dict(q=FAKE + 4), {}, 1),
    (dict(out=None), {}, 1), (dict(bt=None), {}, 1), (dict(sl=FAKE + 2), {}, 1), (dict(mb=0), {}, 1), (dict(msl=-1), {}, 1),
    (dict(scale=float("nan")), {}, 1), (dict(odt=0), {}, 2), (dict(dt=2, odt=2), {}, 2), (dict(k=None), {}, 1),
    (dict(ks=None), {}, 1), (dict(vs=None), {}, 1), (dict(ks=7 * FAR + 1), {}, 1), (dict(vs=7 * FAR + 64), {}, 1),
    ({}, dict(kv_dtype=1), 2), ({}, dict(kv_dtype=0), 2), ({}, dict(head_dim=96), 2), ({}, dict(block_size=64), 2),
    ({}, dict(k_head_scales=FAKE, v_head_scales=FAKE), 1), (dict(n=0, ks=None), {}, 1), (dict(n=0), dict(k_scale=-1.0), 0),
]


def attention(**kw):
    return {**dict(q=FAR, dt=1, n=4, hq=32, k=5 * FAR, v=6 * FAR, ks=7 * FAR, vs=8 * FAR, bt=FAKE, mb=8, sl=FAKE, msl=100, scale=0.1,
                   ws=FAKE, wsb=1 << 30, out=2 * FAR, odt=1, cu=FAKE, qs=FAKE, mq=10), **kw}


@pytest.mark.parametrize("kw,desc_kw,want", ATTENTION + [
    (dict(ws=None), {}, 1), (dict(ws=FAKE + 16), {}, 1), (dict(wsb=100), {}, 1), (dict(n=1 << 20), {}, 2)])
def test_decode_refusals(pa, kw, desc_kw, want):
    a, d = attention(**kw), desc(pa, **desc_kw)
    assert pa.lib().pa_decode_scaled(a["q"], a["dt"], a["n"], a["hq"], a["k"], a["v"], ctypes.byref(d), a["ks"], a["vs"], a["bt"],
                                     a["mb"], a["sl"], a["msl"], a["scale"], a["ws"], a["wsb"], a["out"], a["odt"], None) == want


@pytest.mark.parametrize("kw,desc_kw,want", ATTENTION + [
    (dict(cu=None), {}, 1), (dict(qs=FAKE + 1), {}, 1), (dict(mq=-1), {}, 1), (dict(mq=0), {}, 0)])
def test_chunk_refusals(pa, kw, desc_kw, want):
    a, d = attention(**kw), desc(pa, **desc_kw)
    assert pa.lib().pa_prefill_chunk_scaled(a["q"], a["dt"], a["cu"], a["qs"], a["n"], a["mq"], a["hq"], a["k"], a["v"],
                                            ctypes.byref(d), a["ks"], a["vs"], a["bt"], a["mb"], a["sl"], a["msl"], a["scale"],
                                            a["out"], a["odt"], None) == want


def test_workspace_serves_smaller_batches(pa):
    big = pa.pa_decode_scaled_workspace_bytes(64, 32, 8, 128, 20000)
    assert big > 0
    for n in (1, 2, 7, 63):
        for most in (1, 100, 5000, 20000):
            assert pa.pa_decode_scaled_workspace_bytes(n, 32, 8, 128, most) <= big
    for bad in ((4, 30, 8, 128, 100), (-1, 32, 8, 128, 100), (4, 32, 8, 96, 100), (4, 32, 8, 128, -1), (1 << 20, 32, 8, 128, 100)):
        assert pa.pa_decode_scaled_workspace_bytes(*bad) == 0


def test_model_codes():
    """The test model's e4m3 against torch's: every fp32 near a code, the midpoints, infinities and NaN."""
    v = decode(np.arange(256, dtype=np.uint8))
    v = v[np.isfinite(v)]
    mid = (np.sort(v)[1:] + np.sort(v)[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                        np.nextafter(mid.astype(np.float32), np.float32(-1e9)), [460, 1e9, -1e9, np.inf, -np.inf, 1e-30]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(decode(encode(x)), want)
    assert np.isnan(decode(encode([np.nan]))).all()
    for amax, e in ((448.0, 0), (448.5, 1), (224.0, -1), (0.0, -64), (1e-30, -64), (3e38, 32), (1.0, -8), (0.875, -9)):
        assert power_for(amax) == 2.0 ** e
