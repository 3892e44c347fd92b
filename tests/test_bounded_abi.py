"""Refusals of the bounded-cache calls that need no GPU: every argument is checked on the host before anything is
launched, workspace sizes, and the Python binding's checks of shapes and types."""
import ctypes

import pytest
import torch

FAKE = 0x10000  # a 256-byte aligned non-null address; never dereferenced on these paths


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_writes_gb300 import build_lib
    build_lib.build()
    import paged_kv_cache_writes_gb300 as pa
    return pa


def desc(pa, **kw):
    d = dict(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, kv_dtype=pa.PA_BF16, k_scale=1.0, v_scale=1.0)
    return pa.PaKvCache(**{**d, **kw})


DECODE = [
    (dict(num_seqs=0), {}, 0),                       # zero work
    (dict(num_seqs=-1), {}, 1),
    (dict(hq=30), {}, 1),
    (dict(q=None), {}, 1),
    (dict(q=FAKE + 4), {}, 1),
    (dict(out=None), {}, 1),
    (dict(bt=None), {}, 1),
    (dict(sl=FAKE + 2), {}, 1),
    (dict(mb=0), {}, 1),
    (dict(msl=-1), {}, 1),
    (dict(ps=48), {}, 1),
    (dict(scale=float("inf")), {}, 1),
    (dict(ws=None), {}, 1),
    (dict(ws=FAKE + 16), {}, 1),
    (dict(wsb=100), {}, 1),
    (dict(q_dtype=0), {}, 2),
    (dict(odt=0), {}, 2),
    (dict(num_seqs=1 << 20), {}, 2),
    ({}, dict(head_dim=96), 2),
    ({}, dict(block_size=8), 2),
    ({}, dict(num_blocks=0), 1),
]


def decode_args(**kw):
    a = dict(q=FAKE, q_dtype=1, num_seqs=4, hq=32, k=FAKE, v=FAKE, bt=FAKE, mb=8, sl=FAKE, msl=100, window=50, sinks=4,
             scale=0.1, ps=0, ws=FAKE, wsb=1 << 30, out=FAKE, odt=1, w=FAKE, stride=100, rows=4, wr=None, ff=None, decay=1.0)
    a.update(kw)
    return a


def window(pa, d, **kw):
    a = decode_args(**kw)
    return pa.lib().pa_decode_window(a["q"], a["q_dtype"], a["num_seqs"], a["hq"], a["k"], a["v"], ctypes.byref(d), a["bt"],
                                     a["mb"], a["sl"], a["msl"], a["window"], a["sinks"], a["scale"], a["ps"], a["ws"],
                                     a["wsb"], a["out"], a["odt"], None)


def weights(pa, d, **kw):
    a = decode_args(**kw)
    return pa.lib().pa_decode_weights(a["q"], a["q_dtype"], a["num_seqs"], a["hq"], a["k"], a["v"], ctypes.byref(d),
                                      a["bt"], a["mb"], a["sl"], a["msl"], a["scale"], a["ps"], a["ws"], a["wsb"], a["out"],
                                      a["odt"], a["w"], a["stride"], a["rows"], a["wr"], a["ff"], a["decay"], None)


@pytest.mark.parametrize("kw,desc_kw,want", DECODE + [
    (dict(window=0), {}, 1), (dict(window=-5), {}, 1), (dict(sinks=-1), {}, 1), (dict(window=0, num_seqs=0), {}, 1),
    (dict(msl=2 ** 31 - 1, window=2 ** 31 - 1, mb=2 ** 31 - 1), {}, 2),     # more partitions than a row may have
])
def test_decode_window_refusals(pa, kw, desc_kw, want):
    assert window(pa, desc(pa, **desc_kw), **kw) == want


@pytest.mark.parametrize("kw,desc_kw,want", DECODE + [
    (dict(w=None), {}, 1), (dict(w=FAKE + 4), {}, 1), (dict(stride=99), {}, 1), (dict(rows=3), {}, 1),
    (dict(rows=0, wr=FAKE), {}, 1), (dict(wr=FAKE + 2), {}, 1), (dict(ff=FAKE + 1), {}, 1), (dict(decay=float("nan")), {}, 1),
])
def test_decode_weights_refusals(pa, kw, desc_kw, want):
    assert weights(pa, desc(pa, **desc_kw), **kw) == want


@pytest.mark.parametrize("kw,desc_kw,want", [
    (dict(n=0), {}, 0), (dict(mq=0), {}, 0), (dict(n=-1), {}, 1), (dict(hq=31), {}, 1), (dict(q_dtype=0), {}, 2),
    (dict(cu=None), {}, 1), (dict(qs=FAKE + 2), {}, 1), (dict(out=None), {}, 1), (dict(odt=2), {}, 2), (dict(window=0), {}, 1),
    (dict(window=0, n=0), {}, 1), (dict(sinks=-1), {}, 1), (dict(scale=float("nan")), {}, 1), ({}, dict(head_dim=32), 2),
    (dict(n=1 << 20, mq=1 << 20), {}, 2),
])
def test_prefill_chunk_window_refusals(pa, kw, desc_kw, want):
    a = dict(q=FAKE, q_dtype=1, cu=FAKE, qs=FAKE, n=1, mq=64, hq=32, bt=FAKE, mb=8, sl=FAKE, msl=128, window=50, sinks=4,
             scale=0.1, out=FAKE, odt=1)
    a.update(kw)
    d = desc(pa, **desc_kw)
    assert pa.lib().pa_prefill_chunk_window(a["q"], a["q_dtype"], a["cu"], a["qs"], a["n"], a["mq"], a["hq"], FAKE, FAKE,
                                            ctypes.byref(d), a["bt"], a["mb"], a["sl"], a["msl"], a["window"], a["sinks"],
                                            a["scale"], a["out"], a["odt"], None) == want


@pytest.mark.parametrize("kw,desc_kw,want", [
    (dict(n=0), {}, 0), (dict(n=-1), {}, 1), (dict(mb=0), {}, 1), (dict(msl=-1), {}, 1), (dict(budget=0), {}, 1),
    (dict(sinks=-1), {}, 1), (dict(recent=-1), {}, 1), (dict(sinks=40, recent=20), {}, 1),      # more protected than the budget
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), {}, 1), (dict(bt=None), {}, 1), (dict(sl=None), {}, 1),
    (dict(seen=FAKE + 2), {}, 1), (dict(old=None), {}, 1), (dict(w=None), {}, 1), (dict(p=FAKE + 1), {}, 1),
    (dict(nw=None), {}, 1), (dict(np=None), {}, 1), (dict(nl=None), {}, 1), (dict(stride=99), {}, 1), (dict(rows=3), {}, 1),
    (dict(k=None), {}, 1), (dict(ws=None), {}, 1), (dict(ws=FAKE + 8), {}, 1), (dict(wsb=16), {}, 1),
    (dict(nl=FAKE + 0x100000), {}, 1), (dict(nl=FAKE + 0x100000 + 12), {}, 1), (dict(nl=FAKE + 0x100000 - 12), {}, 1),   # on seq_lens
    (dict(nl=FAKE + 0x200000 - 12), {}, 1), (dict(nl=FAKE + 0x300000 + 4), {}, 1), (dict(nl=FAKE + 0x400000, wr=FAKE + 0x400000), {}, 1),
    (dict(nw=FAKE + 0x500000 + 64), {}, 1), (dict(np=FAKE + 0x600000 - 64), {}, 1),     # shifted against the old ones
    (dict(n=2 ** 31 - 1, rows=2 ** 31 - 1), {}, 1),
    (dict(msl=2 ** 30 + 1, stride=2 ** 31, mb=2 ** 30), {}, 1),
    ({}, dict(block_size=64), 2), ({}, dict(kv_dtype=3), 2),
])
def test_evict_refusals(pa, kw, desc_kw, want):
    a = dict(k=FAKE, v=FAKE, n=4, bt=FAKE, mb=8, sl=FAKE + 0x100000, msl=100, seen=FAKE + 0x200000, old=FAKE + 0x300000, budget=50, sinks=4,
             recent=8, w=FAKE + 0x500000, p=FAKE + 0x600000, nw=FAKE + 0x500000, np=FAKE + 0x600000, stride=100, rows=4, wr=None, nl=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    d = desc(pa, **desc_kw)
    assert pa.lib().pa_evict(a["k"], a["v"], ctypes.byref(d), a["n"], a["bt"], a["mb"], a["sl"], a["msl"], a["seen"], a["old"],
                             a["budget"], a["sinks"], a["recent"], a["w"], a["p"], a["nw"], a["np"], a["stride"], a["rows"],
                             a["wr"], a["nl"], a["ws"], a["wsb"], None) == want


def test_workspace_sizes(pa):
    full = pa.pa_decode_workspace_bytes(64, 64, 8, 128, 8192)
    # a window longer than the context changes nothing; a short one needs as many partitions as the visible tokens
    assert pa.pa_decode_window_workspace_bytes(64, 64, 8, 128, 16, 8192, 100000, 4) >= full
    short = pa.pa_decode_window_workspace_bytes(64, 64, 8, 128, 16, 1 << 20, 1000, 4)
    assert 0 < short <= pa.pa_decode_window_workspace_bytes(64, 64, 8, 128, 16, 8192, 1000, 4) < full
    # one score per query head and token, and the rows' maxima and sums
    assert pa.pa_decode_weights_workspace_bytes(64, 64, 8, 128, 8192) >= full + 64 * 64 * (8192 * 4 + 8)
    for bad in ((-1, 64, 8, 128, 16, 100, 10, 0), (4, 30, 8, 128, 16, 100, 10, 0), (4, 64, 8, 96, 16, 100, 10, 0),
                (4, 64, 8, 128, 16, 100, 0, 0), (4, 64, 8, 128, 16, 100, 10, -1), (4, 64, 8, 128, 24, 100, 10, 0)):
        assert pa.pa_decode_window_workspace_bytes(*bad) == 0
    assert pa.pa_decode_weights_workspace_bytes(4, 30, 8, 128, 100) == 0
    assert pa.pa_decode_weights_workspace_bytes(60000, 30000, 30000, 128, 2 ** 31 - 1, 2 ** 31 - 32) == 0   # past 2^64 bytes
    assert pa.pa_evict_workspace_bytes(4, 8, 100, 0) == 0 and pa.pa_evict_workspace_bytes(4, 0, 100, 5) == 0
    assert pa.pa_evict_workspace_bytes(4, 8, 100, 200) > 0


def test_binding_checks(pa, monkeypatch):
    """The binding refuses tensors that are not on the current device, of another shape or type, before the call."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    d = pa.kv_cache_desc(k)
    with pytest.raises(ValueError, match="descriptor"):
        pa._Args.shapes(None, None, k, k[:3], d, torch.zeros((1, 4)), 1)
    with pytest.raises(ValueError, match="descriptor"):
        pa._Args.shapes(None, None, k[:3], k[:3], d, torch.zeros((1, 4)), 1)
    with pytest.raises(ValueError, match="descriptor"):
        pa._Args.shapes(None, None, k.to(torch.uint8), k.to(torch.uint8), d, torch.zeros((1, 4)), 1)   # a smaller type
    with pytest.raises(ValueError, match="q and out"):
        pa._Args.shapes(torch.zeros((1, 4, 64)), torch.zeros((2, 4, 64)), k, k, d, torch.zeros((1, 4)), 1)
    with pytest.raises(ValueError, match="one row"):
        pa._Args.shapes(None, None, k, k, d, torch.zeros((1, 4)), 2)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    t, n = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    w, p = torch.zeros((1, 2, 64)), torch.zeros((1, 2, 64), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_decode_window(q, k, k, d, t, n, 10, 5, 1, 0.1, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pa.pa_prefill_chunk_window(q, n, n, 1, k, k, d, t, n, 10, 5, 1, 0.1, q)
    with pytest.raises(ValueError, match="num_kv_heads"):
        pa.pa_decode_weights(q, k, k, d, t, n, 10, 0.1, q, torch.zeros((1, 3, 64)))
    with pytest.raises(ValueError, match="one shape"):
        pa.pa_evict(k, k, d, t, n, 10, n, n, 5, 1, 1, w, p, w, p[:, :, :5], n)
    # the checks of one tensor, the device's number aside
    a = pa._Args()
    a.device = -1                       # what a CPU tensor says of itself
    assert a(q, "q") == q.data_ptr() and a.maybe(None, "q") is None and a.of_sequences(None, "n", 1) is None
    with pytest.raises(ValueError, match="one entry per sequence"):
        a.of_sequences(n, "n", 2)
    for bad, why in ((lambda: a(q.transpose(1, 2), "q"), ValueError), (lambda: a.of_sequences(w[0, 0, :1], "n", 1), (TypeError, ValueError)),
                     (lambda: a(w, "w", torch.int32), (TypeError, ValueError))):
        with pytest.raises(why):
            bad()
