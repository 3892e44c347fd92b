"""The attention over a block-scaled cache with infinite and NaN queries.

A row with an infinite or NaN element has no finite score, so it is NaN whatever the keys; the rows beside it are as without
it."""
import math

import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import DT, check
from _scaled import ScaledCache, attend, causal, run_chunks, run_decode

pytestmark = pytest.mark.gpu

OUT = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("qt,out", OUT)
@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 2, 128, 16), (8, 2, 64, 32), (32, 2, 128, 32)])
@pytest.mark.parametrize("scale", [0.09, -0.09])
def test_queries_without_a_value(case, qt, out, hq, hkv, d, bs, scale):
    lens, rows = [1, 1, 2, 90, 700], [1, 1, 2, 50, 300]
    if case == "decode":
        rows = [1] * len(lens)
    c = ScaledCache(lens, hkv, d, bs, seed=hq + d)
    # element 3 of every key is positive: with an infinity there, all of a row's scores are the same infinity
    c.k[..., 3] = torch.where(c.k[..., 3] == 0x7F, c.k[..., 3], (c.k[..., 3] & 0x3F) | 0x30)
    q = (1.5 * torch.randn((sum(rows), hq, d), generator=torch.Generator().manual_seed(1))).to(DT[qt])
    dead = torch.zeros(q.shape[:2], dtype=torch.bool)
    at = 0
    for i, r in enumerate(rows):
        for n, (row, head, bad) in enumerate([(0, 0, math.inf), (0, 1, -math.inf), (r - 1, 3, math.nan), (r // 2, 2, math.inf),
                                              (r // 2, 4, -math.inf)]):
            q[at + row, (head + i) % hq, 3 if n < 2 else (17 * n) % d] = bad
            dead[at + row, (head + i) % hq] = True
        at += r
    if case == "decode":
        o, cu = run_decode(pa, c, q, scale, out), list(range(len(lens) + 1))
    else:
        o, cu = run_chunks(pa, c, q, rows, scale, out)
    o = o.cpu()
    assert torch.isnan(o[dead]).all()
    clean = torch.where(dead[..., None], 0.0, q.float()).to(q.dtype)
    for i, (n, r) in enumerate(zip(lens, rows)):
        a, b = cu[i], cu[i + 1]
        want, bound = attend(clean[a:b], c.rows("k", i, n), c.rows("v", i, n), causal(n, r), scale, out, case == "chunk")
        live = ~dead[a:b]
        check(o[a:b][live], want[live], bound[live], f"sequence {i}: {r} of {n} tokens")
