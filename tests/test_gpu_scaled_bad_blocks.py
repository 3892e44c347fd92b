"""The attention over a block-scaled cache with block ids out of range inside a sequence: reported, and such a key is left
out, like a key behind the end."""
import pytest
import torch

import paged_kv_cache_writes_gb300 as pa
from _bounded import DT, check
from _scaled import ScaledCache, attend, causal, i32

pytestmark = pytest.mark.gpu

OUT = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


@pytest.mark.parametrize("case", ["decode", "chunk"])
@pytest.mark.parametrize("qt,out", OUT)
@pytest.mark.parametrize("d,bs", [(128, 16), (64, 32)])
@pytest.mark.parametrize("bad", [-1, 1 << 29])
def test_keys_of_blocks_out_of_range_are_left_out(case, qt, out, d, bs, bad):
    lens, rows = [100, 700, 33], [100, 260, 20]
    if case == "decode":
        rows = [1] * len(lens)
    c = ScaledCache(lens, 2, d, bs, seed=d)
    good = [torch.ones(n, dtype=torch.bool) for n in lens]
    for i, block in ((0, 0), (0, 2), (1, 5), (1, 700 // bs), (1, 6)):
        c.tables[i, block] = bad
        good[i][block * bs:(block + 1) * bs] = False
    q = (1.5 * torch.randn((sum(rows), 8, d), generator=torch.Generator().manual_seed(2))).to(DT[qt])
    k, v, tables, desc, ks, vs = c.device(pa)
    o = torch.full(q.shape, 7.0, dtype=DT[out], device="cuda")
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    args = (k, v, desc, ks, vs, tables, i32(lens), max(lens), 0.09, o)
    if case == "decode":
        ws = torch.empty(pa.pa_decode_scaled_workspace_bytes(3, 8, 2, d, max(lens)), dtype=torch.uint8, device="cuda")
        pa.pa_decode_scaled(q.cuda(), *args, ws)
    else:
        pa.pa_prefill_chunk_scaled(q.cuda(), i32(cu), i32([n - r for n, r in zip(lens, rows)]), max(rows), *args)
    assert pa.pa_get_device_error() == 4
    tables_host = c.tables
    c.tables = torch.where((tables_host < 0) | (tables_host >= c.num_blocks), 0, tables_host)   # (what is read there is not seen)
    for i, (n, r) in enumerate(zip(lens, rows)):
        parts = []
        for which in "kv":
            x, s = c.rows(which, i, n)
            parts.append((torch.where(good[i][None, :, None], x, 0.0), torch.where(good[i][None], s, 1.0)))
        want, bound = attend(q[cu[i]:cu[i + 1]], *parts, causal(n, r) & good[i][None], 0.09, out, case == "chunk")
        check(o[cu[i]:cu[i + 1]], want, bound, f"sequence {i}: {r} of {n} tokens")
