"""Shapes at the limits of what the bounded-cache calls serve: refused before anything is launched."""
import ctypes

import pytest

import paged_kv_cache_writes_gb300 as pa

FAKE = 0x10000  # never dereferenced: these calls are refused on the host


@pytest.mark.parametrize("group,served", [(1, True), (6144, True), (6145, False), (8192, False), (1 << 20, False)])
@pytest.mark.parametrize("d", [64, 128])
def test_groups_of_decode_weights(group, served, d):
    assert (pa.pa_decode_weights_workspace_bytes(1, group, 1, d, 100) > 0) == served
    assert pa.pa_decode_window_workspace_bytes(1, min(group, 65535), 1, d, 16, 100, 50, 4) > 0
    if not served:
        c = pa.PaKvCache(num_blocks=64, block_size=16, num_kv_heads=1, head_dim=d, kv_dtype=pa.PA_BF16, k_scale=1.0, v_scale=1.0)
        status = pa.lib().pa_decode_weights(FAKE, pa.PA_BF16, 1, group, FAKE, FAKE, ctypes.byref(c), FAKE, 8, FAKE, 100, 0.1, 0,
                                            FAKE, 1 << 40, FAKE, pa.PA_BF16, FAKE, 100, 1, None, None, 1.0, None)
        assert status == 2


@pytest.mark.gpu
def test_the_widest_group():
    import torch
    from _bounded import Cache, attend, check

    c = Cache([70], 1, 64, 16, "bf16", 3)
    k, v, tables, desc = c.device(pa)
    q = torch.randn((1, 6144, 64), generator=torch.Generator().manual_seed(4)).bfloat16()
    o, w = torch.empty((1, 6144, 64), device="cuda"), torch.zeros((1, 1, 70), device="cuda")
    ws = torch.empty(pa.pa_decode_weights_workspace_bytes(1, 6144, 1, 64, 70), dtype=torch.uint8, device="cuda")
    pa.pa_decode_weights(q.cuda(), k, v, desc, tables, torch.tensor([70], dtype=torch.int32, device="cuda"), 70, 0.125, o, w, workspace=ws)
    assert pa.pa_get_device_error() == 0
    ref, bound, a, rel = attend(q, c.rows("k", 0, 70), c.rows("v", 0, 70), torch.ones((1, 70), dtype=bool), 0.125, "bf16", "f32")
    check(o, ref, bound, "output")
    # 6144 terms in order, each rounding at most half a step of the running sum
    check(w[0], a.sum(1), (a * rel[..., None]).sum(1) + 2.0 ** -24 * 6146 * a.sum(1) + 1e-38, "weights")
