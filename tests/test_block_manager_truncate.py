"""Prefix reuse after pa_bm_truncate has kept a shared block in part: once the block's other owners are gone, the truncated
sequence writes behind its kept part, and the block must not be found under its old contents any more."""
import numpy as np
import pytest

import paged_kv_cache_writes_gb300 as pa

IDS = np.array([1, 2, 3, 4], dtype=np.int32)
OTHER = np.array([9, 9], dtype=np.int32)


def filled(bm, ids):
    s = bm.new_sequence()
    slots, _ = bm.append(s, len(ids), ids)
    return s, slots


@pytest.mark.parametrize("how", ["fork", "reuse"])
@pytest.mark.parametrize("new_len", [1, 2, 3])
@pytest.mark.parametrize("given", [False, True])
def test_rewritten_block_is_not_reused(how, new_len, given):
    bm = pa.BlockManager(16, 4)
    a, _ = filled(bm, IDS)
    b = bm.fork(a) if how == "fork" else filled(bm, IDS)[0]
    assert np.array_equal(bm.block_table(a)[0], bm.block_table(b)[0]) and bm.stats().shared_blocks == 1
    bm.truncate(b, new_len)
    bm.free(a)                                             # b is the block's only owner now
    block = bm.block_table(b)[0][0]
    n = 4 - new_len
    slots, pairs = bm.append(b, n, np.full(n, 9, np.int32) if given else None)
    assert len(pairs) == 0 and np.array_equal(slots, block * 4 + np.arange(new_len, 4))   # in place
    c, got = filled(bm, IDS)
    assert (got >= 0).all() and bm.block_table(c)[0][0] != block


@pytest.mark.parametrize("how", ["fork", "reuse"])
def test_block_stays_reusable_until_it_is_rewritten(how):
    """Truncation alone changes no contents: the block is still found, and then the write behind the kept part copies it."""
    bm = pa.BlockManager(16, 4)
    a, _ = filled(bm, IDS)
    b = bm.fork(a) if how == "fork" else filled(bm, IDS)[0]
    bm.truncate(b, 2)
    bm.free(a)
    block = bm.block_table(b)[0][0]
    c, got = filled(bm, IDS)
    assert (got == -1).all() and bm.block_table(c)[0][0] == block
    slots, pairs = bm.append(b, 2, OTHER)
    assert pairs.tolist() == [[block, bm.block_table(b)[0][0]]] and bm.block_table(b)[0][0] != block
    assert np.array_equal(slots, bm.block_table(b)[0][0] * 4 + np.arange(2, 4))
    d, got = filled(bm, IDS)                               # c's block still holds what its name says
    assert (got == -1).all() and bm.block_table(d)[0][0] == block


def test_longer_sequences_and_their_first_blocks():
    bm = pa.BlockManager(32, 4)
    ids = np.arange(12, dtype=np.int32)
    a, _ = filled(bm, ids)
    b = bm.fork(a)
    bm.truncate(b, 6)
    bm.free(a)                                             # the third block goes, the second is b's in part
    first, second = bm.block_table(b)[0]
    bm.append(b, 1, OTHER[:1])
    c, got = filled(bm, ids)
    assert np.array_equal(got >= 0, np.arange(12) >= 4)    # the untouched first block is found, the others are not
    t = bm.block_table(c)[0]
    assert t[0] == first and second not in t
    bm.free(b)
    bm.free(c)
    assert bm.stats().free_blocks == 32 and bm.stats().cached_blocks == 0


def test_an_append_that_is_refused_forgets_nothing():
    bm = pa.BlockManager(2, 4)
    a, _ = filled(bm, IDS)
    b = bm.fork(a)
    bm.truncate(b, 2)
    bm.free(a)
    with pytest.raises(pa.PaError):
        bm.append(b, 11)                                   # needs three blocks, one is free
    assert bm.stats().cached_blocks == 1
    bm.append(b, 0)
    assert bm.stats().cached_blocks == 1                   # nothing written, nothing forgotten
