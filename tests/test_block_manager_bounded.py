"""The block manager under a bounded cache: blocks made a sequence's own before an eviction, blocks behind a shortened
sequence released, blocks that a sliding window has left released out of the middle."""
import numpy as np
import pytest

import paged_kv_cache_writes_gb300 as pa


def filled(bm, n, ids=None):
    s = bm.new_sequence()
    bm.append(s, n, ids)
    return s


def test_unshare_copies_shared_blocks_once():
    bm = pa.BlockManager(32, 16)
    a = filled(bm, 100)                                   # 7 blocks
    b = bm.fork(a)
    before = bm.block_table(b)[0]
    pairs = bm.unshare(b, 50)                             # positions 0..49: 4 blocks
    after, n = bm.block_table(b)
    assert n == 100 and len(pairs) == 4
    assert np.array_equal(pairs[:, 0], before[:4]) and np.array_equal(pairs[:, 1], after[:4])
    assert np.array_equal(after[4:], before[4:]) and not set(after[:4]) & set(before)
    assert np.array_equal(bm.block_table(a)[0], before)
    assert len(bm.unshare(b, 50)) == 0                    # its own now
    assert len(bm.unshare(a, 50)) == 0                    # and the parent's are its own too
    assert bm.stats().shared_blocks == 3
    assert len(bm.unshare(a, 0)) == 0


def test_unshare_without_room_changes_nothing():
    bm = pa.BlockManager(9, 16)
    a = filled(bm, 96)
    b = bm.fork(a)
    before = bm.block_table(b)[0]
    with pytest.raises(pa.PaError) as e:
        bm.unshare(b, 64)                                 # 4 copies, 3 free blocks
    assert e.value.status == 6
    assert np.array_equal(bm.block_table(b)[0], before) and bm.stats().free_blocks == 3
    assert len(bm.unshare(b, 48)) == 3


def test_unshare_refusals():
    bm = pa.BlockManager(16, 16)
    a = filled(bm, 40)
    bm.fork(a)
    for args in ((a, -1), (a, 41), (9, 1)):
        with pytest.raises(pa.PaError):
            bm.unshare(*args)
    import ctypes
    n = ctypes.c_int32(7)
    pairs = np.zeros(2, np.int32)
    assert pa.lib().pa_bm_unshare(bm._h, a, 40, pairs.ctypes.data, 1, ctypes.byref(n)) == 1 and n.value == 3
    assert bm.stats().shared_blocks == 3                  # nothing changed


def test_rewritten_blocks_leave_prefix_reuse():
    bm = pa.BlockManager(64, 16)
    ids = np.arange(64, dtype=np.int32)
    a = filled(bm, 64, ids)
    b = filled(bm, 64, ids)                               # shares all four blocks
    assert bm.stats().shared_blocks == 4 and bm.stats().cached_blocks == 4
    pairs = bm.unshare(b, 20)                             # two blocks of b will be rewritten
    assert len(pairs) == 2
    c = filled(bm, 64, ids)                               # still finds a's
    assert np.array_equal(bm.block_table(c)[0], bm.block_table(a)[0])
    bm.free(c)
    bm.free(b)
    assert len(bm.unshare(a, 64)) == 0 and bm.stats().cached_blocks == 0
    d = filled(bm, 64, ids)
    assert not set(bm.block_table(d)[0]) & set(bm.block_table(a)[0])
    # what a appends now does not stand for the old prefix
    bm.append(a, 16, np.arange(64, 80, dtype=np.int32))
    e = filled(bm, 80, np.arange(80, dtype=np.int32))
    assert bm.block_table(a)[0][4] not in bm.block_table(e)[0]


@pytest.mark.parametrize("new_len,blocks", [(100, 7), (99, 7), (97, 7), (96, 6), (17, 2), (16, 1), (1, 1), (0, 0)])
def test_truncate(new_len, blocks):
    bm = pa.BlockManager(32, 16)
    a = filled(bm, 100)
    table = bm.block_table(a)[0]
    bm.truncate(a, new_len)
    after, n = bm.block_table(a)
    assert n == new_len and np.array_equal(after, table[:blocks])
    assert bm.stats().free_blocks == 32 - blocks
    slots, pairs = bm.append(a, 3)
    t = bm.block_table(a)[0]
    p = np.arange(new_len, new_len + 3)
    assert len(pairs) == 0 and np.array_equal(slots, t[p // 16].astype(np.int64) * 16 + p % 16)


def test_truncate_refusals_and_sharing():
    bm = pa.BlockManager(32, 16)
    a = filled(bm, 40)
    for args in ((a, -1), (a, 41), (5, 0)):
        with pytest.raises(pa.PaError):
            bm.truncate(*args)
    b = bm.fork(a)
    bm.truncate(b, 20)
    assert bm.stats().shared_blocks == 2 and len(bm.block_table(a)[0]) == 3
    slots, pairs = bm.append(b, 1)                        # the last block is shared: copied first
    assert len(pairs) == 1 and pairs[0, 0] == bm.block_table(a)[0][1]


def test_truncated_blocks_leave_prefix_reuse():
    bm = pa.BlockManager(64, 16)
    ids = np.arange(48, dtype=np.int32)
    a = filled(bm, 48, ids)
    bm.truncate(a, 20)                                    # its second block will be written behind
    bm.append(a, 28, ids[::-1][:28].copy())
    b = filled(bm, 48, ids)
    ta, tb = bm.block_table(a)[0], bm.block_table(b)[0]
    assert ta[0] == tb[0] and not set(ta[1:]) & set(tb[1:])
    c = filled(bm, 32, ids[:32])
    bm.truncate(c, 0)                                     # a sequence started over matches again
    bm.append(c, 32, ids[:32])
    assert np.array_equal(bm.block_table(c)[0], tb[:2])


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (40, 5), (64, 32), (33, 100), (500, 4)])
def test_release_window(bs, window, sinks):
    bm = pa.BlockManager(64, bs)
    a = filled(bm, 300)
    table = bm.block_table(a)[0]
    freed = bm.release_window(a, window, sinks)
    after, n = bm.block_table(a)
    assert n == 300 and len(after) == len(table)
    # the next query, at position 300, and every later one: a block stays if and only if one of its tokens is seen
    p = np.arange(300)
    seen = (p < sinks) | (p > 300 - window)
    for j in range(len(table)):
        own = (p // bs) == j
        if seen[own].any() or (j + 1) * bs > 300:
            assert after[j] == table[j]
        else:
            assert after[j] == -1
    assert freed == (after == -1).sum() and bm.stats().free_blocks == 64 - len(table) + freed
    assert bm.release_window(a, window, sinks) == 0
    slots, _ = bm.append(a, 40)                           # it goes on as before
    t = bm.block_table(a)[0]
    q = np.arange(300, 340)
    assert np.array_equal(slots, t[q // bs].astype(np.int64) * bs + q % bs)
    b = bm.fork(a)
    assert np.array_equal(bm.block_table(b)[0], t)
    bm.free(a)
    bm.free(b)
    assert bm.stats().free_blocks == 64


def test_release_window_keeps_others_blocks():
    bm = pa.BlockManager(64, 16)
    a = filled(bm, 160)
    b = bm.fork(a)
    table = bm.block_table(a)[0]
    assert bm.release_window(b, 20, 4) == 7
    assert np.array_equal(bm.block_table(a)[0], table) and bm.stats().free_blocks == 54
    with pytest.raises(pa.PaError):
        bm.truncate(b, 40)                                # would end inside a block it no longer has
    bm.truncate(b, 32)
    for args in ((b, 0, 0), (b, 1, -1), (9, 1, 1)):
        with pytest.raises(pa.PaError):
            bm.release_window(*args)
