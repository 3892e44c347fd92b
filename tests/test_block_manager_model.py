"""The block manager under random calls, against a model that holds what every slot of the pool contains: whatever is shared,
copied, truncated, rewritten by an eviction or released under a window, each sequence finds its own tokens."""
import random

import numpy as np
import pytest

import paged_kv_cache_writes_gb300 as pa

BS, BLOCKS = 4, 48


class Model:
    """A token's content stands for its K and V: a function of its id and everything before it (None of two unknown tokens equal)."""

    def __init__(self, rng):
        self.bm, self.rng = pa.BlockManager(BLOCKS, BS, shuffle_seed=rng.randint(1, 99)), rng
        self.pool = {}                                     # slot -> content
        self.seqs = {}                                     # handle -> contents
        self.gone = {}                                     # handle -> positions whose blocks a window has left
        self.unique = 0

    def fresh(self):
        self.unique += 1
        return ("unique", self.unique)

    def copy(self, pairs):
        for src, dst in np.asarray(pairs).tolist():
            for o in range(BS):
                self.pool[dst * BS + o] = self.pool.get(src * BS + o)

    def new(self):
        s = self.bm.new_sequence()
        self.seqs[s], self.gone[s] = [], set()

    def fork(self, s):
        c = self.bm.fork(s)
        self.seqs[c], self.gone[c] = list(self.seqs[s]), set(self.gone[s])

    def free(self, s):
        self.bm.free(s)
        del self.seqs[s], self.gone[s]

    def append(self, s):
        n, rng = self.rng.randint(0, 11), self.rng
        # most prompts are alike, so that blocks are found again
        ids = rng.choice([[0] * n, [0] * n, [rng.randint(0, 1) for _ in range(n)], None])
        try:
            slots, pairs = self.bm.append(s, n, None if ids is None else np.array(ids, np.int32))
        except pa.PaError as e:
            assert e.status == 6
            return
        self.copy(pairs)
        for i, slot in enumerate(np.asarray(slots).tolist()):
            before = self.seqs[s][-1] if self.seqs[s] else "start"
            content = self.fresh() if ids is None else hash((before, ids[i]))
            self.seqs[s].append(content)
            if slot >= 0:
                self.pool[slot] = content

    def truncate(self, s):
        n = self.rng.randint(0, len(self.seqs[s]))
        keep = -(-n // BS) - 1
        if n % BS and keep * BS in self.gone[s]:
            with pytest.raises(pa.PaError):
                self.bm.truncate(s, n)
            return
        self.bm.truncate(s, n)
        self.seqs[s] = self.seqs[s][:n]
        self.gone[s] = {p for p in self.gone[s] if p < n}

    def evict(self, s):
        """unshare, a rewrite of the first n slots, truncate: as pa_evict leaves the pool."""
        if self.gone[s] or not self.seqs[s]:
            return
        n = self.rng.randint(1, len(self.seqs[s]))
        try:
            pairs = self.bm.unshare(s, n)
        except pa.PaError as e:
            assert e.status == 6
            return
        self.copy(pairs)
        table, _ = self.bm.block_table(s)
        for p in range(n):
            if self.rng.random() < 0.5:
                self.seqs[s][p] = self.fresh()
                self.pool[int(table[p // BS]) * BS + p % BS] = self.seqs[s][p]
        # what follows depends on tokens that are gone: no content of it is that of a prompt
        self.seqs[s][n - 1] = self.fresh()
        self.pool[int(table[(n - 1) // BS]) * BS + (n - 1) % BS] = self.seqs[s][n - 1]
        self.bm.truncate(s, n)
        self.seqs[s] = self.seqs[s][:n]

    def window(self, s):
        w, sinks, n = self.rng.randint(1, 12), self.rng.randint(0, 6), len(self.seqs[s])
        self.bm.release_window(s, w, sinks)
        for b in range(-(-sinks // BS), max(0, n + 1 - w) // BS):
            self.gone[s] |= set(range(b * BS, b * BS + BS))

    def check(self):
        used = set()
        for s, contents in self.seqs.items():
            table, n = self.bm.block_table(s)
            assert n == len(contents) and len(table) == -(-n // BS)
            for p, c in enumerate(contents):
                b = int(table[p // BS])
                assert (b < 0) == (p in self.gone[s])
                if b >= 0:
                    used.add(b)
                    assert self.pool[b * BS + p % BS] == c, (s, p)
        st = self.bm.stats()
        assert st.free_blocks == BLOCKS - len(used) and st.cached_blocks <= len(used)


@pytest.mark.parametrize("seed", range(40))
def test_random_calls(seed):
    rng, most = random.Random(seed), 2 + seed % 4          # with few sequences a block often loses its other owners
    m = Model(rng)
    m.new()
    for _ in range(300):
        if not m.seqs or (len(m.seqs) < most and rng.random() < 0.3):
            m.new()
        s = rng.choice(list(m.seqs))
        op = rng.choices([m.append, m.fork if len(m.seqs) < most else m.free, m.free, m.truncate, m.evict, m.window],
                         [8, 3, 4, 3, 1, 1])[0]
        op(s)
        m.check()
