"""The block manager against a model of what the cache's slots hold.

A slot's K and V depend on its token and on all before it, so a slot holds that whole
prefix; an eviction leaves what no prefix is in the places that it rewrites.  Sequences
come, grow, are cut and go at random over few different tokens, so that prefixes meet
often.  Whatever a prompt is told to find cached must hold its own prefix."""
import numpy as np
import pytest

import paged_kv_cache_241_gb300 as pkv
from test_abi import lib  # noqa: F401  (fixture: the built library, no GPU)


class Model:
    def __init__(self, num_blocks, block_size):
        self.bm = pkv.BlockManager(num_blocks, block_size)
        self.NB, self.BS = num_blocks, block_size
        self.slots = {}     # slot: the prefix that its K and V belong to
        self.seqs = {}      # id: tokens, None in the places of a cut

    def slot(self, seq, p):
        return int(self.bm.slots(seq, p, 1)[0])

    def write(self, seq, p):
        t = self.seqs[seq]
        self.slots[self.slot(seq, p)] = ("cut", seq, p) if None in t[: p + 1] else tuple(t[: p + 1])

    def allocate(self, seq, tokens):
        need = -(-len(tokens) // self.BS)
        try:
            cached = self.bm.allocate(seq, tokens)
        except pkv.PkvError as e:
            assert e.status == pkv.PKV_ERR_OUT_OF_BLOCKS and self.bm.num_free_blocks < need
            return 0
        assert 0 <= cached < len(tokens)
        self.seqs[seq] = list(tokens)
        for p in range(cached):
            assert self.slots[self.slot(seq, p)] == tuple(tokens[: p + 1]), (tokens, cached, p)
        for p in range(cached, len(tokens)):
            self.write(seq, p)
        return cached

    def append(self, seq, token):
        t = self.seqs[seq]
        if len(t) % self.BS == 0 and self.bm.num_free_blocks == 0:
            with pytest.raises(pkv.PkvError):
                self.bm.append(seq, token)
            return
        self.bm.append(seq, token)
        t.append(token)
        self.write(seq, len(t) - 1)

    def evict(self, seq, keep):
        t = self.seqs[seq]
        table = self.bm.block_table(seq, -(-len(t) // self.BS)).tolist()
        rewritten = table[: -(-keep // self.BS)]
        shared = len(t) > keep and any(self.bm.ref_count(b) > 1 for b in rewritten)
        if shared:
            with pytest.raises(pkv.PkvError, match="UNSUPPORTED"):
                self.bm.evict(seq, keep)
            return False
        self.bm.evict(seq, keep)
        if len(t) > keep:
            self.seqs[seq] = [None] * keep
            for p in range(keep):
                self.write(seq, p)
            return True
        return False

    def free(self, seq):
        self.bm.free(seq)
        del self.seqs[seq]

    def check(self):
        held = {}           # block: how many hold it
        for seq, t in self.seqs.items():
            assert self.bm.num_tokens(seq) == len(t)
            for b in self.bm.block_table(seq, -(-len(t) // self.BS)).tolist():
                held[b] = held.get(b, 0) + 1
        for b in range(self.NB):
            assert self.bm.ref_count(b) == held.get(b, 0)
        assert self.bm.num_free_blocks == self.NB - len(held)


@pytest.mark.parametrize("evictions", [False, True])
@pytest.mark.parametrize("seed", range(12))
def test_blocks_found_hold_the_prefix_they_are_found_for(lib, seed, evictions):  # noqa: F811
    rng = np.random.default_rng(seed)
    m = Model(int(rng.choice([12, 30])), int(rng.choice([2, 4])))
    found = cuts = 0
    for step in range(1500):
        what = rng.random()
        ids = list(m.seqs)
        if not ids or (what < 0.25 and len(ids) < 8):
            found += m.allocate(1000 + step, rng.integers(0, 2, int(rng.integers(1, 5 * m.BS))).tolist()) > 0
        elif what < 0.75:
            m.append(int(rng.choice(ids)), int(rng.integers(0, 2)))
        elif what < 0.85 and evictions:
            seq = int(rng.choice(ids))
            cuts += m.evict(seq, int(rng.integers(1, len(m.seqs[seq]) + 2)))
        elif what >= 0.85:
            m.free(int(rng.choice(ids)))
        m.check()
    assert found > 20 and (cuts > 20) == evictions


def test_a_block_is_not_found_for_a_prompt_that_starts_with_its_tokens(lib):  # noqa: F811
    """A sequence grows the tokens of a block that another answers for; the block after
    it still hangs on those, not on the start of a prompt."""
    bm = pkv.BlockManager(16, 4)
    bm.allocate(1, [1, 2, 3, 4])
    bm.allocate(2, [1])
    for t in (2, 3, 4, 5, 6, 7, 8):
        bm.append(2, t)
    assert bm.allocate(3, [5, 6, 7, 8, 9]) == 0
    assert bm.allocate(4, [1, 2, 3, 4, 5, 6, 7, 8, 9]) == 8


def test_evict_releases_a_shared_block_behind_the_budget(lib):  # noqa: F811
    """Two sequences can share a block and not the one before it, where both have the
    same tokens there in blocks of their own."""
    bm = pkv.BlockManager(16, 4)
    bm.allocate(1, [0, 1, 2, 3])
    bm.allocate(2, [0])
    for t in range(1, 10):
        bm.append(2, t)
    assert bm.allocate(3, list(range(8)) + [9]) == 8
    (head, tail, last), theirs = bm.block_table(2, 3).tolist(), bm.block_table(3, 3).tolist()
    assert theirs[:2] == [int(bm.block_table(1, 1)[0]), tail] and theirs[0] != head
    assert [bm.ref_count(b) for b in (head, tail, last)] == [1, 2, 1]
    free = bm.num_free_blocks
    with pytest.raises(pkv.PkvError, match="UNSUPPORTED"):
        bm.evict(2, 5)                                      # it would rewrite the shared block
    bm.evict(2, 3)
    assert bm.block_table(2, 3).tolist() == [head, -1, -1] and bm.num_tokens(2) == 3
    assert [bm.ref_count(b) for b in (head, tail, last)] == [1, 1, 0] and bm.num_free_blocks == free + 1
    assert bm.block_table(3, 3).tolist() == theirs
    assert bm.allocate(4, list(range(8)) + [7]) == 8 and bm.ref_count(tail) == 2
    for seq in (1, 2, 3, 4):
        bm.free(seq)
    assert bm.num_free_blocks == 16
