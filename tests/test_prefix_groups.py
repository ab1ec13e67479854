"""BlockManager.prefix_groups: which sequences read their first blocks together (host)."""
import itertools
import random

import numpy as np
import pytest

import paged_kv_cache_241_gb300 as pkv

BS = 4


def manager(prompts, blocks=400):
    bm = pkv.BlockManager(blocks, BS)
    for i, p in enumerate(prompts):
        bm.allocate(10 * i, p)
    return bm, [10 * i for i in range(len(prompts))]


def check(bm, ids):
    """The groups are of all sequences, once each, and share what they are said to; returns them with what they save."""
    order, starts, shared = bm.prefix_groups(ids)
    assert sorted(order.tolist()) == list(range(len(ids)))
    assert starts[0] == 0 and starts[-1] == len(ids) and (np.diff(starts) > 0).all() and len(shared) == len(starts) - 1
    groups, saved = [], 0
    for g, k in enumerate(shared):
        members = [int(i) for i in order[starts[g]:starts[g + 1]]]
        rows = [bm.block_table(ids[i], 64)[:k].tolist() for i in members]
        assert all(r == rows[0] for r in rows) and all(b >= 0 for b in rows[0])
        assert len(members) > 1 or k == 0
        groups.append((sorted(members), int(k)))
        saved += (len(members) - 1) * int(k)
    return sorted(groups), saved


def tokens(*blocks):
    return [100 * b + i for b in blocks for i in range(BS)]


def test_one_shared_prefix():
    bm, ids = manager([tokens(1, 2, 3) + [7], tokens(1, 2, 3) + [8], tokens(1, 2, 4) + [9]])
    # (three that share two blocks save four readings, two that share three save three)
    assert check(bm, ids) == ([([0, 1, 2], 2)], 4)


def test_two_prompts_and_a_stranger():
    bm, ids = manager([tokens(1, 2) + [1], tokens(5, 6, 7) + [1], tokens(9), tokens(1, 2) + [2], tokens(5, 6, 7) + [2]])
    assert check(bm, ids) == ([([0, 3], 2), ([1, 4], 3), ([2], 0)], 5)


def test_a_deeper_pair_is_taken_out_where_that_saves_more():
    deep = tokens(1, *range(20, 29))
    bm, ids = manager([deep + [1], deep + [2], tokens(1, 2) + [1], tokens(1, 3) + [1]])
    # pair of 10 blocks and pair of 1: 11 readings; all four by one block: 3
    assert check(bm, ids) == ([([0, 1], 10), ([2, 3], 1)], 11)


def test_nothing_shared_and_no_sequences():
    bm, ids = manager([tokens(1), tokens(2), [5]])
    assert check(bm, ids) == ([([0], 0), ([1], 0), ([2], 0)], 0)
    order, starts, shared = bm.prefix_groups([])
    assert order.size == 0 and starts.tolist() == [0] and shared.size == 0


def test_the_same_prompt_twice():
    bm, ids = manager([tokens(1, 2), tokens(1, 2)])
    assert check(bm, ids) == ([([0, 1], 2)], 2)


def test_a_part_of_the_sequences():
    bm, ids = manager([tokens(1, 2) + [1], tokens(1, 2) + [2], tokens(1) + [3], tokens(4)])
    assert check(bm, [ids[3], ids[0], ids[2]]) == ([([0], 0), ([1, 2], 1)], 1)


def test_unknown_and_repeated_sequences_are_refused():
    bm, ids = manager([tokens(1), tokens(2)])
    for bad in ([ids[0], 777], [ids[0], ids[1], ids[0]]):
        with pytest.raises(pkv.PkvError, match="INVALID_ARG"):
            bm.prefix_groups(bad)
    with pytest.raises(ValueError):
        bm.prefix_groups([[ids[0]]])


def partitions(items):
    if not items:
        yield []
        return
    first, rest = items[0], items[1:]
    for k in range(len(rest) + 1):
        for others in itertools.combinations(rest, k):
            left = [x for x in rest if x not in others]
            for p in partitions(left):
                yield [[first, *others], *p]


@pytest.mark.parametrize("seed", range(40))
def test_random_trees_save_what_the_best_partition_does(seed):
    """Against every partition of up to seven sequences."""
    rng = random.Random(seed)
    prompts = []
    for _ in range(rng.randint(1, 7)):
        base = rng.choice(prompts)[: BS * rng.randint(0, 6)] if prompts and rng.random() < 0.8 else []
        prompts.append(base[: len(base) // BS * BS] + tokens(*[rng.randint(1, 3) for _ in range(rng.randint(0, 5))]) + [rng.randint(0, 9)])
    bm, ids = manager(prompts)
    groups, saved = check(bm, ids)
    rows = [bm.block_table(i, 64).tolist() for i in ids]

    def common(some):
        n = 0
        while all(rows[i][n] >= 0 and rows[i][n] == rows[some[0]][n] for i in some):
            n += 1
        return n

    best = max(sum((len(g) - 1) * common(g) for g in p if len(g) > 1) for p in partitions(list(range(len(ids)))))
    assert saved == best


def test_many_sequences_in_a_chain():
    """Each of 300 prompts goes on where the one before it stops: as many ranges inside each other."""
    long = tokens(*range(300))
    bm, ids = manager([long[: BS * (i + 1)] for i in range(300)])
    check(bm, ids)
