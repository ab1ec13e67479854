"""plan_step on the GPU against the step played through on lists, value for value."""
import numpy as np
import pytest
import torch

from oracle import steps

pytestmark = pytest.mark.gpu


class Plan:
    """A batch of sequences over a pool, with everything that the call writes filled with a mark."""

    def __init__(self, lens, new, block=256, free=None, borrowed=None, wide=None, rows=None, seed=0, capacity=None):
        rng = np.random.default_rng(seed)
        S = len(lens)
        have = [max(0, -(-min(L, 1 << 20) // block)) for L in lens]
        after = [max(0, -(-(min(L, 1 << 20) + max(min(n, 1 << 20), 0)) // block)) for L, n in zip(lens, new)]
        self.wide = max(after + [1]) + 1 if wide is None else wide
        need = sum(a - h for a, h, n in zip(after, have, new) if n > 0)
        free = need + 3 if free is None else free
        self.num_blocks = sum(have) + free + 2
        pages = rng.permutation(self.num_blocks).astype(np.int32)
        self.tables = np.full((S, self.wide), -1, np.int32)
        at = 0
        for s, h in enumerate(have):
            h = min(h, self.wide)
            self.tables[s, :h] = pages[at:at + h]
            at += h
        self.capacity = self.num_blocks if capacity is None else capacity
        self.stack = np.full(self.capacity, -7, np.int32)
        self.stack[:free] = pages[at:at + free][:self.capacity]
        self.free = free
        self.lens, self.new, self.block, self.borrowed = lens, new, block, borrowed
        self.rows = sum(max(n, 0) for n in new) if rows is None else rows

    def want(self):
        return steps.plan_step(self.new, self.lens, self.tables, self.stack, self.free, self.rows, self.num_blocks, self.block, self.borrowed)

    def device(self):
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
        S = len(self.lens)
        mark = lambda n: torch.full((n,), 99, dtype=torch.int32, device="cuda")
        return {"new_lens": i32(self.new), "context_lens": i32(self.lens), "block_tables": i32(self.tables), "free_blocks": i32(self.stack),
                "num_free": i32([self.free]), "new_context_lens": mark(S), "new_num_free": mark(1), "slot_mapping": mark(self.rows),
                "positions": mark(self.rows), "cu_seqlens_q": mark(S + 1), "cu_seqlens_k": mark(S + 1), "num_blocks": self.num_blocks,
                "block_size": self.block, "borrowed_blocks": None if self.borrowed is None else i32(self.borrowed),
                "dev_status": torch.zeros(1, dtype=torch.int32, device="cuda")}

    def check(self, pkv, args=None):
        args = self.device() if args is None else args
        pkv.plan_step(**args)
        torch.cuda.synchronize()
        want, status = self.want()
        for name, values in want.items():
            got = args[name].cpu().numpy().reshape(-1).tolist()
            assert got == np.asarray(values, dtype=np.int64).reshape(-1).tolist(), name
        assert int(args["dev_status"].item()) == status
        return args


def random_plan(seed, S, high, new, block, **more):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, high + 1, S).tolist()
    lens = [L // block * block if rng.random() < 0.2 else L for L in lens]
    what = rng.random(S)
    counts = rng.integers(1, new + 1, S)
    n = [-1 if w < 0.15 else 0 if w < 0.3 else int(c) for w, c in zip(what, counts)]
    borrowed = [int(rng.integers(0, L // block + 1)) if rng.random() < 0.5 else 0 for L in lens]
    return Plan(lens, n, block=block, borrowed=borrowed, seed=seed, **more)


@pytest.mark.parametrize("lens,new", [([5, 300], [1, 1]), ([0], [1]), ([256], [1]), ([255, 256, 257], [1, 1, 1]), ([0, 0], [300, 0]),
                                      ([700], [-1]), ([512, 100, 0], [-1, 600, 513]), ([10, 20], [0, 0]), ([0], [0]), ([0], [-1])])
def test_small_steps(lib, lens, new):
    Plan(lens, new).check(lib)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("S,high,new,block", [(64, 2048, 1, 256), (3, 5000, 700, 64), (300, 1000, 40, 128), (257, 3000, 1, 512), (1000, 300, 9, 64)])
def test_random_steps(lib, seed, S, high, new, block):
    random_plan(seed, S, high, new, block).check(lib)


@pytest.mark.parametrize("rows", [1023, 1024, 1025])
def test_about_as_many_rows_as_one_cta_writes(lib, rows):
    Plan([100, 0, 63, 700], [300, rows - 301, 0, 1], block=64).check(lib)


def test_many_sequences_none_with_rows(lib):
    """All of them pause or end: no rows at all."""
    Plan([(37 * s) % 700 for s in range(600)], [-(s % 2) for s in range(600)], block=64, rows=0).check(lib)


@pytest.mark.parametrize("S", [256, 257, 512, 513, 2048, 2049])
def test_as_many_sequences_as_threads(lib, S):
    random_plan(S, S, 600, 2, 64).check(lib)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("free", [0, 1, 7])
@pytest.mark.parametrize("S", [40, 600])
def test_too_few_blocks(lib, seed, free, S):
    """Sequences are refused from the first on that does not find its blocks, unless they need none."""
    random_plan(seed, S, 700, 100, 64, free=free).check(lib)  # (the flag too)


def test_a_refusal_closes_the_stack_for_the_rest(lib):
    """Three of five need a block and the stack has two: the third and the last are refused, the fourth needs none."""
    p = Plan([64, 128, 0, 63, 64], [1, 1, 100, 1, 1], block=64, free=2)
    args = p.check(lib)
    assert int(args["dev_status"].item()) == lib.DEV_NO_BLOCKS
    assert args["new_context_lens"].tolist() == [65, 129, 0, 64, 64] and args["new_num_free"].item() == 0


@pytest.mark.parametrize("pad", [1, 5, 64])
def test_rows_behind_the_last_have_no_slot(lib, pad):
    p = random_plan(3, 50, 600, 1, 256)
    p.rows += pad
    args = p.check(lib)
    assert args["slot_mapping"][-pad:].tolist() == [-1] * pad


@pytest.mark.parametrize("S", [20, 700])
def test_rows_that_do_not_fit(lib, S):
    """Sequences whose rows would end behind the step's are refused; those before are not."""
    p = random_plan(5, S, 600, 30, 64)
    p.rows //= 2
    args = p.check(lib)
    assert int(args["dev_status"].item()) & lib.DEV_BAD_SEQLEN


def test_bad_lengths_touch_nobody_else(lib):
    wide = 4
    lens = [100, -5, 4 * 64 + 1, 200, 256, 30, 2**31 - 1, 60]
    new = [3, 2, 1, 60, 1, -3, 5, 2**31 - 1]
    p = Plan(lens, new, block=64, wide=wide, free=9, borrowed=[0, 1, 9, -2, 3, 0, 0, 0], rows=200)
    args = p.check(lib)
    assert int(args["dev_status"].item()) == lib.DEV_BAD_CONTEXT | lib.DEV_BAD_SEQLEN


@pytest.mark.parametrize("free,capacity", [(-3, 10), (50, 20)])
def test_a_bad_count_of_free_blocks(lib, free, capacity):
    p = Plan([10, 100], [1, 60], block=64, free=20, capacity=capacity)
    p.free = free
    args = p.check(lib)
    assert int(args["dev_status"].item()) & lib.DEV_BAD_BLOCK


def test_a_stack_without_room(lib):
    p = Plan([64 * 5, 64 * 3, 1], [-1, -1, 64], block=64, free=3, capacity=6)
    args = p.check(lib)
    assert int(args["dev_status"].item()) == lib.DEV_BAD_BLOCK


def test_block_ids_out_of_range_give_no_slots(lib):
    p = Plan([10, 70, 64], [1, 2, 70], block=64)
    p.tables[1, 1] = p.num_blocks
    p.stack[p.free - 1] = -4
    args = p.check(lib)
    assert int(args["dev_status"].item()) == lib.DEV_BAD_BLOCK
    assert (args["slot_mapping"] == -1).sum() > 2


@pytest.mark.parametrize("S", [50, 900])
def test_lengths_and_count_in_place(lib, S):
    p = random_plan(8, S, 900, 20, 128)
    args = p.device()
    args["new_context_lens"], args["new_num_free"] = args["context_lens"], args["num_free"]
    p.check(lib, args)


def test_a_call_can_be_repeated(lib):
    p = random_plan(9, 500, 900, 20, 64)
    args = p.check(lib)
    p.check(lib, args)


def test_no_sequences(lib):
    p = Plan([], [], wide=2, free=3)
    args = p.device()
    args["block_tables"] = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    lib.plan_step(**args)
    torch.cuda.synchronize()
    assert args["new_num_free"].item() == 3
    assert args["cu_seqlens_q"].tolist() == [0] and args["cu_seqlens_k"].tolist() == [0]


def test_the_most_sequences(lib):
    random_plan(11, 16384, 300, 3, 64).check(lib)


def test_sums_saturate(lib):
    """Lengths whose sum passes 2^31: the sums stop there, the rest holds."""
    S, wide = 3000, 1 << 14
    p = Plan([0] * S, [1] * S, block=64, wide=wide, free=S)
    p.lens = [64 * wide - 1] * S  # (only each one's last block is looked at)
    p.tables[:, wide - 1] = np.arange(S) % p.num_blocks
    args = p.check(lib)
    assert int(args["dev_status"].item()) == lib.DEV_BAD_SEQLEN
    assert args["cu_seqlens_k"][-1].item() == 2**31 - 1


def test_steps_replayed_from_a_graph(lib):
    """A captured step on lengths in place goes on from where the last one was, as step after step on lists does."""
    S, block, steps_run = 70, 64, 150
    p = Plan([60 + s for s in range(S)], [1] * S, block=block, wide=8, free=3 * S)
    args = p.device()
    args["new_context_lens"], args["new_num_free"] = args["context_lens"], args["num_free"]
    args.pop("dev_status")
    stream = torch.cuda.Stream()
    kept = {k: v.clone() for k, v in args.items() if torch.is_tensor(v)}
    with torch.cuda.stream(stream):
        lib.plan_step(**args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            lib.plan_step(**args)
    torch.cuda.synchronize()
    for k, v in kept.items():
        args[k].copy_(v)
    rng = np.random.default_rng(1)
    for step in range(steps_run):
        new = [int(x) for x in rng.choice([1, 1, 1, 1, 0, -1], S)]
        p.new, p.rows = new, S
        args["new_lens"].copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        want, _ = p.want()
        torch.cuda.synchronize()
        for name, values in want.items():
            assert args[name].cpu().numpy().reshape(-1).tolist() == np.asarray(values).reshape(-1).tolist(), (step, name)
        p.lens, p.free = want["new_context_lens"], want["new_num_free"][0]
        p.tables, p.stack = np.asarray(want["block_tables"], np.int32), np.asarray(want["free_blocks"], np.int32)


def test_agrees_with_the_block_manager(lib):
    """The host's allocator and the device's plan give the same places to the same tokens, up to the blocks' names."""
    block, prompts = 256, [300, 1, 256, 700]
    bm = lib.BlockManager(32, block)
    p = Plan([0] * 4, prompts, block=block, wide=5, free=20)
    args = p.check(lib)
    for s, n in enumerate(prompts):
        bm.allocate(s, list(range(1000 * s, 1000 * s + n)))
    cu = args["cu_seqlens_q"].tolist()
    slots = args["slot_mapping"].cpu().numpy()
    for s, n in enumerate(prompts):
        theirs, ours = bm.slots(s, 0, n), slots[cu[s]:cu[s + 1]]
        assert (theirs % block == ours % block).all()
        assert len(set(zip(theirs // block, ours // block))) == -(-n // block)


# Steps of more than 256 sequences or 1024 rows have two launches.

@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("S,high,new,block,free", [(40, 3000, 1500, 64, None), (700, 900, 120, 128, 30), (3, 100, 20000, 512, None)])
@pytest.mark.parametrize("least", [0, 1025, 16384, 49152, 400000])
def test_many_rows(lib, seed, S, high, new, block, free, least):
    p = random_plan(seed, S, high, new, block, free=free)
    p.rows = max(p.rows, least) + 3 * seed
    p.check(lib)


def test_many_rows_with_bad_lengths(lib):
    wide = 1000
    lens = [100, -5, wide * 64 + 1, 200, 256, 30, 60, 0]
    new = [29000, 2000, 1000, 60, 1, -3, 30000, 70000]
    p = Plan(lens, new, block=64, wide=wide, free=1000, rows=65000)
    p.check(lib)


def test_many_rows_block_ids_out_of_range(lib):
    p = Plan([10, 70, 64], [39000, 18000, 70], block=64)
    p.tables[1, 1] = p.num_blocks
    p.stack[p.free - 5] = -4
    args = p.check(lib)
    assert int(args["dev_status"].item()) == lib.DEV_BAD_BLOCK


def test_many_rows_in_place_and_sums_that_saturate(lib):
    S, wide = 3000, 1 << 14
    p = Plan([0] * S, [1] * S, block=64, wide=wide, free=S, rows=60000)
    p.lens = [64 * wide - 1] * S
    p.tables[:, wide - 1] = np.arange(S) % p.num_blocks
    args = p.device()
    args["new_context_lens"], args["new_num_free"] = args["context_lens"], args["num_free"]
    p.check(lib, args)


@pytest.mark.parametrize("rows", [300, 5000, 60000])
def test_on_streams_and_from_a_graph(lib, rows):
    """Two steps at a time over batches of their own, then both captured and replayed (one CTA, two launches)."""
    plans = [Plan([70 * s % 500 for s in range(30)], [rows // 30 + seed] * 30, block=64, seed=seed) for seed in range(2)]
    args = [p.device() for p in plans]
    wants = [p.want()[0] for p in plans]
    given = [{k: v.clone() for k, v in a.items() if torch.is_tensor(v)} for a in args]
    streams = [torch.cuda.Stream() for _ in plans]
    torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        for a, want in zip(args, wants):
            for name, values in want.items():
                assert a[name].cpu().numpy().reshape(-1).tolist() == np.asarray(values, dtype=np.int64).reshape(-1).tolist(), name

    for _ in range(3):
        for st, a in zip(streams, args):
            lib.plan_step(**a, stream=st)  # (lengths and count are not in place: it can be repeated)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a in args:
            lib.plan_step(**a)
    for a, was in zip(args, given):
        for name, t in was.items():
            a[name].copy_(t)
    graph.replay()
    same()


def test_refusals_of_the_binding(lib):
    a = Plan([5, 300], [1, 1]).device()
    for name in a:
        if not torch.is_tensor(a[name]):
            continue
        with pytest.raises((ValueError, TypeError)):
            lib.plan_step(**{**a, name: a[name].long()})
        if name not in ("free_blocks", "dev_status"):
            with pytest.raises(ValueError):
                lib.plan_step(**{**a, name: torch.cat([a[name], a[name]])})
        with pytest.raises(ValueError):
            lib.plan_step(**{**a, name: a[name].cpu()})
    with pytest.raises(lib.PkvError, match="UNSUPPORTED"):
        lib.plan_step(**{**a, "block_size": 2**32 + 256})
    with pytest.raises(lib.PkvError, match="INVALID_ARG"):
        lib.plan_step(**{**a, "num_blocks": -2**70})
