"""plan_step as a captured loop calls it where it takes two launches: many sequences, lengths and
counts in place, step behind step on the device, against the steps played through on lists."""
import numpy as np
import pytest
import torch

from test_gpu_plan_step import Plan

pytestmark = pytest.mark.gpu

STEPS = 8  # of a graph


class Loop:
    def __init__(self, S, most, block=64, seed=0, room=20):
        self.rng = np.random.default_rng(seed)
        self.S, self.most, self.block = S, most, block
        lens = self.rng.integers(0, 3 * block, S).tolist()
        self.p = Plan(lens, [1] * S, block=block, wide=room, free=4 * S, seed=seed)
        self.p.rows = S * most + 3  # (padded)
        self.args = self.p.device()
        self.args["new_context_lens"], self.args["new_num_free"] = self.args["context_lens"], self.args["num_free"]
        of_step = ("new_lens", "slot_mapping", "positions", "cu_seqlens_q", "cu_seqlens_k", "dev_status")
        self.steps = [{**self.args, **{n: self.args[n].clone() for n in of_step}} for _ in range(STEPS)]
        self.state = [self.args[n] for n in ("context_lens", "block_tables", "free_blocks", "num_free")]

    def draw(self):
        """What the next steps ask for, as their lengths allow, and what each is to leave."""
        wants = []
        for a in self.steps:
            what = self.rng.random(self.S)
            new = [-1 if w < 0.03 else 0 if w < 0.1 else int(self.rng.integers(1, self.most + 1)) for w in what]
            self.p.new = [0 if n > 0 and L + n > self.p.wide * self.block else n for n, L in zip(new, self.p.lens)]
            want, status = self.p.want()
            wants.append((want, status))
            a["new_lens"].copy_(torch.tensor(self.p.new, dtype=torch.int32))
            a["dev_status"].zero_()
            self.p.lens, self.p.free = want["new_context_lens"], want["new_num_free"][0]
            self.p.tables, self.p.stack = np.asarray(want["block_tables"], np.int32), np.asarray(want["free_blocks"], np.int32)
        torch.cuda.synchronize()
        return wants

    def check(self, wants):
        torch.cuda.synchronize()
        for i, (a, (want, status)) in enumerate(zip(self.steps, wants)):
            assert int(a["dev_status"].item()) == status, i
            for name in ("slot_mapping", "positions", "cu_seqlens_q", "cu_seqlens_k"):
                assert a[name].cpu().numpy().tolist() == want[name], (i, name)
        for t, name in zip(self.state, ("new_context_lens", "block_tables", "free_blocks", "new_num_free")):
            assert t.cpu().numpy().reshape(-1).tolist() == np.asarray(wants[-1][0][name]).reshape(-1).tolist(), name


# (as many rows as one CTA of the first launch writes, many of them, and more sequences than threads)
@pytest.mark.parametrize("S,most", [(257, 1), (400, 1), (500, 3), (300, 60), (700, 2), (2500, 1)])
@pytest.mark.parametrize("captured", [True, False])
def test_steps_behind_one_another(lib, S, most, captured):
    loop = Loop(S, most, seed=S)
    kept = [t.clone() for t in loop.state]

    def run():
        for a in loop.steps:
            lib.plan_step(**a)

    if captured:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            run()
            for t, was in zip(loop.state, kept):
                t.copy_(was)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                run()
        torch.cuda.synchronize()
    for _ in range(12):
        wants = loop.draw()
        graph.replay() if captured else run()
        loop.check(wants)
    assert any(not torch.equal(a, b) for a, b in zip(kept, loop.state))


@pytest.mark.parametrize("S", [300, 1000])
def test_what_the_host_wrote_last_is_what_a_step_reads(lib, S):
    """Between steps other work on the stream changes lengths and tables, so that a line of them that an SM
    still has from the step before is another one in memory."""
    p = Plan([5] * S, [1] * S, block=64, wide=8, free=8 * S)
    args = p.device()
    args["new_context_lens"], args["new_num_free"] = args["context_lens"], args["num_free"]
    lens = [torch.full((S,), L, dtype=torch.int32, device="cuda") for L in (5, 63, 64, 130, 400)]
    gen = torch.Generator(device="cuda").manual_seed(S)
    tables = [torch.randint(0, p.num_blocks, (S, 8), generator=gen, dtype=torch.int32, device="cuda") for _ in lens]
    free, stack = args["num_free"].clone(), args["free_blocks"].clone()
    got = []
    for it in range(40):
        i = it % len(lens)
        args["context_lens"].copy_(lens[i])
        args["block_tables"].copy_(tables[i])
        args["num_free"].copy_(free)
        args["free_blocks"].copy_(stack)
        lib.plan_step(**args)
        got.append({n: args[n].clone() for n in ("context_lens", "block_tables", "slot_mapping", "positions", "num_free")})
    torch.cuda.synchronize()
    p.stack = stack.cpu().numpy()
    for it, g in enumerate(got):
        i = it % len(lens)
        p.lens, p.tables = lens[i].tolist(), tables[i].cpu().numpy()
        want, _ = p.want()
        assert g["context_lens"].tolist() == want["new_context_lens"], it
        assert g["num_free"].tolist() == want["new_num_free"], it
        for name in ("slot_mapping", "positions", "block_tables"):
            assert g[name].cpu().numpy().tolist() == want[name], (it, name)
