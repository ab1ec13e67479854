"""paged_decode_shared_attn on batches as a server pads and captures them: groups with nobody in them, rows of q that hold
anything, outputs in the queries' place, very many heads, the longest contexts."""
import pytest
import torch

from test_gpu_decode_shared import Shared, share  # noqa: F401  (the fixture: prefixes are shared however short)

pytestmark = pytest.mark.gpu

both = pytest.mark.parametrize("always", [pytest.param(False, marks=pytest.mark.by_choice), True])


@both
def test_groups_with_nobody_in_them(lib, always):
    """A captured call has as many groups each time: the ones not needed are empty, wherever they are and whatever they share."""
    s = Shared([(3, [1, 70, 2]), (0, [300]), (2, [9] * 20)], 8, 2, 64)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    s.check(lib, group_starts=i32([0, 0, 3, 3, 3, 4, 4, 24, 24]), shared_blocks=i32([5, 3, 0, 4, 0, 1, 2, 0]))


@both
@pytest.mark.parametrize("groups,Hq,Hkv,D", [([(3, [1, 70, None, 5]), (0, [300]), (2, [9] * 20)], 8, 2, 64), ([(0, [5, 9, None])], 4, 4, 64),
                                             ([(40, [1 + i for i in range(40)]), (0, [3000, None])], 16, 4, 128)])
def test_queries_of_others_do_not_matter(lib, groups, Hq, Hkv, D, always):
    """NaN in the rows of sequences without tokens and of some others: the rest keeps its bits."""
    s = Shared(groups, Hq, Hkv, D)
    empty = [i for i, L in enumerate(s.ctx) if L == 0]
    s.check(lib, status=lib.DEV_BAD_CONTEXT)
    want = s.out.clone()
    bad = sorted({*empty, *range(1, len(s.ctx), 3)})
    s.q[bad] = float("nan")
    s.out.fill_(7.0)
    lib.paged_decode_shared_attn(**s.args(lib))
    torch.cuda.synchronize()
    good = [i for i in range(len(s.ctx)) if i not in bad]
    assert torch.equal(s.out[good], want[good])
    for i in bad:
        assert bool((s.out[i] == 7.0).all()) if i in empty else bool(s.out[i].isnan().all())


@both
@pytest.mark.parametrize("groups", [[(3, [1, 70, 5]), (0, [300])], [(60, [1 + i for i in range(40)])]])
def test_outputs_in_the_queries_place(lib, groups, always):
    s = Shared(groups, 8, 2, 64)
    s.check(lib)
    q = s.q.clone()
    lib.paged_decode_shared_attn(**{**s.args(lib), "q": q, "out": q})
    torch.cuda.synchronize()
    assert torch.equal(q, s.out)


@both
@pytest.mark.parametrize("groups,Hq,Hkv,D", [([(2, [1, 70])], 512, 512, 64), ([(0, [100])], 4096, 4096, 64), ([(1, [1, 3])], 2048, 2048, 128),
                                             ([(2, [5, 6, 7])], 4096, 512, 64), ([(3, [40, 1])], 4096, 4096, 64)])
def test_very_many_heads(lib, groups, Hq, Hkv, D, always):
    """More kv heads than warps on the GPU."""
    Shared(groups, Hq, Hkv, D, spare=1).check(lib)


@both
@pytest.mark.parametrize("groups,Hq,Hkv,D,block", [([(16383, [64, 1])], 2, 1, 64, 64), ([(0, [1 << 20])], 8, 1, 128, 512), ([(2047, [512] * 3)], 1, 1, 128, 512)])
def test_the_longest_contexts(lib, groups, Hq, Hkv, D, block, always):
    Shared(groups, Hq, Hkv, D, block).check(lib)
