"""paged_decode_shared_attn where values of attended tokens are infinite: a weight above zero times infinity is infinity,
as in paged_decode_attn, whatever the parts that the weight is taken as."""
import pytest
import torch

from test_gpu_decode_shared import Shared, share  # noqa: F401  (the fixture: prefixes are shared however short)

pytestmark = pytest.mark.gpu

INF = float("inf")


def infinite(s, Hkv, D):
    """Every value of a dim, and single tokens' of others (a prefix's first and last, a tail's first and last)."""
    s.vc[:, :, 0, 7] = torch.where(s.vc[:, :, 0, 7].isnan(), s.vc[:, :, 0, 7], INF)
    d = 8
    for i, L in enumerate(s.ctx):
        for p in sorted({0, 63, L // 2, L - 1} & set(range(L))):
            j, d = i % Hkv, d + 1 if d + 1 < D else 8
            block = int(s.tables[i, p // s.block])
            s.vc[block, p % s.block, j, d] = -INF if p % 2 else INF


# (whether shared, small, short or neither: tables of one and of many blocks)
@pytest.mark.parametrize("wide", [0, 40])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (4, 2, 128), (8, 2, 64), (16, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("groups", [[(0, [1, 5, 100])], [(3, [1, 70, 64]), (0, [300])], [(20, [3 * i + 1 for i in range(40)])]])
@pytest.mark.parametrize("always", [pytest.param(False, marks=pytest.mark.by_choice), True])
def test_values_that_are_infinite(lib, groups, Hq, Hkv, D, wide, always):
    s = Shared(groups, Hq, Hkv, D, wide=wide)
    s.check(lib)
    finite = s.out.clone()
    infinite(s, Hkv, D)
    s.out.fill_(7.0)
    lib.paged_decode_shared_attn(**s.args(lib))
    torch.cuda.synchronize()
    for i, L in enumerate(s.ctx):
        blocks = torch.as_tensor(s.tables[i, :-(-L // s.block)].astype("int64"), device="cuda")
        v = s.vc[blocks].reshape(-1, Hkv, D)[:L]
        up, down = (v == INF).any(0), (v == -INF).any(0)  # [Hkv, D]
        got = s.out[i].view(Hkv, -1, D)
        each = lambda x: x[:, None, :].expand_as(got)
        assert bool((got[each(up & ~down)] == INF).all()), i
        assert bool((got[each(down & ~up)] == -INF).all()), i
        assert bool(got[each(up & down)].isnan().all()), i
        rest = each(~up & ~down)
        assert torch.equal(got[rest], finite[i].view(Hkv, -1, D)[rest]), i
        assert bool(rest.any()) and bool(each(up).any())


@pytest.mark.parametrize("always", [pytest.param(False, marks=pytest.mark.by_choice), True])
@pytest.mark.parametrize("groups", [[(0, [5, 100, 3])], [(2, [1, 70, 64]), (0, [300])]])
@pytest.mark.parametrize("wide", [0, 40])
def test_a_context_whose_logits_are_all_minus_infinity(lib, groups, wide, always):
    """Zero over zero: NaN, and nothing for the others; weights of zero behind it count nothing either."""
    s = Shared(groups, 8, 2, 64, wide=wide)
    s.q.abs_()
    s.check(lib)
    want = s.out.clone()
    last = len(s.ctx) - 1
    for b in range(-(-s.ctx[last] // s.block)):
        s.kc[int(s.tables[last, b])] = -INF
    s.out.fill_(7.0)
    lib.paged_decode_shared_attn(**s.args(lib))
    torch.cuda.synchronize()
    assert bool(s.out[last].isnan().all())
    # (all but the last sequence: it shares nothing)
    assert torch.equal(s.out[:last], want[:last])


@pytest.mark.parametrize("always", [pytest.param(False, marks=pytest.mark.by_choice), True])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (8, 2, 128), (8, 1, 64)])
@pytest.mark.parametrize("groups", [[(0, [5, 100, 3])], [(2, [1, 70, 64]), (0, [300])]])
@pytest.mark.parametrize("wide", [0, 40])
def test_huge_values_of_tokens_that_weigh_nothing(lib, groups, Hq, Hkv, D, wide, always):
    """Zero times the largest bf16 is zero: not a part of a weight that is kept above zero for infinities' sake."""
    s = Shared(groups, Hq, Hkv, D, wide=wide)
    s.q.abs_()
    places = [(int(s.tables[i, p // s.block]), p % s.block) for i, L in enumerate(s.ctx) for p in {0, L // 2} if L > 1]
    for block, at in places:
        s.kc[block, at] = -INF
    outs = []
    for value in (0.0, torch.finfo(torch.bfloat16).max):
        for block, at in places:
            s.vc[block, at] = value
        s.out.fill_(7.0)
        lib.paged_decode_shared_attn(**s.args(lib))
        torch.cuda.synchronize()
        outs.append(s.out.clone())
    some = [i for i, L in enumerate(s.ctx) if L > 2]
    assert bool(outs[0][some].isfinite().all()) and torch.equal(outs[0][some], outs[1][some])
