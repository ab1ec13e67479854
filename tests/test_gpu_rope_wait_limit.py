"""norm_rope_store when the copies of some CTAs never come: their warps give up within the (shortened) limit and say
so, rows and slots are right or as they were, and the next call is as any other."""
import pytest
import torch

from test_gpu_norm_rope import FEW, WHOLE, Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def restored(lib):
    yield
    lib.test_rope_fault(10**9, -1)


@pytest.mark.parametrize("loading", [0, 1, 40])
@pytest.mark.parametrize("T,Hq,Hkv,D", [(FEW + 200, 16, 8, 128), (5000, 5, 2, 64), (WHOLE + 400, 2, 1, 128)])
def test_a_wait_that_runs_out_then_the_next_call(lib, T, Hq, Hkv, D, loading):
    r = Rows(T, Hq, Hkv, D, D)
    kc, vc = r.kc.clone(), r.vc.clone()
    lib.test_rope_fault(2_000_000, loading)
    r.call(lib, k_out=True)
    lib.test_rope_fault(10**9, -1)
    assert int(r.status.item()) == lib.DEV_TIMEOUT
    partly = [x.clone() for x in (r.q_out, r.k_out, r.kc, r.vc)]
    r.status.zero_(), r.kc.copy_(kc), r.vc.copy_(vc), r.q_out.fill_(7.0), r.k_out.fill_(7.0)
    r.check(lib, k_out=True)
    kept = r.slots[r.slots >= 0].long()
    rows = lambda x: x.flatten(1).view(torch.int16)
    for got, want, was in ((partly[0], r.q_out, torch.full_like(r.q_out, 7.0)), (partly[1], r.k_out, torch.full_like(r.k_out, 7.0)),
                           *((g.flatten(0, 1), w.flatten(0, 1), o.flatten(0, 1)) for g, w, o in ((partly[2], r.kc, kc), (partly[3], r.vc, vc)))):
        # (a head at a time: a token may come in halves)
        heads = lambda x: x.reshape(-1, D).view(torch.int16)
        right = (heads(got) == heads(want)).all(1)
        left = (heads(got) == heads(was)).all(1)
        assert bool((right | left).all())
        assert not bool(right.all()) and (loading > 0 or bool(left.all()))
    for got, was in ((partly[2], kc), (partly[3], vc)):
        rest = torch.ones(kc.shape[0] * kc.shape[1], dtype=torch.bool, device="cuda")
        rest[kept] = False
        assert torch.equal(rows(got.flatten(0, 1))[rest], rows(was.flatten(0, 1))[rest])


def test_few_tokens_wait_for_nothing(lib):
    lib.test_rope_fault(2_000_000, 0)
    Rows(FEW, 4, 2, 64).check(lib)
