"""Waits of the prompt key weights that run out, without a fault or a hang (as
test_gpu_wait_limit does for decode): the limit is cut to 2 ms and some CTAs of one
pass load nothing, so that all else in them waits for tiles that never come."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import i32, oracle_caches
from test_gpu_key_weights import Step, assert_weights, prompts, weight_rtol

pytestmark = pytest.mark.gpu

CASES = {
    "whole": dict(new=[1700, 300, 64, 1200], cached=[0, 700, 3, 0], window=1 << 20),
    "window": dict(new=[40, 300, 64, 33], cached=[5000, 700, 9000, 1], window=32),
}


def workspace(lib, b, window):
    return lib.prefill_weights_workspace(b.num_seqs, b.q.shape[0], int(b.new_lens.max()), window, b.num_q_heads,
                                         b.num_kv_heads, b.block_tables.shape[1], b.block_size)


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("loading", [0, 1, 40])
@pytest.mark.parametrize("which", [1, 2])
def test_prompt_wait_runs_out_then_next_call_is_correct(lib, which, loading, D, case):
    c = CASES[case]
    window = c["window"]
    b = prompts(c["new"], c["cached"], 2, 4, D, 95)
    st = Step(lib, b)
    ws = workspace(lib, b, window)
    # denominators of an earlier call, which this one must not take for its own
    other = Step(lib, prompts(c["new"], c["cached"], 2, 4, D, 96))
    other.prefill_weights(window, ws=ws)
    assert other.status_value() == 0
    try:
        lib.test_prompt_fault(2_000_000, which, loading)
        st.prefill_weights(window, ws=ws)
        torch.cuda.synchronize()
    finally:
        lib.test_prompt_fault(1_000_000_000, 1, -1)
    assert st.status_value() & lib.DEV_TIMEOUT
    ekc, _ = oracle_caches(b)
    kw, brought = oracle.prefill_weights(st.sums0, b.q, ekc, b.block_tables, b.cu_seqlens_q, b.cu_seqlens_k, window, b.scale)
    rtol = weight_rtol(b, ekc)
    if which == 1:
        # rows are left out, all of them where no CTA loads; none weighs by the earlier
        # call's denominators
        got, base = st.kw.double().cpu().numpy(), kw - brought
        off = rtol * brought + 2.0**-23 * np.abs(kw)
        assert (got >= base - off).all() and (got <= kw + off).all()
        if loading == 0:
            assert (got == np.where(np.isclose(base, 0.0, atol=1e-12), 0.0, st.sums0)).all()
    st.status.zero_()
    st.kw.copy_(torch.from_numpy(st.sums0))
    st.prefill_weights(window, ws=ws)
    assert st.status_value() == 0
    assert_weights(st.kw, kw, brought, rtol, "prompt weights after a timed-out call")


def test_prompt_limit_does_not_count_the_first_pass(lib):
    """Runs of the first pass take the same steps but not the same time (here 8 ms, up
    to a fifth less): the second pass's CTAs that begin on the SMs that end first must
    not take the others' remaining time for their own waits'."""
    D, H, BS, new = 64, 16, 512, 40960
    seqs = [(1, 639)] * 3000 + [(new, 0)]
    need = [-(-(n + c) // BS) for n, c in seqs]
    tables = np.full((len(seqs), max(need)), -1, np.int32)
    ends = np.cumsum(need)
    for s, (n, end) in enumerate(zip(need, ends)):
        tables[s, :n] = np.arange(end - n, end)
    cu_q, cu_k = (i32(np.concatenate([[0], np.cumsum(x)])) for x in ([n for n, _ in seqs], [n + c for n, c in seqs]))
    gen = torch.Generator(device="cuda").manual_seed(97)
    kc = torch.randn(int(ends[-1]), BS, H, D, generator=gen, device="cuda").bfloat16()
    q = torch.randn(new + 3000, H, D, generator=gen, device="cuda").bfloat16()
    tables = i32(tables)
    ws = lib.prefill_weights_workspace(len(seqs), q.shape[0], new, 1 << 20, H, H, tables.shape[1], BS)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        kw = torch.zeros((kc.shape[0], H, BS), device="cuda")
        lib.paged_prefill_weights(kw, q, kc, tables, cu_q, cu_k, new, 1 << 20, D**-0.5, ws, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        return kw

    want = call()
    try:
        lib.test_prompt_fault(500_000, 1, -1)  # healthy waits last microseconds
        assert torch.equal(call(), want)
    finally:
        lib.test_prompt_fault(1_000_000_000, 1, -1)
