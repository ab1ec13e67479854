"""Waits of the prompt key weights that run out, without a fault or a hang (as
test_gpu_wait_limit does for decode): the limit is cut to 2 ms and some CTAs of one
pass load nothing, so that all else in them waits for tiles that never come."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import oracle_caches
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
