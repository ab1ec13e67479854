"""Key weights and eviction directly behind other calls of the library, and on
blocks that several sequences of a call hold (tolerances: test_gpu_key_weights)."""
import numpy as np
import pytest
import torch

from gpu_util import i32
from test_gpu_key_weights import Step, batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", ["decode", "decode with store", "refused decode"])
@pytest.mark.parametrize("op", ["decode", "prompt", "evict"])
def test_calls_wait_for_the_decode_before_them(lib, op, first):
    """Contexts of one block in a table of several: the decode's second launch has
    nothing to join.  What follows reads the token that the first one stores, or
    moves rows that it reads, so it must not start while that one still runs."""
    b = batch([512 - i % 3 for i in range(76)], 2, 8, 128, 90, block_size=512, max_blocks_pad=3)
    S = b.num_seqs
    st = Step(lib, b, store=False)
    mtb = 1 if first == "refused decode" else b.total_blocks_used
    dws = lib.decode_workspace(S, 16, 8, 128, b.total_blocks_used)
    wws, ids = st.workspace(), b.block_tables.shape[1]
    pws = lib.prefill_weights_workspace(S, S, 1, 4, 16, 8, ids, 512)
    kept = torch.empty((S, 8, 256), dtype=torch.int32, device="cuda")
    new_lens = torch.empty((S,), dtype=torch.int32, device="cuda")
    first_out = torch.empty_like(st.out)
    saved = [t.clone() for t in (st.k_cache, st.v_cache, st.kw)]

    def one():
        args = (st.k_cache, st.v_cache, st.block_tables, st.context_lens, b.scale, dws, mtb)
        if first == "decode with store":
            lib.paged_decode_store_attn(first_out, st.q, st.k, st.v, st.slot_mapping, *args)
        else:
            lib.paged_decode_attn(first_out, st.q, *args)

    def two():
        if op == "decode":
            st.decode_weights(ws=wws)
        elif op == "prompt":
            st.prefill_weights(4, ws=pws)
        else:
            lib.kv_evict(st.k_cache, st.v_cache, st.kw, st.block_tables, st.context_lens, 256, 32, kept, new_lens, st.status)

    def both(between):
        for t, s in zip((st.k_cache, st.v_cache, st.kw), saved):
            t.copy_(s)
        for t in (st.out, first_out, kept, new_lens):
            t.fill_(7)
        torch.cuda.synchronize()
        one()
        between()
        two()
        torch.cuda.synchronize()
        return [t.clone() for t in (first_out, st.out, st.kw, st.k_cache, st.v_cache, kept, new_lens)]

    want = both(torch.cuda.synchronize)
    for _ in range(20):
        for a, c in zip(both(lambda: None), want):
            assert torch.equal(a, c)
    assert st.status_value() == 0
