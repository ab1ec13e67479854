"""Key weights and eviction directly behind other calls of the library, and on
blocks that several sequences of a call hold (tolerances: test_gpu_key_weights)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import i32, oracle_caches
from test_gpu_key_weights import Step, assert_weights, batch, prompts, weight_rtol

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


# ------------------------------------- one sequence's own key, another's cached one

def check_shared(st, tables, call, oracle_call):
    """`call` ten times on stale sums (NaN where a token arrives), against the oracle.
    A slot has an addition for each sequence at most, each off by 2^-24 of its result,
    which is no more than the last one's."""
    b = st.b
    ekc, _ = oracle_caches(b)
    kw, brought = oracle_call(st.sums0, ekc, tables)
    assert np.isfinite(kw[np.unique(tables[tables >= 0])][:, :, :1]).all()
    st.block_tables.copy_(i32(tables))
    for _ in range(10):
        st.kw.copy_(torch.from_numpy(st.sums0))
        call()
        assert st.status_value() == 0
        got = st.kw.double().cpu().numpy()
        bound = weight_rtol(b, ekc) * brought + b.num_seqs * 2.0**-24 * np.abs(kw)
        bad = ~(np.abs(got - kw) <= bound) & ~(np.isnan(got) & np.isnan(kw))
        assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside; the first at {np.argwhere(bad)[0]}"


def stale_sums(b, tables, first_own):
    """Running sums, NaN in the slots of tokens that the call brings."""
    sums = np.random.default_rng(5).random((b.num_blocks, b.num_kv_heads, b.block_size), dtype=np.float32)
    for s, (c, L) in enumerate(zip(first_own, b.context_lens)):
        p = np.arange(c, int(L))
        sums[tables[s, p // b.block_size], :, p % b.block_size] = np.nan
    return sums


@pytest.mark.parametrize("owner", ["first", "last"])
@pytest.mark.parametrize("window", [1, 40, 1 << 20])
@pytest.mark.parametrize("G,D,bs", [(2, 64, 64), (1, 128, 128), (8, 64, 256)])
def test_prompt_owner_of_a_prefix_and_those_that_find_it_in_one_call(lib, G, D, bs, window, owner):
    """Full blocks get their keys when a prompt is admitted, so the prompts admitted
    behind it hold its blocks before the call that fills them."""
    new = [3 * bs + 70, 5, bs + 9, 1, 200, 33]
    cached = [0] + [2 * bs] * 5
    at = 0
    if owner == "last":
        new, cached, at = new[::-1], cached[::-1], 5
    b = prompts(new, cached, G, 4, D, 91, block_size=bs)
    tables = np.array(b.block_tables)
    tables[:, :2] = tables[at, :2]
    st = Step(lib, b, sums=stale_sums(b, tables, cached))
    check_shared(st, tables, lambda: st.prefill_weights(window),
                 lambda sums, kc, t: oracle.prefill_weights(sums, b.q, kc, t, b.cu_seqlens_q, b.cu_seqlens_k, window, b.scale))


@pytest.mark.parametrize("owner", ["first", "last"])
def test_prompt_found_whole_computes_its_last_token_again(lib, owner):
    """The last token of a prompt whose blocks were all found is another sequence's
    key (here still its own): the slot collects from both."""
    new, cached = [512, 1, 1], [0, 255, 511]
    at = 0
    if owner == "last":
        new, cached, at = new[::-1], cached[::-1], 2
    b = prompts(new, cached, 2, 4, 64, 92)
    tables = np.array(b.block_tables)
    for s in range(3):
        n = (new[s] + cached[s]) // 256
        tables[s, :n] = tables[at, :n]
    st = Step(lib, b, sums=stale_sums(b, tables, cached))
    check_shared(st, tables, lambda: st.prefill_weights(1 << 20),
                 lambda sums, kc, t: oracle.prefill_weights(sums, b.q, kc, t, b.cu_seqlens_q, b.cu_seqlens_k, 1 << 20, b.scale))


@pytest.mark.parametrize("newest", ["first", "last"])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_decode_whose_newest_slot_is_in_a_shared_block(lib, G, newest):
    lens = [256, 300, 256, 900]
    if newest == "last":
        lens = lens[::-1]
    b = batch(lens, G, 4, 64, 93)
    tables = np.array(b.block_tables)
    tables[:, 0] = tables[0, 0]
    st = Step(lib, b, sums=stale_sums(b, tables, [L - 1 for L in lens]))
    check_shared(st, tables, st.decode_weights,
                 lambda sums, kc, t: oracle.decode_weights(sums, b.q, kc, t, b.context_lens, b.scale))


# ---------------------------------------------------------------- two calls at a time

def test_prompts_on_two_streams(lib):
    """Each pass takes all of an SM's tensor memory; calls on two streams take turns."""
    shapes = [([900, 300, 64, 1200], [100, 0, 700, 0]), ([33, 1500, 257], [2000, 0, 31])]
    steps = [Step(lib, prompts(new, cached, 2, 2, 128, 94 + i)) for i, (new, cached) in enumerate(shapes)]
    windows = (1 << 20, 48)
    want, spaces = [], []
    for st, window in zip(steps, windows):
        b = st.b
        spaces.append(lib.prefill_weights_workspace(b.num_seqs, b.q.shape[0], int(b.new_lens.max()), window, b.num_q_heads,
                                                    b.num_kv_heads, b.block_tables.shape[1], b.block_size))
        st.prefill_weights(window, ws=spaces[-1])
        want.append(st.kw.clone())
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for st in steps:
            st.kw.copy_(torch.from_numpy(st.sums0))
        torch.cuda.synchronize()
        for st, window, ws, stream in zip(steps, windows, spaces, streams):
            st.prefill_weights(window, ws=ws, stream=stream)
        torch.cuda.synchronize()
        for st, kw in zip(steps, want):
            assert torch.equal(st.kw, kw) and st.status_value() == 0


@pytest.mark.parametrize("S", [639, 641, 1300])
def test_prompts_of_more_sequences_than_a_cta_has_threads(lib, S):
    """Every thread of a CTA counts the work of one sequence, of two or three."""
    rng = np.random.default_rng(S)
    b = prompts(rng.integers(1, 40, S).tolist(), rng.integers(0, 60, S).tolist(), 2, 2, 64, 98, block_size=64)
    st = Step(lib, b)
    st.prefill_weights(16)
    assert st.status_value() == 0
    ekc, _ = oracle_caches(b)
    kw, brought = oracle.prefill_weights(st.sums0, b.q, ekc, b.block_tables, b.cu_seqlens_q, b.cu_seqlens_k, 16, b.scale)
    assert_weights(st.kw, kw, brought, weight_rtol(b, ekc), f"{S} sequences")
