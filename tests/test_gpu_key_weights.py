"""Key weights and eviction on the GPU against the float64 oracle.

Tolerances, derived: a weight is exp(z - log sum), z = scale * sum of D products
that are exact in fp32 and summed in fp32 in some order.  The tensor cores' sum
may truncate where IEEE rounds, so each of the D additions is off by at most
2^-23 of the sum of magnitudes A = max_p sum_d |q_d k_d|, z by
scale * A * D * 2^-23, and z and the log sum by that each; the products with
log2(e), the two exponentials, the sums and the reciprocal add under 2^-17
(2^-24 |z log2 e| with |z| < 32, a few 2^-22 each).  A key's sum then has one
fp32 addition: 2^-24 of the result.  The attention output's bound is the other
attention tests' (bf16 output, fp32 accumulation, weights rounded to bf16).
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from gpu_util import DeviceBatch, assert_close, bf16, bits, i32, oracle_caches

pytestmark = pytest.mark.gpu


def weight_rtol(b, keys):
    """Relative bound on a weight of this batch (see above)."""
    q = np.abs(oracle.bf16_bits_to_f64(b.q)).max(axis=(0, 1))
    k = oracle.bf16_bits_to_f64(keys)
    k = np.abs(np.where(np.isfinite(k), k, 0.0)).max(axis=(0, 1, 2))
    # (an upper bound on A: the largest |q_d| times the largest |k_d|, dim by dim, and
    # no sum of products of such draws comes near it, so Cauchy-Schwarz below is used)
    qn = np.sqrt((oracle.bf16_bits_to_f64(b.q) ** 2).sum(-1).max())
    kk = oracle.bf16_bits_to_f64(keys)
    kn = np.sqrt((np.where(np.isfinite(kk), kk, 0.0) ** 2).sum(-1).max())
    A = min(float((q * k).sum()), float(qn * kn))
    return 2 * abs(b.scale) * A * b.head_dim * 2.0**-23 + 2.0**-17


def assert_weights(got, want, brought, rtol, what):
    got = got.double().cpu().numpy()
    bound = rtol * brought + 2.0**-23 * np.abs(want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    err = np.where(same, 0.0, np.abs(got - want))
    bad = ~same & ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} outside; worst "
                           f"{np.nanmax(np.where(bad, err / np.maximum(bound, 1e-300), 0))} of the bound")


def sums_for(b, seed=0):
    """Running sums of earlier steps, for every slot of the pool (stale ones too)."""
    return np.random.default_rng(seed).random((b.num_blocks, b.num_kv_heads, b.block_size), dtype=np.float32)


class Step(DeviceBatch):
    def __init__(self, lib, b, store=True, sums=None):
        super().__init__(lib, b, store=store)
        self.sums0 = sums_for(b) if sums is None else sums
        self.kw = torch.from_numpy(self.sums0.copy()).cuda()
        self.out = torch.full((b.q.shape[0], b.num_q_heads, b.head_dim), 7.0, dtype=torch.bfloat16, device="cuda")

    def workspace(self, mtb=None):
        b = self.b
        return self.pkv.decode_weights_workspace(b.num_seqs, b.num_q_heads, b.num_kv_heads, b.head_dim, b.block_size,
                                                 b.total_blocks_used if mtb is None else mtb)

    def decode_weights(self, mtb=None, fused=False, ws=None, stream=None):
        b = self.b
        mtb = b.total_blocks_used if mtb is None else mtb
        new = dict(k=self.k, v=self.v, slot_mapping=self.slot_mapping) if fused else {}
        self.pkv.paged_decode_weights_attn(self.out, self.kw, self.q, self.k_cache, self.v_cache, self.block_tables,
                                           self.context_lens, b.scale, self.workspace(mtb) if ws is None else ws, mtb,
                                           dev_status=self.status, stream=stream, **new)

    def prefill_weights(self, window, ws=None, stream=None):
        b = self.b
        mq = int(b.new_lens.max())
        if ws is None:
            ws = self.pkv.prefill_weights_workspace(b.num_seqs, b.q.shape[0], mq, window, b.num_q_heads, b.num_kv_heads,
                                                    b.block_tables.shape[1], b.block_size)
        self.pkv.paged_prefill_weights(self.kw, self.q, self.k_cache, self.block_tables, self.cu_q, self.cu_k, mq, window,
                                       b.scale, ws, dev_status=self.status, stream=stream)


def check_decode(lib, b, fused=False, mtb=None):
    st = Step(lib, b, store=not fused)
    st.decode_weights(mtb, fused)
    assert st.status_value() == 0
    ekc, evc = oracle_caches(b)
    want = oracle.paged_decode_attn(b.q, ekc, evc, b.block_tables, b.context_lens, b.scale)
    assert_close(st.out.double().cpu().numpy(), want, f"out {b.name}")
    kw, brought = oracle.decode_weights(st.sums0, b.q, ekc, b.block_tables, b.context_lens, b.scale)
    assert_weights(st.kw, kw, brought, weight_rtol(b, ekc), f"weights {b.name}")
    if fused:
        assert np.array_equal(bits(st.k_cache), ekc) and np.array_equal(bits(st.v_cache), evc)
    return st


def batch(lens, G=2, Hkv=2, D=64, seed=1, **kw):
    return wl.build_batch("kw", "decode", seed, [L - 1 for L in lens], [1] * len(lens), G * Hkv, Hkv, D, **kw)


# ------------------------------------------------------------------------ decode

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("fused", [False, True])
def test_decode_edge_lengths(lib, D, G, fused):
    check_decode(lib, batch([1, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 511, 513, 1000], G, 2, D, 10 + G + D,
                            num_blocks=40, max_blocks_pad=3, stale="nan"), fused)


@pytest.mark.parametrize("bs", [64, 128, 512])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_decode_block_sizes(lib, bs, Hkv):
    check_decode(lib, batch([1, bs - 1, bs, bs + 1, 3 * bs + 5, 700], 4, Hkv, 128, bs, block_size=bs, stale="nan"), True)


@pytest.mark.parametrize("mtb", [1 << 5, 1 << 9, 1 << 13])
def test_decode_with_a_loose_block_bound(lib, mtb):
    # The bound sizes the workspace, nothing else: results stay right.
    check_decode(lib, batch([1, 300, 2000, 1537], 2, 4, 128, 5), mtb=mtb)


def test_decode_many_sequences(lib):
    L = np.random.default_rng(8).integers(1, 90, size=1500)
    check_decode(lib, batch(L.tolist(), 2, 1, 64, 8, block_size=64), True)


def test_decode_long_sequence(lib):
    check_decode(lib, batch([20011, 3], 8, 1, 128, 9, block_size=64), True)


@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_decode_zero_and_negative_scale(lib, scale):
    check_decode(lib, dataclasses.replace(batch([1, 63, 257, 700], 2, 2, 64, 17), scale=scale))


def test_decode_is_the_decode_and_repeats_bit_for_bit(lib):
    b = batch([1, 300, 2048, 777], 4, 2, 128, 21)
    st = Step(lib, b)
    ws = st.workspace()
    st.decode_weights(ws=ws)
    first, kw = st.out.clone(), st.kw.clone()
    assert_close(first.double().cpu().numpy(), st.decode().double().cpu().numpy(), "against paged_decode_attn")
    st.kw.copy_(torch.from_numpy(st.sums0))
    st.decode_weights(ws=ws)
    assert torch.equal(first, st.out) and torch.equal(kw, st.kw)
    # once more: everything but the newest keys collects a second time
    st.decode_weights(ws=ws)
    blk, off = (st.slot_mapping // 256).long(), (st.slot_mapping % 256).long()
    assert torch.equal(st.kw[blk, :, off], kw[blk, :, off])
    assert (st.kw >= kw).all() and (st.kw > kw).any()


def test_decode_leaves_padded_rows_and_flags_them(lib):
    b = batch([5, 300, 70], 2, 2, 64, 22)
    st = Step(lib, b)
    st.context_lens[1] = 0
    st.block_tables[1] = -1
    st.decode_weights()
    assert st.status_value() == lib.DEV_BAD_CONTEXT
    # (how a sequence is split depends on the others' lengths: compared with the oracle, not bit for bit)
    ekc, evc = oracle_caches(b)
    want = oracle.paged_decode_attn(b.q, ekc, evc, b.block_tables, b.context_lens, b.scale)
    assert_close(st.out[[0, 2]].double().cpu().numpy(), want[[0, 2]], "beside a padded row")
    assert (st.out[1] == 7.0).all()
    kw, brought = oracle.decode_weights(st.sums0, b.q, ekc, b.block_tables, b.context_lens, b.scale)
    kw[b.block_tables[1]], brought[b.block_tables[1]] = st.sums0[b.block_tables[1]], 0.0
    assert_weights(st.kw, kw, brought, weight_rtol(b, ekc), "beside a padded row")


def test_decode_flags_bad_blocks_and_a_short_workspace_bound(lib):
    b = batch([5, 600, 70], 2, 2, 64, 23)
    ref = Step(lib, b)
    ref.decode_weights()
    for bad in (-1, b.num_blocks, 1 << 30):
        st = Step(lib, b)
        st.block_tables[1, 1] = bad
        st.decode_weights()
        assert st.status_value() == lib.DEV_BAD_BLOCK
        assert torch.equal(st.out[[0, 2]], ref.out[[0, 2]])
        other = np.setdiff1d(np.arange(b.num_blocks), b.block_tables[1])
        assert torch.equal(st.kw[other], ref.kw[other])
    st = Step(lib, b)
    st.decode_weights(mtb=2)
    # (in tiles of 32 tokens, 2 blocks of 256 hold 16; the batch has 1 + 19 + 3)
    assert st.status_value() == lib.DEV_WORKSPACE
    assert (st.out == 7.0).all() and np.array_equal(st.kw.cpu().numpy(), st.sums0)


def test_decode_context_longer_than_the_table(lib):
    b = batch([512], 2, 2, 64, 24)
    st = Step(lib, b)
    st.context_lens[0] = 513
    st.decode_weights()
    assert st.status_value() == lib.DEV_BAD_CONTEXT
    ekc, evc = oracle_caches(b)
    _, brought = oracle.decode_weights(st.sums0, b.q, ekc, b.block_tables, b.context_lens, b.scale)
    assert_weights(st.kw, st.sums0 + brought, brought, weight_rtol(b, ekc), "clamped: all added")


def test_decode_stops_at_lengths_that_add_up_past_32_bits(lib):
    """The sum of the tiles of all sequences is 2^32 less a few: far more than the
    workspace has room for, and negative in 32 bits."""
    S, blocks = 1024, 131070
    b = batch([5], 1, 1, 128, 19, block_size=512)
    st = Step(lib, b)
    q = torch.zeros((S, 1, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    tables = torch.zeros((S, blocks), dtype=torch.int32, device="cuda")
    lens = torch.full((S,), blocks * 512, dtype=torch.int32, device="cuda")
    assert S * (blocks * 512 // 16) > 2**31 and (S * (blocks * 512 // 16)) % 2**32 > 2**31
    ws = lib.decode_weights_workspace(S, 1, 1, 128, 512, 4)
    before = st.kw.clone()
    lib.paged_decode_weights_attn(out, st.kw, q, st.k_cache, st.v_cache, tables, lens, 1.0, ws, 4, dev_status=st.status)
    assert st.status_value() == lib.DEV_WORKSPACE
    assert (out == 7.0).all() and torch.equal(before, st.kw)


def test_decode_join_with_more_parts_than_ctas(lib):
    """512 sequences of eight kv heads: the second launch has four CTAs for each,
    the longest takes five parts and a bit."""
    check_decode(lib, batch([1] * 300 + [5400] + [70] * 210 + [4097], 1, 8, 64, 20, block_size=64))


def test_decode_nan_stays_in_its_sequence(lib):
    b = batch([40, 300], 2, 2, 64, 25)
    st = Step(lib, b)
    ref = Step(lib, b)
    ref.decode_weights()
    st.k_cache[int(b.block_tables[0, 0]), 3, 1] = float("nan")
    st.decode_weights()
    assert torch.equal(st.out[1], ref.out[1])
    assert torch.isnan(st.out[0, 2:]).all() and torch.equal(st.out[0, :2], ref.out[0, :2])
    blk = int(b.block_tables[0, 0])
    assert torch.isnan(st.kw[blk, 1, :40]).all() and torch.equal(st.kw[blk, 0], ref.kw[blk, 0])


def test_decode_slots_of_the_fused_store(lib):
    b = batch([5, 300, 70], 2, 2, 64, 26)
    st = Step(lib, b, store=False)
    before = st.k_cache.clone()
    st.slot_mapping[0] = -1                      # attended to, not stored
    st.slot_mapping[2] = b.num_blocks * 256      # out of range
    st.decode_weights(fused=True)
    assert st.status_value() == lib.DEV_BAD_SLOT
    ref = Step(lib, b)
    ref.decode_weights()
    assert torch.equal(st.out, ref.out) and torch.equal(st.kw, ref.kw)
    changed = (st.k_cache != before).flatten(2).any(-1).nonzero().tolist()
    assert changed == [[int(b.slot_mapping[1]) // 256, int(b.slot_mapping[1]) % 256]]


def test_decode_shared_prefix_collects_from_every_sequence(lib):
    b = batch([300, 280], 2, 2, 64, 27)
    st = Step(lib, b)
    st.block_tables[1, 0] = st.block_tables[0, 0]
    tables = np.array(b.block_tables)
    tables[1, 0] = tables[0, 0]
    st.decode_weights()
    assert st.status_value() == 0
    ekc, _ = oracle_caches(b)
    kw, brought = oracle.decode_weights(st.sums0, b.q, ekc, tables, b.context_lens, b.scale)
    assert_weights(st.kw, kw, brought, weight_rtol(b, ekc), "shared block")


# ------------------------------------------------------------------------ prompts

def check_prefill(lib, b, window):
    st = Step(lib, b)
    st.prefill_weights(window)
    assert st.status_value() == 0
    ekc, _ = oracle_caches(b)
    kw, brought = oracle.prefill_weights(st.sums0, b.q, ekc, b.block_tables, b.cu_seqlens_q, b.cu_seqlens_k, window, b.scale)
    assert_weights(st.kw, kw, brought, weight_rtol(b, ekc), f"weights {b.name} window {window}")
    return st


def prompts(new, cached, G=2, Hkv=2, D=64, seed=1, **kw):
    return wl.build_batch("pw", "prefill", seed, cached, new, G * Hkv, Hkv, D, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("window", [1, 19, 64, 1 << 20])
def test_prefill_lengths(lib, D, G, window):
    check_prefill(lib, prompts([1, 2, 16, 63, 64, 65, 127, 128, 129, 200], [0, 300, 5, 0, 64, 1, 127, 128, 0, 57], G, 2, D,
                               40 + G, stale="nan"), window)


@pytest.mark.parametrize("bs", [64, 128, 512])
@pytest.mark.parametrize("window", [33, 1 << 31])
def test_prefill_block_sizes(lib, bs, window):
    check_prefill(lib, prompts([1, bs, 130, 70], [bs - 1, 0, 2 * bs + 3, 0], 4, 3, 128, bs, block_size=bs, stale="nan",
                               max_blocks_pad=2), window)


@pytest.mark.parametrize("window", [32, 1 << 20])
def test_prefill_longer_prompts(lib, window):
    check_prefill(lib, prompts([700, 300], [1500, 0], 2, 1, 128, 50), window)


@pytest.mark.parametrize("G,Hkv,cached", [(1, 4, 0), (2, 2, 300), (8, 1, 0)])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_rows_of_many_tiles(lib, D, G, Hkv, cached):
    """More row tiles than any ring of the kernel has slots, most of whose products
    no row or key is hidden from, in heads of unlike lengths."""
    check_prefill(lib, prompts([1700, 129, 960, 1301], [cached, 0, cached, 7], G, Hkv, D, 36), 1 << 20)


def test_prefill_long_cache_few_queries(lib):
    check_prefill(lib, prompts([5, 40], [9000, 4090], 8, 1, 64, 51, block_size=64), 8)


def test_prefill_one_query_is_the_decode_step(lib):
    b = batch([1, 300, 777, 64], 4, 2, 128, 52)
    one, two = Step(lib, b), Step(lib, b)
    one.decode_weights()
    two.prefill_weights(3)
    rtol = weight_rtol(b, oracle_caches(b)[0])
    assert torch.allclose(one.kw, two.kw, rtol=2 * rtol, atol=1e-12)


@pytest.mark.parametrize("scale", [0.0, -0.125])
def test_prefill_zero_and_negative_scale(lib, scale):
    check_prefill(lib, dataclasses.replace(prompts([70, 150], [0, 90], 2, 2, 64, 53), scale=scale), 40)


def test_prefill_empty_chunks_change_nothing(lib):
    b = prompts([30, 7, 50], [20, 400, 0], 2, 2, 64, 54)
    ref = Step(lib, b)
    ref.prefill_weights(16)
    st = Step(lib, b)
    # the middle sequence brings nothing this time (its rows are left out of the packing)
    cu_q, cu_k = np.array([0, 30, 30, 80]), np.array(b.cu_seqlens_k)
    st.cu_q = i32(cu_q)
    st.q = torch.cat([st.q[:30], st.q[37:]]).contiguous()
    st.b = dataclasses.replace(b, q=np.concatenate([b.q[:30], b.q[37:]]))
    st.cu_k = i32([0, cu_k[1], cu_k[1] + 400, cu_k[1] + 400 + cu_k[3] - cu_k[2]])
    st.prefill_weights(16)
    assert st.status_value() == 0
    mine = b.block_tables[1][b.block_tables[1] >= 0]
    assert np.array_equal(st.kw[mine].cpu().numpy(), st.sums0[mine])
    other = np.setdiff1d(np.arange(b.num_blocks), mine)
    assert torch.equal(st.kw[other], ref.kw[other])


def test_prefill_flags_lengths_and_blocks(lib):
    b = prompts([30, 7, 50], [20, 600, 0], 2, 2, 64, 55)
    ref = Step(lib, b)
    ref.prefill_weights(16)
    mine = b.block_tables[1][b.block_tables[1] >= 0]
    other = np.setdiff1d(np.arange(b.num_blocks), mine)
    # more keys than the table holds; fewer keys than queries
    for len_k in (b.block_tables.shape[1] * 256 + 1, 6):
        st = Step(lib, b)
        ck = np.array(b.cu_seqlens_k)
        ck[2:] += len_k - (ck[2] - ck[1])
        st.cu_k = i32(ck)
        st.prefill_weights(16)
        assert st.status_value() == lib.DEV_BAD_SEQLEN
        assert np.array_equal(st.kw[mine].cpu().numpy(), st.sums0[mine])
        assert torch.equal(st.kw[other], ref.kw[other])
    for bad in (-1, b.num_blocks, 1 << 30):
        st = Step(lib, b)
        st.block_tables[1, 1] = bad
        st.prefill_weights(16)
        assert st.status_value() == lib.DEV_BAD_BLOCK
        assert torch.equal(st.kw[other], ref.kw[other])
        gone = int(b.block_tables[1, 1])
        assert np.array_equal(st.kw[gone].cpu().numpy(), st.sums0[gone])


def test_prefill_more_queries_than_stated(lib):
    b = prompts([30, 50], [0, 0], 2, 2, 64, 56)
    st = Step(lib, b)
    ws = lib.prefill_weights_workspace(2, 80, 30, 16, 4, 2, b.block_tables.shape[1], 256)
    lib.paged_prefill_weights(st.kw, st.q, st.k_cache, st.block_tables, st.cu_q, st.cu_k, 30, 16, b.scale, ws, st.status)
    assert st.status_value() == lib.DEV_BAD_SEQLEN
    mine = b.block_tables[1][b.block_tables[1] >= 0]
    assert np.array_equal(st.kw[mine].cpu().numpy(), st.sums0[mine])


def test_prefill_chunks_add_up_to_the_whole(lib):
    # Two chunks, every query counted, against the prompt at once.
    whole = prompts([300], [0], 2, 2, 64, 57)
    ref = Step(lib, whole)
    ref.prefill_weights(1 << 20)
    st = Step(lib, whole)
    row = dict(block_tables=st.block_tables, scale=whole.scale)
    for lo, hi in ((0, 170), (170, 300)):
        ws = lib.prefill_weights_workspace(1, hi - lo, hi - lo, 1 << 20, 4, 2, 2, 256)
        lib.paged_prefill_weights(st.kw, st.q[lo:hi].contiguous(), st.k_cache, row["block_tables"], i32([0, hi - lo]),
                                  i32([0, hi]), hi - lo, 1 << 20, row["scale"], ws, st.status)
    assert st.status_value() == 0
    used = whole.block_tables[0]
    rtol = weight_rtol(whole, oracle_caches(whole)[0])
    a, b_ = st.kw[used].transpose(1, 2).reshape(-1, 2)[:300], ref.kw[used].transpose(1, 2).reshape(-1, 2)[:300]
    assert torch.allclose(a, b_, rtol=2 * rtol, atol=0)


# ----------------------------------------------------------------------- eviction

def check_evict(lib, b, budget, recent, sums):
    st = Step(lib, b, sums=sums)
    ekc, evc = oracle_caches(b)
    kept = torch.full((b.num_seqs, b.num_kv_heads, budget), 99, dtype=torch.int32, device="cuda")
    new_lens = torch.full((b.num_seqs,), 99, dtype=torch.int32, device="cuda")
    lib.kv_evict(st.k_cache, st.v_cache, st.kw, st.block_tables, st.context_lens, budget, recent, kept, new_lens, st.status)
    assert st.status_value() == 0
    kc, vc, kw, want, lens = oracle.kv_evict(ekc, evc, st.sums0, b.block_tables, b.context_lens, budget, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(new_lens.cpu().numpy(), lens)
    assert np.array_equal(bits(st.k_cache), kc) and np.array_equal(bits(st.v_cache), vc)
    assert np.array_equal(st.kw.cpu().numpy().view(np.uint32), kw.astype(np.float32).view(np.uint32))
    return st


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (33, 0), (64, 7), (64, 64), (300, 1), (300, 150), (300, 299), (2000, 3)])
def test_evict_lengths(lib, D, budget, recent):
    b = batch([1, 32, 33, 34, 63, 64, 65, 299, 300, 301, 302, 450, 601, 1100], 2, 2, D, 60, stale="nan")
    check_evict(lib, b, budget, recent, sums_for(b, 1))


@pytest.mark.parametrize("bs,Hkv", [(64, 1), (128, 3), (512, 2)])
def test_evict_block_sizes(lib, bs, Hkv):
    b = batch([bs, bs + 1, 5 * bs + 17, 1500], 1, Hkv, 64, 61, block_size=bs, max_blocks_pad=2)
    check_evict(lib, b, bs, bs // 3, sums_for(b, 2))


def special(kind, b):
    s = sums_for(b, 3)
    rng = np.random.default_rng(4)
    if kind == "equal":
        s[:] = 0.25
    elif kind == "zeros":
        s[:] = np.where(rng.random(s.shape) < 0.5, 0.0, -0.0)
    elif kind == "few":
        s[:] = rng.integers(0, 4, s.shape)
    elif kind == "tiny":
        s[:] = s * 1e-40                          # subnormals keep their order
    elif kind == "odd":
        s[:] = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 3.4e38, -3.4e38], np.float32), s.shape)
    elif kind == "near":
        s[:] = (np.float32(1.0).view(np.uint32) + rng.integers(0, 40, s.shape).astype(np.uint32)).view(np.float32)
    return s


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "tiny", "odd", "near"])
def test_evict_ties_and_special_weights(lib, kind):
    b = batch([700, 2500, 130], 1, 2, 64, 62)
    check_evict(lib, b, 128, 16, special(kind, b))


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_evict_where_all_or_none_of_the_places_free_up(lib, order):
    b = batch([1500, 515], 1, 2, 64, 63)
    s = sums_for(b, 5)
    for t, L in zip(b.block_tables, b.context_lens):
        p = np.arange(int(L))
        s[t[p // 256], :, p % 256] = (p if order == "rising" else -p)[:, None]
    check_evict(lib, b, 512, 100, s)


def test_evict_long_context(lib):
    b = batch([40000, 70], 1, 1, 64, 64, block_size=512)
    check_evict(lib, b, 3000, 500, sums_for(b, 6))
    check_evict(lib, b, 39990, 20000, sums_for(b, 7))


@pytest.mark.parametrize("kind", ["few", "zeros"])
def test_evict_more_candidates_than_the_key_cache_holds(lib, kind):
    b = batch([70000, 45001], 1, 1, 64, 66, block_size=512)
    check_evict(lib, b, 30011, 77, special(kind, b))


@pytest.mark.parametrize("pad,lens", [(384, [70000, 300]), (512, [140000]), (1978, [35333]), (876, [600000])])
@pytest.mark.parametrize("kind", ["few", "random"])
def test_evict_with_a_long_table(lib, pad, lens, kind):
    """Tables up to the 2^20 tokens that a call may have, of contexts shorter and as long."""
    b = batch(lens, 1, 1, 64, 68, block_size=512, max_blocks_pad=pad)
    assert b.block_tables.shape[1] * 512 <= 1 << 20
    check_evict(lib, b, 5003, 77, sums_for(b, 8) if kind == "random" else special(kind, b))


def test_evict_bad_sequences_are_left_as_they_were(lib):
    b = batch([300, 600, 700, 40, 500], 2, 2, 64, 65)
    st = Step(lib, b)
    before = st.k_cache.clone(), st.v_cache.clone(), st.kw.clone()
    st.block_tables[0, 1] = b.num_blocks
    st.context_lens[1] = -5
    st.context_lens[2] = b.block_tables.shape[1] * 256 + 1
    st.context_lens[3] = 0
    kept = torch.full((5, 2, 128), 99, dtype=torch.int32, device="cuda")
    new_lens = torch.full((5,), 99, dtype=torch.int32, device="cuda")
    lib.kv_evict(st.k_cache, st.v_cache, st.kw, st.block_tables, st.context_lens, 128, 16, kept, new_lens, st.status)
    assert st.status_value() == lib.DEV_BAD_BLOCK | lib.DEV_BAD_CONTEXT
    assert (kept[:4] == -1).all() and (kept[4] >= 0).all()
    assert new_lens.tolist() == [300, -5, b.block_tables.shape[1] * 256 + 1, 0, 128]
    mine = b.block_tables[4][b.block_tables[4] >= 0]
    other = np.setdiff1d(np.arange(b.num_blocks), mine)
    for a, c in zip(before, (st.k_cache, st.v_cache, st.kw)):
        assert torch.equal(a[other].view(torch.uint8), c[other].view(torch.uint8))


def test_evict_outputs_are_there_for_the_next_kernel_when_nothing_moves(lib):
    """All sequences within the budget: the second launch has nothing to do, and must
    not let the stream go on before the first one has written its outputs."""
    S, Hkv, budget = 512, 8, 8192
    kc, vc = (torch.zeros((S, 64, Hkv, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kw = torch.zeros((S, Hkv, 64), device="cuda")
    tables = torch.arange(S, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = (torch.arange(S, device="cuda") % 64 + 1).int()
    kept = torch.empty((S, Hkv, budget), dtype=torch.int32, device="cuda")
    new_lens = torch.empty((S,), dtype=torch.int32, device="cuda")
    at = torch.arange(budget, dtype=torch.int32, device="cuda")
    want = torch.where(at < lens[:, None], at, -1)[:, None, :]
    seen = torch.empty_like(kept)
    for _ in range(20):
        kept.fill_(99)
        new_lens.fill_(99)
        lib.kv_evict(kc, vc, kw, tables, lens, budget, 16, kept, new_lens)
        lens_seen = new_lens.clone()
        seen.copy_(kept)
        assert torch.equal(lens_seen, lens) and (seen == want).all()


def off_by_one(t):
    """The same values 4 bytes past a 16-byte boundary."""
    flat = torch.empty(t.numel() + 1, device=t.device, dtype=t.dtype)
    moved = flat[1:].view(t.shape)
    moved.copy_(t)
    return moved


def test_sums_that_are_aligned_to_their_values_alone(lib):
    b = batch([300, 1100, 64], 4, 2, 64, 67)
    ref, st = Step(lib, b), Step(lib, b)
    st.kw = off_by_one(st.kw)
    outs = []
    for x in (ref, st):
        kept = torch.empty((3, 2, 200), dtype=torch.int32, device="cuda")
        new_lens = torch.empty((3,), dtype=torch.int32, device="cuda")
        x.decode_weights()
        x.prefill_weights(4)
        lib.kv_evict(x.k_cache, x.v_cache, x.kw, x.block_tables, x.context_lens, 200, 30, kept, new_lens, x.status)
        assert x.status_value() == 0
        outs.append((x.out, x.kw, x.k_cache, x.v_cache, kept))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


def test_prefill_is_the_same_every_time(lib):
    # Tiles cut between CTAs are joined by whichever finishes last, in one order.
    b = prompts([900, 300, 64, 1200], [100, 0, 700, 0], 2, 2, 128, 68)
    st = Step(lib, b)
    ws = lib.prefill_weights_workspace(4, b.q.shape[0], 1200, 1 << 20, 4, 2, b.block_tables.shape[1], 256)
    want = None
    for window in (1 << 20, 48) * 10:
        st.kw.copy_(torch.from_numpy(st.sums0))
        st.prefill_weights(window, ws=ws)
        if want is None:
            want = {}
        if window not in want:
            want[window] = st.kw.clone()
        assert torch.equal(st.kw, want[window])
    assert st.status_value() == 0


def test_workspaces_serve_calls_of_other_sizes(lib):
    # One workspace of each kind, as large as any call needs, for a mix of calls.
    dws = lib.decode_weights_workspace(8, 16, 2, 128, 64, 400)
    pws = lib.prefill_weights_workspace(8, 2000, 2000, 1 << 20, 16, 2, 64, 512)
    for seed in range(6):
        rng = np.random.default_rng(seed)
        G, D, bs = int(rng.choice([1, 2, 4, 8])), int(rng.choice([64, 128])), int(rng.choice([64, 256]))
        lens = rng.integers(1, 700, size=int(rng.integers(1, 8))).tolist()
        b = batch(lens, G, 2, D, seed, block_size=bs)
        st, ref = Step(lib, b), Step(lib, b)
        st.decode_weights(ws=dws)
        ref.decode_weights()
        assert torch.equal(st.out, ref.out) and torch.equal(st.kw, ref.kw)
        b = prompts(lens, rng.integers(0, 300, size=len(lens)).tolist(), G, 2, D, seed, block_size=bs)
        st, ref = Step(lib, b), Step(lib, b)
        window = int(rng.choice([3, 40, 1 << 20]))
        st.prefill_weights(window, ws=pws)
        ref.prefill_weights(window)
        assert torch.equal(st.kw, ref.kw)


# ------------------------------------------------- streams, graphs, calls together

def test_two_streams_with_workspaces_of_their_own(lib):
    steps = [Step(lib, batch([900, 1300, 64], 4, 2, 128, 70 + i)) for i in range(2)]
    want = []
    for st in steps:
        st.decode_weights()
        want.append((st.out.clone(), st.kw.clone()))
        st.kw.copy_(torch.from_numpy(st.sums0))
        st.out.fill_(7.0)
    spaces = [st.workspace() for st in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for st, ws, stream in zip(steps, spaces, streams):
        st.decode_weights(ws=ws, stream=stream)
    torch.cuda.synchronize()
    for st, (out, kw) in zip(steps, want):
        assert torch.equal(st.out, out) and torch.equal(st.kw, kw)


def test_captured_and_replayed(lib):
    b = batch([900, 1300, 64], 4, 2, 128, 72, num_blocks=16)
    st = Step(lib, b)
    ws = st.workspace(20)
    kept = torch.empty((3, 2, 256), dtype=torch.int32, device="cuda")
    new_lens = torch.empty((3,), dtype=torch.int32, device="cuda")
    pws = lib.prefill_weights_workspace(3, 3, 1, 4, 8, 2, b.block_tables.shape[1], 256)

    def go():
        st.decode_weights(mtb=20, ws=ws)
        lib.paged_prefill_weights(st.kw, st.q, st.k_cache, st.block_tables, st.cu_q, st.cu_k, 1, 4, b.scale, pws, st.status)
        lib.kv_evict(st.k_cache, st.v_cache, st.kw, st.block_tables, st.context_lens, 256, 32, kept, new_lens, st.status)

    saved = st.k_cache.clone(), st.v_cache.clone(), st.kw.clone(), st.context_lens.clone()

    def reset(lens):
        for t, s in zip((st.k_cache, st.v_cache, st.kw), saved):
            t.copy_(s)
        st.context_lens.copy_(i32(lens))
        st.cu_k.copy_(i32(np.concatenate([[0], np.cumsum(lens)])))

    def outputs():
        return [t.clone() for t in (st.out, st.kw, st.k_cache, st.v_cache, kept, new_lens)]

    results = []
    for lens in ([900, 1300, 64], [700, 1111, 1]):
        reset(lens)
        go()
        results.append(outputs())
    reset([900, 1300, 64])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for lens, want in zip(([900, 1300, 64], [700, 1111, 1]), results):
        for _ in range(2):
            reset(lens)
            g.replay()
            for a, c in zip(outputs(), want):
                assert torch.equal(a, c)
    assert st.status_value() == 0


def test_blocks_past_32_bits_of_elements(lib):
    """The same batch in the last blocks of caches of more than 2^32 values each."""
    b = batch([900, 1300, 64], 2, 8, 128, 74, block_size=512)
    ref, st = Step(lib, b), Step(lib, b)
    NB, per = b.num_blocks, 512 * 8 * 128
    big = (1 << 32) // per + 2 * NB
    assert (big - NB) * per > 1 << 32
    for name in ("k_cache", "v_cache", "kw"):
        small = getattr(st, name)
        pool = torch.empty((big, *small.shape[1:]), dtype=small.dtype, device="cuda")
        pool[big - NB:].copy_(small)
        setattr(st, name, pool)
    st.block_tables = torch.where(st.block_tables >= 0, st.block_tables + (big - NB), -1).int()
    st.slot_mapping = (st.slot_mapping + (big - NB) * 512).int()
    outs = []
    for x in (ref, st):
        kept = torch.empty((3, 8, 256), dtype=torch.int32, device="cuda")
        new_lens = torch.empty((3,), dtype=torch.int32, device="cuda")
        x.decode_weights(fused=True)
        x.prefill_weights(1)
        lib.kv_evict(x.k_cache, x.v_cache, x.kw, x.block_tables, x.context_lens, 256, 32, kept, new_lens, x.status)
        assert x.status_value() == 0
        outs.append((x.out, x.kw[-NB:], x.k_cache[-NB:], x.v_cache[-NB:], kept, new_lens))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


@pytest.mark.parametrize("before", ["kernel", "copy", "memset", "two streams", "nothing"])
@pytest.mark.parametrize("op", ["decode", "prompt", "evict"])
def test_calls_wait_for_what_is_before_them(lib, op, before):
    """The first launch of a call may start under the tail of what precedes it on the
    stream, whatever that is, and must see all of its results: inputs that slow work
    has just written, eagerly and in a captured graph."""
    b = batch([900, 1300, 64], 4, 2, 128, 73, num_blocks=16)
    st = Step(lib, b)
    ws = st.workspace(20)
    pws = lib.prefill_weights_workspace(3, 3, 1, 4, 8, 2, b.block_tables.shape[1], 256)
    kept = torch.empty((3, 2, 256), dtype=torch.int32, device="cuda")
    new_lens = torch.empty((3,), dtype=torch.int32, device="cuda")
    inputs = st.context_lens, st.cu_k, st.q, st.kw, st.k_cache, st.v_cache
    true = [x.clone() for x in inputs]
    slow, other = torch.rand((2048, 2048), device="cuda"), torch.empty((2048, 2048), device="cuda")
    side = torch.cuda.Stream()

    def spoil():
        for x in inputs:
            x.zero_()
        for x in (st.out, kept, new_lens):
            x.fill_(7)
        torch.cuda.synchronize()

    def feed():
        for _ in range(10):
            torch.mm(slow, slow, out=other)
        for x, y in zip(inputs, true):
            torch.add(y, 0, out=x) if before == "kernel" else x.copy_(y)

    def go():
        if before == "two streams":
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                feed()
            other.add_(1.0)
            torch.cuda.current_stream().wait_stream(side)
        elif before != "nothing":
            feed()
        if before == "memset":
            st.out.zero_()
        if op == "decode":
            st.decode_weights(mtb=20, ws=ws)
        elif op == "prompt":
            lib.paged_prefill_weights(st.kw, st.q, st.k_cache, st.block_tables, st.cu_q, st.cu_k, 1, 4, b.scale, pws, st.status)
        else:
            lib.kv_evict(st.k_cache, st.v_cache, st.kw, st.block_tables, st.context_lens, 256, 32, kept, new_lens, st.status)

    def outputs():
        torch.cuda.synchronize()
        return [x.clone() for x in (st.out, st.kw, st.k_cache, st.v_cache, kept, new_lens)]

    def start():
        spoil()
        if before == "nothing":
            for x, y in zip(inputs, true):
                x.copy_(y)
            torch.cuda.synchronize()

    spoil()
    feed()
    torch.cuda.synchronize()
    if before == "memset":
        st.out.zero_()
    before, kind = "nothing", before
    go()
    want = outputs()
    before = kind
    for _ in range(3):
        start()
        go()
        for x, y in zip(outputs(), want):
            assert torch.equal(x, y)
    g = torch.cuda.CUDAGraph()
    start()
    with torch.cuda.graph(g):
        go()
    for _ in range(3):
        start()
        g.replay()
        for x, y in zip(outputs(), want):
            assert torch.equal(x, y)
    assert st.status_value() == 0


def test_a_sequence_goes_on_in_a_bounded_cache(lib):
    """Prompts, their weights, eviction, decode steps that store and collect, and
    eviction again whenever a budget's worth and a block has filled up; the block
    manager gives the blocks back.  Every step against the oracle on the cache as
    it stands."""
    rng = np.random.default_rng(80)
    Hq, Hkv, D, BS, budget, recent, NB = 4, 2, 64, 64, 128, 24, 24
    scale = 0.125
    bm = lib.BlockManager(NB, BS)
    lens = [300, 150]
    pool = wl.normal_bf16(rng, (2, NB, BS, Hkv, D))
    kc, vc = bf16(pool[0]), bf16(pool[1])
    kw = torch.full((NB, Hkv, BS), float("nan"), device="cuda")   # whatever the pool held
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for s, n in enumerate(lens):
        assert bm.allocate(s, rng.integers(0, 50000, n)) == 0

    def tables(width=6):
        return np.stack([bm.block_table(s, width) for s in range(2)])

    # the prompts: K and V stored, attended, the last 32 queries counted
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = (wl.normal_bf16(rng, (sum(lens), h, D)) for h in (Hq, Hkv, Hkv))
    slots = np.concatenate([bm.slots(s, 0, n) for s, n in enumerate(lens)])
    lib.kv_store(bf16(k), bf16(v), kc, vc, i32(slots), status)
    out = torch.empty((sum(lens), Hq, D), dtype=torch.bfloat16, device="cuda")
    t = tables()
    lib.paged_prefill_attn(out, bf16(q), kc, vc, i32(t), i32(cu), i32(cu), max(lens), scale, dev_status=status)
    ws = lib.prefill_weights_workspace(2, sum(lens), max(lens), 32, Hq, Hkv, 6, BS)
    lib.paged_prefill_weights(kw, bf16(q), kc, i32(t), i32(cu), i32(cu), max(lens), 32, scale, ws, status)
    want, brought = oracle.prefill_weights(np.full((NB, Hkv, BS), np.nan), q, bits(kc), t, cu, cu, 32, scale)
    b = batch([2], seed=1)
    b = dataclasses.replace(b, q=q, scale=scale)
    assert_weights(kw, want, brought, weight_rtol(b, bits(kc)), "prompt")
    dws = lib.decode_weights_workspace(2, Hq, Hkv, D, BS, 12)
    evictions = 0
    for step in range(150):
        ctx = np.array([bm.num_tokens(s) for s in range(2)], np.int32)
        if (ctx > budget + BS).any() or step == 0:
            t = tables()
            kept = torch.empty((2, Hkv, budget), dtype=torch.int32, device="cuda")
            new_lens = torch.empty((2,), dtype=torch.int32, device="cuda")
            before = bits(kc), bits(vc), kw.cpu().numpy()
            for s in range(2):
                bm.evict(s, budget)
            lib.kv_evict(kc, vc, kw, i32(t), i32(ctx), budget, recent, kept, new_lens, status)
            ekc, evc, ekw, ekept, elens = oracle.kv_evict(*before, t, ctx, budget, recent)
            assert np.array_equal(bits(kc), ekc) and np.array_equal(bits(vc), evc)
            assert np.array_equal(kw.cpu().numpy(), ekw, equal_nan=True) and np.array_equal(kept.cpu().numpy(), ekept)
            assert [bm.num_tokens(s) for s in range(2)] == elens.tolist() == new_lens.tolist()
            assert bm.num_free_blocks == NB - 2 * 2
            evictions += 1
        for s in range(2):
            bm.append(s, int(rng.integers(0, 50000)))
        ctx = np.array([bm.num_tokens(s) for s in range(2)], np.int32)
        t = tables()
        slots = np.array([bm.slots(s, int(ctx[s]) - 1, 1)[0] for s in range(2)], np.int32)
        q, k, v = (wl.normal_bf16(rng, (2, h, D)) for h in (Hq, Hkv, Hkv))
        check = step % 25 in (0, 24)
        ekc, evc = oracle.kv_store(bits(kc), bits(vc), k, v, slots) if check else (None, None)
        sums = kw.cpu().numpy() if check else None
        out = torch.empty((2, Hq, D), dtype=torch.bfloat16, device="cuda")
        lib.paged_decode_weights_attn(out, kw, bf16(q), kc, vc, i32(t), i32(ctx), scale, dws, 12, k=bf16(k), v=bf16(v),
                                      slot_mapping=i32(slots), dev_status=status)
        if check:
            assert np.array_equal(bits(kc), ekc) and np.array_equal(bits(vc), evc)
            assert_close(out.double().cpu().numpy(), oracle.paged_decode_attn(q, ekc, evc, t, ctx, scale), f"step {step}")
            want, brought = oracle.decode_weights(sums, q, ekc, t, ctx, scale)
            assert_weights(kw, want, brought, weight_rtol(dataclasses.replace(b, q=q), ekc), f"step {step}")
    assert evictions >= 3
    assert int(status.item()) == 0
