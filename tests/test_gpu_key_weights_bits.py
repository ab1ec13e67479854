"""How many bits of a weight reach the output of decode with key weights.

Every sequence has keys of two kinds, k and k / 2, so two weights a head, and values
that almost cancel between the two: what is left shows any rounding of the weights.
Bound: the output is rounded to bf16 (2^-8 of itself); before that, a weight is off by
rtol (weight_rtol of test_gpu_key_weights, with its own sum of magnitudes) and by 2^-18
where it meets its value, and the products of the length's values are summed in fp32, the
tensor cores' truncating: off by 2^-23 of the sum of magnitudes for each of the
additions, of which the longest chain here has fewer than 64 (16 keys a product, joined
by runs).  A weight rounded to bf16 would be off by up to 2^-9, alike for all keys of a
kind: 8 to 30 times this bound."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import workloads as wl
from gpu_util import bf16, i32
from test_gpu_key_weights import batch

pytestmark = pytest.mark.gpu


def two_kinds(G, D, lens, seed):
    """A batch of such sequences: its caches hold all tokens already."""
    b = batch(lens, G, 2, D, seed)
    rng = np.random.default_rng(seed)
    q = 0.5 * rng.standard_normal((len(lens), 2 * G, D)).astype(np.float32)
    q = wl.f32_to_bf16_bits(q)
    k = oracle.bf16_bits_to_f64(wl.normal_bf16(rng, (2, D)))
    qf = oracle.bf16_bits_to_f64(q)
    kc, vc = np.zeros(b.k_cache.shape, np.uint16), np.zeros(b.v_cache.shape, np.uint16)
    for s, L in enumerate(lens):
        half = rng.permutation(L) < L // 2             # the keys k / 2
        p = np.arange(L)
        blk, off = b.block_tables[s, p // 256], p % 256
        for j in range(2):
            kc[blk, off, j] = wl.f32_to_bf16_bits((np.where(half, 0.5, 1.0)[:, None] * k[j]).astype(np.float32))
            z = b.scale * (qf[s, j * G:(j + 1) * G] @ k[j])
            ratio = np.exp(z / 2) * (L - L // 2) / max(1, L // 2)   # all weights of k to all of k / 2
            v = np.repeat(np.exp2(rng.integers(-2, 3, D // G)), G) * rng.choice([-1.0, 1.0], D)
            other = -v * np.tile(ratio, D // G)
            vc[blk, off, j] = wl.f32_to_bf16_bits(np.where(half[:, None], other, v).astype(np.float32))
    return dataclasses.replace(b, q=q, k_cache=kc, v_cache=vc)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_weights_meet_their_values_in_more_than_bf16(lib, G, D):
    lens = [2, 3, 17, 64, 200, 257, 300, 512]
    b = two_kinds(G, D, lens, 100 + G)
    qf, K, V = (oracle.bf16_bits_to_f64(x) for x in (b.q, b.k_cache, b.v_cache))
    want = oracle.paged_decode_attn(b.q, b.k_cache, b.v_cache, b.block_tables, b.context_lens, b.scale)
    bound = np.empty_like(want)
    for s, L in enumerate(lens):
        blk, off = b.block_tables[s, np.arange(L) // 256], np.arange(L) % 256
        for h in range(2 * G):
            keys, values = K[blk, off, h // G], V[blk, off, h // G]
            w = np.exp(b.scale * (keys @ qf[s, h]))
            w /= w.sum()
            A = (np.abs(keys) @ np.abs(qf[s, h])).max()
            rtol = 2 * b.scale * A * D * 2.0**-23 + 2.0**-17
            bound[s, h] = 2.0**-8 * np.abs(want[s, h]) + (w @ np.abs(values)) * (rtol + 2.0**-18 + 64 * 2.0**-23)
    out = torch.empty(b.q.shape, dtype=torch.bfloat16, device="cuda")
    kw = torch.zeros((b.num_blocks, 2, 256), device="cuda")
    ws = lib.decode_weights_workspace(len(lens), 2 * G, 2, D, 256, b.total_blocks_used)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.paged_decode_weights_attn(out, kw, bf16(b.q), bf16(b.k_cache), bf16(b.v_cache), i32(b.block_tables),
                                  i32(b.context_lens), b.scale, ws, b.total_blocks_used, dev_status=status)
    assert int(status.item()) == 0
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= bound).all(), f"worst {np.max(err / bound)} of the bound"
