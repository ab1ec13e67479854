"""Float64 oracle for the key weights and the eviction that goes by them.

TEST INFRASTRUCTURE ONLY (see attention.py).  Plain loops over sequences,
queries, heads and positions, from the definitions:

* the weight of key p for query head h is softmax_p(scale <q_h, k_p>); a kv
  head's key collects the sum over the query heads of its group;
* a call adds to the sums of keys that were there before it and sets the sums
  of the tokens that it brings (decode: the newest token; a prompt chunk: its
  own tokens): those start at zero before any sequence of the call adds to them,
  so that a slot which one sequence brings and another has cached, or several
  bring, gets the weights of all;
* eviction keeps the last `recent` positions and, of the others, the
  budget - recent with the largest sums (NaN as -inf, lowest position first
  among equals); kept positions below budget - recent stay, the kept ones
  behind them fill the free places in order, the recent ones follow in order.

key_weights: float64 [NB, Hkv, BS].
"""
from __future__ import annotations

import numpy as np

from .attention import bf16_bits_to_f64, gather_sequence, kv_head_of


def softmax_weights(q_vec, keys, scale):
    s = scale * (keys @ q_vec)
    w = np.exp(s - s.max())
    return w / w.sum()


def place_of(block_table_row, pos, block_size):
    return int(block_table_row[pos // block_size]), pos % block_size


def decode_weights(key_weights, q, k_cache, block_tables, context_lens, scale):
    """(key_weights after the step, what it contributed); the caches already hold the newest tokens."""
    after = np.array(key_weights, dtype=np.float64)
    brought = np.zeros_like(after)
    NB, BS, Hkv, D = k_cache.shape
    Hq = q.shape[1]
    qf = bf16_bits_to_f64(q)
    for s, L in enumerate(context_lens):
        b, o = place_of(block_tables[s], int(L) - 1, BS)
        after[b, :, o] = 0.0
    for s, L in enumerate(context_lens):
        L = int(L)
        keys = bf16_bits_to_f64(gather_sequence(k_cache, block_tables[s], L))
        a = np.zeros((Hkv, L))
        for h in range(Hq):
            j = kv_head_of(h, Hq, Hkv)
            a[j] += softmax_weights(qf[s, h], keys[:, j], scale)
        for p in range(L):
            b, o = place_of(block_tables[s], p, BS)
            after[b, :, o] += a[:, p]
            brought[b, :, o] += a[:, p]
    return after, brought


def prefill_weights(key_weights, q, k_cache, block_tables, cu_seqlens_q, cu_seqlens_k, window, scale):
    """As decode_weights, for the last `window` queries of every prompt chunk."""
    after = np.array(key_weights, dtype=np.float64)
    brought = np.zeros_like(after)
    NB, BS, Hkv, D = k_cache.shape
    Hq = q.shape[1]
    qf = bf16_bits_to_f64(q)
    for s in range(len(cu_seqlens_q) - 1):
        L = int(cu_seqlens_k[s + 1] - cu_seqlens_k[s])
        for p in range(L - int(cu_seqlens_q[s + 1] - cu_seqlens_q[s]), L):
            b, o = place_of(block_tables[s], p, BS)
            after[b, :, o] = 0.0
    for s in range(len(cu_seqlens_q) - 1):
        q0, n = int(cu_seqlens_q[s]), int(cu_seqlens_q[s + 1] - cu_seqlens_q[s])
        L = int(cu_seqlens_k[s + 1] - cu_seqlens_k[s])
        if n == 0:
            continue
        c = L - n
        keys = bf16_bits_to_f64(gather_sequence(k_cache, block_tables[s], L))
        a = np.zeros((Hkv, L))
        for i in range(max(0, n - window), n):
            for h in range(Hq):
                j = kv_head_of(h, Hq, Hkv)
                a[j, : c + i + 1] += softmax_weights(qf[q0 + i, h], keys[: c + i + 1, j], scale)
        for p in range(L):
            b, o = place_of(block_tables[s], p, BS)
            after[b, :, o] += a[:, p]
            brought[b, :, o] += a[:, p]
    return after, brought


def evict_map(weights, L, budget, recent):
    """For one kv head: the old position of what ends at each of the `budget` places (-1: none)."""
    if L <= budget:
        return np.array(list(range(L)) + [-1] * (budget - L), dtype=np.int32)
    heavy = budget - recent
    w = [(-np.inf if np.isnan(x) else float(x)) for x in weights[: L - recent]]
    best = sorted(range(L - recent), key=lambda p: (-w[p], p))[:heavy]
    stay = {p for p in best if p < heavy}
    movers = sorted(p for p in best if p >= heavy)
    out, m = [], 0
    for place in range(heavy):
        if place in stay:
            out.append(place)
        else:
            out.append(movers[m])
            m += 1
    assert m == len(movers)
    return np.array(out + list(range(L - recent, L)), dtype=np.int32)


def kv_evict(k_cache, v_cache, key_weights, block_tables, context_lens, budget, recent):
    """(k_cache, v_cache, key_weights, kept, new_lens) after the eviction."""
    kc, vc, kw = (np.array(x, copy=True) for x in (k_cache, v_cache, key_weights))
    NB, BS, Hkv, D = k_cache.shape
    kept = np.empty((len(context_lens), Hkv, budget), dtype=np.int32)
    for s, L in enumerate(context_lens):
        L = int(L)
        places = [place_of(block_tables[s], p, BS) for p in range(L)]
        for j in range(Hkv):
            kept[s, j] = evict_map([key_weights[b, j, o] for b, o in places], L, budget, recent)
            if L <= budget:
                continue
            for i, src in enumerate(kept[s, j]):
                (b, o), (b0, o0) = places[i], places[src]
                kc[b, o, j], vc[b, o, j], kw[b, j, o] = k_cache[b0, o0, j], v_cache[b0, o0, j], key_weights[b0, j, o0]
    return kc, vc, kw, kept, np.minimum(np.asarray(context_lens), budget).astype(np.int32)
