"""Plain oracles of the calls around attention: a step's blocks and slots, and the
norm, rotation and store of its projections.

TEST INFRASTRUCTURE ONLY (see attention.py).  From the definitions: the step is
played through sequence after sequence and token after token on Python lists; a
head is normed and turned value by value in float64.
"""
from __future__ import annotations

import math

import numpy as np

BAD_BLOCK, BAD_CONTEXT, BAD_SEQLEN, NO_BLOCKS = 0x2, 0x4, 0x20, 0x40
MOST = 2**31 - 1


def plan_step(new_lens, context_lens, block_tables, free_blocks, num_free, num_rows, num_blocks,
              block_size, borrowed=None):
    """What the step leaves: a dict of lists by the call's names, and its status bits."""
    BS = block_size
    tables = [list(map(int, row)) for row in block_tables]
    memory = list(map(int, free_blocks))
    room = (len(tables[0]) if tables else 0) * BS
    status = 0
    count = int(num_free)
    if not 0 <= count <= len(memory):
        status |= BAD_BLOCK
        count = min(max(count, 0), len(memory))
    S = len(new_lens)
    lens = [int(x) for x in context_lens]
    left_out = []
    for s in range(S):
        L, n = lens[s], int(new_lens[s])
        bad = L < 0 or L > room
        if n < -1:
            status |= BAD_SEQLEN
        bad = bad or L + max(n, 0) > room
        left_out.append(bad)
        if bad:
            status |= BAD_CONTEXT
        have = -(-L // BS) if 0 <= L <= room else 0
        b = 0 if borrowed is None else int(borrowed[s])
        if not 0 <= b <= have:
            status |= BAD_CONTEXT
            b = min(max(b, 0), have)
        if n == -1 and not bad:
            for i in range(b, have):
                if count < len(memory):
                    memory[count] = tables[s][i]
                    count += 1
                else:
                    status |= BAD_BLOCK
    slots, positions, cu_q, cu_k, after = [], [], [0], [0], []
    closed, wanted, top = False, 0, count
    for s in range(S):
        L, n = lens[s], max(int(new_lens[s]), 0)
        start = L if 0 <= L <= room else 0
        have = -(-start // BS)
        need = -(-(start + n) // BS) - have if n and not left_out[s] else 0
        wanted += need
        refused = left_out[s]
        if need and wanted > top:
            status |= NO_BLOCKS
            refused = True
        if n and cu_q[-1] + n > num_rows:
            status |= BAD_SEQLEN
            refused = True
        if not refused:
            for i in range(need):
                count -= 1
                tables[s][have + i] = memory[count]
        for p in range(start, start + min(n, max(0, num_rows - len(slots)))):
            slot = -1
            if not refused:
                block = tables[s][p // BS]
                if 0 <= block < num_blocks:
                    slot = block * BS + p % BS
                else:
                    status |= BAD_BLOCK
            slots.append(slot)
            positions.append(p)
        after.append(0 if new_lens[s] == -1 and not left_out[s] else L if refused else L + n)
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + (0 if refused else after[-1]))
    pad = num_rows - len(slots)
    if cu_q[-1] > MOST or cu_k[-1] > MOST:
        status |= BAD_SEQLEN
    return {"block_tables": tables, "free_blocks": memory, "new_num_free": [count],
            "new_context_lens": after, "slot_mapping": slots + [-1] * pad,
            "positions": positions + [0] * pad, "cu_seqlens_q": [min(x, MOST) for x in cu_q],
            "cu_seqlens_k": [min(x, MOST) for x in cu_k]}, status


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False, amplitude=1.0):
    """x [T, H, D] float64 -> the same, each head normed (with weight) and turned."""
    out = np.array(x, dtype=np.float64)
    T, H, D = out.shape
    half = len(inv_freq)
    for t in range(T):
        for h in range(H):
            y = out[t, h]
            if weight is not None:
                y *= np.asarray(weight, dtype=np.float64) / math.sqrt(float(np.mean(y * y)) + eps)
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                angle = int(positions[t]) * float(inv_freq[i])
                c, s = amplitude * math.cos(angle), amplitude * math.sin(angle)
                y[a], y[b] = y[a] * c - y[b] * s, y[b] * c + y[a] * s
    return out
