"""What is measured of the operators that carry a step from its projections to its attention.

Three operators around the paged cache [num_blocks, block_size, Hkv, D]:

  plan    which blocks the step's new tokens get: block tables, slots, positions and
          prefix sums from the sequences' lengths and a stack of free blocks
  rotate  the norm of each head's query and key, the rotation by position and the
          store of K and V through the slots, in one pass over the projections
  shared  one new token per sequence attends over its pages, where groups of
          sequences begin with the same blocks

`own` is set from outside: False runs the plain forms (elementary operations in 32
bits, in 64 for angles), True the framework's calls.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ the cases

def listed():
    def plan(name, seqs, low, high, new, ending, idle, block, pad):
        return {"name": name, "op": "plan", "seqs": seqs, "low": low, "high": high, "new": new, "ending": ending,
                "idle": idle, "block": block, "pad": pad, "scarce": False, "pick": 1}

    def rotate(name, seqs, low, high, heads, **more):
        q_heads, kv_heads, dim, block = heads
        return dict({"name": name, "op": "rotate", "seqs": seqs, "low": low, "high": high, "far": 4096, "q_heads": q_heads,
                     "kv_heads": kv_heads, "dim": dim, "block": block, "rotary": dim, "interleaved": False, "norm": True,
                     "scaling": "none", "packed": True, "store": True, "pick": 1}, **more)

    def shared(name, seqs, groups, prefix_low, prefix_high, low, high, heads):
        q_heads, kv_heads, dim, block = heads
        return {"name": name, "op": "shared", "seqs": seqs, "groups": groups, "prefix_low": prefix_low, "prefix_high": prefix_high,
                "low": low, "high": high, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "block": block, "pick": 1}

    return [
        # Two short chats, a token each: latency alone.
        plan("plan 2 decode", 2, 5, 300, 1, 0.0, 0.0, 256, 0),
        # A running batch of decode rows, padded to the size its graph was captured for; some sequences end, some pause.
        plan("plan 64 running", 64, 128, 2048, 1, 0.1, 0.1, 256, 7),
        # Whole prompts and further chunks for many sequences at once, beside those that end.
        plan("plan 500 prompts", 500, 1, 4096, 1024, 0.05, 0.05, 64, 0),
        # Two rows of a small model: latency alone.
        rotate("rotate 2 rows", 2, 1, 1, (4, 2, 64, 256)),
        # The decode rows of a running batch.
        rotate("rotate 64 rows", 64, 1, 1, (16, 8, 128, 256)),
        # A batch of fresh prompts.
        rotate("rotate 16 prompts", 16, 64, 4096, (16, 8, 128, 256)),
        # Chunks of long documents: half of the head rotated, neighbouring dims paired, frequencies stretched, no norm.
        rotate("rotate 11 far chunks", 11, 300, 1500, (32, 8, 128, 128), far=1 << 20, rotary=64, interleaved=True, norm=False,
               scaling="yarn"),
        # Two short chats after the same instructions on a small model.
        shared("shared 2 short", 2, 1, 256, 256, 1, 40, (4, 2, 64, 256)),
        # A running batch behind one system prompt.
        shared("shared 64 system", 64, 1, 2048, 2048, 64, 1024, (16, 8, 128, 256)),
        # Several system prompts of different lengths and groups of different sizes, odd lengths, small pages.
        shared("shared 50 in 6", 50, 6, 200, 4000, 1, 700, (32, 8, 64, 64)),
        # Samples of answers about one long document, eight query heads to a kv head.
        shared("shared 16 document", 16, 1, 32000, 32000, 1, 300, (64, 8, 128, 128)),
        # Many chats behind a long common context, four query heads to a kv head.
        shared("shared 128 context", 128, 1, 8192, 8192, 1, 512, (32, 8, 128, 256)),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["plan", "rotate", "shared"])
    pick = rng.randrange(1 << 20)
    if op == "plan":
        seqs = _log(rng, 1, 1000)
        high = _log(rng, 2, 8192)
        return {"op": op, "seqs": seqs, "low": max(1, int(high * rng.random())), "high": high, "new": rng.choice([1, 1, _log(rng, 2, min(2048, 250000 // seqs))]),
                "ending": rng.choice([0.0, 0.1, 0.5]), "idle": rng.choice([0.0, 0.1, 0.5]), "block": rng.choice([64, 128, 256, 512]),
                "pad": rng.choice([0, 0, 1, 63]), "scarce": rng.random() < 0.25, "pick": pick}
    kv_heads = rng.choice([1, 2, 4, 8])
    case = {"op": op, "kv_heads": kv_heads, "q_heads": kv_heads * rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]),
            "block": rng.choice([64, 128, 256, 512]), "pick": pick}
    if op == "rotate":
        seqs = _log(rng, 1, 256)
        # (at most about the values of the listed prompts)
        most = max(1, (1 << 27) // (seqs * (case["q_heads"] + 2 * kv_heads) * case["dim"]))
        high = rng.choice([1, _log(rng, 1, min(4096, most))])
        case.update(seqs=seqs, low=max(1, int(high * rng.random())), high=high, far=_log(rng, 1, 1 << 20),
                    rotary=min(case["dim"], rng.choice([16, 32, 48, 64, 96, 128, 128])), interleaved=rng.random() < 0.5, norm=rng.random() < 0.7,
                    scaling=rng.choice(["none", "none", "linear", "yarn"]), packed=rng.random() < 0.7, store=rng.random() < 0.8)
    else:
        seqs = _log(rng, 1, 192)
        # (at most about the padded tokens of the largest listed case, fewer with more query heads)
        tokens = 1000000 * 32 // max(32, case["q_heads"])
        prefix = _log(rng, 64, min(32768, max(64, tokens * 9 // 10 // seqs)))
        high = _log(rng, 1, max(1, min(2048, tokens // seqs - prefix)))
        case.update(seqs=seqs, groups=rng.randint(1, max(1, min(seqs, 8))), prefix_low=int(prefix * rng.random()), prefix_high=prefix,
                    low=max(1, int(high * rng.random())), high=high)
    return case


def _between(rng, low, high, count):
    """`count` whole numbers, the two ends first."""
    return ([high, low] + [rng.randint(low, high) for _ in range(count)])[:count]


def _plan_lens(case):
    """What each sequence holds, how many leading blocks of it are another's, and its new tokens (-1: it ends)."""
    rng = random.Random(case["pick"])
    ctx = _between(rng, case["low"], case["high"], case["seqs"])
    new, borrowed = [], []
    for s, L in enumerate(ctx):
        what = rng.random()
        n = rng.randint(1, case["new"])
        new.append(-1 if what < case["ending"] else 0 if what < case["ending"] + case["idle"] else n)
        if case["new"] > 1 and rng.random() < 0.5:
            # A fresh prompt: all that it has is what was found in the cache.
            ctx[s] = rng.choice([0, L // case["block"] * case["block"]])
        borrowed.append(min(rng.choice([0, 0, 1, 2]), ctx[s] // case["block"]))
    return ctx, borrowed, new


def _lens(case):
    return _between(random.Random(case["pick"]), case["low"], case["high"], case["seqs"])


def _groups(case):
    """First sequence of each group (and the end), the blocks its sequences share, every sequence's length."""
    rng = random.Random(case["pick"] + 1)
    S, n, BS = case["seqs"], case["groups"], case["block"]
    starts = [0] + sorted(rng.sample(range(1, S), n - 1)) + [S]
    blocks = [tokens // BS for tokens in _between(rng, case["prefix_low"], case["prefix_high"], n)]
    ctx = _lens(case)
    for g in range(n):
        for s in range(starts[g], starts[g + 1]):
            ctx[s] += blocks[g] * BS
    return starts, blocks, ctx


def work(case):
    if case["op"] == "plan":
        ctx, borrowed, new = _plan_lens(case)
        BS, S, rows = case["block"], case["seqs"], sum(max(n, 0) for n in new) + case["pad"]
        given = sum(-(-L // BS) - b for L, b, n in zip(ctx, borrowed, new) if n < 0)
        taken = sum(-(-(L + n) // BS) - -(-L // BS) for L, n in zip(ctx, new) if n > 0)
        # lengths, borrowed and new counts read; blocks given back and taken, read and written; slots, positions, lengths, sums written
        return {"bytes": 12 * S + 8 * (given + taken) + 8 * rows + 12 * S, "flops": 0}
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rotate":
        rows = sum(_lens(case))
        # q, k, v read and written (without a store v stays where it is); positions and slots
        heads = Hq + Hkv + (Hkv if case["store"] else 0)
        return {"bytes": rows * (4 * heads * D + 8), "flops": rows * (Hq + Hkv) * (3 * case["rotary"] + (4 * D if case["norm"] else 0))}
    starts, blocks, ctx = _groups(case)
    once = sum(blocks) * case["block"]
    shared = sum((starts[g + 1] - starts[g]) * blocks[g] for g in range(len(blocks))) * case["block"]
    # K and V of the shared blocks once, of the others for each sequence; q and out
    return {"bytes": (once + sum(ctx) - shared) * Hkv * 4 * D + 4 * len(ctx) * Hq * D, "flops": 4 * sum(ctx) * Hq * D}


# ----------------------------------------------------------------- the inputs

def _device(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"plan": _prepare_plan, "rotate": _prepare_rotate, "shared": _prepare_shared}[case["op"]](case, gen)


def _prepare_plan(case, gen):
    S, BS = case["seqs"], case["block"]
    ctx, borrowed, new = _plan_lens(case)
    need = [-(-L // BS) for L in ctx]
    wide = max(-(-(L + max(n, 0)) // BS) for L, n in zip(ctx, new)) + 1
    taken = sum(-(-(L + n) // BS) - -(-L // BS) for L, n in zip(ctx, new) if n > 0)
    given = sum(h - b for h, b, n in zip(need, borrowed, new) if n < 0)
    free = max(0, taken - given) // 2 if case["scarce"] else taken + 5
    NB = sum(need) + free + 1
    pages = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32)
    tables = torch.full((S, wide), -1, dtype=torch.int32)
    host = pages.cpu()
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = host[at:at + n]
        at += n
    stack = torch.full((NB,), -1, dtype=torch.int32, device="cuda")
    stack[:free] = pages[at:at + free]
    rows = sum(max(n, 0) for n in new) + case["pad"]

    def room(count):
        return torch.empty(count, dtype=torch.int32, device="cuda")

    return {"case": case, "num_blocks": NB, "context_lens": _device(ctx), "borrowed": _device(borrowed), "new_lens": _device(new),
            "block_tables": tables.cuda(), "free_blocks": stack, "num_free": _device([free]), "new_context_lens": room(S),
            "new_num_free": room(1), "slot_mapping": room(rows), "positions": room(rows), "cu_q": room(S + 1), "cu_k": room(S + 1)}


def _frequencies(case):
    """Radians per position of each pair, in 64 bits, and what the rotated values are multiplied by."""
    R = case["rotary"]
    i = torch.arange(0, R, 2, dtype=torch.float64)
    freq = 1e6 ** (-i / R)
    if case["scaling"] == "linear":
        return freq / 4.0, 1.0
    if case["scaling"] == "yarn":
        # Slow pairs are stretched by 32, fast ones kept, those between them blended.
        turns = 32768 * freq / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return freq / 32.0 * (1 - keep) + freq * keep, 0.1 * math.log(32.0) + 1.0
    return freq, 1.0


def _prepare_rotate(case, gen):
    Hq, Hkv, D, BS = case["q_heads"], case["kv_heads"], case["dim"], case["block"]
    rng = random.Random(case["pick"] + 2)
    lens = _lens(case)
    T = sum(lens)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    # Projections as models have them: a few dims far larger than the rest, heads of different sizes.
    size = torch.exp(0.7 * normal(Hq + 2 * Hkv, D))
    rows = (normal(T, Hq + 2 * Hkv, D) * size).to(torch.bfloat16)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    if not case["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    first = [rng.randint(0, case["far"]) for _ in lens]
    positions = torch.cat([torch.arange(f, f + n, dtype=torch.int32) for f, n in zip(first, lens)]).cuda()
    freq, amplitude = _frequencies(case)
    state = {"case": case, "q": q, "k": k, "v": v, "positions": positions, "freq": freq.cuda(), "amplitude": amplitude,
             "q_out": torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")}
    if case["norm"]:
        state.update(q_weight=torch.exp(0.3 * normal(D)).to(torch.bfloat16), k_weight=torch.exp(0.3 * normal(D)).to(torch.bfloat16))
    if case["store"]:
        NB = -(-T // BS) + 2
        pages = torch.randperm(NB, generator=gen, device="cuda")
        t = torch.arange(T, device="cuda")
        slots = pages[t // BS] * BS + t % BS
        # Rows that pad a batch have no slot.
        slots[1:][torch.rand(T - 1, generator=gen, device="cuda") < 0.02] = -1
        state.update(slot_mapping=slots.to(torch.int32), k_cache=normal(NB, BS, Hkv, D).to(torch.bfloat16), v_cache=normal(NB, BS, Hkv, D).to(torch.bfloat16))
    else:
        state["k_out"] = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    if own:
        import paged_kv_cache_241_gb300 as pkv

        state["turns"] = pkv.rope_turns(freq, "cuda")
    return state


def _prepare_shared(case, gen):
    S, Hq, Hkv, D, BS = case["seqs"], case["q_heads"], case["kv_heads"], case["dim"], case["block"]
    starts, blocks, ctx = _groups(case)
    need = [-(-L // BS) for L in ctx]
    group = [g for g in range(len(blocks)) for _ in range(starts[g], starts[g + 1])]
    NB = sum(blocks) + sum(n - blocks[g] for n, g in zip(need, group)) + 2  # a pool has blocks that no sequence holds
    pages = torch.randperm(NB, generator=gen, device="cuda").to(torch.int32).cpu()
    tables = torch.full((S, max(need)), -1, dtype=torch.int32)
    at = 0
    for g, n in enumerate(blocks):
        tables[starts[g]:starts[g + 1], :n] = pages[at:at + n]
        at += n
    for s, n in enumerate(need):
        rest = n - blocks[group[s]]
        tables[s, n - rest:n] = pages[at:at + rest]
        at += rest

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    # A few tokens draw attention from everybody, as a text's first ones and its separators do.
    lean = 0.6 * normal(Hkv, D)
    heavy = torch.rand(NB, BS, 1, 1, generator=gen, device="cuda") < 0.02
    k_cache = normal(NB, BS, Hkv, D)
    k_cache = torch.where(heavy, k_cache + lean, k_cache).to(torch.bfloat16)
    q = (normal(S, Hkv, Hq // Hkv, D) + lean[:, None, :]).reshape(S, Hq, D).to(torch.bfloat16)
    state = {"case": case, "block_tables": tables.cuda(), "context_lens": _device(ctx), "group_starts": _device(starts), "shared_blocks": _device(blocks),
             "spare_block": int(pages[-1]), "longest": max(ctx), "k_cache": k_cache, "v_cache": normal(NB, BS, Hkv, D).to(torch.bfloat16), "q": q,
             "scale": 1.0 / math.sqrt(D), "out": torch.empty(S, Hq, D, dtype=torch.bfloat16, device="cuda")}
    if own:
        import paged_kv_cache_241_gb300 as pkv

        state["workspace"] = pkv.decode_shared_workspace(S, len(blocks), Hq, Hkv, D, "cuda")
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if op == "plan":
        return _plan_own(state) if own else _plan_plain(state)
    if op == "rotate":
        return _rotate_own(state) if own else _rotate_plain(state)
    return _shared_own(state) if own else _shared_plain(state)


def _plan_own(state):
    import paged_kv_cache_241_gb300 as pkv

    pkv.plan_step(state["new_lens"], state["context_lens"], state["block_tables"], state["free_blocks"], state["num_free"], state["new_context_lens"],
                  state["new_num_free"], state["slot_mapping"], state["positions"], state["cu_q"], state["cu_k"], state["num_blocks"],
                  state["case"]["block"], borrowed_blocks=state["borrowed"])
    return _plan_outputs(state)


def _plan_outputs(state):
    return {x: state[x] for x in ("block_tables", "free_blocks", "new_context_lens", "new_num_free", "slot_mapping", "positions", "cu_q", "cu_k")}


def _rotate_own(state):
    import paged_kv_cache_241_gb300 as pkv

    case = state["case"]
    pkv.norm_rope_store(state["q_out"], state["q"], state["k"], state["v"], state["positions"], state["turns"], k_cache=state.get("k_cache"),
                        v_cache=state.get("v_cache"), slot_mapping=state.get("slot_mapping"), k_out=state.get("k_out"), q_weight=state.get("q_weight"),
                        k_weight=state.get("k_weight"), eps=1e-6, interleaved=case["interleaved"], amplitude=state["amplitude"])
    return _rotate_outputs(state)


def _rotate_outputs(state):
    return {x: state[x] for x in ("q_out", "k_out", "k_cache", "v_cache") if x in state}


def _shared_own(state):
    import paged_kv_cache_241_gb300 as pkv

    pkv.paged_decode_shared_attn(state["out"], state["q"], state["k_cache"], state["v_cache"], state["block_tables"], state["context_lens"],
                                 state["group_starts"], state["shared_blocks"], state["scale"], state["workspace"])
    return state["out"]


# ------------------------------------------------------------- the plain forms

def _plan_plain(state):
    BS = state["case"]["block"]
    n, L, tables, stack = state["new_lens"].long(), state["context_lens"].long(), state["block_tables"], state["free_blocks"]
    S, wide = tables.shape
    held = (L + BS - 1) // BS
    ends = n < 0
    # Blocks of sequences that end go onto the stack, in the order of the sequences.
    column = torch.arange(wide, device="cuda")
    back = ends[:, None] & (column >= state["borrowed"].long()[:, None]) & (column < held[:, None])
    rank = back.flatten().cumsum(0) - 1
    there = state["num_free"].long() + rank
    spare = torch.cat([stack, stack[:1]])  # (one more place, for what is not given back)
    spare[torch.where(back.flatten(), there, stack.shape[0])] = tables.flatten()
    stack.copy_(spare[:-1])
    left = state["num_free"].long() + back.sum()
    # The others take theirs from its top; from the first that does not find enough on, nobody takes any.
    n = n.clamp(min=0)
    need = torch.where(n > 0, (L + n + BS - 1) // BS - held, 0)
    before = need.cumsum(0) - need
    fits = (need == 0) | (before + need <= left)
    new = (column >= held[:, None]) & (column < (held + need)[:, None]) & fits[:, None]
    at = left - 1 - before[:, None] - (column - held[:, None])
    tables.copy_(torch.where(new, stack[torch.where(new, at, 0)], tables))
    state["new_num_free"].copy_(left - torch.where(fits, need, 0).sum())
    after = torch.where(ends, 0, torch.where(fits, L + n, L))
    state["new_context_lens"].copy_(after)
    # Rows, in the order of the sequences; behind the last one: no slot.
    last = n.cumsum(0)
    state["cu_q"][0] = 0
    state["cu_q"][1:] = last
    state["cu_k"][0] = 0
    state["cu_k"][1:] = torch.where(fits, after, 0).cumsum(0)
    t = torch.arange(state["slot_mapping"].shape[0], device="cuda")
    s = torch.searchsorted(last, t, right=True)
    real = s < S
    s = s.clamp(max=S - 1)
    pos = torch.where(real, L[s] + t - (last - n)[s], 0)
    state["positions"].copy_(pos)
    slot = tables[s, (pos // BS).clamp(max=wide - 1)].long() * BS + pos % BS
    state["slot_mapping"].copy_(torch.where(real & fits[s], slot, -1))
    return _plan_outputs(state)


def _rotate_plain(state):
    case = state["case"]
    R = case["rotary"]
    angle = state["positions"].double()[:, None] * state["freq"]
    cos, sin = (torch.cos(angle) * state["amplitude"]).float()[:, None], (torch.sin(angle) * state["amplitude"]).float()[:, None]

    def rotated(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        a, b = (x[..., 0:R:2], x[..., 1:R:2]) if case["interleaved"] else (x[..., : R // 2], x[..., R // 2 : R])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([turned, x[..., R:]], -1).to(torch.bfloat16)

    state["q_out"].copy_(rotated(state["q"], state.get("q_weight")))
    k = rotated(state["k"], state.get("k_weight"))
    if case["store"]:
        # (in the place of a row without a slot: the first row, which has one, once more)
        row = torch.where(state["slot_mapping"] >= 0, torch.arange(k.shape[0], device="cuda"), 0)
        slots = state["slot_mapping"][row].long()
        state["k_cache"].flatten(0, 1)[slots] = k[row]
        state["v_cache"].flatten(0, 1)[slots] = state["v"][row]
    else:
        state["k_out"].copy_(k)
    return _rotate_outputs(state)


def _shared_plain(state):
    case = state["case"]
    S, Hkv, D, BS = case["seqs"], case["kv_heads"], case["dim"], case["block"]
    pos = torch.arange(state["longest"], device="cuda")
    valid = pos < state["context_lens"][:, None]
    slot = torch.where(valid, state["block_tables"].long()[:, pos // BS] * BS + pos % BS, state["spare_block"] * BS)
    k = state["k_cache"].flatten(0, 1)[slot].transpose(1, 2).float()
    z = torch.matmul(state["q"].float().view(S, Hkv, -1, D), k.transpose(2, 3)) * state["scale"]
    del k
    z = z.masked_fill(~valid[:, None, None, :], -math.inf)
    w = torch.exp(z - z.amax(-1, keepdim=True))
    w = w / w.sum(-1, keepdim=True)
    v = state["v_cache"].flatten(0, 1)[slot].transpose(1, 2).float()
    state["out"].copy_(torch.matmul(w, v).view(S, -1, D).to(torch.bfloat16))
    return state["out"]


# ------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"plan": _plan_exact, "rotate": _rotate_exact, "shared": _shared_exact}[case["op"]](state)


def _plan_exact(state):
    """The step played through on the host, token after token."""
    BS = state["case"]["block"]
    tables, lens, new = state["block_tables"].tolist(), state["context_lens"].tolist(), state["new_lens"].tolist()
    borrowed, memory = state["borrowed"].tolist(), state["free_blocks"].tolist()
    stack = memory[: state["num_free"].item()]
    for s, L in enumerate(lens):
        if new[s] == -1:
            stack.extend(tables[s][borrowed[s] : (L + BS - 1) // BS])
    memory[: len(stack)] = stack
    slots, positions, cu_q, cu_k, after, closed = [], [], [0], [0], [], False
    for s, L in enumerate(lens):
        n = max(new[s], 0)
        have = (L + BS - 1) // BS
        want = (L + n + BS - 1) // BS - have if n else 0
        closed = closed or want > len(stack)
        refused = closed and want > 0
        for i in range(0 if refused else want):
            tables[s][have + i] = stack.pop()
        for p in range(L, L + n):
            slots.append(-1 if refused else tables[s][p // BS] * BS + p % BS)
            positions.append(p)
        after.append(0 if new[s] == -1 else L if refused else L + n)
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + (0 if refused else after[-1]))
    pad = state["slot_mapping"].shape[0] - len(slots)
    return {"block_tables": _device(tables), "free_blocks": _device(memory), "new_context_lens": _device(after), "new_num_free": _device([len(stack)]),
            "slot_mapping": _device(slots + [-1] * pad), "positions": _device(positions + [0] * pad), "cu_q": _device(cu_q), "cu_k": _device(cu_k)}


def _rotate_exact(state):
    """Pairs as complex numbers, multiplied by exp(i angle)."""
    case = state["case"]
    R, D = case["rotary"], case["dim"]
    half = torch.arange(R // 2, device="cuda")
    first, second = (2 * half, 2 * half + 1) if case["interleaved"] else (half, half + R // 2)
    angle = state["positions"].to(torch.float64)[:, None] * state["freq"]
    turn = torch.polar(torch.full_like(angle, state["amplitude"]), angle)

    def head(x, weight):
        y = x.to(torch.float64).clone()
        if weight is not None:
            y *= weight.to(torch.float64) / torch.sqrt(y.square().sum(-1) / D + 1e-6)[:, None]
        z = torch.complex(y[:, first], y[:, second]) * turn
        y[:, first], y[:, second] = z.real, z.imag
        return y

    def heads(x, weight):
        return torch.stack([head(x[:, h], weight) for h in range(x.shape[1])], 1)

    got = {"q_out": heads(state["q"], state.get("q_weight"))}
    k = heads(state["k"], state.get("k_weight"))
    if not case["store"]:
        return dict(got, k_out=k)
    kept = (state["slot_mapping"] >= 0).nonzero()[:, 0]
    slots = state["slot_mapping"][kept].long()
    for name, rows in (("k_cache", k), ("v_cache", state["v"])):
        cache = state[name].to(torch.float64)
        cache.view(-1, *cache.shape[2:])[slots] = rows[kept].to(torch.float64)
        got[name] = cache
    return got


def _shared_exact(state):
    """Every sequence by itself, over all of its context."""
    case = state["case"]
    S, Hkv, D, BS = case["seqs"], case["kv_heads"], case["dim"], case["block"]
    out = torch.empty(S, case["q_heads"], D, dtype=torch.float64, device="cuda")
    for s, L in enumerate(state["context_lens"].tolist()):
        blocks = state["block_tables"][s, : -(-L // BS)].long()
        k = state["k_cache"][blocks].reshape(-1, Hkv, D)[:L].to(torch.float64)
        v = state["v_cache"][blocks].reshape(-1, Hkv, D)[:L].to(torch.float64)
        q = state["q"][s].to(torch.float64).view(Hkv, -1, D)
        w = torch.softmax(torch.einsum("jgd,pjd->jgp", q, k) * state["scale"], -1)
        out[s] = torch.einsum("jgp,pjd->jgd", w, v).view(-1, D)
    return out
