"""What is measured of the operators that bound a sequence's cache by the attention its keys receive.

Three operators over the paged cache [num_blocks, block_size, Hkv, D] and the
running sums of attention weight key_weights [num_blocks, Hkv, block_size]:

  decode   one new token per sequence attends over its pages; the weight each
           key receives (summed over the query heads of its kv head) is added
           to its sum, and the newest key's sum is set
  prompt   the weight that the last `window` queries of each prompt chunk give
           to each key: added for keys cached before the chunk, set for its own
  evict    keeps, per sequence and kv head, the `recent` last tokens and the
           heaviest others, `budget` in all, moving rows inside the pages

`own` is set from outside: False runs the plain forms (elementary operations
in 32 bits on padded batches), True the framework's calls.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ the cases

def listed():
    def case(name, op, seqs, low, high, heads, **more):
        q_heads, kv_heads, dim, block = heads
        return dict({"name": name, "op": op, "seqs": seqs, "low": low, "high": high, "spread": "flat",
                     "pick": 1, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "block": block}, **more)

    return [
        # Two short chats on a small model: a single block and a crossing into the second; latency alone.
        case("decode 2 short", "decode", 2, 5, 300, (4, 2, 64, 256), store=False),
        # The ordinary decode step of a running batch, its new tokens stored by the same call.
        case("decode 64 fused store", "decode", 64, 128, 2048, (16, 8, 128, 256), store=True),
        # A skewed batch with long contexts, four query heads to a kv head.
        case("decode 64 skewed", "decode", 64, 256, 8192, (32, 8, 128, 256), spread="log", store=False),
        # One long document on odd lengths and small pages, eight query heads to a kv head.
        case("decode 2 long g8", "decode", 2, 24001, 32701, (64, 8, 128, 64), store=True),
        # A short prompt on a small model, all of its queries.
        case("prompt 2 short", "prompt", 2, 17, 130, (4, 2, 64, 256), cached=0, window=1 << 20),
        # A batch of fresh prompts of which the last 32 queries speak for the tokens to come.
        case("prompt 16 window 32", "prompt", 16, 64, 4096, (16, 8, 128, 256), cached=0, window=32),
        # A further chunk of long prompts whose first part is cached, four query heads to a kv head.
        case("prompt 12 chunked", "prompt", 12, 100, 512, (32, 8, 64, 128), cached=7800, window=64),
        # Whole prompts: every query counts.
        case("prompt 8 whole", "prompt", 8, 300, 2048, (16, 8, 128, 256), cached=0, window=1 << 20),
        # Two chats on a small model at their limit.
        case("evict 2 short", "evict", 2, 100, 321, (4, 2, 64, 256), budget=256, recent=32),
        # A running batch of which each sequence has filled another page beyond its budget.
        case("evict 64 running", "evict", 64, 1025, 1280, (16, 8, 128, 256), budget=1024, recent=128),
        # Long prompts cut down to what the decode steps are to read.
        case("evict 16 prompts", "evict", 16, 2000, 16384, (32, 8, 128, 256), spread="log", budget=2048, recent=64),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """A case between the listed ones: at most about half a million padded tokens of eight heads of 128."""
    op = rng.choice(["decode", "prompt", "evict"])
    kv_heads = rng.choice([1, 2, 4, 8])
    case = {"op": op, "spread": rng.choice(["flat", "log"]), "pick": rng.randrange(1 << 20), "kv_heads": kv_heads,
            "q_heads": kv_heads * rng.choice([1, 2, 4, 8]), "dim": rng.choice([64, 128]), "block": rng.choice([64, 128, 256, 512])}
    if op == "decode":
        seqs = _log(rng, 1, 128)
        high = _log(rng, 16, min(32768, 262144 // seqs))
        case.update(store=rng.random() < 0.5)
    elif op == "prompt":
        seqs = _log(rng, 1, 24)
        high = _log(rng, 16, min(2048, 8192 // seqs))
        window = rng.choice([1, 16, 32, 64, 1 << 20])
        cached = 0 if rng.random() < 0.5 else _log(rng, 1, min(8192, 65536 // seqs) if window <= 64 else 1024)
        case.update(window=window, cached=cached)
    else:
        seqs = _log(rng, 1, 64)
        high = _log(rng, 64, min(16384, 131072 // seqs))
        budget = _log(rng, 32, high)
        case.update(budget=budget, recent=rng.choice([0, 1, min(32, budget), budget // 8, budget // 2]))
    case.update(seqs=seqs, low=max(1, int(high * rng.uniform(0.02, 1.0))), high=high)
    return case


def _lens(case):
    """Tokens of each sequence (prompt: new tokens): the two ends first, the others spread between them."""
    rng = random.Random(case["pick"])
    low, high = case["low"], case["high"]
    some = [_log(rng, low, high) if case["spread"] == "log" else rng.randint(low, high) for _ in range(case["seqs"])]
    return ([high, low] + some)[: case["seqs"]]


def _cached(case):
    """Prompt: tokens cached before the chunk, another number for each sequence."""
    rng = random.Random(case["pick"] + 1)
    return [rng.randint(case["cached"] // 2, case["cached"]) for _ in range(case["seqs"])]


def _contexts(case):
    lens = _lens(case)
    return [n + c for n, c in zip(lens, _cached(case))] if case["op"] == "prompt" else lens


def work(case):
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["dim"]
    lens, ctx = _lens(case), _contexts(case)
    tokens = sum(ctx)
    if case["op"] == "decode":
        # K, V, the sums read and written; q and out
        return {"bytes": tokens * Hkv * (4 * D + 8) + 4 * len(lens) * Hq * D, "flops": 4 * tokens * Hq * D}
    if case["op"] == "prompt":
        # K, the sums written (and read, for the cached keys), the q rows that count; one product per pair
        rows = [min(n, case["window"]) for n in lens]
        pairs = sum(r * c - r * (r - 1) // 2 for r, c in zip(rows, ctx))
        return {"bytes": tokens * Hkv * (2 * D + 4) + 4 * Hkv * (tokens - sum(lens)) + 2 * sum(rows) * Hq * D, "flops": 2 * pairs * Hq * D}
    moved = read = 0
    for L in lens:
        if L > case["budget"]:
            heavy = case["budget"] - case["recent"]
            # of `heavy` kept tokens that are spread evenly, the ones behind the first `heavy` places move
            moved += case["recent"] + heavy * (1.0 - heavy / max(1, L - case["recent"]))
            read += L - case["recent"]
    # the sums read; rows of K and V and their sums read and written; what was kept
    return {"bytes": Hkv * (4 * read + moved * 2 * (4 * D + 4) + 4 * case["budget"] * len(lens)), "flops": 0}


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    S, Hq, Hkv, D, BS = case["seqs"], case["q_heads"], case["kv_heads"], case["dim"], case["block"]
    ctx = _contexts(case)
    need = [-(-L // BS) for L in ctx]
    NB = sum(need) + 2  # a pool has blocks that no sequence holds
    pages = torch.randperm(NB, generator=gen, device=dev).to(torch.int32).tolist()
    tables = torch.full((S, max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = torch.tensor(pages[at:at + n], dtype=torch.int32)
        at += n

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(torch.bfloat16)

    state = {"case": case, "block_tables": tables.to(dev), "spare_block": pages[-1], "context_lens": torch.tensor(ctx, dtype=torch.int32, device=dev),
             "k_cache": normal(NB, BS, Hkv, D), "v_cache": normal(NB, BS, Hkv, D), "scale": 1.0 / math.sqrt(D), "longest": max(ctx), "total_blocks": sum(need)}
    # A few tokens draw attention from everybody, as a text's first ones and its separators do.
    lean = 0.6 * torch.randn(Hkv, D, generator=gen, device=dev)
    heavy = torch.rand(NB, BS, 1, 1, generator=gen, device=dev) < 0.02
    state["k_cache"] = torch.where(heavy, state["k_cache"] + lean, state["k_cache"]).to(torch.bfloat16)
    # Sums of many steps: most small, a few large, some keys that nothing has attended to yet.
    sums = torch.empty(NB, Hkv, BS, device=dev).exponential_(1.0, generator=gen).pow_(3)
    sums[torch.rand(NB, Hkv, BS, generator=gen, device=dev) < 0.05] = 0.0

    def queries(rows):
        q = torch.randn(rows, Hkv, Hq // Hkv, D, generator=gen, device=dev) + lean[:, None, :]
        return q.reshape(rows, Hq, D).to(torch.bfloat16)

    if case["op"] == "decode":
        state.update(key_weights=sums, q=queries(S), out=torch.empty(S, Hq, D, dtype=torch.bfloat16, device=dev))
        if case["store"]:
            last = torch.tensor([L - 1 for L in ctx])
            slots = tables[torch.arange(S), last // BS].long() * BS + last % BS
            state.update(k=normal(S, Hkv, D), v=normal(S, Hkv, D), slot_mapping=slots.to(torch.int32).to(dev))
        if own:
            import paged_kv_cache_241_gb300 as pkv

            state["workspace"] = pkv.decode_weights_workspace(S, Hq, Hkv, D, BS, sum(need), dev)
    elif case["op"] == "prompt":
        lens = _lens(case)
        cu_q = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
        cu_k = torch.tensor([0] + ctx).cumsum(0).to(torch.int32)
        state.update(key_weights=sums, q=queries(sum(lens)), cu_q=cu_q.to(dev), cu_k=cu_k.to(dev), longest_q=max(lens))
        if own:
            import paged_kv_cache_241_gb300 as pkv

            state["workspace"] = pkv.prefill_weights_workspace(S, sum(lens), max(lens), case["window"], Hq, Hkv, max(need), BS, dev)
    else:
        # What the decode steps before the eviction have left; the eviction itself moves the sums with their rows.
        state.update(sums=sums, key_weights=torch.empty_like(sums), kept=torch.empty(S, Hkv, case["budget"], dtype=torch.int32, device=dev),
                     new_lens=torch.empty(S, dtype=torch.int32, device=dev))
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if case["op"] == "decode":
        return _decode_own(state) if own else _decode_plain(state)
    if case["op"] == "prompt":
        return _prompt_own(state) if own else _prompt_plain(state)
    state["key_weights"].copy_(state["sums"])
    return _evict_own(state) if own else _evict_plain(state)


def _decode_own(state):
    import paged_kv_cache_241_gb300 as pkv

    pkv.paged_decode_weights_attn(state["out"], state["key_weights"], state["q"], state["k_cache"], state["v_cache"], state["block_tables"],
                                  state["context_lens"], state["scale"], state["workspace"], state["total_blocks"],
                                  k=state.get("k"), v=state.get("v"), slot_mapping=state.get("slot_mapping"))
    return _decode_outputs(state, state["out"])


def _prompt_own(state):
    import paged_kv_cache_241_gb300 as pkv

    pkv.paged_prefill_weights(state["key_weights"], state["q"], state["k_cache"], state["block_tables"], state["cu_q"], state["cu_k"],
                              state["longest_q"], state["case"]["window"], state["scale"], state["workspace"])
    return state["key_weights"]


def _evict_own(state):
    import paged_kv_cache_241_gb300 as pkv

    case = state["case"]
    pkv.kv_evict(state["k_cache"], state["v_cache"], state["key_weights"], state["block_tables"], state["context_lens"], case["budget"],
                 case["recent"], state["kept"], state["new_lens"])
    return _evict_outputs(state, state["kept"], state["new_lens"])


def _decode_outputs(state, out):
    got = {"out": out, "key_weights": state["key_weights"]}
    return dict(got, k_cache=state["k_cache"], v_cache=state["v_cache"]) if state["case"]["store"] else got


def _evict_outputs(state, kept, new_lens):
    return {"k_cache": state["k_cache"], "v_cache": state["v_cache"], "key_weights": state["key_weights"], "kept": kept, "new_lens": new_lens}


# ------------------------------------------------------------- the plain forms

def _places(state):
    """Positions 0 .. longest-1 of every sequence: whether they hold a token [S, L], and their slot
    (positions without one: a slot of the block that no sequence holds)."""
    BS = state["case"]["block"]
    pos = torch.arange(state["longest"], device="cuda")
    valid = pos < state["context_lens"][:, None]
    slot = state["block_tables"].long()[:, pos // BS] * BS + pos % BS
    return pos, valid, torch.where(valid, slot, state["spare_block"] * BS)


def _sums_at(case, slot):
    """Index of a slot's sum, for each kv head, in key_weights.view(-1): [S, Hkv, L]."""
    BS, Hkv = case["block"], case["kv_heads"]
    return ((slot // BS)[:, None, :] * Hkv + torch.arange(Hkv, device="cuda")[:, None]) * BS + (slot % BS)[:, None, :]


def _rows(cache, slot):
    """Cache rows [S, Hkv, L, D] in 32 bits."""
    return cache.flatten(0, 1)[slot].transpose(1, 2).float()


def _softmax(z):
    z = torch.exp(z - z.amax(-1, keepdim=True))
    return z / z.sum(-1, keepdim=True)


def _collect(state, slot, valid, old, brought):
    """Adds `brought` [S, Hkv, L] to the sums where `old` [S, L], sets them where not; places without a token stay."""
    at = _sums_at(state["case"], slot)
    sums = state["key_weights"].view(-1)
    before = sums[at]
    after = torch.where(old[:, None, :], before + brought, brought)
    sums[at] = torch.where(valid[:, None, :], after, before)


def _decode_plain(state):
    case = state["case"]
    S, Hkv, D = case["seqs"], case["kv_heads"], case["dim"]
    if case["store"]:
        state["k_cache"].flatten(0, 1)[state["slot_mapping"].long()] = state["k"]
        state["v_cache"].flatten(0, 1)[state["slot_mapping"].long()] = state["v"]
    pos, valid, slot = _places(state)
    q = state["q"].float().view(S, Hkv, -1, D)
    z = torch.matmul(q, _rows(state["k_cache"], slot).transpose(2, 3)) * state["scale"]
    w = _softmax(z.masked_fill(~valid[:, None, None, :], -math.inf))
    out = torch.matmul(w, _rows(state["v_cache"], slot)).view(S, -1, D).to(torch.bfloat16)
    _collect(state, slot, valid, pos < state["context_lens"][:, None] - 1, w.sum(2))
    return _decode_outputs(state, out)


def _prompt_plain(state):
    case = state["case"]
    S, Hkv, D = case["seqs"], case["kv_heads"], case["dim"]
    pos, valid, slot = _places(state)
    n = (state["cu_q"][1:] - state["cu_q"][:-1]).long()[:, None]
    cached = state["context_lens"].long()[:, None] - n
    i = torch.arange(state["longest_q"] - min(case["window"], state["longest_q"]), state["longest_q"], device="cuda") - state["longest_q"] + n
    counts = i >= 0  # [S, R]: the queries that count, the last ones of each sequence
    q = state["q"][state["cu_q"][:-1].long()[:, None] + i.clamp(min=0)].float().view(S, i.shape[1], Hkv, -1, D).permute(0, 2, 3, 1, 4)
    z = torch.matmul(q.flatten(2, 3), _rows(state["k_cache"], slot).transpose(2, 3)) * state["scale"]
    sees = pos <= (cached + i.clamp(min=0))[:, :, None]
    z = z.view(S, Hkv, -1, i.shape[1], pos.shape[0]).masked_fill(~sees[:, None, None], -math.inf)
    w = _softmax(z).masked_fill(~counts[:, None, None, :, None], 0.0)
    _collect(state, slot, valid, pos < cached, w.sum((2, 3)))
    return state["key_weights"]


def _evict_plain(state):
    case = state["case"]
    budget, recent = case["budget"], case["recent"]
    heavy = budget - recent
    pos, valid, slot = _places(state)
    L = state["context_lens"].long()[:, None, None]
    at = _sums_at(case, slot)
    sums = state["key_weights"].view(-1)[at]
    cuts = L > budget
    # The heaviest of the tokens before the recent ones, the first of equals first.
    rank_by = torch.where(torch.isnan(sums), -math.inf, sums) + 0.0
    candidate = (pos < L - recent).expand_as(sums)
    order = torch.sort(rank_by.masked_fill(~candidate, -math.inf), dim=-1, descending=True, stable=True).indices
    order = torch.gather(order, 2, torch.sort(torch.gather(candidate, 2, order).logical_not().to(torch.uint8), dim=-1, stable=True).indices)
    kept = torch.zeros_like(candidate).scatter_(2, order[..., :heavy], True) & candidate
    # The k-th kept token behind the first `heavy` places takes the k-th free one of them.
    hole, mover = ~kept & (pos < heavy), kept & (pos >= heavy)
    by_rank = torch.zeros(*sums.shape[:2], pos.shape[0] + 1, dtype=torch.long, device="cuda")
    by_rank.scatter_(2, torch.where(mover, mover.cumsum(2) - 1, pos.shape[0]), pos.expand_as(sums))
    place = torch.arange(budget, device="cuda")
    inside = place.clamp(max=pos.shape[0] - 1)
    filled = torch.gather(by_rank, 2, (hole.cumsum(2) - 1).clamp(min=0))[..., inside]
    source = torch.where(place >= heavy, place + L - budget, torch.where(hole[..., inside], filled, place))
    source = torch.where(cuts, source, torch.where(place < L, place, -1))
    # Rows move with their sums; a place that keeps its token, or has none, is left alone.
    moves = cuts & (source != place)
    spare = (pos[:1] * 0 + state["spare_block"] * case["block"])
    slots = torch.cat([slot, spare.expand(slot.shape[0], 1)], 1)[:, None, :].expand(-1, case["kv_heads"], -1)
    src = torch.gather(slots, 2, torch.where(moves, source, pos.shape[0]))
    dst = torch.gather(slots, 2, torch.where(moves, place, pos.shape[0]))
    head = torch.arange(case["kv_heads"], device="cuda")[:, None]
    rows_from, rows_to = src * case["kv_heads"] + head, dst * case["kv_heads"] + head
    for cache in (state["k_cache"], state["v_cache"]):
        rows = cache.flatten(0, 2)
        rows[rows_to] = rows[rows_from]
    BS = case["block"]
    flat = state["key_weights"].view(-1)
    flat[(dst // BS * case["kv_heads"] + head) * BS + dst % BS] = flat[(src // BS * case["kv_heads"] + head) * BS + src % BS]
    return _evict_outputs(state, source.to(torch.int32), torch.minimum(state["context_lens"], torch.full_like(state["context_lens"], budget)))


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """One sequence at a time, from the definitions."""
    state = prepare(case, seed)
    BS, Hkv, Hq, D = case["block"], case["kv_heads"], case["q_heads"], case["dim"]
    tables, ctx = state["block_tables"].cpu().long(), _contexts(case)
    pages = [(tables[s, torch.arange(L) // BS].cuda(), (torch.arange(L) % BS).cuda()) for s, L in enumerate(ctx)]
    if case["op"] == "decode":
        sums = state["key_weights"].double()
        outs = []
        for s, (blk, off) in enumerate(pages):
            if case["store"]:
                state["k_cache"][blk[-1], off[-1]] = state["k"][s]
                state["v_cache"][blk[-1], off[-1]] = state["v"][s]
            K, V = state["k_cache"][blk, off].double(), state["v_cache"][blk, off].double()
            w = torch.softmax(state["scale"] * torch.einsum("jgd,pjd->jgp", state["q"][s].double().view(Hkv, -1, D), K), -1)
            outs.append(torch.einsum("jgp,pjd->jgd", w, V).reshape(Hq, D))
            sums[blk[-1], :, off[-1]] = 0.0
            sums[blk, :, off] += w.sum(1).T
        got = {"out": torch.stack(outs), "key_weights": sums}
        return dict(got, k_cache=state["k_cache"], v_cache=state["v_cache"]) if case["store"] else got
    if case["op"] == "prompt":
        sums = state["key_weights"].double()
        first = 0
        for (blk, off), L, n in zip(pages, ctx, _lens(case)):
            R = min(n, case["window"])
            q = state["q"][first + n - R:first + n].double().view(R, Hkv, -1, D)
            first += n
            late = torch.arange(L, device="cuda") > torch.arange(L - R, L, device="cuda")[:, None]
            K = state["k_cache"][blk, off].double()
            sums[blk[L - n:], :, off[L - n:]] = 0.0
            for j in range(Hkv):
                z = state["scale"] * torch.einsum("igd,pd->gip", q[:, j], K[:, j])
                sums[blk, j, off] += torch.softmax(z.masked_fill(late, -math.inf), -1).sum((0, 1))
        return sums
    # Eviction moves values and computes none: position by position, on the host.
    budget, recent = case["budget"], case["recent"]
    before = state["sums"].cpu()
    kept = torch.full((case["seqs"], Hkv, budget), -1, dtype=torch.int32)
    after = state["sums"].double()
    for s, ((blk, off), L) in enumerate(zip(pages, ctx)):
        if L <= budget:
            kept[s, :, :L] = torch.arange(L, dtype=torch.int32)
            continue
        heavy = budget - recent
        for j in range(Hkv):
            a = before[blk.cpu(), j, off.cpu()].tolist()
            best = set(sorted(range(L - recent), key=lambda p: (-a[p], p))[:heavy])
            coming = iter(sorted(p for p in best if p >= heavy))
            kept[s, j] = torch.tensor([p if p in best else next(coming) for p in range(heavy)] + list(range(L - recent, L)), dtype=torch.int32)
            to, source = torch.arange(budget), kept[s, j].long()
            b, o = blk.cpu(), off.cpu()
            for cache in (state["k_cache"], state["v_cache"]):
                cache[b[to], o[to], j] = cache[b[source], o[source], j]
            after[b[to], j, o[to]] = after[b[source], j, o[source]]
    return {"k_cache": state["k_cache"], "v_cache": state["v_cache"], "key_weights": after, "kept": kept,
            "new_lens": torch.tensor([min(L, budget) for L in ctx], dtype=torch.int32)}
