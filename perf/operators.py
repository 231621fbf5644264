"""Timed calls of the operators that put new tokens into the paged cache and attend from them.

One serving step of a batch whose requests have tokens in the cache and bring new ones:

* ``tables``  the requests' block tables grow by blocks off the free list, and each new token gets its
              cache slot (from the requests' lengths);
* ``append``  the new tokens' keys and values go into the cache at their slots;
* ``attend``  each new token's queries attend over the request's cached tokens and the chunk's tokens
              up to itself (or, ``full``, over all states that an encoder left in the cache).

Head layouts, lengths and the block size of 16 tokens are those of the decode workloads in
``fca_workloads`` (4/1/64, 32/8/128 and 64/8/128 heads; prompts of 128, 1024, 2048 and 32768 tokens), or
generic.  Queries, keys and values are views of one packed projection output, as a model has them.
"""
import math
import random

import torch

own = False

BLOCK = 16


def listed():
    return [
        # a decode step's tables: one token each, most requests inside their last block
        {"name": "tables_decode", "op": "tables", "requests": 256, "new_lo": 1, "new_hi": 1, "had_lo": 1,
         "had_hi": 4096, "padded": 0, "shape": 1},
        # a step of prompts of uneven length beside decodes, in slots padded for a captured graph
        {"name": "tables_mixed", "op": "tables", "requests": 1000, "new_lo": 0, "new_hi": 37, "had_lo": 0,
         "had_hi": 6000, "padded": 777, "shape": 2},
        # many prompts at once, from nothing
        {"name": "tables_prompts", "op": "tables", "requests": 2048, "new_lo": 16, "new_hi": 240, "had_lo": 0,
         "had_hi": 0, "padded": 0, "shape": 3},
        # the tokens of one decode step, one for each request
        {"name": "append_decode", "op": "append", "requests": 256, "run": 1, "padded": 0, "blocks": 4096,
         "hkv": 8, "d": 128, "shape": 4},
        # an odd number of tokens in short runs, padded
        {"name": "append_odd", "op": "append", "requests": 83, "run": 25, "padded": 93, "blocks": 1024, "hkv": 4,
         "d": 64, "shape": 5},
        # the prompts of the 16-prompt workload in one step
        {"name": "append_prompts", "op": "append", "requests": 16, "run": 2048, "padded": 0, "blocks": 3000,
         "hkv": 8, "d": 128, "shape": 6},
        # the smallest heads, a few new tokens each: the call's latency
        {"name": "attend_tiny", "op": "attend", "requests": 8, "new_lo": 1, "new_hi": 8, "had_lo": 100, "had_hi": 160,
         "decodes": 0, "shared": 0, "hq": 4, "hkv": 1, "d": 64, "full": False, "lse": True, "replan": False, "shape": 7},
        # drafted tokens of many requests verified at once, under a shared prompt: bound by the cache's bytes
        {"name": "attend_verify", "op": "attend", "requests": 64, "new_lo": 5, "new_hi": 5, "had_lo": 1500, "had_hi": 8000,
         "decodes": 0, "shared": 1024, "hq": 32, "hkv": 8, "d": 128, "full": False, "lse": True, "replan": False, "shape": 8},
        # whole prompts from nothing: bound by the matrix products
        {"name": "attend_prompts", "op": "attend", "requests": 16, "new_lo": 2048, "new_hi": 2048, "had_lo": 0, "had_hi": 0,
         "decodes": 0, "shared": 0, "hq": 32, "hkv": 8, "d": 128, "full": False, "lse": False, "replan": False, "shape": 9},
        # one prompt's chunk beside decodes, the step's first layer: the work lists are made anew too
        {"name": "attend_mixed", "op": "attend", "requests": 1, "new_lo": 1999, "new_hi": 1999, "had_lo": 6001, "had_hi": 6001,
         "decodes": 95, "shared": 0, "hq": 64, "hkv": 8, "d": 128, "full": False, "lse": False, "replan": True, "shape": 10},
        # a chunk of a long document
        {"name": "attend_long", "op": "attend", "requests": 1, "new_lo": 4096, "new_hi": 4096, "had_lo": 32768, "had_hi": 32768,
         "decodes": 0, "shared": 0, "hq": 32, "hkv": 8, "d": 128, "full": False, "lse": False, "replan": False, "shape": 11},
        # decoder tokens over an encoder's states, one of the requests with none
        {"name": "attend_encoder", "op": "attend", "requests": 25, "new_lo": 7, "new_hi": 440, "had_lo": 700, "had_hi": 1500,
         "decodes": 0, "shared": 0, "hq": 16, "hkv": 16, "d": 64, "full": True, "lse": True, "replan": False, "shape": 12},
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(max(lo, 0.5)), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend"])
    shape = rng.randrange(1 << 30)
    if op == "tables":
        r = _log(rng, 1, 2500)
        hi = _log(rng, 1, max(1, min(4000, 250000 // r)))
        return {"op": op, "requests": r, "new_lo": rng.choice([0, 1, hi]), "new_hi": hi, "had_lo": 0,
                "had_hi": rng.choice([0, _log(rng, 1, 8000)]), "padded": rng.choice([0, _log(rng, 1, 1000)]), "shape": shape}
    if op == "append":
        r = _log(rng, 1, 512)
        run = _log(rng, 1, 30000 // r)
        return {"op": op, "requests": r, "run": run, "padded": rng.choice([0, _log(rng, 1, 500)]),
                "blocks": r * (-(-run // BLOCK) + 1) + rng.randrange(1, 900), "hkv": rng.choice([1, 2, 4, 5, 8]),
                "d": rng.choice([64, 128]), "shape": shape}
    hq, hkv = rng.choice([(4, 1), (8, 2), (16, 16), (28, 4), (24, 8), (32, 8), (64, 8), (16, 1)])
    full = rng.random() < 0.25
    r = _log(rng, 1, 64)
    new = _log(rng, 1, max(1, 4000 // r))
    had = _log(rng, 16, max(32, min(32000, 200000 // r)))
    shared = 0 if full else rng.choice([0, 0, had // 2 // BLOCK * BLOCK])
    return {"op": op, "requests": r, "new_lo": max(1, new // 3), "new_hi": new, "had_lo": max(shared, had // 2), "had_hi": had,
            "decodes": rng.choice([0, 0, _log(rng, 1, 64)]), "shared": shared, "hq": hq, "hkv": hkv,
            "d": rng.choice([64, 128]), "full": full, "lse": rng.random() < 0.5, "replan": rng.random() < 0.3, "shape": shape}


def _lengths(case):
    """(cached, new) tokens of each request, the same for every seed."""
    rng = random.Random(case["shape"])
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["requests"])]
    had = [rng.randint(case["had_lo"], case["had_hi"]) for _ in range(case["requests"])]
    for _ in range(case.get("decodes", 0)):
        new.append(1)
        had.append(rng.randint(max(1, case["had_lo"] // 8), max(1, case["had_hi"] // 2)))
    if case.get("full") and len(had) > 1:
        had[1] = 0
    return had, new


def _blocks(n):
    return -(-n // BLOCK)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = random.Random(seed)

    def normal(*size):
        return torch.randn(size, generator=gen, device="cuda", dtype=torch.float32).bfloat16()

    s = {"op": case["op"], "case": case}
    if case["op"] == "tables":
        had, new = _lengths(case)
        r = len(had)
        held = [_blocks(c) for c in had]
        grown = sum(_blocks(c + n) - _blocks(c) for c, n in zip(had, new))
        width = max(_blocks(c + n) for c, n in zip(had, new)) + 3
        skip = host.randrange(1, 50)                       # blocks that earlier steps took off the list
        pool = sum(held) + grown + skip + 100
        ids = torch.randperm(pool, generator=gen, device="cuda").int()
        at = _offsets(held)
        tables = torch.zeros(r, width, dtype=torch.int32, device="cuda")
        col = torch.arange(width, device="cuda")[None]
        start = torch.tensor(at[:-1], device="cuda")[:, None]
        count = torch.tensor(held, device="cuda")[:, None]
        tables = torch.where(col < count, ids[(start + col).clamp(max=pool - 1)], tables).contiguous()
        tokens = sum(new)
        s.update(pool=pool, tables=tables, had=_ints(had), new=_ints(new), free=ids[at[-1]:].contiguous(),
                 free_next=_ints([skip]), seq=_ints([0] * r), starts=_ints([0] * (r + 1)),
                 slots=_ints([0]).expand(tokens + case["padded"]).contiguous(), free_after=_ints([0]))
        return s
    hkv, d = case["hkv"], case["d"]
    if case["op"] == "append":
        r, run, nb = case["requests"], case["run"], case["blocks"]
        per = _blocks(run) + 1 if run > 1 else 1
        order = torch.randperm(nb, generator=gen, device="cuda")
        first = torch.randint(0, BLOCK, (r, 1), generator=gen, device="cuda")
        pos = first + torch.arange(run, device="cuda")[None]
        slots = order[(torch.arange(r, device="cuda")[:, None] * per + pos // BLOCK)] * BLOCK + pos % BLOCK
        slots = torch.cat([slots.reshape(-1), torch.full((case["padded"],), -1, device="cuda")]).int()
        tokens = r * run + case["padded"]
        packed = normal(tokens, (2 * hkv + 4 * hkv) * d)   # a projection's output: queries, keys, values
        k = packed[:, 4 * hkv * d:5 * hkv * d].view(tokens, hkv, d)
        v = packed[:, 5 * hkv * d:].view(tokens, hkv, d)
        s.update(tokens=r * run, slots=slots, k=k, v=v, pool=nb, k_cache=normal(nb, BLOCK, hkv, d),
                 v_cache=normal(nb, BLOCK, hkv, d))
        return s
    had, new = _lengths(case)
    hq, full = case["hq"], case["full"]
    seq = had if full else [c + n for c, n in zip(had, new)]
    common = case["shared"] // BLOCK
    lead = [common if c >= case["shared"] else 0 for c in had]
    pool = common + sum(_blocks(l) - p for l, p in zip(seq, lead)) + 5
    ids = torch.randperm(pool, generator=gen, device="cuda").int()
    width = max(_blocks(l) for l in seq) + 2
    tables = ids[torch.randint(0, pool, (len(seq), width), generator=gen, device="cuda")]
    at = common
    for r, (l, p) in enumerate(zip(seq, lead)):
        tables[r, :p] = ids[:p]
        n = _blocks(l) - p
        tables[r, p:p + n] = ids[at:at + n]
        at += n
    tokens = sum(new)
    packed = normal(tokens, (hq + 2 * hkv) * d)
    s.update(seq_host=seq, new_host=new, tables=tables, seq=_ints(seq), starts=_ints(_offsets(new)), tokens=tokens, pool=pool,
             q=packed[:, :hq * d].view(tokens, hq, d), k_cache=normal(pool, BLOCK, hkv, d), v_cache=normal(pool, BLOCK, hkv, d),
             out=torch.empty(tokens, hq, d, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(tokens, hq, dtype=torch.float32, device="cuda") if case["lse"] else None)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] == "attend":
        # the step's work lists, which every layer of the step uses
        import shared_prefix_kv_fca_b200 as fca
        s["plan"] = fca.fca_chunk_plan(s["tables"], s["seq"], s["starts"], s["tokens"], s["pool"], case["hq"], case["hkv"],
                                       case["d"], full=case["full"])
    return s


def _tables(s):
    had, new, free, tables = s["had"].long(), s["new"].long(), s["free"], s["tables"]
    held, seq = (had + BLOCK - 1) // BLOCK, had + new
    need = (seq + BLOCK - 1) // BLOCK - held
    take = s["free_next"].long() + torch.cumsum(need, 0) - need
    ends = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    col = torch.arange(tables.shape[1], device=tables.device)[None]
    grown = (col >= held[:, None]) & (col < (held + need)[:, None])
    pick = (take[:, None] + col - held[:, None]).clamp(0, free.numel() - 1)
    tables.copy_(torch.where(grown, free[pick], tables))
    t = torch.arange(s["slots"].numel(), device=tables.device)
    r = torch.searchsorted(ends, t, right=True).clamp(max=had.numel() - 1)
    pos = (had[r] + t - starts[r]).clamp(max=tables.shape[1] * BLOCK - 1)
    slots = tables[r, pos // BLOCK].long() * BLOCK + pos % BLOCK
    s["slots"].copy_(torch.where(t < ends[-1], slots, -1))
    s["seq"].copy_(seq)
    s["starts"].copy_(starts)
    s["free_after"].copy_(s["free_next"] + need.sum())


def _append(s):
    n = s["tokens"]
    at = s["slots"][:n].long()
    s["k_cache"].view(-1, *s["k"].shape[1:])[at] = s["k"][:n]
    s["v_cache"].view(-1, *s["v"].shape[1:])[at] = s["v"][:n]


def _attend(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g, at = hq // hkv, 0
    for r, (length, n) in enumerate(zip(s["seq_host"], s["new_host"])):
        rows = slice(at, at + n)
        at += n
        ids = s["tables"][r, :_blocks(length)].long()
        k = s["k_cache"][ids].view(-1, hkv, d)[:length].float().permute(1, 2, 0)
        v = s["v_cache"][ids].view(-1, hkv, d)[:length].float().permute(1, 0, 2)
        q = s["q"][rows].float().view(n, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, n * g, d)
        if length == 0:
            s["out"][rows] = 0
            if s["lse"] is not None:
                s["lse"][rows] = -math.inf
            continue
        score = torch.matmul(q, k).mul_(1.0 / math.sqrt(d)).view(hkv, n, g, length)
        if not case["full"]:
            last = torch.arange(length - n, length, device=q.device)
            hidden = torch.arange(length, device=q.device)[None] > last[:, None]
            score.masked_fill_(hidden[None, :, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        total = score.sub_(top).exp_().sum(-1, keepdim=True)
        o = torch.matmul(score.view(hkv, n * g, length), v).view(hkv, n, g, d) / total
        s["out"][rows] = o.permute(1, 0, 2, 3).reshape(n, hq, d).bfloat16()
        if s["lse"] is not None:
            s["lse"][rows] = (top + total.log()).permute(1, 0, 2, 3).reshape(n, hq)


def run(state):
    s, op = state, state["op"]
    if op == "tables":
        if own:
            import shared_prefix_kv_fca_b200 as fca
            fca.fca_extend_tables(s["tables"], s["had"], s["new"], s["free"], s["free_next"], s["pool"], s["seq"], s["starts"],
                                  s["slots"], free_after=s["free_after"])
        else:
            _tables(s)
        return s["tables"], s["seq"], s["starts"], s["slots"], s["free_after"]
    if op == "append":
        if own:
            import shared_prefix_kv_fca_b200 as fca
            fca.fca_append_kv(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["pool"])
        else:
            _append(s)
        return s["k_cache"], s["v_cache"]
    if own:
        import shared_prefix_kv_fca_b200 as fca
        if s["case"]["replan"]:
            fca.fca_chunk_plan_update(s["plan"], s["tables"], s["seq"], s["starts"])
        fca.fca_chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["plan"], s["out"], s["lse"])
    else:
        _attend(s)
    return s["out"] if s["lse"] is None else (s["out"], s["lse"])


def work(case):
    if case["op"] == "append":
        n = case["requests"] * case["run"]
        return {"bytes": 2 * 2 * n * case["hkv"] * case["d"] * 2 + 4 * (n + case["padded"]), "flops": 0}
    had, new = _lengths(case)
    if case["op"] == "tables":
        r, tokens = len(had), sum(new)
        grown = sum(_blocks(c + n) - _blocks(c) for c, n in zip(had, new))
        inside = sum(1 for c, n in zip(had, new) if n and c % BLOCK)
        # lengths in, list entries in, table entries out, last blocks in; lengths, starts, slots and the count out
        return {"bytes": 4 * (2 * r + 2 * grown + inside + 2 * r + 1 + tokens + case["padded"] + 2), "flops": 0}
    hq, hkv, d, full = case["hq"], case["hkv"], case["d"], case["full"]
    seq = had if full else [c + n for c, n in zip(had, new)]
    seen = sum(n * l if full else n * (l - n) + n * (n + 1) // 2 for l, n in zip(seq, new))
    sharing = [c for c in had if c >= case["shared"]]
    states = sum(seq) - max(0, len(sharing) - 1) * case["shared"]      # a shared prompt's states are read once
    rows = sum(new) * hq
    return {"bytes": 2 * 2 * states * hkv * d + 2 * 2 * rows * d + (4 * rows if case["lse"] else 0),
            "flops": 4 * d * hq * seen}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        at = s["slots"].long()[:, None, None]
        for cache, rows in ((k, s["k"]), (v, s["v"])):
            flat = cache.view(-1, case["hkv"], case["d"])
            keep = slice(0, case["requests"] * case["run"])
            flat.scatter_(0, at[keep].expand(-1, case["hkv"], case["d"]), rows[keep].double())
        return k, v
    if case["op"] == "tables":
        had, new = s["had"].tolist(), s["new"].tolist()
        tables, free, at = s["tables"].tolist(), s["free"].tolist(), int(s["free_next"][0])
        starts, slots = [0], []
        for r, (c, n) in enumerate(zip(had, new)):
            for p in range(c, c + n):
                if p % BLOCK == 0:
                    tables[r][p // BLOCK] = free[at]
                    at += 1
                slots.append(tables[r][p // BLOCK] * BLOCK + p % BLOCK)
            starts.append(len(slots))
        slots += [-1] * (s["slots"].numel() - len(slots))
        return _ints(tables), _ints([c + n for c, n in zip(had, new)]), _ints(starts), _ints(slots), _ints([at])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.zeros(s["tokens"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], hq), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for r, (length, n) in enumerate(zip(s["seq_host"], s["new_host"])):
        where = torch.arange(length, device="cuda")
        slot = s["tables"][r].long()[where // BLOCK] * BLOCK + where % BLOCK
        for h in range(hkv if length else 0):
            k = s["k_cache"].view(-1, hkv, d)[slot, h].double()
            v = s["v_cache"].view(-1, hkv, d)[slot, h].double()
            q = s["q"][first:first + n, h * g:(h + 1) * g].double()
            score = torch.einsum("tgd,sd->gts", q, k) / math.sqrt(d)
            if not case["full"]:
                score += torch.full((n, length), -math.inf, dtype=torch.float64, device="cuda").triu(length - n + 1)
            total = torch.logsumexp(score, -1)
            lse[first:first + n, h * g:(h + 1) * g] = total.T
            out[first:first + n, h * g:(h + 1) * g] = torch.einsum("gts,sd->tgd", (score - total[..., None]).exp(), v)
        first += n
    return out if s["lse"] is None else (out, lse)
