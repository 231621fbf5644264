"""Calls for new tokens, on the GPU, as programs make them: buffers cut back to back out of one
allocation, and whole steps captured in a graph and replayed with other lengths."""
import math

import pytest

from test_chunk_gpu import BLOCK, Batch, blocks, check, table_step

pytestmark = pytest.mark.gpu


class Arena:
    """Pieces of one allocation, back to back; one taken `back` bytes early overlaps the one before it."""

    def __init__(self, size):
        import torch
        self.bytes, self.at = torch.zeros(size, dtype=torch.uint8, device="cuda"), 0

    def take(self, shape, dtype, back=0):
        import torch
        n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
        start = self.at - back
        self.at = start + n
        return self.bytes[start:self.at].view(dtype).view(shape)


def refused(call):
    import shared_prefix_kv_fca_b200 as fca
    with pytest.raises(fca.FcaError, match="INVALID_ARG"):
        call()


def test_tables_in_buffers_that_touch():
    import torch
    import shared_prefix_kv_fca_b200 as fca
    had, new, width = [5, 16, 0, 31], [20, 1, 40, 3], 6
    s, want = table_step(had, new, width, seed=5)
    R = len(had)
    shapes = {"tables": (R, width), "seq": (R,), "starts": (R + 1,), "slots": (s["slots"],), "after": (1,), "status": (1,),
              "cached": (R,), "fresh": (R,), "free": (len(s["free"]),), "next": (1,)}
    values = {"tables": s["tables"], "cached": had, "fresh": new, "free": s["free"], "next": [s["skip"]]}

    def laid_out(order, moved=None):
        arena = Arena(4096)
        t = {n: arena.take(shapes[n], torch.int32, 4 if n == moved else 0) for n in order}
        for n, v in values.items():
            t[n].copy_(torch.tensor(v, dtype=torch.int32))
        before = arena.bytes.clone()

        def call():
            fca.fca_extend_tables(t["tables"], t["cached"], t["fresh"], t["free"], t["next"], s["pool"], t["seq"], t["starts"],
                                  t["slots"], free_after=t["after"], dev_status=t["status"])
        return arena, t, before, call

    names = list(shapes)
    for order in (names, names[::-1], names[3:] + names[:3]):
        arena, t, _, call = laid_out(order)
        call()
        got = {n: t[n].tolist() for n in names}
        assert got["tables"] == want["tables"] and got["seq"] == want["seq"] and got["starts"] == want["starts"]
        assert got["slots"] == want["slots"] and got["after"] == [want["after"]] and got["status"] == [0]
        assert got["cached"] == had and got["fresh"] == new and got["free"] == s["free"] and got["next"] == [s["skip"]]
        assert not arena.bytes[arena.at:].any()
        for prev, n in zip(order, order[1:]):           # one element into the piece before it
            arena, t, before, call = laid_out(order, n)
            if not {prev, n} & set(names[:6]):
                continue                                # inputs may share memory
            if len({prev, n} & {"after", "next"}) == 2:
                continue                                # the list position may be updated in place
            refused(call)
            torch.cuda.synchronize()
            assert torch.equal(arena.bytes, before), (prev, n)


def test_rows_and_caches_that_touch():
    import torch
    import shared_prefix_kv_fca_b200 as fca
    T, hkv, d, pool = 20, 2, 64, 9
    g = torch.Generator(device="cuda").manual_seed(6)
    shapes = {"k_cache": (pool, BLOCK, hkv, d), "k": (T, hkv, d), "v_cache": (pool, BLOCK, hkv, d), "v": (T, hkv, d)}
    slots = torch.randperm(pool * BLOCK, generator=g, device="cuda")[:T].int()
    for moved in (None, "k", "v_cache", "v"):
        arena = Arena(1 << 18)
        t = {n: arena.take(x, torch.bfloat16, 16 if n == moved else 0) for n, x in shapes.items()}
        own = arena.take((T,), torch.int32)
        own.copy_(slots)
        for x in t.values():
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        before = arena.bytes.clone()
        want = {n: x.clone() for n, x in t.items()}

        def call():
            fca.fca_append_kv(t["k"], t["v"], own, t["k_cache"], t["v_cache"], pool)
        if moved:
            refused(call)
            torch.cuda.synchronize()
            assert torch.equal(arena.bytes, before), moved
            continue
        call()
        for c, x in (("k_cache", "k"), ("v_cache", "v")):
            want[c].view(-1, hkv, d)[slots.long()] = want[x]
        assert all(torch.equal(t[n], want[n]) for n in t) and torch.equal(own, slots)
        assert not arena.bytes[arena.at:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_in_buffers_that_touch(d):
    import torch
    import shared_prefix_kv_fca_b200 as fca
    b = Batch([200, 45], [30, 45], 4, 2, d, seed=7, packed=False)
    shapes = {"out": b.out.shape, "k": b.k.shape, "lse": b.lse.shape, "q": b.q.shape, "v": b.v.shape}
    names = list(shapes)
    with b.plan() as plan:
        for order in (names, names[::-1]):
            for moved in [None] + order[1:]:
                arena = Arena(1 << 22)
                t = {n: arena.take(shapes[n], torch.float32 if n == "lse" else torch.bfloat16, 16 if n == moved else 0)
                     for n in order}
                for n, x in (("q", b.q), ("k", b.k), ("v", b.v)):
                    t[n].copy_(x)
                before = arena.bytes.clone()

                def call():
                    fca.fca_chunk_attention(t["q"], t["k"], t["v"], plan, t["out"], t["lse"], b.scale)
                if moved and {moved, order[order.index(moved) - 1]} & {"out", "lse"}:
                    refused(call)
                    torch.cuda.synchronize()
                    assert torch.equal(arena.bytes, before), moved
                elif moved is None:
                    call()
                    b.out, b.lse = t["out"], t["lse"]
                    check(b, what=f"{order}")
                    assert torch.equal(t["q"], b.q) and not arena.bytes[arena.at:].any()
                    for n, x in (("k", b.k), ("v", b.v)):
                        assert torch.equal(t[n].view(torch.int16), x.view(torch.int16))
        # an output inside a cache that starts where the queries do
        q = b.k.view(-1)[:b.q.numel()].view(b.q.shape)
        before = b.k.clone()
        inside = b.k.view(-1)[-b.q.numel():].view(b.q.shape)
        assert inside.data_ptr() >= q.data_ptr() + q.numel() * 2
        refused(lambda: fca.fca_chunk_attention(q, b.k, b.v, plan, inside, None, b.scale))
        lse = b.k.view(-1)[-b.lse.numel() * 2:].view(torch.float32).view(b.lse.shape)
        refused(lambda: fca.fca_chunk_attention(q, b.k, b.v, plan, b.out, lse, b.scale))
        torch.cuda.synchronize()
        assert torch.equal(before.view(torch.int16), b.k.view(torch.int16))


@pytest.mark.parametrize("large", [False, True], ids=["one_launch", "two_launches"])
def test_a_captured_step_of_tables_and_writes(large):
    """The graph is replayed over a run of steps whose lengths change; a step that cannot be made changes nothing."""
    import random
    import torch
    import shared_prefix_kv_fca_b200 as fca
    rng = random.Random(large)
    R, most, hkv, d = (1500, 40, 1, 64) if large else (7, 60, 2, 64)
    steps = [[rng.choice([0, 1, 1, rng.randrange(most)]) for _ in range(R)] for _ in range(4)]
    cap = max(map(sum, steps)) + 11
    assert (cap > 4096) == large                    # the longest step that is one launch
    width = blocks(sum(max(s) for s in steps)) + 1
    pool = sum(blocks(sum(s[r] for s in steps)) for r in range(R)) + 5
    g = torch.Generator(device="cuda").manual_seed(8)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")      # noqa: E731
    tables, lens, fresh, nxt, starts, slots, status = z(R, width), z(R), z(R), z(1), z(R + 1), z(cap), z(1)
    free = torch.randperm(pool, generator=g, device="cuda").int()
    k, v = (torch.zeros(cap, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    caches = [torch.zeros(pool, BLOCK, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step():
        fca.fca_extend_tables(tables, lens, fresh, free, nxt, pool, lens, starts, slots, dev_status=status)
        fca.fca_append_kv(k, v, slots, *caches, pool, dev_status=status)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                      # no new tokens
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
            step()
    torch.cuda.synchronize()
    had, taken, ids = [0] * R, 0, free.tolist()
    table = [[0] * width for _ in range(R)]
    want = [c.clone() for c in caches]
    for new in steps:
        fresh.copy_(torch.tensor(new, dtype=torch.int32))
        for x in (k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        where, edges = [], [0]
        for r, n in enumerate(new):
            for p in range(had[r], had[r] + n):
                if p % BLOCK == 0:
                    table[r][p // BLOCK] = ids[taken]
                    taken += 1
                where.append(table[r][p // BLOCK] * BLOCK + p % BLOCK)
            had[r] += n
            edges.append(len(where))
        at = torch.tensor(where, dtype=torch.long, device="cuda")
        for c, x in zip(want, (k, v)):
            c.view(-1, hkv, d)[at] = x[:len(where)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert tables.tolist() == table and lens.tolist() == had and nxt.item() == taken and starts.tolist() == edges
        assert slots.tolist() == where + [-1] * (cap - len(where)) and status.item() == 0
        assert all(torch.equal(c, w) for c, w in zip(caches, want))
    fresh.copy_(torch.tensor([width * BLOCK] + [0] * (R - 1), dtype=torch.int32))     # longer than the table
    fresh[0] += 1
    graph.replay()
    torch.cuda.synchronize()
    assert status.item() & 8 and tables.tolist() == table and lens.tolist() == had and nxt.item() == taken
    assert set(starts.tolist()) == {0} and set(slots.tolist()) == {-1}
    assert all(torch.equal(c, w) for c, w in zip(caches, want))
    del graph
