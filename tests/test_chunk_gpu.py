"""New tokens in the paged cache, on the GPU: fca_extend_tables, fca_append_kv
and fca_chunk_attention against plain 64-bit definitions.

Tolerance of an attention output (bf16), element by element, with
o = sum_j w_j v_j over the visible tokens and A = sum_j w_j |v_j|:

* the weights are rounded to bf16 before the product with V, each by at most
  2^-8 of itself, and the result is divided by the sum of the rounded weights:
  at most 2 * 2^-8 * A;
* scores, exponentials and sums are held in 32 bits: a score is off by at most
  B = D 2^-23 max_j sum_i |q_i k_ji| scale, an exponential by 2^-20 more, a
  sum of n terms by n 2^-24: (2 B + 2^-19 + n 2^-23) A, small beside the above;
* the final rounding: 2^-8 |o| plus 2^-8 of all of the above.

Over a row's D elements the roundings of the weights, each at most 2^-8 and
taken as uniform and independent, add up to a vector of expected square
2^-16 / 3 sum_j w_j^2 |v_j|^2; a row may be off by six times the root of that
(and the terms above), which is far less than A for a row that averages many
tokens, and so shows a token that is wrong among thousands.

lse (fp32): B + 2^-20 + n 2^-24, plus 2^-23 |lse| for its own arithmetic.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

BLOCK = 16


def _torch():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch


def blocks(n):
    return -(-n // BLOCK)


class Batch:
    """A paged cache holding requests of given lengths; every slot that no
    token sits in is NaN."""

    def __init__(self, seq, new, hq, hkv, d, seed=0, spare=3, base=0, pool=None, pad_rows=0, packed=True):
        torch = _torch()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.seq_h, self.new_h, self.hq, self.hkv, self.d = list(seq), list(new), hq, hkv, d
        need = sum(blocks(l) for l in seq)
        self.pool = pool if pool else base + need + spare
        ids = base + torch.randperm(self.pool - base, generator=g, device="cuda")[:need] if not pool else \
            base + torch.randperm(need, generator=g, device="cuda")
        width = max([blocks(l) for l in seq] + [1]) + 2
        self.tables = torch.full((len(seq), width), -7, dtype=torch.int32, device="cuda")   # never read
        shape = (self.pool, BLOCK, hkv, d)
        if pool:
            self.k, self.v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        else:
            self.k, self.v = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.slot, at = [], 0
        for r, l in enumerate(seq):
            n = blocks(l)
            row = ids[at:at + n]
            at += n
            self.tables[r, :n] = row.int()
            self.k[row], self.v[row] = float("nan"), float("nan")
            p = torch.arange(l, device="cuda")
            s = row[p // BLOCK] * BLOCK + p % BLOCK
            self.slot.append(s)
            for c in (self.k, self.v):
                c.view(-1, hkv, d)[s] = torch.randn(l, hkv, d, generator=g, device="cuda").bfloat16()
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        self.starts_h = starts
        self.T = starts[-1] + pad_rows
        self.seq = torch.tensor(seq, dtype=torch.int32, device="cuda")
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        if packed:
            qkv = torch.randn(self.T, (hq + 2 * hkv) * d, generator=g, device="cuda").bfloat16()
            self.q = qkv[:, :hq * d].view(self.T, hq, d)
        else:
            self.q = torch.randn(self.T, hq, d, generator=g, device="cuda").bfloat16()
        self.out = torch.full((self.T, hq, d), 7.25, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, hq), 7.25, dtype=torch.float32, device="cuda")
        self.scale = 1 / math.sqrt(d)

    def plan(self, full=False):
        import shared_prefix_kv_fca_b200 as fca
        return fca.fca_chunk_plan(self.tables, self.seq, self.starts, self.T, self.pool, self.hq, self.hkv, self.d, full=full)

    def attend(self, plan, lse=True, stream=None):
        import shared_prefix_kv_fca_b200 as fca
        fca.fca_chunk_attention(self.q, self.k, self.v, plan, self.out, self.lse if lse else None, self.scale, stream=stream)


def reference(b, r, full):
    """(o, A, lse, B, N) of request r in 64 bits: [n, hq, d], [n, hq, d], and [n, hq] each."""
    torch = _torch()
    n, l, g = b.new_h[r], b.seq_h[r], b.hq // b.hkv
    s0 = b.starts_h[r]
    q = b.q[s0:s0 + n].double().view(n, b.hkv, g, b.d)
    k, v = (c.view(-1, b.hkv, b.d)[b.slot[r]].double() for c in (b.k, b.v))
    o = torch.zeros(n, b.hkv, g, b.d, dtype=torch.float64, device="cuda")
    a, lse = torch.zeros_like(o), torch.full((n, b.hkv, g), -math.inf, dtype=torch.float64, device="cuda")
    top, norm = torch.zeros_like(lse), torch.zeros_like(lse)
    pos = torch.arange(n, device="cuda") + (l - n)
    sees = torch.ones(n, l, dtype=torch.bool, device="cuda") if full else \
        torch.arange(l, device="cuda")[None] <= pos[:, None]
    for h in range(b.hkv if l else 0):
        s = torch.einsum("ngd,ld->ngl", q[:, h], k[:, h]) * b.scale
        s = s.masked_fill(~sees[:, None], -math.inf)
        lse[:, h] = torch.logsumexp(s, -1)
        w = (s - lse[:, h][..., None]).exp().masked_fill(~sees[:, None], 0.0)
        vf = v[:, h]
        if not bool(torch.isfinite(vf).all()):      # a token that a row does not see has no part in it
            vz = torch.where(torch.isfinite(vf), vf, torch.zeros_like(vf))
            o[:, h] = torch.einsum("ngl,ld->ngd", w, vz)
            special = ~torch.isfinite(vf)
            hit = torch.einsum("nl,ld->nd", sees.double(), special.double()) > 0
            o[:, h] = torch.where(hit[:, None], torch.full_like(o[:, h], math.nan), o[:, h])
            vf = vz
        else:
            o[:, h] = torch.einsum("ngl,ld->ngd", w, vf)
        a[:, h] = torch.einsum("ngl,ld->ngd", w, vf.abs())
        norm[:, h] = torch.einsum("ngl,l->ng", w * w, (vf * vf).sum(-1)).sqrt()
        big = torch.einsum("ngd,ld->ngl", q[:, h].abs(), k[:, h].abs()).masked_fill(~sees[:, None], 0.0)
        top[:, h] = big.amax(-1) * b.scale
    shape = (n, b.hq, b.d)
    return o.view(shape), a.view(shape), lse.view(n, b.hq), top.view(n, b.hq) * b.d * 2.0 ** -23, norm.view(n, b.hq)


def check(b, full=False, lse=True, what=""):
    torch = _torch()
    for r, (n, l) in enumerate(zip(b.new_h, b.seq_h)):
        if n == 0:
            continue
        s0 = b.starts_h[r]
        o, a, ref, err, norm = reference(b, r, full)
        got = b.out[s0:s0 + n].double()
        tol = (2 * 2.0 ** -8 + 2 * err[..., None] + 2.0 ** -19 + l * 2.0 ** -23) * a
        tol = tol + 2.0 ** -8 * (o.abs() + tol) + 1e-30
        nan = torch.isnan(o)
        assert bool((~torch.isfinite(got) == nan).all()), f"{what}: request {r}: finite elsewhere than it should be"
        off = ((got - o).abs() / tol).masked_fill(nan, 0)
        assert bool((off <= 1).all()), f"{what}: request {r} (n {n}, L {l}): {off.max().item():.3f} of the tolerance"
        rest = (2 * err + 2.0 ** -19 + l * 2.0 ** -23) * a.norm(dim=-1) + 2.0 ** -8 * o.masked_fill(nan, 0).norm(dim=-1)
        tol = 6 * 2.0 ** -8 / math.sqrt(3) * norm * (1 + 2.0 ** -8) + rest + 1e-30
        off = (got - o).masked_fill(nan, 0).norm(dim=-1) / tol
        assert bool((off <= 1).all()), f"{what}: request {r} (n {n}, L {l}): a row is {off.max().item():.3f} of its tolerance"
        if lse:
            have = b.lse[s0:s0 + n].double()
            none = torch.isinf(ref)
            assert bool((torch.isinf(have) == none).all()), f"{what}: request {r}: lse"
            tol = err + 2.0 ** -20 + l * 2.0 ** -24 + 2.0 ** -23 * ref.abs()
            off = ((have - ref).abs() / tol).masked_fill(none, 0)
            assert bool((off <= 1).all()), f"{what}: request {r}: lse {off.max().item():.3f} of the tolerance"
    rest = b.starts_h[-1]
    assert bool((b.out[rest:] == 7.25).all()) and bool((b.lse[rest:] == 7.25).all()), f"{what}: rows behind the last"


HEADS = [(4, 1, 64), (8, 2, 128), (4, 4, 64), (6, 2, 128), (10, 2, 64), (7, 1, 128), (16, 1, 128), (32, 8, 128)]

LENGTHS = {
    "one": ([1], [1]),
    "one_behind": ([2], [1]),
    "stage_edges": ([127, 128, 129, 255, 256, 257], [1, 1, 1, 1, 1, 1]),
    "page_edges": ([15, 16, 17, 31, 33], [15, 16, 1, 31, 2]),
    "prompts": ([1, 5, 64, 65, 130, 300], [1, 5, 64, 65, 130, 300]),
    "tail": ([700, 1023, 40], [65, 2, 40]),
    "no_rows": ([10, 300, 17], [0, 3, 0]),
    "decodes": ([50, 333, 1000, 16], [1, 1, 1, 1]),
}


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("name", sorted(LENGTHS))
def test_attention_matches_the_definition(heads, name):
    import shared_prefix_kv_fca_b200 as fca
    seq, new = LENGTHS[name]
    b = Batch(seq, new, *heads, seed=len(name), pad_rows=3)
    with b.plan() as plan:
        b.attend(plan)
        assert fca.fca_chunk_check_status(plan) == 0
    check(b, what=f"{name} {heads}")


@pytest.mark.parametrize("heads", [(4, 1, 64), (6, 2, 128), (16, 16, 64)], ids=lambda h: "x".join(map(str, h)))
def test_full_attention_over_states_of_another_length(heads):
    # as many rows as one likes over any number of states, none among them
    b = Batch([300, 0, 1, 129, 40], [7, 5, 300, 1, 90], *heads, seed=3, pad_rows=1)
    with b.plan(full=True) as plan:
        b.attend(plan)
        check(b, full=True, what=f"full {heads}")
        b.out.fill_(7.25)
        b.lse.fill_(7.25)
        b.attend(plan, lse=False)           # the same outputs without lse
        check(b, full=True, lse=False, what="full without lse")
        assert bool((b.out[7:12] == 0).all()) and bool((b.lse == 7.25).all())


@pytest.mark.parametrize("seed", range(6))
def test_attention_on_random_batches(seed):
    import random
    rng = random.Random(seed)
    heads = rng.choice(HEADS)
    new = [rng.choice([0, 1, 1, 2, 9, rng.randrange(1, 400)]) for _ in range(rng.randrange(1, 20))] + [3]
    had = [rng.choice([0, 1, rng.randrange(3000)]) for _ in new]
    b = Batch([h + n for h, n in zip(had, new)], new, *heads, seed=seed)
    with b.plan() as plan:
        b.attend(plan)
    check(b, what=f"seed {seed} {heads}")


@pytest.mark.parametrize("d", [64, 128])
def test_long_rows_are_cut_and_joined(d):
    # one request, few rows, a long cache: every tile is cut into many pieces
    b = Batch([20000], [3], 8, 2, d, seed=1)
    with b.plan() as plan:
        b.attend(plan)
        check(b, what="long")
        first = b.out.clone(), b.lse.clone()
        for _ in range(3):                  # the same bits every time
            b.attend(plan)
            assert bool((b.out == first[0]).all()) and bool((b.lse == first[1]).all())
    # whole prompts whose tiles are cut
    b = Batch([2500, 70], [2500, 70], 8, 2, d, seed=2)
    with b.plan() as plan:
        b.attend(plan)
    check(b, what="cut prompts")


@pytest.mark.parametrize("hq,hkv,d,full", [(64, 8, 64, False), (32, 8, 128, False), (16, 16, 64, True), (12, 4, 128, False)])
def test_many_items_a_cta(hq, hkv, d, full):
    # hundreds of short requests: every CTA walks a long list of short items, whole
    # tiles, half tiles and single rows mixed, again and again
    import random
    import shared_prefix_kv_fca_b200 as fca
    rng = random.Random(d + hq)
    new = [rng.choice([1, 2, 17, 18, 33, 56, 70]) for _ in range(300)]
    seq = [rng.choice([0, 1, 40, 130, 300]) if full else n + rng.choice([0, 9, 18, 120, 250]) for n in new]
    b = Batch(seq, new, hq, hkv, d, seed=d)
    with b.plan(full=full) as plan:
        for _ in range(20):
            b.attend(plan)
        assert fca.fca_chunk_check_status(plan) == 0
    check(b, full=full, what="many items")


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows_over_long_caches(d):
    # items of many stages, one after the other, whose last block is only partly filled: the
    # slots behind it are cleared while other stages are under way
    import random
    rng = random.Random(d)
    new = [rng.randint(2, 8) for _ in range(50)]
    b = Batch([n + rng.randint(1984, 3969) for n in new], new, 16, 16, d, seed=d)
    with b.plan() as plan:
        for _ in range(3):
            b.out.fill_(7.25)
            b.attend(plan)
            check(b, what="few rows, long caches")


@pytest.mark.parametrize("d", [64, 128])
def test_scores_far_apart(d):
    # maxima that jump by thousands in the log domain from one stage to the
    # next, upwards and downwards, and rows whose weight sits on one token
    torch = _torch()
    b = Batch([900], [200], 4, 1, d, seed=5)
    k = b.k.view(-1, 1, d)
    factor = torch.ones(900, device="cuda")
    factor[:128], factor[128:256], factor[256:384], factor[400], factor[890] = 0.01, 3.0, 40.0, 300.0, 900.0
    k[b.slot[0]] = (k[b.slot[0]].float() * factor[:, None, None]).bfloat16()
    with b.plan() as plan:
        b.attend(plan)
    check(b, what="far apart")


def test_what_a_row_does_not_see_has_no_part_in_it():
    torch = _torch()
    for d in (64, 128):
        b = Batch([333, 40], [40, 40], 4, 2, d, seed=6)
        k, v = (c.view(-1, 2, d) for c in (b.k, b.v))
        s = b.slot[0]
        v[s[310], 0, 3] = float("nan")      # seen by the last 23 rows only
        v[s[320], 1, 5] = float("inf")
        k[s[325], 1, :] = float("nan")
        k[s[325], 1, 0] = 0
        with b.plan() as plan:
            b.attend(plan)
        rows = torch.arange(40, device="cuda") + 293
        o = b.out[:40].float().view(40, 2, 2, d)
        bad = ~torch.isfinite(o)
        want = torch.zeros_like(bad)
        want[rows >= 310, 0, :, 3] = True
        want[rows >= 320, 1, :, 5] = True
        want[rows >= 325, 1] = True
        assert bool((bad == want).all()), d
        # everything else as if those tokens were not there
        v[s[310], 0, 3], v[s[320], 1, 5] = 0, 0
        k[s[325], 1, :] = 0
        ref = Batch([333, 40], [40, 40], 4, 2, d, seed=6)
        ref.k, ref.v, ref.out, ref.lse = b.k, b.v, b.out, b.lse
        o_ref, a, _, err, _ = reference(ref, 0, False)
        off = ((b.out[:40].double() - o_ref).abs() / ((2 ** -7 + 2 * err[..., None] + 2 ** -12) * a + 2 ** -8 * o_ref.abs()))
        early = torch.arange(40, device="cuda") < 17
        assert bool((off[early] <= 1).all())


def test_what_rows_do_not_see_behind_a_long_cache():
    # the last token's value is not finite: the rows before it are computed again, from all of a
    # long cache, of which a CTA has as much as 30000 tokens
    _torch()
    import shared_prefix_kv_fca_b200 as fca
    b = Batch([30000], [64], 592, 148, 64, seed=22)
    b.v.view(-1, 148, 64)[b.slot[0][-1], :, 50] = float("nan")
    with b.plan() as plan:
        b.attend(plan)
        assert fca.fca_chunk_check_status(plan) == 0
        check(b, what="one value at the end")


def test_what_a_row_does_see_stays_in_it():
    # inf and NaN in tokens that every row sees: out is not finite there, elsewhere as ever
    torch = _torch()
    b = Batch([5000, 300], [70, 300], 8, 2, 128, seed=7)
    v = b.v.view(-1, 2, 128)
    v[b.slot[0][17], 0, 3] = float("nan")
    v[b.slot[0][4000], 1, 9] = float("inf")
    with b.plan() as plan:
        b.attend(plan)
    o = b.out[:70].float().view(70, 2, 4, 128)
    bad = ~torch.isfinite(o)
    want = torch.zeros_like(bad)
    want[:, 0, :, 3] = True
    want[:, 1, :, 9] = True
    assert bool((bad == want).all())
    assert bool((o[:, 1, :, 9] == float("inf")).all())
    b.new_h[0] = 0
    check(b, what="the request beside")


def test_nothing_to_attend():
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    for rows in (0, 5):                     # no rows at all, and rows that belong to no request
        b = Batch([40, 0], [0, 0], 4, 1, 64, seed=1, pad_rows=rows)
        with b.plan() as plan:
            b.attend(plan)
            plan.update(b.tables, b.seq, b.starts)
            b.attend(plan)
            assert fca.fca_chunk_check_status(plan) == 0
        assert bool((b.out == 7.25).all()) and bool((b.lse == 7.25).all())


def test_as_many_requests_as_there_may_be():
    # 16384 requests: the sums' and the shared memory's full size
    import random
    import shared_prefix_kv_fca_b200 as fca
    rng = random.Random(2)
    had = [rng.choice([0, 15, 16, 31, 3]) for _ in range(16384)]
    new = [rng.choice([0, 1, 1, 2]) for _ in had]
    s, want = table_step(had, new, 4, seed=3, slots=sum(new) + 9)
    got = run_tables(s, had, new)
    for key in want:
        assert got[key] == want[key], key
    torch = _torch()
    b = Batch([max(h + n, 1) for h, n in zip(had, new)], new, 2, 1, 64, seed=4)
    with b.plan() as plan:
        b.attend(plan)
        assert fca.fca_chunk_check_status(plan) == 0
    # every row at once: at most 33 tokens, gathered into a rectangle
    lens = torch.tensor(b.seq_h, device="cuda")
    owner = torch.repeat_interleave(torch.arange(16384, device="cuda"), torch.tensor(new, device="cuda"))
    first = torch.tensor(b.starts_h[:-1], device="cuda")
    pos = lens[owner] - torch.tensor(new, device="cuda")[owner] + torch.arange(b.T, device="cuda") - first[owner]
    j = torch.arange(64, device="cuda")
    slot = b.tables.long()[owner][:, (j // BLOCK).clamp(max=b.tables.shape[1] - 1)] * BLOCK + j % BLOCK
    sees = j[None] <= pos[:, None]
    slot = torch.where(sees, slot, slot[:, :1])
    k, v = (c.view(-1, 64)[slot].double() for c in (b.k, b.v))
    w = torch.einsum("thd,tld->thl", b.q.double(), k) * b.scale
    w = torch.softmax(w.masked_fill(~sees[:, None], -math.inf), -1)
    ref, a = torch.einsum("thl,tld->thd", w, v), torch.einsum("thl,tld->thd", w, v.abs())
    off = (b.out.double() - ref).abs() / ((2.0 ** -7 + 2.0 ** -12) * a * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs())
    assert bool((off <= 1).all()), off.max().item()


def test_offsets_beyond_32_bits():
    torch = _torch()
    hkv, d = 8, 128
    pool = 2 ** 31 // (BLOCK * hkv * d) + 200         # more than 2^31 elements a cache
    b = Batch([300, 77], [300, 20], 8, hkv, d, seed=8, base=pool - 30, pool=pool)
    with b.plan() as plan:
        b.attend(plan)
    check(b, what="large cache")
    import shared_prefix_kv_fca_b200 as fca
    slots = torch.tensor([pool * BLOCK - 1, -1, 5], dtype=torch.int32, device="cuda")
    new = torch.randn(3, hkv, d, device="cuda").bfloat16()
    fca.fca_append_kv(new, new * 2, slots, b.k, b.v, pool)
    assert bool((b.k.view(-1, hkv, d)[-1] == new[0]).all()) and bool((b.v.view(-1, hkv, d)[5] == new[2] * 2).all())


def test_a_plan_updated_and_captured():
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    steps = [([200, 900, 3], [40, 1, 3]), ([201, 905, 0], [1, 5, 0]), ([240, 905, 64], [38, 0, 6])]
    b = [Batch(s, n, 8, 2, 128, seed=20 + i, pool=None) for i, (s, n) in enumerate(steps)]
    T, width, pool = 50, max(x.tables.shape[1] for x in b), max(x.pool for x in b)
    tables = torch.full((3, width), -7, dtype=torch.int32, device="cuda")
    seq, starts = torch.ones(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(pool, BLOCK, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(T, 8, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(T, 8, device="cuda")
    tables.fill_(0)
    plan = fca.fca_chunk_plan(tables, seq, starts, T, pool, 8, 2, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()

    def step():
        fca.fca_chunk_plan_update(plan, tables, seq, starts)
        fca.fca_chunk_attention(q, k, v, plan, out, lse)

    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
            step()
    torch.cuda.synchronize()
    for x in b + b[:1]:
        tables.fill_(-3)
        tables[:, :x.tables.shape[1]] = x.tables
        seq.copy_(x.seq)
        starts.copy_(x.starts)
        k.fill_(float("nan"))
        v.fill_(float("nan"))
        k[:x.pool], v[:x.pool] = x.k, x.v
        q[:x.T] = x.q
        out.fill_(7.25)
        lse.fill_(7.25)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert fca.fca_chunk_check_status(plan) == 0
        assert bool((out[x.T:] == 7.25).all()) and bool((lse[x.T:] == 7.25).all())
        x.out, x.lse = out[:x.T].clone(), lse[:x.T].clone()
        check(x, what="replayed")
    plan.close()


def test_a_captured_attention_runs_after_updates_outside_the_graph():
    # the plan has no cut tiles when the graph is made, and has some when it is replayed
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    b = Batch([9000, 40], [3, 2], 8, 2, 128, seed=21)
    short = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    with fca.fca_chunk_plan(b.tables, short, b.starts, b.T, b.pool, b.hq, b.hkv, b.d) as plan:
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.attend(plan)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side, capture_error_mode="thread_local"):
            b.attend(plan)
        plan.update(b.tables, b.seq, b.starts)
        b.out.fill_(7.25)
        b.lse.fill_(7.25)
        graph.replay()
        torch.cuda.synchronize()
        check(b, what="replayed")
        assert fca.fca_chunk_check_status(plan) == 0
        del graph


def test_bad_steps_are_refused_or_flagged():
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    b = Batch([40, 100], [4, 5], 4, 1, 64, seed=9)

    def status(**kw):
        a = dict(tables=b.tables, seq=b.seq, starts=b.starts)
        a.update(kw)
        with pytest.raises(fca.FcaError) as e:
            fca.fca_chunk_plan(a["tables"], a["seq"], a["starts"], b.T, b.pool, 4, 1, 64)
        return e.value.status

    def ints(*v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    worse = b.tables.clone()
    worse[1, 2] = b.pool
    assert status(tables=worse) == 2
    worse[1, 2] = -1
    assert status(tables=worse) == 2
    assert status(seq=ints(40, 4)) == 1                 # fewer tokens than rows
    assert status(seq=ints(40, 10 ** 6)) == 1
    assert status(seq=ints(-1, 100)) == 1
    assert status(starts=ints(0, 5, 4)) == 1
    assert status(starts=ints(1, 5, 9)) == 1
    assert status(starts=ints(0, 5, b.T + 1)) == 1
    # an update of a kept plan flags what building would refuse
    with b.plan() as plan:
        for kw, bit, zero in ((dict(tables=worse), 16, 1), (dict(seq=ints(3, 100)), 8, 0), (dict(starts=ints(0, 4, 99)), 8, None)):
            a = dict(tables=b.tables, seq=b.seq, starts=b.starts)
            a.update(kw)
            b.out.fill_(7.25)
            b.lse.fill_(7.25)
            plan.update(a["tables"], a["seq"], a["starts"])
            b.attend(plan)
            with pytest.raises(fca.FcaError) as e:
                fca.fca_chunk_check_status(plan)
            assert e.value.status == 6 and f"{bit:#x}" in str(e.value)
            if zero is None:
                assert bool((b.out == 7.25).all()) and bool((b.lse == 7.25).all())
                continue
            rows = slice(b.starts_h[zero], b.starts_h[zero + 1])
            assert bool((b.out[rows] == 0).all()) and bool((b.lse[rows] == -math.inf).all())
            other = Batch([40, 100], [4, 5], 4, 1, 64, seed=9)
            other.out, other.lse = b.out, b.lse
            other.new_h[zero] = 0           # the other request is served
            check(other, what="beside a refused one")
        plan.update(b.tables, b.seq, b.starts)
        b.attend(plan)
        assert fca.fca_chunk_check_status(plan) == 0
        check(b, what="after refusals")


# ------------------------------------------------------------------ tables

def table_step(had, new, width, seed=0, skip=3, spare=5, slots=None):
    """Inputs of one step and its outcome by the definition, on the host."""
    import random
    rng = random.Random(seed)
    held = [blocks(c) for c in had]
    grown = sum(blocks(c + n) - blocks(c) for c, n in zip(had, new))
    pool = sum(held) + grown + skip + spare
    ids = list(range(pool))
    rng.shuffle(ids)
    tables, at = [], 0
    for h in held:
        tables.append(ids[at:at + h] + [-9] * (width - h))
        at += h
    free = ids[at:]
    want = [list(t) for t in tables]
    nxt, starts, where = skip, [0], []
    for r, (c, n) in enumerate(zip(had, new)):
        for p in range(c, c + n):
            if p % BLOCK == 0:
                want[r][p // BLOCK] = free[nxt]
                nxt += 1
            where.append(want[r][p // BLOCK] * BLOCK + p % BLOCK)
        starts.append(len(where))
    total = len(where) if slots is None else slots
    where += [-1] * (total - len(where))
    return dict(tables=tables, free=free, skip=skip, pool=pool, slots=total), \
        dict(tables=want, seq=[c + n for c, n in zip(had, new)], starts=starts, slots=where, after=nxt)


def run_tables(s, had, new, in_place=False, status=None):
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca

    def ints(v, shape=None):
        t = torch.tensor(v, dtype=torch.int32, device="cuda")
        return t if shape is None else t.reshape(shape)

    tables = ints(s["tables"], (len(had), -1)) if had else torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    cached, fresh, free, nxt = ints(had), ints(new), ints(s["free"]), ints([s["skip"]])
    seq = cached if in_place else ints([-5] * len(had))
    starts, slots = ints([-5] * (len(had) + 1)), ints([-5] * s["slots"])
    after = None if in_place else ints([-5])
    fca.fca_extend_tables(tables, cached, fresh, free, nxt, s["pool"], seq, starts, slots, free_after=after, dev_status=status)
    got = dict(tables=tables.tolist(), seq=seq.tolist(), starts=starts.tolist(), slots=slots.tolist(),
               after=(nxt if in_place else after).item())
    if not in_place:
        assert cached.tolist() == had and nxt.item() == s["skip"]
    assert fresh.tolist() == new and free.tolist() == s["free"]
    return got


STEPS = {
    "none": ([], [], 0),
    "one": ([0], [1], 0),
    "inside": ([5], [3], 0),
    "page_end": ([15, 16, 17, 31, 32], [1, 1, 15, 2, 0], 0),
    "decode": (list(range(1, 300)), [1] * 299, 7),
    "nothing_new": ([3, 0, 40], [0, 0, 0], 4),
    "prompts": ([0] * 9, [1, 16, 17, 300, 0, 64, 2000, 5, 15], 0),
    "large": ([(7 * i) % 90 for i in range(1500)], [(13 * i) % 23 for i in range(1500)], 100),
    "long": ([10, 3], [40000, 9], 33),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", sorted(STEPS))
def test_tables_match_the_definition(name, in_place):
    torch = _torch()
    had, new, pad = STEPS[name]
    width = max([blocks(c + n) for c, n in zip(had, new)] + [1]) + 2
    s, want = table_step(had, new, width, seed=len(name), slots=sum(new) + pad)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_tables(s, had, new, in_place, status)
    for key in want:
        assert got[key] == want[key], key
    assert status.item() == 0


@pytest.mark.parametrize("large", [False, True])
def test_a_step_that_cannot_be_made_is_refused_whole(large):
    torch = _torch()
    n = 600 if large else 4
    had, new = [20] * n, [29] * n                   # two blocks each, the first token inside the last one
    width = 4
    for what, bit in (("negative", 8), ("cached", 8), ("long", 8), ("blocks", 64), ("slots", 128), ("free_id", 16),
                      ("free_id_high", 16), ("last_block", 16), ("next", 64)):
        h, m = list(had), list(new)
        s, _ = table_step(had, new, width, seed=1)
        if what == "negative":
            m[n // 2] = -1
        elif what == "cached":
            h[n - 1] = -4
        elif what == "long":
            m[1] = width * BLOCK - 19
            s["slots"] += 1000
        elif what == "blocks":
            s["free"] = s["free"][:s["skip"] + 2 * n - 1]
        elif what == "slots":
            s["slots"] -= 1
        elif what == "free_id":
            s["free"][s["skip"] + 2 * n - 1] = -1
        elif what == "free_id_high":
            s["free"][s["skip"]] = s["pool"]
        elif what == "last_block":
            s["tables"][n - 1][1] = s["pool"] + 5
        elif what == "next":
            s["skip"] = -1
        for in_place in (False, True):
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            got = run_tables(s, h, m, in_place, status)
            assert status.item() == bit, what
            assert got["tables"] == s["tables"] and got["seq"] == h and got["after"] == s["skip"], what
            assert set(got["starts"]) == {0} and set(got["slots"]) == {-1}, what
            run_tables(s, h, m)                     # without a status word


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("hkv,d", [(1, 64), (8, 128), (5, 64), (3, 128)])
@pytest.mark.parametrize("T", [1, 7, 500])
def test_append_writes_rows_to_their_slots(hkv, d, T):
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    g = torch.Generator(device="cuda").manual_seed(T)
    pool = 60
    qkv = torch.randn(T, 3 * hkv * d + 16, generator=g, device="cuda").bfloat16()
    k = qkv[:, 8:8 + hkv * d].view(T, hkv, d)
    v = qkv[:, 16 + hkv * d:16 + 2 * hkv * d].view(T, hkv, d)
    slots = torch.randperm(pool * BLOCK, generator=g, device="cuda")[:T].int()
    slots[T // 2] = -1 if T > 1 else slots[0]
    caches = [torch.randn(pool + 2, BLOCK, hkv, d, generator=g, device="cuda").bfloat16() for _ in range(2)]
    want = [c.clone() for c in caches]
    for c, x in zip(want, (k, v)):
        keep = slots >= 0
        c.view(-1, hkv, d)[slots[keep].long()] = x[keep]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fca.fca_append_kv(k, v, slots, *caches, pool, dev_status=status)
    assert all(bool((c == w).all()) for c, w in zip(caches, want)) and status.item() == 0
    # slots behind the cache are skipped and flagged
    slots[T - 1] = pool * BLOCK
    fca.fca_append_kv(k, v, slots, *caches, pool, dev_status=status)
    fca.fca_append_kv(k, v, slots, *caches, pool)
    assert all(bool((c == w).all()) for c, w in zip(caches, want)) and status.item() == 16
    fca.fca_append_kv(k[:0], v[:0], slots[:0], *caches, pool)


# ---------------------------------------------------------------- together

def test_a_serving_run():
    """Prompts taken in chunks beside decodes, then decoded: tables, slots,
    cache and outputs of every step against attention over the tokens' own
    keys and values, the last one also by fca_decode."""
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    hq, hkv, d, R, pool, width = 8, 2, 128, 5, 220, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    total = [700, 33, 400, 16, 1]
    chunks = [[300, 33, 0, 16, 0], [300, 0, 399, 0, 1], [100, 0, 1, 0, 0]] + [[1] * R] * 3
    keys = [[torch.randn(t + 4, hkv, d, generator=g, device="cuda").bfloat16() for t in total] for _ in range(2)]
    cap = max(sum(c) for c in chunks) + 5
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")      # noqa: E731
    tables, lens, fresh, nxt, starts, slots, status = z(R, width), z(R), z(R), z(1), z(R + 1), z(cap), z(1)
    free = torch.randperm(pool, generator=g, device="cuda").int()
    caches = [torch.full((pool, BLOCK, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plan, had = None, [0] * R
    for chunk in chunks:
        q = torch.randn(cap, hq, d, generator=g, device="cuda").bfloat16()
        new = [torch.zeros(cap, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        at = 0
        for r, n in enumerate(chunk):
            for x, own in zip(new, keys):
                x[at:at + n] = own[r][had[r]:had[r] + n]
            at += n
        fresh.copy_(torch.tensor(chunk, dtype=torch.int32))
        fca.fca_extend_tables(tables, lens, fresh, free, nxt, pool, lens, starts, slots, dev_status=status)
        fca.fca_append_kv(*new, slots, *caches, pool, dev_status=status)
        if plan is None:
            plan = fca.fca_chunk_plan(tables, lens, starts, cap, pool, hq, hkv, d)
        else:
            plan.update(tables, lens, starts)
        out = torch.full((cap, hq, d), 7.25, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((cap, hq), 7.25, device="cuda")
        fca.fca_chunk_attention(q, *caches, plan, out, lse)
        had = [h + n for h, n in zip(had, chunk)]
        assert status.item() == 0 and fca.fca_chunk_check_status(plan) == 0
        assert lens.tolist() == had and nxt.item() == sum(blocks(h) for h in had)
        b = Batch.__new__(Batch)
        b.seq_h, b.new_h, b.hq, b.hkv, b.d, b.scale = had, chunk, hq, hkv, d, 1 / math.sqrt(d)
        b.starts_h = starts.tolist()
        b.q, b.out, b.lse = q, out, lse
        b.k, b.v = (torch.cat([own[r][:had[r]] for r in range(R)]) for own in keys)
        edge = [0]
        for h in had:
            edge.append(edge[-1] + h)
        b.slot = [torch.arange(edge[r], edge[r + 1], device="cuda") for r in range(R)]
        check(b, what=f"chunk {chunk}")
    # the last step again by the decode of the same cache: each within its own
    # bound of the exact value, so within twice the bound of each other
    with fca.fca_plan(tables, lens, pool, hq, hkv, d) as dec:
        o2, l2 = torch.empty(R, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(R, hq, device="cuda")
        fca.fca_decode(q[:R].contiguous(), *caches, dec, o2, l2)
        b.out, b.lse = torch.cat([o2, out[R:]]), torch.cat([l2, lse[R:]])
        check(b, what="decode")
    plan.close()


def test_on_a_stream_of_ones_own():
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    side = torch.cuda.Stream()
    b = Batch([500, 60], [30, 60], 8, 2, 64, seed=30)
    torch.cuda.synchronize()
    plan = fca.fca_chunk_plan(b.tables, b.seq, b.starts, b.T, b.pool, 8, 2, 64, stream=side)
    plan.update(b.tables, b.seq, b.starts, stream=side)
    b.attend(plan, stream=side)
    assert fca.fca_chunk_check_status(plan, stream=side) == 0
    check(b, what="side stream")
    plan.close()


def test_two_plans_at_once():
    # plans have their own workspaces: attentions of two plans may overlap
    torch = _torch()
    b = [Batch([9000 + i], [2], 8, 2, 128, seed=40 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in b]
    plans = [x.plan() for x in b]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, p, s in zip(b, plans, streams):
            x.attend(p, stream=s)
    torch.cuda.synchronize()
    for x, p in zip(b, plans):
        check(x, what="two plans")
        p.close()


def test_attention_in_place_is_refused():
    torch = _torch()
    import shared_prefix_kv_fca_b200 as fca
    b = Batch([40, 17], [3, 17], 8, 2, 64, seed=23, packed=False)
    with b.plan() as plan:
        flat = torch.zeros(b.T * b.hq * b.d + 8, dtype=torch.bfloat16, device="cuda")
        for out in (b.q, flat[:-8].view(b.q.shape)):
            q = b.q if out is b.q else flat[8:].view(b.q.shape)
            before = q.clone()
            with pytest.raises(fca.FcaError, match="INVALID_ARG"):
                fca.fca_chunk_attention(q, b.k, b.v, plan, out, b.lse, b.scale)
            assert torch.equal(q, before)
        lse = flat[:b.T * b.hq * 2].view(torch.float32).view(b.T, b.hq)
        with pytest.raises(fca.FcaError, match="INVALID_ARG"):
            fca.fca_chunk_attention(b.q, b.k, b.v, plan, flat[:-8].view(b.q.shape), lse, b.scale)
        b.attend(plan)
        check(b, what="after refusals")
