"""fca_chunk_attention, on the GPU: rows that are computed again over a cache of 1.6 million tokens.

Every request's table repeats a few blocks and ends in one of its own, so 1.6 million tokens
take no memory; the last token of one request has a value that is not finite.  The rows before
it do not see that token and are computed again from all the others, one request to an SM,
which takes two seconds, twice as long as any wait in the kernel may last.

Tolerance (as for any output): weights rounded to 2^-8 on either side of the division, scores
off by err, sums of n terms by n 2^-23 of themselves, the output rounded by 2^-8:
(2^-7 + 2 err + 2^-19 + n 2^-23) A + 2^-8 (|o| + all that), A = sum_j w_j |v_j|.  n 2^-23 is 0.19 here, so
the values lie in [1, 2) and their mean is known to that; what the rows see is told apart by
a value of 1000 in the own block's tokens, whose weight is raised to be a half.
"""
import math

import pytest

pytestmark = pytest.mark.gpu


def test_rows_computed_again_take_as_long_as_they_need():
    import torch
    import shared_prefix_kv_fca_b200 as fca
    R = torch.cuda.get_device_properties(0).multi_processor_count
    L, n, G, D, common = 1_600_000, 16, 16, 128, 64
    g = torch.Generator(device="cuda").manual_seed(31)
    pool, width = common + R, L // 16
    k = torch.randn(pool, 16, 1, D, generator=g, device="cuda").bfloat16()
    v = (1 + torch.rand(pool, 16, 1, D, generator=g, device="cuda")).bfloat16()
    tables = torch.randint(0, common, (R, width), generator=g, device="cuda", dtype=torch.int32)
    tables[:, -1] = common + torch.arange(R, device="cuda", dtype=torch.int32)
    q = torch.randn(R * n, G, D, generator=g, device="cuda").bfloat16()
    # token 0 of each own block: its key is along one direction that all queries have, its value is 1000
    q[:, :, 0] = 8
    k[:, :, :, 0] = 0
    k[common:, 0, 0, :] = 0
    k[common:, 0, 0, 0] = math.log(L) * math.sqrt(D) / 8        # score log(L), about what the others come to together
    v[common:, 0] = 1000
    v[common + 3, 15, 0, 7] = float("nan")
    out = torch.full((R * n, G, D), 7.25, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((R * n, G), 7.25, device="cuda")
    seq = torch.full((R,), L, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, R * n + 1, n, device="cuda", dtype=torch.int32)
    with fca.fca_chunk_plan(tables, seq, starts, R * n, pool, G, 1, D) as plan:
        fca.fca_chunk_attention(q, k, v, plan, out, lse)
        assert fca.fca_chunk_check_status(plan) == 0
    scale = 1 / math.sqrt(D)
    for r in (0, 3, R - 1):
        count = torch.bincount(tables[r, :-1].long(), minlength=common).double()
        sees = torch.arange(16, device="cuda")[None] <= torch.arange(n, device="cuda")[:, None]
        often = torch.cat([count.repeat_interleave(16).expand(n, -1), sees.double()], 1)        # [n, tokens that differ]
        kk, vv = (torch.cat([c[:common], c[common + r][None]]).view(-1, D).double() for c in (k, v))
        vv = vv.nan_to_num(0)
        qq = q[r * n:(r + 1) * n].double()
        s = torch.einsum("thd,ld->thl", qq, kk) * scale + often.log()[:, None]
        ref = torch.logsumexp(s, -1)
        w = (s - ref[..., None]).exp()
        o = torch.einsum("thl,ld->thd", w, vv)
        err = torch.einsum("thd,ld->thl", qq.abs(), kk.abs()).amax(-1) * scale * D * 2.0 ** -23
        tol = (2.0 ** -7 + 2 * err[..., None] + 2.0 ** -19 + L * 2.0 ** -23) * o         # all values are positive
        tol = tol + 2.0 ** -8 * (o + tol)
        got = out[r * n:(r + 1) * n].double()
        if r == 3:
            assert bool(got[15, :, 7].isnan().all())
            got[15, :, 7] = o[15, :, 7]
        assert bool(((got - o).abs() <= tol).all()), r
        off = (lse[r * n:(r + 1) * n].double() - ref).abs() - (err + 2.0 ** -20 + L * 2.0 ** -24 + 2.0 ** -23 * ref.abs())
        assert bool((off <= 0).all()), r
