"""fca_chunk_attention, on the GPU: an output is a weighted mean of the values that its row sees.

P V applies weights r_j that are rounded to bf16; the output is
sum_j r_j v_j / sum_j r_j.  Where all tokens have the same value c that is c, whatever the
weights: r_j c is exact in fp32 (two bf16 factors), and sums of n positive terms are off by
2 n 2^-23 of themselves at most, numerator and denominator together, even if every
addition truncates.  For n <= 4000 that is below 2^-9, and c in [1, 2) is a bf16 number whose
neighbours are at least 2^-8 c away: the rounded output has to be c itself.  Divided by the sum
of the weights before rounding it would be off by up to 2^-8 where few tokens carry a row.
"""
import pytest

from test_chunk_gpu import Batch

pytestmark = pytest.mark.gpu

HEADS = [(4, 1, 64), (6, 2, 128), (8, 2, 128), (16, 16, 64)]


@pytest.mark.parametrize("spread", [1, 4])      # of the scores: many tokens carry a row, or few
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("seq,new", [([900, 300, 129], [200, 300, 2]), ([4000], [3])], ids=["chunks", "cut"])
def test_equal_values_come_out_as_they_are(seq, new, heads, spread):
    import torch
    import shared_prefix_kv_fca_b200 as fca
    hq, hkv, d = heads
    b = Batch(seq, new, *heads, seed=11)
    g = torch.Generator(device="cuda").manual_seed(12)
    c = (1 + torch.randint(0, 128, (hkv, d), generator=g, device="cuda") / 128).bfloat16()
    for s in b.slot:
        b.v.view(-1, hkv, d)[s] = c
        b.k.view(-1, hkv, d)[s] *= spread
    with b.plan() as plan:
        b.attend(plan)
        assert fca.fca_chunk_check_status(plan) == 0
    assert torch.equal(b.out, c.repeat_interleave(hq // hkv, 0).expand(b.T, hq, d))
