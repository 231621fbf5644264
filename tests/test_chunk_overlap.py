"""Which buffers fca_chunk_attention may be given, without a GPU: addresses that are never read,
and a plan that holds nothing but its sizes.  What passes the checks ends at the missing device
(FCA_ERR_CUDA), so the tests run where there is none."""
import ctypes

import pytest
import torch

import shared_prefix_kv_fca_b200 as fca
from shared_prefix_kv_fca_b200 import build as fbuild

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the stand-in plan must not be launched")

T, HQ, HKV, D, NB, STRIDE = 5, 8, 2, 64, 12, 8 * 64 + 16
REFUSED, NO_DEVICE = 1, 4
UNIT = 1 << 20
SIZES = {"q": ((T - 1) * STRIDE + HQ * D) * 2, "k": NB * 16 * HKV * D * 2, "v": NB * 16 * HKV * D * 2,
         "out": T * HQ * D * 2, "lse": T * HQ * 4}


def attend(**at):
    """The call's status, buffers a megabyte apart where `at` does not say otherwise."""
    fbuild.build()
    plan = (ctypes.c_int32 * 1024)()
    plan[1], plan[2], plan[3], plan[4] = 1, T, 4, NB            # device, then R, T, max_blocks, num_blocks,
    plan[5], plan[6], plan[7], plan[8] = HQ, HKV, D, HQ // HKV  # Hq, Hkv, D, G
    a = {n: UNIT * (i + 1) for i, n in enumerate(SIZES)}
    a.update(at)
    return fca.load_library().fca_chunk_attention(a["q"], STRIDE, a["k"], a["v"], ctypes.addressof(plan), a["out"], a["lse"],
                                                  0.125, None)


def test_buffers_of_their_own_pass():
    assert attend() == NO_DEVICE
    assert attend(lse=None) == NO_DEVICE
    # read alone: queries and caches may share memory
    assert attend(k=UNIT, v=UNIT) == attend(v=2 * UNIT) == NO_DEVICE


@pytest.mark.parametrize("same", [(), ("q", "k"), ("q", "v"), ("k", "v"), ("q", "k", "v")], ids="-".join)
@pytest.mark.parametrize("output", ["out", "lse"])
def test_an_output_beside_a_buffer_passes_and_inside_is_refused(output, same):
    for name in ("q", "k", "v"):
        base = {n: 16 * UNIT for n in same}                     # inputs that start at one address
        start = 16 * UNIT if name in same else UNIT * (1 + list(SIZES).index(name))
        end = start + max([SIZES[n] for n in same] if name in same else [SIZES[name]])
        for where, status in ((start - SIZES[output], NO_DEVICE), (start - SIZES[output] + 16, REFUSED), (start, REFUSED),
                              (end - 16, REFUSED), (end, NO_DEVICE)):
            assert attend(**base, **{output: where}) == status, (name, where - start)


def test_outputs_may_touch_but_not_overlap():
    out = UNIT * 8
    assert attend(out=out, lse=out + SIZES["out"]) == attend(out=out, lse=out - SIZES["lse"]) == NO_DEVICE
    assert attend(out=out, lse=out + SIZES["out"] - 4) == attend(out=out, lse=out - SIZES["lse"] + 4) == REFUSED
