"""What can only be read off the chunk attention's source: how its warps wait.

A bounded wait may answer lanes of a warp differently (it is given up just as the phase
completes).  The warps of the tiles and of the products vote, load and store tensor memory
as whole warps, so a lane that left alone would keep the others in such a step without a
limit: every wait of theirs has to be one of the whole warp.  That happens in the moment of a
failure only, which no test brings about.
"""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def kernel():
    src = open(os.path.join(ROOT, "shared_prefix_kv_fca_b200", "csrc", "fca_chunk.cu")).read()
    return src, src[src.index("    k_chunk(const __grid_constant__"):src.index("k_chunk_merge(")]


def test_warps_that_act_as_one_wait_as_one():
    src, body = kernel()
    assert re.search(r"bool warp_wait\([^)]*\) \{\s*return __all_sync\(0xffffffffu, dev::mbar_wait\(", src)
    tile = body[body.index("a tile's warpgroup"):body.index("regs_dec<kRegsOthers>")]
    products = body[body.index("MMA issue"):body.index("every MMA of this warp has retired")]
    for part in (tile, products):
        assert "warp_wait(" in part and "dev::mbar_wait(" not in part and "mbar_try_wait" not in part


def test_waits_of_one_lane_are_shared_with_its_warp():
    # the loading warps: lane 0 waits, and all lanes take its answer before they go on
    _, body = kernel()
    loads = body[body.index("TMA loads"):body.index("never leave with copies in flight")]
    waits = [m.start() for m in re.finditer(r"dev::mbar_wait\(", loads)]
    shared = [m.start() for m in re.finditer(r"ok = __shfl_sync\(0xffffffffu, ok, 0\);", loads)]
    assert len(waits) == len(shared) == 2
    for w, s in zip(waits, shared):
        assert w < s and "if (lane == 0)" in loads[w - 200:w] and "break" not in loads[w:s] and "return" not in loads[w:s]
