"""Host-side checks of the calls for new tokens, without a GPU: the binding's
(through a stand-in library and CPU tensors that stand in for CUDA ones) and
the C entry points' own."""
import ctypes
import re
import os
import types

import pytest
import torch

import shared_prefix_kv_fca_b200 as fca
from shared_prefix_kv_fca_b200 import build as fbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
R, T, HQ, HKV, D, NB, MB = 3, 9, 8, 2, 64, 40, 6
BF = torch.bfloat16


class FakeLib:
    def __init__(self):
        self.calls, self.args = [], {}

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            self.args[name] = args
            if name == "fca_chunk_plan":
                args[12]._obj.value = 4321
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLib()
    monkeypatch.setattr(fca, "load_library", lambda: fake)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))
    return fake


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def tensors():
    qkv = torch.zeros(T, (HQ + 2 * HKV) * D, dtype=BF)
    return types.SimpleNamespace(
        q=qkv[:, :HQ * D].view(T, HQ, D), kn=qkv[:, HQ * D:(HQ + HKV) * D].view(T, HKV, D),
        vn=qkv[:, (HQ + HKV) * D:].view(T, HKV, D), k=torch.zeros(NB, 16, HKV, D, dtype=BF),
        v=torch.zeros(NB, 16, HKV, D, dtype=BF), out=torch.zeros(T, HQ, D, dtype=BF), lse=torch.zeros(T, HQ),
        bt=ints(R, MB), had=ints(R), new=ints(R), free=ints(NB), nxt=ints(1), seq=ints(R), starts=ints(R + 1),
        slots=ints(T), status=ints(1))


def extend(t):
    fca.fca_extend_tables(t.bt, t.had, t.new, t.free, t.nxt, NB, t.seq, t.starts, t.slots, dev_status=t.status, stream=0)


def append(t):
    fca.fca_append_kv(t.kn, t.vn, t.slots, t.k, t.v, NB, dev_status=t.status, stream=0)


def make_plan(t):
    return fca.fca_chunk_plan(t.bt, t.seq, t.starts, T, NB, HQ, HKV, D, stream=0)


def attend(t, plan):
    fca.fca_chunk_attention(t.q, t.k, t.v, plan, t.out, t.lse, 0.125, stream=0)


def test_valid_calls_pass_through(lib):
    t = tensors()
    extend(t)
    assert lib.args["fca_extend_tables"][13] == t.nxt.data_ptr()        # in place without free_after
    append(t)
    assert lib.args["fca_append_kv"][1] == lib.args["fca_append_kv"][3] == (HQ + 2 * HKV) * D
    plan = make_plan(t)
    attend(t, plan)
    assert lib.args["fca_chunk_attention"][1] == (HQ + 2 * HKV) * D
    plan.update(t.bt, t.seq, t.starts, stream=0)
    t.q, t.lse = t.q.contiguous(), None
    attend(t, plan)
    assert lib.args["fca_chunk_attention"][1] == HQ * D
    fca.fca_chunk_check_status(plan, stream=0)
    plan.close()
    assert lib.calls == ["fca_extend_tables", "fca_append_kv", "fca_chunk_plan", "fca_chunk_attention",
                         "fca_chunk_plan_update", "fca_chunk_attention", "fca_chunk_check_status",
                         "fca_chunk_plan_destroy"]


BAD = {
    "extend": [("bt", ints(R + 1, MB)), ("bt", ints(R * MB)), ("had", torch.zeros(R)),
               ("new", ints(R + 1)), ("seq", ints(2 * R)[::2]), ("starts", ints(R)), ("slots", ints(T, 1)),
               ("free", ints(1, NB)), ("nxt", ints(0)), ("status", torch.zeros(1))],
    "append": [("kn", torch.zeros(T, HKV * D, dtype=BF)), ("vn", torch.zeros(T + 1, HKV, D, dtype=BF)),
               ("vn", torch.zeros(T, HKV, D)), ("kn", torch.zeros(T, D, HKV, dtype=BF).transpose(1, 2)),
               ("kn", torch.zeros(T, HKV * D + 4, dtype=BF)[:, :HKV * D].view(T, HKV, D)),
               ("vn", torch.zeros(1, HKV, D, dtype=BF).expand(T, HKV, D)), ("slots", ints(T + 1)),
               ("k", torch.zeros(NB - 1, 16, HKV, D, dtype=BF)), ("v", torch.zeros(NB, 16, HKV + 1, D, dtype=BF)),
               ("k", torch.zeros(NB, 16, HKV, D)), ("status", ints(0))],
    "plan": [("bt", ints(R + 1, MB)), ("seq", ints(R + 1)), ("starts", ints(R)), ("starts", torch.zeros(R + 1)),
             ("bt", ints(R, 2 * MB)[:, ::2])],
    "attend": [("q", torch.zeros(T + 1, HQ, D, dtype=BF)), ("q", torch.zeros(T, HQ, D)),
               ("q", torch.zeros(T, HQ, D + 8, dtype=BF)[:, :, :D]), ("out", torch.zeros(T, 2 * HQ, D, dtype=BF)[:, ::2]),
               ("out", torch.zeros(T - 1, HQ, D, dtype=BF)), ("lse", torch.zeros(T, HQ + 1)),
               ("lse", torch.zeros(T, HQ, dtype=torch.float64)), ("k", torch.zeros(NB - 1, 16, HKV, D, dtype=BF)),
               ("v", torch.zeros(NB, 8, HKV, D, dtype=BF))],
}


@pytest.mark.parametrize("call,name,value", [(c, n, v) for c, l in BAD.items() for n, v in l],
                         ids=[f"{c}-{n}-{i}" for c, l in BAD.items() for i, (n, v) in enumerate(l)])
def test_tensors_that_do_not_fit_are_refused(lib, call, name, value):
    t = tensors()
    plan = make_plan(t)
    plan_calls = list(lib.calls)
    setattr(t, name, value)
    with pytest.raises(ValueError):
        {"extend": lambda: extend(t), "append": lambda: append(t), "attend": lambda: attend(t, plan),
         "plan": lambda: plan.update(t.bt, t.seq, t.starts, stream=0)}[call]()
    if call == "plan":
        with pytest.raises(ValueError):
            make_plan(t)
    assert lib.calls == plan_calls          # nothing reached the library
    plan.handle = None


class OnDevice:
    """A CPU tensor that reports itself as living on CUDA device `idx`."""

    def __init__(self, t, idx):
        self._t = t
        self.device = torch.device("cuda", idx)

    def __getattr__(self, name):
        return getattr(self._t, name)


def test_buffers_on_another_device_are_refused(lib):
    for call, names in ((extend, ["bt", "had", "free", "nxt", "seq", "slots", "status"]),
                        (append, ["kn", "vn", "slots", "k", "v", "status"])):
        for name in names:
            t = tensors()
            for n, x in vars(t).items():
                setattr(t, n, OnDevice(x, 1 if n == name else 0))
            with pytest.raises(ValueError, match="one device"):
                call(t)
    t = tensors()
    plan = make_plan(t)
    plan.device = 1
    for name in ("q", "k", "v", "out", "lse"):
        t = tensors()
        for n, x in vars(t).items():
            setattr(t, n, OnDevice(x, 0))
        with pytest.raises(ValueError, match="plan belongs to cuda:1"):
            attend(t, plan)
        setattr(t, name, OnDevice(getattr(t, name)._t, 1))
        with pytest.raises(ValueError, match="one device"):
            attend(t, plan)
    assert lib.calls == ["fca_chunk_plan"]
    plan.handle = None


def test_the_flag_is_the_headers():
    src = open(os.path.join(ROOT, "include", "fca.h")).read()
    assert int(re.search(r"#define\s+FCA_CHUNK_FULL\s+(\d+)u", src).group(1)) == fca.FCA_CHUNK_FULL


def test_entry_points_check_before_the_device():
    fbuild.build()
    lib = fca.load_library()
    p, q, n = 1 << 20, 1 << 24, None        # never dereferenced
    #                      bt mb had new R free nf next NB seq starts slots ns after status stream
    good = [p, 4, p, p, 2, p, 8, p, 8, q, p, p, 5, q, n, n]
    for at, v in ((0, n), (1, 0), (2, n), (3, n), (4, -1), (5, n), (6, -1), (7, n), (8, 0), (9, n), (10, n), (11, n),
                  (12, -1), (13, n), (0, p + 2), (9, p + 4), (11, p + 1), (14, p + 3)):
        a = list(good)
        a[at] = v
        assert lib.fca_extend_tables(*a) == 1, (at, v)
    for at, v in ((4, 16385), (8, 1 << 27), (1, 1 << 27), (12, (1 << 30) + 1)):
        a = list(good)
        a[at] = v
        assert lib.fca_extend_tables(*a) == 3, (at, v)
    #       k stride v stride slots T NB Hkv D kc vc status stream
    good = [p, 128, p, 128, p, 3, 8, 2, 64, q, q, n, n]
    for at, v in ((0, n), (1, 127), (1, 120), (3, 132), (2, n), (4, n), (5, -1), (6, 0), (7, 0), (9, n), (10, n), (0, p + 8),
                  (9, q + 4), (4, p + 2), (11, p + 2)):
        a = list(good)
        a[at] = v
        assert lib.fca_append_kv(*a) == 1, (at, v)
    for at, v in ((8, 96), (6, 1 << 27)):
        a = list(good)
        a[at] = v
        assert lib.fca_append_kv(*a) == 3, (at, v)
    a = list(good)
    a[5] = 0
    assert lib.fca_append_kv(*a) == 0       # no rows: nothing to do
    h = ctypes.c_void_p()
    #       bt mb seq starts R T block NB Hq Hkv D flags out stream
    good = [p, 4, p, p, 2, 5, 16, 8, 4, 1, 64, 0, ctypes.byref(h), n]
    for at, v in ((0, n), (1, 0), (2, n), (3, n), (4, 0), (5, -1), (7, 0), (8, 0), (9, 0), (9, 3), (11, 2), (12, n), (0, p + 1)):
        a = list(good)
        a[at] = v
        assert lib.fca_chunk_plan(*a) == 1, (at, v)
    for at, v in ((6, 32), (10, 96), (8, 17), (4, 16385), (1, (1 << 20) + 1), (7, 1 << 27)):
        a = list(good)
        a[at] = v
        assert lib.fca_chunk_plan(*a) == 3, (at, v)
    assert h.value is None
    assert lib.fca_chunk_plan_update(n, p, 4, p, p, 2, n) == 1
    assert lib.fca_chunk_attention(p, 64, p, p, n, p, n, 0.1, n) == 1
    assert lib.fca_chunk_check_status(n, n, None) == 1
    assert lib.fca_chunk_plan_destroy(n) == 0


def test_outputs_that_overlap_other_buffers_are_refused():
    fbuild.build()
    lib = fca.load_library()
    at = [None] + [i << 16 for i in range(1, 11)]       # never dereferenced
    #      bt     mb cached new   R  free  nf  next  NB  seq    starts slots  ns after  status stream
    good = [at[1], 4, at[2], at[3], 5, at[4], 8, at[5], 8, at[6], at[7], at[8], 9, at[9], at[10], None]
    sizes = {0: 20, 2: 5, 3: 5, 5: 8, 7: 1, 9: 5, 10: 6, 11: 9, 13: 1, 14: 1}
    outputs = (0, 9, 10, 11, 13, 14)
    for x in outputs:
        for y in sizes:
            if x == y:
                continue
            a = list(good)
            a[x] = a[y] + 4 * (sizes[y] - 1)            # on the other's last element
            if a[x] == a[y] and (x, y) == (13, 7):
                continue                                # the list position may be updated in place
            assert lib.fca_extend_tables(*a) == 1, (x, y)


def test_caches_that_overlap_rows_are_refused():
    fbuild.build()
    lib = fca.load_library()
    k, v, slots, kc, vc = (i << 24 for i in range(1, 6))
    #       k  stride v  stride slots T NB Hkv D kc vc status stream; a cache has 8 * 16 * 256 bytes
    good = [k, 384, v, 384, slots, 3, 8, 2, 64, kc, vc, None, None]
    for at, where in ((10, kc), (10, kc + 32752), (9, k + 1536 + 240), (10, k), (9, v + 16), (10, slots), (9, slots - 32752)):
        a = list(good)
        a[at] = where
        assert lib.fca_append_kv(*a) == 1, (at, where)
