"""The int4 and mixture-of-experts calls: what the C entries refuse before any device
work, and what the binding hands to them (CPU only)."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


class Recorder:
    """Stands for the library: keeps the arguments of the last call as the C side would
    see them, converted by the declared types."""

    def __init__(self, declared):
        self.declared, self.name, self.args = declared, None, None

    def __getattr__(self, name):
        def call(*args):
            assert len(args) == len(self.declared[name])
            self.name = name
            self.args = [t(a).value if t is ctypes.c_int64 else a for t, a in zip(self.declared[name], args)]
            return 0
        return call


@pytest.fixture
def recorder(q, monkeypatch):
    r = Recorder(q.EXPORTED)
    monkeypatch.setattr(q, "lib", r)
    monkeypatch.setattr(q, "_require", lambda t, what: None)
    monkeypatch.setattr(q, "_stream", lambda t: None)
    return r


@pytest.mark.parametrize("group_size", [96, 100, 4096, 2 ** 63 - 1, 2 ** 64 + 32, 2 ** 80])
def test_a_group_size_beyond_the_row_means_one_group(q, recorder, group_size):
    """Any value from K on is one group per row; what reaches the C call is in range and says so."""
    e, n, m, k = 3, 5, 2, 96
    w, s = torch.zeros((e, n, k // 2), dtype=torch.uint8), torch.ones((e, n, 1), dtype=torch.bfloat16)
    x = torch.zeros((m, k), dtype=torch.bfloat16)
    q.int4_gemm(w[0], s[0], x, group_size=group_size)
    assert recorder.name == "qlinear_int4_gemm" and recorder.args[9] == k
    q.int4_grouped_gemm(w, s, x, torch.zeros(e + 1, dtype=torch.int32), torch.zeros(e, dtype=torch.int32),
                        group_size=group_size)
    assert recorder.name == "qlinear_int4_grouped_gemm" and recorder.args[14] == k


@pytest.mark.parametrize("group_size", [32, 64])
def test_a_group_size_inside_the_row_is_passed_on(q, recorder, group_size):
    w, s = torch.zeros((5, 48), dtype=torch.uint8), torch.ones((5, -(-96 // group_size)), dtype=torch.bfloat16)
    q.int4_gemm(w, s, torch.zeros((2, 96), dtype=torch.bfloat16), group_size=group_size)
    assert recorder.args[9] == group_size


def test_int4_refusals(q):
    L = q.lib

    def dense(w=FAKE, s=FAKE, x=FAKE, out=FAKE, dt=0, m=2, n=8, k=64, g=32):
        return L.qlinear_int4_gemm(w, s, None, x, out, dt, m, n, k, g, 1.0, None, None)

    def grouped(w=FAKE, s=FAKE, x=FAKE, off=FAKE, ids=FAKE, out=FAKE, dt=0, g=3, most=2, e=3, t=2, n=8, k=64, size=32):
        return L.qlinear_int4_grouped_gemm(w, s, None, x, off, ids, out, dt, g, most, e, t, n, k, size, None)

    for kw in (dict(w=None), dict(s=None), dict(x=None), dict(out=None), dict(dt=2), dict(dt=7), dict(m=-1), dict(n=0),
               dict(k=0), dict(k=1 << 23, g=1 << 23), dict(g=0), dict(g=-32), dict(g=16), dict(g=48), dict(g=63),
               dict(s=ODD), dict(x=ODD), dict(out=ODD), dict(n=1 << 60)):
        assert dense(**kw) == q.ERR_INVALID_ARG, kw
    for kw in (dict(w=None), dict(off=None), dict(ids=None), dict(dt=2), dict(g=0), dict(g=65536), dict(most=-1), dict(e=0),
               dict(t=-1), dict(t=(1 << 30) + 1), dict(n=0), dict(k=0), dict(size=0), dict(size=16), dict(size=33),
               dict(off=ODD), dict(ids=ODD), dict(x=ODD), dict(e=1 << 60)):
        assert grouped(**kw) == q.ERR_INVALID_ARG, kw


def test_expert_call_refusals(q):
    L, bad = q.lib, q.ERR_INVALID_ARG
    need = ctypes.c_int64(-1)
    for t, e, k in ((-1, 8, 2), (4, 0, 1), (4, 1025, 2), (4, 8, 0), (4, 8, 9), (4, 100, 65), (1 << 31, 8, 1)):
        assert L.qlinear_moe_route(FAKE, 0, FAKE, FAKE, t, e, k, 1, None) == bad
        assert L.qlinear_moe_route_backward(FAKE, 0, FAKE, FAKE, FAKE, t, e, k, 1, None) == bad
    assert L.qlinear_moe_route(FAKE, 2, FAKE, FAKE, 4, 8, 2, 1, None) == bad
    assert L.qlinear_moe_route(ODD, 1, FAKE, FAKE, 4, 8, 2, 1, None) == bad
    for slots, e in ((-1, 8), (1 << 31, 8), (8, 0), (8, 1025)):
        assert L.qlinear_moe_sort_workspace_size(slots, e, ctypes.byref(need)) == bad and need.value == 0
        assert L.qlinear_moe_sort(FAKE, FAKE, FAKE, FAKE, slots, e, FAKE, 1 << 20, None) == bad
    assert L.qlinear_moe_sort_workspace_size(9000, 8, ctypes.byref(need)) == 0 and need.value > 0
    for ws, size in ((FAKE, need.value - 1), (None, 0), (None, need.value), (ODD, need.value)):
        assert L.qlinear_moe_sort(FAKE, FAKE, FAKE, FAKE, 9000, 8, ws, size, None) == bad
    for t, k, h in ((-1, 2, 8), (4, 0, 8), (4, 65, 8), (4, 2, 0), (1 << 30, 2, 8), (4, 2, 1 << 60)):
        assert L.qlinear_moe_gather(FAKE, FAKE, FAKE, 0, t, k, h, None) == bad
        assert L.qlinear_moe_combine(FAKE, 0, FAKE, None, FAKE, 0, t, k, h, None) == bad
        assert L.qlinear_moe_combine_backward(FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, t, k, h, None) == bad
    assert L.qlinear_moe_combine(FAKE, 0, FAKE, None, FAKE, 2, 4, 2, 8, None) == bad
    assert L.qlinear_moe_combine(FAKE, 1, FAKE, ODD, FAKE, 0, 4, 2, 8, None) == bad
    for m, f in ((-1, 8), (4, 0), (1 << 62, 8)):
        assert L.qlinear_swiglu(FAKE, FAKE, 0, m, f, None) == bad
        assert L.qlinear_swiglu_backward(FAKE, FAKE, FAKE, 0, m, f, None) == bad
    assert L.qlinear_swiglu(ODD, FAKE, 1, 4, 8, None) == bad
