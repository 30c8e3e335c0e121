"""The gated product, the adapters and the block norm: what the C entries refuse before any device work,
and what the binding refuses and hands to them (CPU only)."""

import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced: every call below fails validation first
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def q():
    import weight_quantized_linear_amd as q
    return q


def test_gated_refusals(q):
    L = q.lib

    def gated(w=FAKE, fmt=2, x=FAKE, c=None, cd=0, out=FAKE, od=0, pre=None, pd=0, m=2, f=8, k=64, act=2):
        return L.qlinear_gated_gemm(w, fmt, x, c, cd, out, od, pre, pd, m, f, k, 1.0, 1.0, act, None)

    def back(dy=FAKE, dd=0, pre=FAKE, pd=0, dpre=FAKE, m=2, f=8, act=2):
        return L.qlinear_gated_backward(dy, dd, pre, pd, dpre, m, f, act, None)

    for kw in (dict(w=None), dict(x=None), dict(out=None), dict(fmt=1), dict(fmt=3), dict(fmt=-1), dict(od=2), dict(c=FAKE, cd=2),
               dict(pre=FAKE, pd=5), dict(m=-1), dict(f=0), dict(k=0), dict(act=0), dict(act=4), dict(w=ODD), dict(x=ODD),
               dict(out=TWO), dict(od=1, out=ODD), dict(c=TWO), dict(pre=TWO), dict(f=1 << 60), dict(m=1 << 60)):
        assert gated(**kw) == q.ERR_INVALID_ARG, kw
    for kw in (dict(dy=None), dict(pre=None), dict(dpre=None), dict(dd=2), dict(pd=2), dict(m=-1), dict(f=0), dict(act=0),
               dict(act=4), dict(dy=TWO), dict(pre=TWO), dict(dpre=ODD), dict(m=1 << 60)):
        assert back(**kw) == q.ERR_INVALID_ARG, kw
    for call in (L.qlinear_bf16_gemm_grad_x, L.qlinear_bf16_gemm_grad_w):
        for args in ((None, FAKE, FAKE, 0, 2, 8, 4), (FAKE, None, FAKE, 0, 2, 8, 4), (FAKE, FAKE, None, 0, 2, 8, 4),
                     (FAKE, FAKE, FAKE, 2, 2, 8, 4), (FAKE, FAKE, FAKE, 0, -1, 8, 4), (FAKE, FAKE, FAKE, 0, 2, 0, 4),
                     (FAKE, FAKE, FAKE, 0, 2, 8, 0), (ODD, FAKE, FAKE, 0, 2, 8, 4), (FAKE, FAKE, TWO, 0, 2, 8, 4),
                     (FAKE, FAKE, FAKE, 0, 1 << 40, 1 << 40, 4)):
            assert call(*args, None, 0, None) == q.ERR_INVALID_ARG, args
        for ws, size in ((None, 16), (FAKE, -1), (TWO, 64)):
            assert call(FAKE, FAKE, FAKE, 0, 2, 8, 4, ws, size, None) == q.ERR_INVALID_ARG
    need = ctypes.c_int64(-1)
    for m, n, k in ((-1, 8, 4), (2, 0, 4), (2, 8, 0), (1 << 40, 1 << 40, 4)):
        assert L.qlinear_bf16_gemm_grad_workspace_size(m, n, k, ctypes.byref(need), None) == q.ERR_INVALID_ARG
    assert L.qlinear_bf16_gemm_grad_workspace_size(2, 8, 4, None, None) == q.ERR_INVALID_ARG


def test_lora_refusals(q):
    L, need = q.lib, ctypes.c_int64(-1)
    assert L.qlinear_lora_workspace_size(2, 30, 64, 8, ctypes.byref(need)) == 0 and need.value >= 30 * 8 * 4
    size = need.value

    def fwd(x=FAKE, a=FAKE, b=FAKE, off=FAKE, ids=FAKE, s=None, base=None, out=FAKE, od=0, z=None, g=2, l=3, t=30, n=16, k=64,
            r=8, ws=FAKE, wb=size):
        return L.qlinear_lora_gemm(x, a, b, off, ids, s, base, out, od, z, g, l, t, n, k, r, ws, wb, None)

    sizes = (dict(g=0), dict(g=4097), dict(l=0), dict(l=4097), dict(t=-1), dict(t=(1 << 30) + 1), dict(n=0), dict(n=(1 << 20) + 1),
             dict(k=0), dict(k=(1 << 20) + 1), dict(r=0), dict(r=257))
    for kw in (dict(x=None), dict(a=None), dict(b=None), dict(off=None), dict(ids=None), dict(out=None), dict(od=2), dict(x=ODD),
               dict(a=ODD), dict(b=ODD), dict(off=TWO), dict(ids=TWO), dict(s=TWO), dict(base=TWO), dict(out=TWO),
               dict(z=ctypes.c_void_p(0x10004)), dict(wb=size - 1), dict(ws=None, wb=0), dict(ws=None), dict(ws=TWO), *sizes):
        assert fwd(**kw) == q.ERR_INVALID_ARG, kw
    assert L.qlinear_lora_workspace_size(2, 30, 64, 8, None) == q.ERR_INVALID_ARG
    assert L.qlinear_lora_workspace_size(0, 30, 64, 8, ctypes.byref(need)) == q.ERR_INVALID_ARG and need.value == 0
    assert L.qlinear_lora_backward_workspace_size(2, 3, 30, 16, 64, 8, ctypes.byref(need)) == 0 and need.value > 0
    back_size = need.value

    def back(dy=FAKE, x=FAKE, z=FAKE, a=FAKE, b=FAKE, off=FAKE, ids=FAKE, s=None, base=None, dx=FAKE, xd=0, da=FAKE, db=FAKE,
             pd=0, g=2, l=3, t=30, n=16, k=64, r=8, ws=FAKE, wb=back_size):
        return L.qlinear_lora_gemm_backward(dy, x, z, a, b, off, ids, s, base, dx, xd, da, db, pd, g, l, t, n, k, r, ws, wb, None)

    for kw in (dict(dy=None), dict(x=None), dict(z=None), dict(a=None), dict(b=None), dict(off=None), dict(ids=None), dict(dx=None),
               dict(da=None), dict(db=None), dict(xd=2), dict(pd=2), dict(dy=ODD), dict(z=TWO), dict(dx=TWO), dict(da=TWO),
               dict(db=TWO), dict(base=TWO), dict(wb=back_size - 1), dict(ws=None, wb=0), dict(ws=TWO), *sizes):
        assert back(**kw) == q.ERR_INVALID_ARG, kw


def test_norm_refusals(q):
    L, need = q.lib, ctypes.c_int64(-1)

    def fwd(res=FAKE, rd=0, w=FAKE, pd=0, block=FAKE, d=0, wo=FAKE, gate=FAKE, gates=2, r2=FAKE, out=FAKE, t=4, h=64, eps=1e-6):
        return L.qlinear_block_norm(res, rd, w, pd, block, d, wo, gate, gates, r2, out, t, h, 1.0, eps, None)

    both = (dict(rd=2), dict(pd=2), dict(d=2), dict(rd=1, d=0), dict(gates=0), dict(gates=3), dict(gates=-1), dict(gate=None),
            dict(t=-1), dict(h=0), dict(h=16385), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(t=1 << 60))
    for kw in (dict(res=None), dict(w=None), dict(out=None), dict(block=None), dict(r2=None), dict(block=None, r2=None),
               dict(block=None, r2=None, wo=None), dict(res=TWO), dict(w=TWO), dict(block=TWO), dict(wo=TWO), dict(gate=TWO),
               dict(r2=TWO), dict(out=TWO), *both):
        assert fwd(**kw) == q.ERR_INVALID_ARG, kw
    assert L.qlinear_block_norm_backward_workspace_size(4, 64, 1, 1, ctypes.byref(need)) == 0 and need.value > 0
    size = need.value

    def back(dy=FAKE, d=0, dr=None, r2=FAKE, rd=0, w=FAKE, pd=0, block=FAKE, wo=FAKE, gate=FAKE, gates=2, dres=FAKE, db=FAKE,
             dw=FAKE, dwo=FAKE, dg=FAKE, t=4, h=64, eps=1e-6, ws=FAKE, wb=size):
        return L.qlinear_block_norm_backward(dy, d, dr, r2, rd, w, pd, block, wo, gate, gates, dres, db, dw, dwo, dg, t, h, 1.0,
                                             eps, ws, wb, None)

    for kw in (dict(dy=None), dict(r2=None), dict(w=None), dict(dres=None), dict(dw=None), dict(db=None), dict(dwo=None),
               dict(dg=None), dict(block=None), dict(wo=None), dict(dr=TWO), dict(dres=TWO), dict(dg=TWO), dict(wb=size - 1),
               dict(ws=None, wb=0), dict(ws=TWO), *both):
        assert back(**kw) == q.ERR_INVALID_ARG, kw
    for t, h in ((-1, 8), (4, 0), (4, 16385)):
        assert L.qlinear_block_norm_backward_workspace_size(t, h, 1, 1, ctypes.byref(need)) == q.ERR_INVALID_ARG
    assert L.qlinear_block_norm_backward_workspace_size(0, 8, 1, 1, ctypes.byref(need)) == 0 and need.value == 0


class Recorder:
    """Stands for the library: keeps the last call's arguments."""

    def __init__(self, lib):
        self.lib, self.name, self.args = lib, None, None

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return getattr(self.lib, name)

        def call(*args):
            self.name, self.args = name, args
            return 0
        return call


@pytest.fixture
def recorder(q, monkeypatch):
    r = Recorder(q.lib)
    monkeypatch.setattr(q, "lib", r)
    monkeypatch.setattr(q, "_require", lambda t, what: None)
    monkeypatch.setattr(q, "_stream", lambda t: None)
    return r


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_what_the_binding_passes(q, recorder):
    q.gated_gemm(bf(16, 32), bf(3, 32), alpha=2.0, activation="gelu_tanh", addend=torch.zeros(3, 16))
    assert recorder.name == "qlinear_gated_gemm" and recorder.args[1] == q.WEIGHT_BF16 and recorder.args[4] == q.F32
    assert recorder.args[9:16] == (3, 8, 32, 2.0, 2.0, 3, None)
    q.gated_gemm(torch.zeros((16, 32), dtype=torch.uint8), bf(3, 32), alpha=2.0, alpha_up=0.5)
    assert recorder.args[1] == q.WEIGHT_FP8 and recorder.args[12:15] == (2.0, 0.5, 2)
    off, ids = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    q.lora_gemm(bf(5, 32), bf(4, 8, 32), bf(4, 24, 8), off, ids)
    assert recorder.name == "qlinear_lora_gemm" and recorder.args[10:16] == (2, 4, 5, 24, 32, 8)
    q.block_norm(bf(6, 32), bf(32), block=bf(6, 32), gate=bf(3, 32))
    assert recorder.name == "qlinear_block_norm" and recorder.args[8] == 3 and recorder.args[11:13] == (6, 32)
    q.block_norm(bf(6, 32), bf(32), block=bf(6, 32), gate=bf(32))
    assert recorder.args[8] == 1
    y, r = q.block_norm(res := bf(6, 32), bf(32))
    assert recorder.args[4] is None and recorder.args[9] is None and r is res


def test_what_the_binding_refuses(q, recorder):
    off, ids = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x, a, b = bf(5, 32), bf(4, 8, 32), bf(4, 24, 8)
    meta = torch.zeros((5, 32), dtype=torch.bfloat16, device="meta")
    wrong = [
        lambda: q.gated_gemm(bf(15, 32), bf(3, 32)),
        lambda: q.gated_gemm(bf(16, 32), bf(3, 31)),
        lambda: q.gated_gemm(bf(16, 32), torch.zeros(3, 32)),
        lambda: q.gated_gemm(torch.zeros(16, 32), bf(3, 32)),
        lambda: q.gated_gemm(bf(16, 32), bf(3, 32), activation="none"),
        lambda: q.gated_gemm(bf(16, 32), bf(3, 32), out_dtype=torch.float16),
        lambda: q.gated_gemm(bf(16, 32), bf(3, 32), addend=bf(3, 8)),
        lambda: q.gated_gemm(bf(16, 32), bf(3, 32), return_pre=True, pre_dtype=torch.float16),
        lambda: q.gated_gemm(bf(16, 32), meta[:3]),
        lambda: q.gated_gemm_backward(bf(3, 8), bf(3, 8), bf(16, 32), bf(3, 32)),
        lambda: q.gated_gemm_backward(bf(3, 8), bf(3, 16), torch.zeros((16, 32), dtype=torch.uint8), bf(3, 32)),
        lambda: q.bf16_gemm_grad_x(bf(3, 8), bf(9, 4)),
        lambda: q.bf16_gemm_grad_w(bf(3, 8), bf(4, 8)),
        lambda: q.lora_gemm(x, a, bf(4, 24, 7), off, ids),
        lambda: q.lora_gemm(x, a, bf(3, 24, 8), off, ids),
        lambda: q.lora_gemm(bf(5, 31), a, b, off, ids),
        lambda: q.lora_gemm(x, a, b, off[:2], ids),
        lambda: q.lora_gemm(x, a, b, off.long(), ids),
        lambda: q.lora_gemm(x, a, b, off, ids.long()),
        lambda: q.lora_gemm(x, a, b, off, ids, scale=torch.ones(3)),
        lambda: q.lora_gemm(x, a, b, off, ids, scale=bf(4)),
        lambda: q.lora_gemm(x, a, b, off, ids, base=torch.zeros(5, 24)),
        lambda: q.lora_gemm(x, a, b, off, ids, out_dtype=torch.int32),
        lambda: q.lora_gemm(meta, a, b, off, ids),
        lambda: q.lora_gemm_backward(bf(5, 23), x, torch.zeros(5, 8), a, b, off, ids),
        lambda: q.lora_gemm_backward(bf(5, 24), x, bf(5, 8), a, b, off, ids),
        lambda: q.lora_gemm_backward(bf(5, 24), x, torch.zeros(5, 8), a, b, off, ids, base=torch.zeros(5, 32)),
        lambda: q.block_norm(bf(6, 32), bf(31)),
        lambda: q.block_norm(bf(6, 32), bf(32), gate=bf(1, 32)),
        lambda: q.block_norm(bf(6, 32), bf(32), block_weight=bf(32)),
        lambda: q.block_norm(bf(6, 32), bf(32), block=bf(6, 32), gate=bf(4, 32)),
        lambda: q.block_norm(bf(6, 32), bf(32), block=bf(6, 32), gate=torch.zeros(1, 32)),
        lambda: q.block_norm(bf(6, 32), bf(32), block=bf(6, 32), block_weight=torch.zeros(32)),
        lambda: q.block_norm(bf(6, 32), bf(32), residual_out=bf(6, 32)),
        lambda: q.block_norm(bf(6, 32), bf(32), block=bf(6, 32), out_dtype=torch.float32),
        lambda: q.block_norm_backward(torch.zeros(6, 32), None, torch.zeros(6, 32), bf(32), block=bf(6, 32)),
        lambda: q.block_norm_backward(bf(6, 32), torch.zeros(6, 32), bf(6, 32), bf(32)),
    ]
    for n, call in enumerate(wrong):
        recorder.name = None
        with pytest.raises((TypeError, ValueError)):
            call()
        assert recorder.name is None, n


def test_strided_operands_are_refused(q):
    with pytest.raises(ValueError):
        q.gated_gemm(bf(16, 32), bf(3, 32))  # not on a device
