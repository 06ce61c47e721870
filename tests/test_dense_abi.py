"""Refusals of the norms, the gated projection and the 8-bit product: status codes before any
CUDA call, and the binding's checks of tensors (no GPU needed)."""
import ctypes

import pytest
import torch

P, I64, SZ, F32, I32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float,
                        ctypes.c_int)
OK = 1 << 20                       # 16-byte aligned address, never read
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_moe_nvfp4_b200 import build
    return ctypes.CDLL(build.build())


def entry(lib, name, types, args):
    """call(**changes): the entry point with `args` (a dict in order) and those changes."""
    f = getattr(lib, name)
    f.restype, f.argtypes = I32, types + [P]

    def call(**over):
        assert set(over) <= set(args)
        return f(*dict(args, **over).values(), None)
    return call


def test_pre_norm(lib):
    call = entry(lib, "moe_nvfp4_pre_norm", [P, P, I64, I64, F32, P],
                 dict(x=OK, w=OK, T=4, H=64, eps=1e-5, out=OK))
    assert call(T=0, x=None, out=None) == 0           # nothing to do, nothing enqueued
    for bad in (dict(x=None), dict(w=None), dict(out=None), dict(T=-1), dict(H=0), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(x=OK + 2), dict(w=OK + 8),
                dict(out=OK + 4)):
        assert call(**bad) == -1, bad
    assert call(H=60) == -2 and call(H=32768 + 8) == -2 and call(T=1 << 40) == -2


def test_rows_to_8_bits(lib):
    norm = entry(lib, "moe_nvfp4_pre_norm_int8", [P, P, I64, I64, F32, P, P],
                 dict(x=OK, w=OK, T=4, H=64, eps=1e-5, codes=OK, scales=OK))
    quant = entry(lib, "nvfp4_int8_quantize", [P, I64, I64, P, P],
                  dict(x=OK, T=4, H=64, codes=OK, scales=OK))
    for call in (norm, quant):
        assert call(T=0, x=None, codes=None, scales=None) == 0
        for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(T=-1), dict(H=0),
                    dict(x=OK + 2), dict(codes=OK + 8), dict(scales=OK + 2)):
            assert call(**bad) == -1, bad
        assert call(H=72) == -2 and call(H=32768 + 16) == -2
    assert norm(w=None) == -1 and norm(eps=0.0) == -1


def test_post_norm(lib):
    call = entry(lib, "moe_nvfp4_post_norm", [P, P, P, P, I64, I64, I64, I64, F32, F32, P, P, P],
                 dict(y=OK, w=OK, res=OK, gate=None, T=4, H=64, gr=0, gc=0, eps=1e-5, a=1.0,
                      w2=None, out=OK, nxt=None))
    assert call(T=0, y=None, res=None, out=None) == 0
    for bad in (dict(y=None), dict(w=None), dict(res=None), dict(out=None), dict(w2=OK),
                dict(nxt=OK), dict(w2=OK + 2, nxt=OK), dict(w2=OK, nxt=OK + 8), dict(eps=0.0),
                dict(gate=OK), dict(gate=OK, gr=2, gc=64), dict(gate=OK, gr=4, gc=2),
                dict(gr=4, gc=64), dict(gate=OK + 2, gr=1, gc=64), dict(gate=OK + 1, gr=4, gc=1)):
        assert call(**bad) == -1, bad
    assert call(H=60) == -2


def test_norm_gradients(lib):
    size = lib.moe_nvfp4_norm_backward_workspace_size
    size.restype, size.argtypes = SZ, [I64, I64]
    assert size(4, 64) > 0 and size(100000, 6144) < 64 << 20   # bounded by the CTAs, not T
    assert size(-1, 64) == 0 and size(4, 0) == 0
    pre = entry(lib, "moe_nvfp4_pre_norm_backward", [P, P, P, P, I64, I64, F32, P, P, P, SZ],
                dict(dy=OK, x=OK, w=OK, dskip=None, T=4, H=64, eps=1e-5, dx=OK, dw=OK, ws=OK,
                     ws_bytes=1 << 30))
    post = entry(lib, "moe_nvfp4_post_norm_backward",
                 [P, P, P, P, I64, I64, I64, I64, F32, F32, P, P, P, P, P, SZ],
                 dict(dy=OK, x=OK, w=OK, gate=None, T=4, H=64, gr=0, gc=0, eps=1e-5, a=1.0,
                      dx=OK, dw=OK, dg=None, dr=None, ws=OK, ws_bytes=1 << 30))
    for call in (pre, post):
        for bad in (dict(dy=None), dict(x=None), dict(w=None), dict(dx=None), dict(dw=None),
                    dict(dy=OK + 2), dict(dw=OK + 2), dict(T=-1), dict(eps=0.0)):
            assert call(**bad) == -1, bad
        assert call(H=60) == -2
        assert call(ws=None) == -3 and call(ws=OK + 4) == -3
        assert call(ws_bytes=size(4, 64) - 1) == -3
    assert pre(dskip=OK + 2) == -1
    for bad in (dict(dg=OK), dict(gate=OK, gr=1, gc=64), dict(gate=OK, gr=4, gc=64),
                dict(gate=OK, gr=1, gc=64, dg=OK + 2), dict(dr=OK + 2),
                dict(gate=OK, gr=3, gc=64, dg=OK)):
        assert post(**bad) == -1, bad


def test_gate_up(lib):
    fwd = entry(lib, "moe_nvfp4_gate_up", [P, P, I64, I64, I64, I32, P, P, P],
                dict(x=OK, w=OK, T=4, H=64, I=32, act=0, h=OK, gu=None, flag=None))
    assert fwd(T=0, x=None, h=None) == 0
    for bad in (dict(x=None), dict(w=None), dict(h=None), dict(T=-1), dict(H=0), dict(I=0),
                dict(act=2), dict(act=-1), dict(x=OK + 2), dict(w=OK + 2), dict(h=OK + 2),
                dict(gu=OK + 2), dict(flag=OK + 2)):
        assert fwd(**bad) == -1, bad
    for bad in (dict(H=60), dict(I=12), dict(H=65544), dict(I=65544), dict(T=1 << 30),
                dict(T=(1 << 28) + 1, I=32768)):
        assert fwd(**bad) == -2, bad
    size = lib.moe_nvfp4_gate_up_backward_workspace_size
    size.restype, size.argtypes = SZ, [I64, I64]
    assert size(4, 32) == 4 * 64 * 2 and size(0, 32) == 0 and size(3, 8) == 256
    bwd = entry(lib, "moe_nvfp4_gate_up_backward",
                [P, P, P, P, I64, I64, I64, I32, P, P, P, SZ, P],
                dict(dh=OK, x=OK, w=OK, gu=OK, T=4, H=64, I=32, act=0, dx=OK, dw=OK, ws=OK,
                     ws_bytes=1 << 30, flag=None))
    assert bwd(T=0, dw=None) == 0
    for bad in (dict(dh=None), dict(gu=None), dict(x=None), dict(w=None), dict(dx=None, dw=None),
                dict(act=7), dict(dx=OK + 2), dict(dw=OK + 2), dict(gu=OK + 2), dict(flag=OK + 1)):
        assert bwd(**bad) == -1, bad
    assert bwd(H=60) == -2 and bwd(I=12) == -2
    assert bwd(ws=None) == -3 and bwd(ws=OK + 8) == -3 and bwd(ws_bytes=size(4, 32) - 1) == -3


def test_int8_matmul(lib):
    call = entry(lib, "nvfp4_int8_matmul", [P, P, P, P, I64, I64, I64, P, P],
                 dict(a=OK, sa=OK, w=OK, sw=OK, T=4, N=64, K=64, out=OK, flag=None))
    assert call(T=0, a=None, sa=None, out=None) == 0
    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(out=None),
                dict(T=-1), dict(N=0), dict(K=0), dict(a=OK + 8), dict(w=OK + 8), dict(sw=OK + 4),
                dict(sa=OK + 2), dict(out=OK + 2), dict(flag=OK + 2)):
        assert call(**bad) == -1, bad
    for bad in (dict(K=72), dict(N=12), dict(K=32784), dict(N=(1 << 24) + 8), dict(T=1 << 30),
                dict(T=(1 << 24), N=(1 << 20) + 8)):
        assert call(**bad) == -2, bad


def test_binding_checks_tensors(lib):
    """Wrong types, shapes, strides and devices are refused before the library is called."""
    import bit_quantized_moe_nvfp4_b200 as nv
    bf = torch.bfloat16
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(64, dtype=bf)
    i8, f = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    calls = [lambda: nv.moe_nvfp4_pre_norm(x, w, 1e-5), lambda: nv.moe_nvfp4_pre_norm(x[0], w, 1e-5),
             lambda: nv.moe_nvfp4_pre_norm_int8(x, w, 1e-5),
             lambda: nv.moe_nvfp4_post_norm(x, w, x, 1e-5),
             lambda: nv.moe_nvfp4_post_norm_backward(x, x, w, 1e-5),
             lambda: nv.moe_nvfp4_pre_norm_backward(x, x, w, 1e-5),
             lambda: nv.moe_nvfp4_gate_up(x, x), lambda: nv.nvfp4_int8_quantize(x),
             lambda: nv.moe_nvfp4_gate_up_backward(x[:, :2], x, x, x[:, :4]),
             lambda: nv.nvfp4_int8_matmul(i8, f, i8, f), lambda: nv.nvfp4_int8_matmul(x, f, i8, f)]
    for c in calls:
        with pytest.raises(ValueError):
            c()


def test_the_timeout_hooks(lib):
    gate = entry(lib, "nvfp4_selftest_gate_up_timeout", [P, P, I64, I64, I64, P, P, P],
                 dict(x=OK, w=OK, T=4, H=64, I=32, h=OK, gu=None, flag=OK))
    prod = entry(lib, "nvfp4_selftest_int8_matmul_timeout", [P, P, P, P, I64, I64, I64, P, P],
                 dict(a=OK, sa=OK, w=OK, sw=OK, T=4, N=64, K=64, out=OK, flag=OK))
    for call in (gate, prod):
        for bad in (dict(flag=None), dict(flag=OK + 2), dict(T=0), dict(T=-1), dict(w=None)):
            assert call(**bad) == -1, bad
        assert call(T=1 << 30) == -2
    assert gate(x=OK + 2) == -1 and gate(I=12) == -2
    assert prod(out=OK + 8) == -1 and prod(K=72) == -2
