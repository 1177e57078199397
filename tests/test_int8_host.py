"""Host-side checks of the 8-bit calls (no GPU, nothing launched): the C ABI's
refusals with addresses that are never read, and the binding's with host
tensors."""
import os

import pytest
import torch

import bit_nf4_quantized_07_amd as q

if not os.path.exists(q.LIB_PATH):
    pytest.skip("libqlora.so not built", allow_module_level=True)

lib = q.load_library()
D = 0x7f0000000000
MIS = D + 4
bf, f32, i8 = torch.bfloat16, torch.float32, torch.int8


@pytest.mark.parametrize("fn", [lib.int8_quantize, lib.int8_quantize_fp32])
def test_quantize_validation(fn):
    assert fn(None, 4, 64, D, D, None) == q.ERR_NULL
    assert fn(D, 4, 64, None, D, None) == q.ERR_NULL
    assert fn(D, 4, 64, D, None, None) == q.ERR_NULL
    for M, K in ((0, 64), (-1, 64), (4, 0), (4, 24), (1 << 22, 16), (4, (1 << 24) + 16),
                 (1 << 21, 1 << 14)):
        assert fn(D, M, K, D, D, None) == q.ERR_SHAPE, (M, K)
    assert fn(MIS, 4, 64, D, D, None) == q.ERR_ALIGN
    assert fn(D, 4, 64, MIS, D, None) == q.ERR_ALIGN
    assert fn(D, 4, 64, D, MIS, None) == q.ERR_ALIGN


def test_dequant_validation():
    f = lib.int8_dequant
    assert f(D, D, 4, 64, 0, None, None) == q.ERR_NULL
    assert f(D, D, 4, 64, 32, D, None) == q.ERR_UNSUPPORTED
    assert f(D, D, 4, 80, 64, D, None) == q.ERR_SHAPE
    assert f(D, D, 4, 72, 0, D, None) == q.ERR_SHAPE
    assert f(D, MIS, 4, 64, 0, D, None) == q.ERR_ALIGN


def test_gating_validation():
    f = lib.silu_mul_fwd_int8
    ok = [D, D, 4, 64, None, D, D, D, D, D, D, None]
    for i in (0, 1, 5, 6):
        assert f(*(None if j == i else v for j, v in enumerate(ok))) == q.ERR_NULL
    for i in (7, 8, 9, 10):       # G and Up are kept both or not at all
        assert f(*(None if j == i else v for j, v in enumerate(ok))) == q.ERR_NULL
    assert f(D, D, 4, 96, None, D, D, None, None, None, None, None) == q.ERR_SHAPE
    assert f(D, D, 0, 64, None, D, D, None, None, None, None, None) == q.ERR_SHAPE
    assert f(D, D, 4, 64, MIS, D, D, None, None, None, None, None) == q.ERR_ALIGN
    g = lib.silu_mul_bwd_int8
    assert g(D, D, D, D, D, 4, 64, D, None, None) == q.ERR_NULL
    assert g(D, D, D, D, D, 4, 32, D, D, None) == q.ERR_SHAPE
    assert g(D, D, MIS, D, D, 4, 64, D, D, None) == q.ERR_ALIGN


def _fwd(**kw):
    a = dict(Xc=D, Xs=D, M=32, K=256, N=128, Wc=D, Ws=D, A=D, B=D, r=8, alpha=16.0, Y=D, T=None, ws=D,
             wsb=1 << 30)
    a.update(kw)
    return lib.int8_linear_fwd(*a.values(), None)


def _bwd(**kw):
    a = dict(dY=D, Xc=D, Xs=D, M=32, K=256, N=128, Wc=D, Ws=D, A=D, B=D, r=8, alpha=16.0, T=None, dX=D,
             dA=D, dB=D, flags=0, ws=D, wsb=1 << 30)
    a.update(kw)
    return lib.int8_linear_bwd(*a.values(), None)


@pytest.mark.parametrize("fn", [_fwd, _bwd])
def test_linear_validation(fn):
    for name in ("Xc", "Xs", "Wc", "Ws", "A", "B"):
        assert fn(**{name: None}) == q.ERR_NULL, name
        assert fn(**{name: MIS}) == q.ERR_ALIGN, name
    assert fn(M=0) == q.ERR_SHAPE
    assert fn(K=96) == q.ERR_SHAPE
    assert fn(N=132) == q.ERR_SHAPE
    assert fn(r=257) == q.ERR_SHAPE
    assert fn(r=-8) == q.ERR_SHAPE
    assert fn(K=(1 << 17) + 64) == q.ERR_SHAPE          # the whole sums would leave 32 bits
    assert fn(M=1 << 20, K=1 << 11) == q.ERR_SHAPE      # 2 GiB of codes
    assert fn(M=1 << 16, N=1 << 14) == q.ERR_SHAPE      # 2 GiB of Y
    assert fn(N=1 << 15, K=1 << 16) == q.ERR_SHAPE      # 2 GiB of weight
    assert fn(alpha=float("nan")) == q.ERR_ARG
    assert fn(ws=None) == q.ERR_WORKSPACE
    assert fn(wsb=64) == q.ERR_WORKSPACE
    assert fn(ws=MIS) == q.ERR_ALIGN


def test_forward_only_validation():
    assert _fwd(Y=None) == q.ERR_NULL
    assert _fwd(Y=MIS) == q.ERR_ALIGN
    assert _fwd(T=MIS) == q.ERR_ALIGN
    assert _fwd(r=0) == q.ERR_ARG                       # A and B beside no rank
    assert _fwd(r=0, A=None, B=None, T=D) == q.ERR_ARG


def test_backward_only_validation():
    for name in ("dY", "dA", "dB"):
        assert _bwd(**{name: None}) == q.ERR_NULL, name
        assert _bwd(**{name: MIS}) == q.ERR_ALIGN, name
    assert _bwd(r=0) == q.ERR_SHAPE
    assert _bwd(flags=2) == q.ERR_ARG
    assert _bwd(dX=MIS) == q.ERR_ALIGN
    assert _bwd(N=1 << 14, K=1 << 16) == q.ERR_SHAPE    # 2 GiB of the base's bf16 copy
    f = lib.qlora_linear_bwd_int8
    a = [D, D, D, 32, 256, 128, D, D, D, D, D, D, 8, 16.0, None, D, D, D, 0, D, 1 << 30, None]
    for i in (6, 7, 8, 9):
        assert f(*(None if j == i else v for j, v in enumerate(a))) == q.ERR_NULL
        assert f(*(MIS if j == i else v for j, v in enumerate(a))) == q.ERR_ALIGN
    g = lib.qlora_linear_bwd_bf16_int8
    b = [D, D, D, 32, 256, 128, D, D, D, 8, 16.0, None, D, D, D, 0, D, 1 << 30, None]
    assert g(*(None if j == 6 else v for j, v in enumerate(b))) == q.ERR_NULL
    assert g(*(MIS if j == 6 else v for j, v in enumerate(b))) == q.ERR_ALIGN


def test_workspace_sizes():
    w = lib.int8_linear_workspace_bytes
    assert w(0, 256, 128, 8, q.BASE_INT8, 0) == 0
    assert w(32, 256, 128, 8, q.BASE_NF4, 0) == 0       # the forward has the 8-bit base alone
    assert w(32, 256, 128, 8, 3, 1) == 0
    assert w(32, 256, 128, 8, -1, 1) == 0
    for base in (q.BASE_INT8, q.BASE_NF4, q.BASE_BF16):
        assert w(32, 256, 128, 8, base, 1) > 0
        assert w(32, 256, 128, 5, base, 1) > w(32, 256, 128, 8, base, 1)   # padded copies
    assert w(2048, 4096, 4096, 16, q.BASE_INT8, 1) >= 2 * 4096 * 4096     # the base's bf16 copy


def _t8(rows, cols, blocks=False):
    scale = torch.zeros(rows, cols // 64, dtype=f32) if blocks else torch.zeros(rows, dtype=f32)
    return q.Int8Tensor(torch.zeros(rows, cols, dtype=i8), scale)


def _raises(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


M, K, N, R = 16, 256, 128, 8


def test_binding_refuses_quantize():
    X = torch.zeros(M, K, dtype=bf)
    _raises("X: a 2-D tensor", q.int8_quantize, X[0])
    _raises("X: dtype", q.int8_quantize, X.half())
    _raises("X: not contiguous", q.int8_quantize, torch.zeros(K, M, dtype=bf).t())
    _raises("codes_out: shape", q.int8_quantize, X, codes_out=torch.zeros(M, K + 16, dtype=i8))
    _raises("scale_out: dtype", q.int8_quantize, X, scale_out=torch.zeros(M, dtype=bf))
    _raises("not on a CUDA", q.int8_quantize, X)
    _raises("an Int8Tensor", q.int8_dequant, X)
    _raises("scale: shape", q.int8_dequant, q.Int8Tensor(torch.zeros(M, K, dtype=i8), torch.zeros(M + 1)))
    _raises("blocks of 64", q.int8_dequant, q.Int8Tensor(torch.zeros(M, 80, dtype=i8), torch.zeros(M, 1)))
    _raises("out: dtype", q.int8_dequant, _t8(M, K), out=torch.zeros(M, K))
    _raises("not on a CUDA", q.int8_dequant, _t8(M, K, True))


def test_binding_refuses_linear():
    A, B = torch.zeros(R, K, dtype=bf), torch.zeros(N, R, dtype=bf)
    f = lambda **kw: q.linear_fwd_int8(kw.get("X", _t8(M, K)), kw.get("W", _t8(N, K)), kw.get("A", A),
                                       kw.get("B", B), 16.0, out=kw.get("out"), T_out=kw.get("T_out"))
    _raises("X: an Int8Tensor", f, X=A)
    _raises("X.scale: shape", f, X=_t8(M, K, True))
    _raises("W: an Int8Tensor", f, W=(A, B))
    _raises("weight has K", f, W=_t8(N, K + 64))
    _raises("A: shape", f, A=torch.zeros(R, K + 64, dtype=bf))
    _raises("B: shape", f, B=torch.zeros(N, R + 8, dtype=bf))
    _raises("B: missing", f, B=None)
    _raises("A: a bf16", f, A=None)
    _raises("out: shape", f, out=torch.zeros(M, N + 8, dtype=bf))
    _raises("T_out: dtype", f, T_out=torch.zeros(M, R, dtype=bf))
    _raises("T_out: given", f, A=None, B=None, T_out=torch.zeros(M, R))
    _raises("not on a CUDA", f)
    dY = torch.zeros(M, N, dtype=bf)
    g = lambda **kw: q.linear_bwd_int8(kw.get("dY", dY), kw.get("X", _t8(M, K)), kw.get("W", _t8(N, K)),
                                       A, B, 16.0, T=kw.get("T"), need_dX=kw.get("need_dX", True),
                                       accumulate_into=kw.get("acc"), dX_out=kw.get("dX_out"),
                                       dA_out=kw.get("dA_out"), dB_out=kw.get("dB_out"))
    _raises("dY: shape", g, dY=torch.zeros(M, N + 8, dtype=bf))
    _raises("X: an Int8Tensor", g, X=dY)
    _raises("T: dtype", g, T=torch.zeros(M, R, dtype=bf))                       # 8-bit base: fp32
    _raises("T: dtype", g, W=torch.zeros(N, K, dtype=bf), T=torch.zeros(M, R))   # bf16 base: bf16
    _raises("weight has K", g, W=_t8(N, K + 64))
    _raises("W: shape", g, W=torch.zeros(N, K + 64, dtype=bf))
    _raises("dX: shape", g, acc=torch.zeros(M, K + 64, dtype=bf))
    _raises("dX_out: given", g, acc=torch.zeros(M, K, dtype=bf), dX_out=torch.zeros(M, K, dtype=bf))
    _raises("need_dX", g, need_dX=False, dX_out=torch.zeros(M, K, dtype=bf))
    _raises("dA: dtype", g, dA_out=torch.zeros(R, K, dtype=bf))
    _raises("dB: shape", g, dB_out=torch.zeros(N, R + 8))
    _raises("not on a CUDA", g)


def test_binding_refuses_gating():
    G = torch.zeros(M, K, dtype=bf)
    _raises("Up: shape", q.silu_mul_fwd_int8, G, torch.zeros(M, K + 64, dtype=bf))
    _raises("G: a 2-D", q.silu_mul_fwd_int8, G[0], G)
    _raises("out: dtype", q.silu_mul_fwd_int8, G, G, out=torch.zeros(M, K))
    _raises("not on a CUDA", q.silu_mul_fwd_int8, G, G)
    _raises("G: an Int8Tensor", q.silu_mul_bwd_int8, G, G, _t8(M, K, True))
    _raises("Up.scale: shape", q.silu_mul_bwd_int8, G, _t8(M, K, True), _t8(M, K))
    _raises("Up: shape", q.silu_mul_bwd_int8, G, _t8(M, K, True), _t8(M, K + 64, True))
    _raises("dH: dtype", q.silu_mul_bwd_int8, G.float(), _t8(M, K, True), _t8(M, K, True))
    _raises("not on a CUDA", q.silu_mul_bwd_int8, G, _t8(M, K, True), _t8(M, K, True))
