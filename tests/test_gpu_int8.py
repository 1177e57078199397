"""Activations and weights in 8 bits on the GPU, against numpy in 64 bits.

Tolerances are worst cases, counted: a rounding to fp32 is off by at most 2^-24
of the value, one to bf16 by 2^-8; a sum of n terms in fp32 by n 2^-23 of the
sum of magnitudes (a step may cut instead of round).
"""
import numpy as np
import pytest

from oracle import int8 as o8

import gpu_helpers as h

pytestmark = pytest.mark.gpu

F32, BF = 2.0 ** -24, 2.0 ** -8


def _q():
    import bit_nf4_quantized_07_amd as q
    return q


def _bits(x):
    """fp64 -> bf16 bits (numpy)."""
    t = h.torch()
    return t.from_numpy(np.ascontiguousarray(x, np.float32)).bfloat16().view(t.int16).numpy().view(np.uint16)


def _activations(g, M, K):
    x = g.standard_normal((M, K)) * np.exp(0.5 * g.standard_normal((M, 1)))
    x[:, g.random(K) < 0.02] *= 9.0
    return x


def _assert_within(got, ref, tol, name):
    got = np.asarray(got, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    ok = ~np.isnan(ref)
    err = np.abs(got - ref)[ok]
    worst = (err - np.broadcast_to(tol, ref.shape)[ok]).max() if err.size else 0.0
    h.log(f"  {name}: largest error {err.max() if err.size else 0:.3e}, over its bound by {worst:.3e}")
    assert worst <= 0.0, f"{name}: over its bound by {worst:.3e}"


# ---- rows and blocks of codes ------------------------------------------------

SIZES = [(1, 16), (3, 48), (7, 1024), (5, 1040), (2, 4096), (129, 4112), (3, 11008), (2, 16384),
         (2, 16400), (1, 65536), (2, 65552), (1, 131072)]


def _nasty(g, M, K):
    """Rows of zeros, ties, the type's extremes and non-finite values among others."""
    x = _activations(g, M, K)
    x[0] = g.integers(-254, 255, K)
    x[0, 0] = 254.0                          # 127 x / a = x / 2: ties wherever x is odd
    if M > 1:
        x[1] = 0.0
    if M > 2:
        x[2] *= 2.0 ** -125                  # largest magnitude near the smallest normal
    if M > 6:
        x[3] = np.clip(x[3], -1, 1) * 3.3e38
        x[4, K // 2] = np.inf
        x[5, K - 1] = np.nan
        x[6] = g.integers(-3, 4, K) * 2.0 ** -133   # subnormal bf16
    return x


@pytest.mark.parametrize("M,K", SIZES)
def test_rows_from_bf16_are_exact(M, K):
    q, t = _q(), h.torch()
    bits = _bits(_nasty(np.random.default_rng(M * 7919 + K), M, K))
    X = q.int8_quantize(h.dev_bf16(bits))
    codes, scale = o8.quantize_rows(h.f64(bits))
    assert np.array_equal(h.host(X.codes), codes)
    assert np.array_equal(h.host(X.scale), scale, equal_nan=True)
    back = h.host_bf16_bits(q.int8_dequant(X))
    with np.errstate(invalid="ignore"):
        want = (codes.astype(np.float32) * scale[:, None])
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(h.f64(back)), nan)
    assert np.array_equal(back[~nan], _bits(want)[~nan])


@pytest.mark.parametrize("M,K", [(5, 48), (130, 4096), (3, 11008), (1, 65552)])
def test_rows_from_fp32(M, K):
    q, t = _q(), h.torch()
    x = _activations(np.random.default_rng(K), M, K).astype(np.float32)
    x[0] = 0.0
    if M > 2:
        x[1] *= np.float32(2.0 ** -120)
        x[2] *= np.float32(2.0 ** 120)
    X = q.int8_quantize(h.dev_f32(x))
    a = np.abs(x).max(1)
    assert np.array_equal(h.host(X.scale), a / np.float32(127.0))
    safe = np.where(a == 0, 1.0, a).astype(np.float64)
    n = 127.0 * x.astype(np.float64) / safe[:, None]
    # the quotient is rounded to fp32 (2^-24 of up to 127) before it is rounded whole
    assert np.abs(h.host(X.codes) - n).max() <= 0.5 + 128 * F32


def test_out_tensors_and_another_stream():
    q, t = _q(), h.torch()
    X = t.randn(33, 512, device="cuda").bfloat16()
    want = q.int8_quantize(X)
    codes, scale = t.empty(33, 512, dtype=t.int8, device="cuda"), t.empty(33, device="cuda")
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(s):
        got = q.int8_quantize(X, codes_out=codes, scale_out=scale)
    s.synchronize()
    assert got.codes is codes and got.scale is scale
    assert t.equal(codes, want.codes) and t.equal(scale, want.scale)
    with pytest.raises(ValueError, match="overlaps"):
        q.int8_quantize(X, codes_out=X.view(t.int8).reshape(-1)[: 33 * 512].reshape(33, 512))
    whole = t.zeros(2 * 33 * 512, dtype=t.int8, device="cuda")
    inside = q.Int8Tensor(whole[: 33 * 512].reshape(33, 512), want.scale)
    with pytest.raises(ValueError, match="overlaps"):
        q.int8_dequant(inside, out=whole.view(t.bfloat16).reshape(33, 512))


# ---- gating -------------------------------------------------------------------

# The fast exponential's error: the argument times log2 e rounds within 2^-24 of
# itself (|g| log2 e 2^-24 of the result, |g| <= 30 here: 44 2^-24), v_exp_f32
# within 2^-22; the sum, the reciprocal and the products three roundings each.
GATE = 80 * F32


@pytest.mark.parametrize("M,I", [(1, 64), (3, 192), (9, 1024), (4, 1088), (5, 4096), (2, 11008),
                                 (2, 16448), (1, 28672), (1, 65600)])
@pytest.mark.parametrize("save", [True, False])
def test_gating_forward(M, I, save):
    q, t = _q(), h.torch()
    g = np.random.default_rng(M + I)
    G, U = (np.clip(_activations(g, M, I), -30, 30) for _ in range(2))
    if M > 2:
        G[1] = 0.0
        U[2, I // 2] = np.nan
    Gb, Ub = _bits(G), _bits(U)
    dG, dU = h.dev_bf16(Gb), h.dev_bf16(Ub)
    out = t.full((M, I), 7.0, dtype=t.bfloat16, device="cuda")
    H, G8, U8 = q.silu_mul_fwd_int8(dG, dU, save=save, out=out)
    assert np.array_equal(h.host_bf16_bits(out), h.host_bf16_bits(q.silu_mul_fwd(dG, dU)))
    ref = o8.silu(h.f64(Gb)) * h.f64(Ub)
    bad = ~np.isfinite(ref).all(1)
    a = np.abs(np.where(bad[:, None], 0.0, ref)).max(1)
    scale = h.host(H.scale).astype(np.float64)
    assert np.array_equal(np.isnan(scale), bad)
    assert np.all(np.abs(scale - a / 127.0)[~bad] <= (a / 127.0)[~bad] * (GATE + F32))
    codes = h.host(H.codes).astype(np.float64)
    assert np.all(codes[bad] == 0) and np.all(codes[a == 0] == 0)
    ok = ~bad & (a > 0)
    n = 127.0 * ref[ok] / a[ok][:, None]
    # half a step, and up to 127 times the value's and the maximum's own error
    assert np.abs(codes[ok] - n).max() <= 0.5 + 127 * (2 * GATE + 2 * F32)
    if not save:
        assert G8 is None and U8 is None
        return
    for got, bits in ((G8, Gb), (U8, Ub)):
        c, s = o8.quantize_rows(h.f64(bits), 64)
        assert np.array_equal(h.host(got.codes), c)
        assert np.array_equal(h.host(got.scale), s, equal_nan=True)
    with np.errstate(invalid="ignore"):
        want = _bits(np.float32(1) * h.host(G8.codes).reshape(M, -1, 64) * h.host(G8.scale)[..., None])
    assert np.array_equal(h.host_bf16_bits(q.int8_dequant(G8)), want.reshape(M, I))


@pytest.mark.parametrize("M,I", [(1, 64), (7, 192), (33, 1024), (3, 11008)])
def test_gating_backward(M, I):
    q, t = _q(), h.torch()
    g = np.random.default_rng(31 * M + I)
    G8, U8 = (q.Int8Tensor(*map(lambda v: t.from_numpy(v).cuda(), o8.quantize_rows(
        np.clip(_activations(g, M, I), -30, 30), 64))) for _ in range(2))
    dHb = _bits(g.standard_normal((M, I)))
    dG, dU = q.silu_mul_bwd_int8(h.dev_bf16(dHb), G8, U8)
    # the kept values are fp32 products of code and scale
    gv = (h.host(G8.codes).reshape(M, -1, 64) * h.host(G8.scale)[..., None]).reshape(M, I).astype(np.float64)
    uv = (h.host(U8.codes).reshape(M, -1, 64) * h.host(U8.scale)[..., None]).reshape(M, I).astype(np.float64)
    rG, rU = o8.silu_mul_grad(h.f64(dHb), gv, uv)
    sig = 1.0 / (1.0 + np.exp(-gv))
    # 1 + g (1 - sig) cancels: its error counts the two terms' magnitudes
    mag = np.abs(h.f64(dHb) * uv * sig) * (1.0 + np.abs(gv) * (1.0 + 2 * sig))
    _assert_within(h.host_bf16_f64(dG), rG, np.abs(rG) * BF + mag * GATE * 2 * (1 + BF) + 1e-40, "dG")
    _assert_within(h.host_bf16_f64(dU), rU, np.abs(rU) * (BF + 2 * GATE) + 1e-40, "dU")


# ---- the layer ----------------------------------------------------------------

class _Layer:
    """A layer's tensors on both sides."""

    def __init__(self, M, K, N, r, seed=0):
        q, t = _q(), h.torch()
        g = np.random.default_rng([seed, M, K, N, r])
        self.M, self.K, self.N, self.r = M, K, N, r
        self.xc, self.xs = o8.quantize_rows(h.f64(_bits(_activations(g, M, K))))
        self.wc, self.ws = o8.quantize_rows(h.f64(_bits(0.02 * g.standard_normal((N, K)))))
        self.A = _bits(g.uniform(-1, 1, (r, K)) / np.sqrt(K))
        self.B = _bits(0.05 * g.standard_normal((N, r)))
        self.dY = _bits(0.1 * g.standard_normal((M, N)))
        self.alpha = 1.7 * max(r, 1)
        self.s = float(np.float32(np.float32(self.alpha) / np.float32(max(r, 1))))
        dev = lambda v: t.from_numpy(v).cuda()
        self.X, self.W = q.Int8Tensor(dev(self.xc), dev(self.xs)), q.Int8Tensor(dev(self.wc), dev(self.ws))
        self.dA, self.dB, self.ddY = h.dev_bf16(self.A), h.dev_bf16(self.B), h.dev_bf16(self.dY)

    def x(self):
        return o8.values(self.xc, self.xs)

    def w(self):
        return o8.values(self.wc, self.ws)

    def check_fwd(self, Y, T):
        X, W, A, B = self.x(), self.w(), h.f64(self.A), h.f64(self.B)
        base, absb = X @ W.T, np.abs(X) @ np.abs(W).T
        # whole sums; three roundings to fp32, and those of up to 16 partial sums
        tol = absb * 20 * F32
        ref = base
        if self.r:
            refT, absT = X @ A.T, np.abs(X) @ np.abs(A).T
            tolT = absT * (self.K + 16) * 2 * F32 + np.abs(refT) * 2 * F32
            if T is not None:
                _assert_within(h.host(T), refT, tolT, "T")
            ref = base + self.s * refT @ B.T
            # T's own error, its two bf16 terms (2^-16), the sum over r of both
            tol = tol + abs(self.s) * ((tolT + absT * (2.0 ** -16 + (2 * self.r + 20) * 2 * F32)) @ np.abs(B).T)
        _assert_within(h.host_bf16_f64(Y), ref, np.abs(ref) * BF + tol * (1 + BF), "Y")

    def check_bwd(self, dX, dA, dB, T, W, what="", dX0=None, Wtol=BF):
        """W: the base's values; Wtol: how far its bf16 copy may be from them."""
        X, A, B, dY = self.x(), h.f64(self.A), h.f64(self.B), h.f64(self.dY)
        U, absU = dY @ B, np.abs(dY) @ np.abs(B)
        tolU = absU * (self.N + 16) * 2 * F32
        if dX is not None:
            ref = dY @ W + self.s * U @ A + (0.0 if dX0 is None else dX0)
            absX = np.abs(dY) @ np.abs(W)
            # W's bf16 copy; U and s A in bf16; the sums in fp32
            tol = absX * (Wtol + (self.N + 40) * 2 * F32) + self.s * (
                tolU + absU * (2 * BF + BF * BF + 4 * self.r * F32)) @ np.abs(A)
            tol = tol + (0.0 if dX0 is None else np.abs(dX0) * 2 * F32)
            _assert_within(h.host_bf16_f64(dX), ref, np.abs(ref) * BF + tol * (1 + BF), what + "dX")
        n = 2 * F32 * (3 * self.M + 40)
        refA = self.s * U.T @ X
        _assert_within(h.host(dA), refA, self.s * (tolU.T @ np.abs(X) + absU.T @ np.abs(X) * n), what + "dA")
        refB = self.s * dY.T @ T
        _assert_within(h.host(dB), refB, self.s * (np.abs(dY).T @ np.abs(T)) * n, what + "dB")


LAYERS = [(1, 64, 8, 8), (20, 32768, 40, 8), (40, 16448, 72, 32), (1, 4096, 512, 16), (3, 2048, 136, 8), (16, 1024, 264, 16), (16, 512, 4104, 32), (7, 640, 72, 24), (2, 128, 24, 0), (5, 192, 40, 3), (16, 256, 256, 8),
          (16, 832, 1000, 64), (16, 320, 4104, 256), (17, 64, 8, 8), (17, 256, 136, 16), (33, 448, 72, 24),
          (64, 1024, 520, 0), (100, 4096, 264, 12), (129, 512, 1032, 128), (257, 320, 776, 16),
          (300, 2048, 2056, 256), (700, 576, 1304, 40), (1030, 1152, 2824, 8)]


@pytest.mark.parametrize("M,K,N,r", LAYERS)
def test_forward(M, K, N, r):
    q, t = _q(), h.torch()
    L = _Layer(M, K, N, r)
    args = (L.X, L.W, L.dA, L.dB, L.alpha) if r else (L.X, L.W)
    Y, T = q.linear_fwd_int8(*args)
    assert (T is None) == (r == 0)
    L.check_fwd(Y, T)
    # the same bits again, without T, into the caller's tensors and workspace
    out = t.full((M, N), 3.0, dtype=t.bfloat16, device="cuda")
    Y2, T2 = q.linear_fwd_int8(*args, save_T=False, out=out, workspace=q.Workspace())
    assert T2 is None and Y2 is out and t.equal(out, Y)


@pytest.mark.parametrize("N,form", [(40000, "two blocks of rows"), (16376, "one block, many")])
def test_forward_small_wide(N, form):
    L = _Layer(3, 128, N, 8)
    L.check_fwd(*_q().linear_fwd_int8(L.X, L.W, L.dA, L.dB, L.alpha))


def test_forward_large_tiles():
    """Sizes at which each of the large tiles is taken, against sampled rows."""
    q, t = _q(), h.torch()
    for M, K, N, r in ((2048, 1024, 4096, 16), (4100, 512, 5000, 16), (513, 640, 8200, 0)):
        g = t.Generator("cuda")
        g.manual_seed(M)
        X = q.int8_quantize(t.randn(M, K, device="cuda", generator=g).bfloat16())
        W = q.int8_quantize(0.02 * t.randn(N, K, device="cuda", generator=g))
        A = (t.randn(max(r, 1), K, device="cuda", generator=g) / 32).bfloat16()
        B = (t.randn(N, max(r, 1), device="cuda", generator=g) / 16).bfloat16()
        Y, T = q.linear_fwd_int8(X, W, *((A, B, 2.0 * r) if r else ()))
        xv, wv = X.codes.double() * X.scale.double()[:, None], W.codes.double() * W.scale.double()[:, None]
        ref, tol = xv @ wv.t(), (xv.abs() @ wv.abs().t()) * 20 * F32
        if r:
            ref = ref + 2.0 * (xv @ A.double().t()) @ B.double().t()
            tol = tol + 2.0 * ((xv.abs() @ A.double().abs().t()) * (2.0 ** -16 + (K + 2 * r + 36) * 2 * F32)) @ B.double().abs().t()
        err = (Y.double() - ref).abs() - ref.abs() * BF - tol * (1 + BF)
        assert float(err.max()) <= 0.0, (M, K, N, r, float(err.max()))


def test_forward_non_finite_rows():
    """A token that stands for NaN spoils its own row alone; an infinite adapter
    weight gives the product's infinity or NaN, not the terms'."""
    q, t = _q(), h.torch()
    for M in (3, 40):
        L = _Layer(M, 256, 136, 8)
        xs = L.xs.copy()
        xs[1] = np.nan
        xc = L.xc.copy()
        xc[1] = 0
        X = q.Int8Tensor(t.from_numpy(xc).cuda(), t.from_numpy(xs).cuda())
        Y, T = q.linear_fwd_int8(X, L.W, L.dA, L.dB, L.alpha)
        want, _ = q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, L.alpha)
        assert bool(Y[1].isnan().all()) and bool(T[1].isnan().all())
        keep = [m for m in range(M) if m != 1]
        assert t.equal(Y[keep], want[keep])
        B = L.dB.clone()
        B[5, 2] = float("inf")
        Y, T = q.linear_fwd_int8(L.X, L.W, L.dA, B, L.alpha)
        assert t.equal(Y[:, 5].float(), t.sign(T[:, 2]) * float("inf"))
        assert bool(Y[:, 6].isfinite().all())


BWD = [(1, 64, 8, 8), (4, 128, 16648, 16), (70, 64, 8200, 24), (5, 192, 40, 3), (16, 256, 256, 8), (33, 448, 72, 24), (100, 1024, 264, 16),
       (129, 512, 1032, 128), (300, 320, 776, 256), (1030, 576, 512, 12)]


@pytest.mark.parametrize("M,K,N,r", BWD)
def test_backward_int8_base(M, K, N, r):
    q, t = _q(), h.torch()
    L = _Layer(M, K, N, r)
    _, T = q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, L.alpha)
    got = q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha, T=T)
    L.check_bwd(*got, h.host(T).astype(np.float64), L.w())
    # T computed again; dX left out
    dX, dA, dB = q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha, need_dX=False)
    assert dX is None and t.equal(dA, got[1])
    absT = np.abs(L.x()) @ np.abs(h.f64(L.A)).T
    refB, n = L.s * h.f64(L.dY).T @ (L.x() @ h.f64(L.A).T), 2 * F32 * (3 * M + K + 60)
    _assert_within(h.host(dB), refB, L.s * (np.abs(h.f64(L.dY)).T @ absT) * n, "dB from codes")
    # added to a dX, everything into the caller's tensors; twice the same bits
    dX0 = t.randn(M, K, device="cuda").bfloat16()
    for _ in range(2):
        acc = dX0.clone()
        oA, oB = t.full((r, K), 9.0, device="cuda"), t.full((N, r), 9.0, device="cuda")
        dX, dA, dB = q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha, T=T, accumulate_into=acc,
                                       dA_out=oA, dB_out=oB, workspace=q.Workspace())
        assert dX is acc and t.equal(oA, got[1]) and t.equal(oB, got[2])
        L.check_bwd(dX, dA, dB, h.host(T).astype(np.float64), L.w(), "added: ", dX0=h.host_bf16_f64(dX0))


@pytest.mark.parametrize("M,K,N,r", [(5, 192, 40, 3), (100, 1024, 264, 16), (1030, 576, 512, 12)])
def test_backward_nf4_and_bf16_base(M, K, N, r):
    q, t = _q(), h.torch()
    L = _Layer(M, K, N, r)
    g = np.random.default_rng(K)
    W0 = (0.02 * g.standard_normal((N, K))).astype(np.float32)
    ow = h.OracleWeight(W0)
    qw = q.quantize(h.dev_f32(W0))
    Tb = _bits(L.x() @ h.f64(L.A).T)
    dX, dA, dB = q.linear_bwd_int8(L.ddY, L.X, qw, L.dA, L.dB, L.alpha, T=h.dev_bf16(Tb))
    L.check_bwd(dX, dA, dB, h.f64(Tb), h.f64(ow.w_bf16()), "NF4: ", Wtol=0.0)
    # the base's own backward gives the same dX from the same dY (A in place of X: not read for dX)
    dX2, _, _ = q.linear_bwd(L.ddY, t.zeros(M, K, dtype=t.bfloat16, device="cuda"), qw, L.dA, L.dB, L.alpha,
                             T=h.dev_bf16(Tb))
    # U and the products in another order: both within the same bound of the same values
    h.assert_close(h.host_bf16_f64(dX2), h.host_bf16_f64(dX), "NF4: dX beside linear_bwd's")
    Wb = _bits(W0)
    dX, dA, dB = q.linear_bwd_int8(L.ddY, L.X, h.dev_bf16(Wb), L.dA, L.dB, L.alpha)
    refT = L.x() @ h.f64(L.A).T
    X, A, B, dY = L.x(), h.f64(L.A), h.f64(L.B), h.f64(L.dY)
    U, absU = dY @ B, np.abs(dY) @ np.abs(B)
    absT = np.abs(X) @ np.abs(A).T
    _assert_within(h.host(dB), L.s * dY.T @ refT, L.s * (np.abs(dY).T @ absT) * 2 * F32 * (3 * M + K + 60), "bf16: dB")
    ref = dY @ h.f64(Wb) + L.s * U @ A
    tol = np.abs(dY) @ np.abs(h.f64(Wb)) * (N + 40) * 2 * F32 + L.s * (
        absU * ((N + 16) * 2 * F32 + 2 * BF + BF * BF + 4 * r * F32)) @ np.abs(A)
    _assert_within(h.host_bf16_f64(dX), ref, np.abs(ref) * BF + tol * (1 + BF), "bf16: dX")


DX = [(1, 64, 8), (3, 4096, 4104), (16, 8192, 1000), (40, 320, 72), (100, 2048, 2056), (130, 4160, 520), (7, 1088, 4096), (100, 2112, 512), (128, 64, 768),
      (257, 1088, 4096), (300, 4096, 1544), (512, 11008, 264), (511, 576, 8200), (513, 320, 72), (700, 2112, 776),
      (1100, 4096, 1032), (2100, 4160, 328), (4100, 4096, 200)]


@pytest.mark.parametrize("M,K,N", DX)
def test_input_gradient(M, K, N):
    """dX on every base at few and many tokens, with outputs that end inside a step
    and features that end inside a tile, alone and added to what is there."""
    q, t = _q(), h.torch()
    g = t.Generator("cuda")
    g.manual_seed(M + K + N)
    rnd = lambda *s: t.randn(*s, device="cuda", generator=g)
    r = 8
    X, W0 = q.int8_quantize(rnd(M, K).bfloat16()), 0.02 * rnd(N, K)
    A, B, dY = (rnd(r, K) / 32).bfloat16(), (rnd(N, r) / 16).bfloat16(), rnd(M, N).bfloat16()
    dX0 = rnd(M, K).bfloat16()
    W8, W4 = q.int8_quantize(W0), q.quantize(W0)
    # NF4 decodes to a bf16 value; codes are rounded to one (within half a step)
    for W, v, wtol in ((W8, W8.codes.double() * W8.scale.double()[:, None], BF),
                       (W4, q.nf4_dequant(W4).double(), BF), (W0.bfloat16(), W0.bfloat16().double(), 0.0)):
        T = rnd(M, r)
        T = T if W is W8 else T.bfloat16()
        dX = q.linear_bwd_int8(dY, X, W, A, B, 2.0 * r, T=T)[0]
        U, absU = dY.double() @ B.double(), dY.double().abs() @ B.double().abs()
        ref = dY.double() @ v + 2.0 * U @ A.double()
        # the weight's rounding; U and 2 A in bf16; the sums in fp32, the splits' too
        tol = dY.double().abs() @ v.abs() * (wtol + (N + 40) * 2 * F32) + 2.0 * (
            absU * ((N + 16) * 2 * F32 + 2 * BF + BF * BF + 4 * r * F32)) @ A.double().abs()
        err = (dX.double() - ref).abs() - ref.abs() * BF - tol * (1 + BF)
        assert float(err.max()) <= 0.0, (type(W).__name__, float(err.max()))
        acc = dX0.clone()
        q.linear_bwd_int8(dY, X, W, A, B, 2.0 * r, T=T, accumulate_into=acc)
        ref = ref + dX0.double()
        tol = tol + dX0.double().abs() * 2 * F32
        err = (acc.double() - ref).abs() - ref.abs() * BF - tol * (1 + BF)
        assert float(err.max()) <= 0.0, (type(W).__name__, "added", float(err.max()))


@pytest.mark.parametrize("M,N", [(3, 136), (40, 264), (600, 264), (600, 256)])
def test_backward_non_finite_rows(M, N):
    """An infinity in a token's dY reaches that token's dX alone, a token kept as NaN
    dA alone (T is given), a base row of NaN dX alone."""
    q, t = _q(), h.torch()
    L = _Layer(M, 256, N, 8)
    _, T = q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, L.alpha)
    run = lambda dY, X, W: q.linear_bwd_int8(dY, X, W, L.dA, L.dB, L.alpha, T=T)
    dX, dA, dB = run(L.ddY, L.X, L.W)
    dY = L.ddY.clone()
    dY[1, 9] = float("inf")
    gX, gA, gB = run(dY, L.X, L.W)
    keep = [m for m in range(M) if m != 1]
    cols = [n for n in range(N) if n != 9]
    assert t.equal(gX[keep], dX[keep]) and not bool(gX[1].isfinite().any())
    assert not bool(gA.isfinite().any()) and t.equal(gB[cols], dB[cols]) and not bool(gB[9].isfinite().any())
    xs = L.X.scale.clone()
    xs[1] = float("nan")
    gX, gA, gB = run(L.ddY, q.Int8Tensor(L.X.codes, xs), L.W)
    assert t.equal(gX, dX) and t.equal(gB, dB) and bool(gA.isnan().all())
    ws = L.W.scale.clone()
    ws[N - 1] = float("nan")
    gX, gA, gB = run(L.ddY, L.X, q.Int8Tensor(L.W.codes, ws))
    assert bool(gX.isnan().all()) and t.equal(gA, dA) and t.equal(gB, dB)


@pytest.mark.parametrize("base,K,N", [("int8", 32768, 32760), ("nf4", 65536, 65528)])
def test_input_gradient_of_the_largest_bases(base, K, N):
    """Weights just under the size limits, against sampled features."""
    q, t = _q(), h.torch()
    if t.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GiB of free memory")
    M, r = 9, 8
    g = t.Generator("cuda")
    g.manual_seed(K)
    W0 = t.empty(N, K, device="cuda").normal_(std=0.02, generator=g)
    cols = [0, 63, 64, 257, K // 2 + 5, K - 1]
    W = q.int8_quantize(W0) if base == "int8" else q.quantize(W0)
    del W0
    rnd = lambda *s: t.randn(*s, device="cuda", generator=g)
    X, A, B = q.int8_quantize(rnd(M, K).bfloat16()), (rnd(r, K) / 32).bfloat16(), (rnd(N, r) / 16).bfloat16()
    dY, T = rnd(M, N).bfloat16(), rnd(M, r)
    dX = q.linear_bwd_int8(dY, X, W, A, B, 2.0 * r, T=T if base == "int8" else T.bfloat16())[0]
    v = W.codes[:, cols].double() * W.scale.double()[:, None] if base == "int8" else q.nf4_dequant(W)[:, cols].double()
    U, absU = dY.double() @ B.double(), dY.double().abs() @ B.double().abs()
    a = A[:, cols].double()
    ref = dY.double() @ v + 2.0 * U @ a
    # the bound of test_input_gradient
    tol = dY.double().abs() @ v.abs() * (BF + (N + 40) * 2 * F32) + 2.0 * (
        absU * ((N + 16) * 2 * F32 + 2 * BF + BF * BF + 4 * r * F32)) @ a.abs()
    err = (dX[:, cols].double() - ref).abs() - ref.abs() * BF - tol * (1 + BF)
    assert float(err.max()) <= 0.0, float(err.max())
    # and not only within the bound: the errors are independent roundings
    assert float((dX[:, cols].double() - ref).norm() / ref.norm()) <= 2 * BF


def test_gradient_against_differences():
    """dA and dB of L = sum(dY Y) against differences of the forward's formula in
    64 bits (L is linear in A and in B alone, so a difference is exact)."""
    q = _q()
    L = _Layer(40, 256, 72, 8)
    _, T = q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, L.alpha)
    _, dA, dB = q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha, T=T)
    X, A, B, dY = L.x(), h.f64(L.A), h.f64(L.B), h.f64(L.dY)
    f = lambda a, b: float((dY * (L.s * (X @ a.T) @ b.T)).sum())
    g = np.random.default_rng(1)
    for got, at in ((h.host(dA), 0), (h.host(dB), 1)):
        for _ in range(12):
            i = tuple(g.integers(0, n) for n in got.shape)
            d = np.zeros(got.shape)
            d[i] = 1.0
            num = (f(A + d, B) - f(A - d, B)) / 2 if at == 0 else (f(A, B + d) - f(A, B - d)) / 2
            # one value of an fp32 sum over 40 tokens: far below 1e-4 of the gradient's size
            assert abs(got[i] - num) <= 1e-4 * np.abs(got).max()


def test_outputs_that_overlap_are_refused():
    q, t = _q(), h.torch()
    L = _Layer(32, 64, 64, 64)
    with pytest.raises(ValueError, match="overlaps"):
        q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, 1.0, out=L.dB.reshape(-1)[: 32 * 64].reshape(32, 64))
    with pytest.raises(ValueError, match="overlaps"):
        q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, 1.0, dX_out=L.ddY.reshape(32, 64))
    o = t.empty(64, 64, device="cuda")
    with pytest.raises(ValueError, match="overlaps"):
        q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, 1.0, dA_out=o, dB_out=o)


def test_small_workspace_is_refused():
    q, t = _q(), h.torch()
    L = _Layer(32, 64, 64, 8)

    class Small:
        def get(self, nbytes, stream=None):
            return t.empty(nbytes - 1, dtype=t.uint8, device="cuda"), nbytes - 1

    with pytest.raises(q.QLoRAError, match="workspace"):
        q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, 1.0, workspace=Small())
    with pytest.raises(q.QLoRAError, match="workspace"):
        q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, 1.0, workspace=Small())


@pytest.mark.parametrize("M", [4, 160])
def test_mlp_block_captured_and_replayed(M):
    """Gate and up projections, gating, down projection and the whole backward, all
    in 8 bits: eager against the formulas step by step, then captured once and
    replayed on other inputs."""
    q, t = _q(), h.torch()
    K, I, r = 256, 448, 8
    g = t.Generator("cuda")
    g.manual_seed(M)
    rnd = lambda *s, std=1.0: t.randn(*s, device="cuda", generator=g) * std
    Wg, Wu, Wd = (q.int8_quantize(rnd(*s, std=0.06)) for s in ((I, K), (I, K), (K, I)))
    lo = [(rnd(r, i, std=0.06).bfloat16(), rnd(o, r, std=0.1).bfloat16()) for o, i in ((I, K), (I, K), (K, I))]
    x, dy = rnd(M, K).bfloat16(), rnd(M, K).bfloat16()

    def step():
        X = q.int8_quantize(x)
        G, Tg = q.linear_fwd_int8(X, Wg, *lo[0], 16.0)
        U, Tu = q.linear_fwd_int8(X, Wu, *lo[1], 16.0)
        H, G8, U8 = q.silu_mul_fwd_int8(G, U)
        Y, Td = q.linear_fwd_int8(H, Wd, *lo[2], 16.0)
        dH, dAd, dBd = q.linear_bwd_int8(dy, H, Wd, *lo[2], 16.0, T=Td)
        dG, dU = q.silu_mul_bwd_int8(dH, G8, U8)
        dX, dAg, dBg = q.linear_bwd_int8(dG, X, Wg, *lo[0], 16.0, T=Tg)
        dX, dAu, dBu = q.linear_bwd_int8(dU, X, Wu, *lo[1], 16.0, T=Tu, accumulate_into=dX)
        return [Y, dX, dAg, dBg, dAu, dBu, dAd, dBd, X.codes, X.scale, H.codes, H.scale, G8.codes, U8.codes]

    got = step()
    f = lambda v: v.double()
    val = lambda c, s: c.double() * s.double()[:, None]

    def ref():
        """The same block in 64 bits from the unquantised input."""
        W = [val(*w) for w in (Wg, Wu, Wd)]
        A, B = [f(a) for a, _ in lo], [f(b) for _, b in lo]
        G = f(x) @ W[0].t() + 2.0 * f(x) @ A[0].t() @ B[0].t()
        U = f(x) @ W[1].t() + 2.0 * f(x) @ A[1].t() @ B[1].t()
        p = t.sigmoid(G)
        H = G * p * U
        Y = H @ W[2].t() + 2.0 * H @ A[2].t() @ B[2].t()
        dH = f(dy) @ W[2] + 2.0 * f(dy) @ B[2] @ A[2]
        dG, dU = dH * U * (p + G * p * (1 - p)), dH * G * p
        dX = sum(d @ W[i] + 2.0 * d @ B[i] @ A[i] for i, d in ((0, dG), (1, dU)))
        return [Y, dX] + [v for i, (d, X) in enumerate(((dG, f(x)), (dU, f(x)), (f(dy), H)))
                          for v in (2.0 * (d @ B[i]).t() @ X, 2.0 * d.t() @ (X @ A[i].t()))]

    # A stored row is within half a step, scale / 2 <= max / 254 of each value; on
    # rows of K normal values (max / rms about 3.2) that is 3.2 / 254 / sqrt(3) =
    # 0.8 % of the row in the 2-norm, and H's heavier tails (max / rms up to 12)
    # 2.8 %.  A gradient passes at most three such stores.
    for name, a, b in zip(("Y", "dX", "dAg", "dBg", "dAu", "dBu", "dAd", "dBd"), got, ref()):
        rel = float((a.double() - b).norm() / b.norm())
        h.log(f"  {name}: {rel:.3e}")
        assert rel <= 0.06, (name, rel)

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        held = step()
    for k in range(3):
        x.copy_(rnd(M, K).bfloat16())
        dy.copy_(rnd(M, K).bfloat16())
        graph.replay()
        t.cuda.synchronize()
        replayed = [v.clone() for v in held]
        for a, b in zip(replayed, step()):
            assert t.equal(a, b)


@pytest.mark.parametrize("M,N", [(20, 264), (20, 512), (200, 512), (300, 264)])
def test_backward_on_other_bases_captured_and_replayed(M, N):
    """An NF4 and a bf16 base at token counts that decode it in dX's tile and that
    copy it, captured in two graphs that share a Workspace and are replayed in turn."""
    q, t = _q(), h.torch()
    K, r = 320, 8
    g = t.Generator("cuda")
    g.manual_seed(M + N)
    rnd = lambda *s: t.randn(*s, device="cuda", generator=g)
    W0 = 0.05 * rnd(N, K)
    A, B = (0.06 * rnd(r, K)).bfloat16(), (0.1 * rnd(N, r)).bfloat16()
    x, dY, T, dX0 = rnd(M, K).bfloat16(), rnd(M, N).bfloat16(), rnd(M, r).bfloat16(), rnd(M, K).bfloat16()
    X, ws = q.int8_quantize(x), q.Workspace()

    def step(W, acc):
        return q.linear_bwd_int8(dY, X, W, A, B, 16.0, T=T, accumulate_into=acc, workspace=ws)

    graphs = []
    for W in (q.quantize(W0), W0.bfloat16()):
        acc = dX0.clone()
        side = t.cuda.Stream()
        side.wait_stream(t.cuda.current_stream())
        with t.cuda.stream(side):
            step(W, acc.clone())
        t.cuda.current_stream().wait_stream(side)
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            held = step(W, acc)
        graphs.append((W, acc, graph, held))
    for k in range(3):
        dY.copy_(rnd(M, N).bfloat16())
        T.copy_(rnd(M, r).bfloat16())
        q.int8_quantize(rnd(M, K).bfloat16(), codes_out=X.codes, scale_out=X.scale)
        for W, acc, graph, held in graphs:
            acc.copy_(dX0)
            graph.replay()
            got = [v.clone() for v in held]
            for a, b in zip(got, q.linear_bwd_int8(dY, X, W, A, B, 16.0, T=T, accumulate_into=dX0.clone())):
                assert t.equal(a, b)


def test_workspace_that_grows_after_a_capture():
    """The graph's scratch memory stays its own when a later call needs more."""
    q, t = _q(), h.torch()
    L, big = _Layer(24, 256, 136, 8), _Layer(600, 512, 264, 64)
    ws = q.Workspace()
    run = lambda: q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha, workspace=ws)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        run()
    t.cuda.current_stream().wait_stream(side)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        held = run()
    n, at = ws.buf.numel(), ws.buf.data_ptr()
    q.linear_bwd_int8(big.ddY, big.X, big.W, big.dA, big.dB, big.alpha, workspace=ws)
    t.cuda.synchronize()
    assert ws.buf.numel() > n
    others = [t.full((n,), 77, dtype=t.uint8, device="cuda") for _ in range(8)]
    assert all(o.data_ptr() != at for o in others)
    graph.replay()
    t.cuda.synchronize()
    assert all(bool((o == 77).all()) for o in others)
    for a, b in zip(held, q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha)):
        assert t.equal(a, b)


def test_rows_past_32_bit_offsets():
    """Elementwise calls on more than 2^31 elements: sampled rows equal the same
    rows by themselves."""
    q, t = _q(), h.torch()
    M, I = 66000, 32768                              # 2.16e9 elements
    if t.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GiB of free memory")
    g = t.Generator("cuda")
    g.manual_seed(5)
    rows = [0, 65534, 65535, 65536, 65537, M - 1]
    rnd = lambda: t.empty(M, I, dtype=t.bfloat16, device="cuda").normal_(generator=g)
    G, U = rnd(), rnd()
    H, G8, U8 = q.silu_mul_fwd_int8(G, U)
    want = q.silu_mul_fwd_int8(G[rows].contiguous(), U[rows].contiguous())
    for a, b in zip((H, G8, U8), want):
        assert t.equal(a.codes[rows], b.codes) and t.equal(a.scale[rows], b.scale)
    del H
    dG, dU = q.silu_mul_bwd_int8(G, G8, U8)
    wG, wU = q.silu_mul_bwd_int8(G[rows].contiguous(), want[1], want[2])
    assert t.equal(dG[rows], wG) and t.equal(dU[rows], wU)
    del dG, dU, G8, U8, U
    X = q.int8_quantize(G)
    one = q.int8_quantize(G[rows].contiguous())
    assert t.equal(X.codes[rows], one.codes) and t.equal(X.scale[rows], one.scale)
    assert t.equal(q.int8_dequant(X, out=G)[rows], q.int8_dequant(one))


def test_two_streams_at_once():
    q, t = _q(), h.torch()
    layers = [_Layer(200, 512, 520, 16, seed=k) for k in range(2)]
    want = [(q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, L.alpha)[0],
             *q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha)) for L in layers]
    streams = [t.cuda.Stream() for _ in layers]
    t.cuda.synchronize()
    got = [None, None]
    for _ in range(4):
        for k, (L, s) in enumerate(zip(layers, streams)):
            with t.cuda.stream(s):
                got[k] = (q.linear_fwd_int8(L.X, L.W, L.dA, L.dB, L.alpha)[0],
                          *q.linear_bwd_int8(L.ddY, L.X, L.W, L.dA, L.dB, L.alpha))
        t.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(t.equal(u, v) for u, v in zip(a, b))
