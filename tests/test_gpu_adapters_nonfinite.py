"""Infinities, NaN and values next to the largest in the batched adapters, on
the GPU: T and U enter the matrix products as sums of bf16 terms, and the
products have to be what the formulas give in 64 bits for them, not what the
terms' own infinities or signs would make of them.

Finite values are compared within 2^-7 of the sum of absolute values: a
rounding to bf16 (2^-8), the terms (2^-16) and fp32 sums of up to 300 products
(300 2^-23 < 2^-14)."""
import numpy as np
import pytest

import qlora_workloads as wl
from gpu_helpers import dev_bf16, dev_f32, f64, host, host_bf16_f64, log
from test_gpu_adapters import Case

pytestmark = pytest.mark.gpu
t = pytest.importorskip("torch")

BF16_MAX = (2 - 2.0 ** -7) * 2.0 ** 127


def bits(a):
    return wl.round_to_bf16_bits(np.asarray(a, np.float32))


def put(c, **operands):
    for k, v in operands.items():
        setattr(c, k, v)
        c.d[k] = dev_f32(v) if k == "scale" else dev_bf16(v)


def same(name, got, want, sums):
    """Infinities and NaN where `want`, rounded to the output's type, has them,
    finite values within 2^-7 of `sums`."""
    got = np.asarray(got, np.float64)
    if name in ("out", "dX"):    # half a step above bf16's largest rounds to an infinity
        with np.errstate(invalid="ignore"):
            want = np.where(np.abs(want) >= BF16_MAX + 2.0 ** 119, np.sign(want) * np.inf, want)
    for kind, f in (("NaN", np.isnan), ("+inf", np.isposinf), ("-inf", np.isneginf)):
        bad = f(got) != f(want)
        assert not bad.any(), f"{name}: {kind} differs at {int(bad.sum())} of {bad.size}"
    ok = np.isfinite(want)
    assert np.all(np.abs(got - np.where(ok, want, 0))[ok] <= (2.0 ** -7 * sums + 2.0 ** -120)[ok]), name


def formulas(c, T, base=True):
    """(out, dX, dA, dB) and their sums of absolute values, in 64 bits, from the
    T that the forward gave."""
    X, Y, dY, A, B = (f64(getattr(c, k)) for k in ("X", "Y", "dY", "A", "B"))
    out, dX = Y.copy(), f64(c.dX0).copy()
    so, sx = np.abs(out), np.abs(dX)
    dA, dB, sa, sb = (np.zeros(v.shape) for v in (A, B, A, B))
    keep = c.keep if c.mask is None else c.mask * c.keep
    Xd = X * c.keep if c.mask is None else np.where(c.mask, X, 0.0) * c.keep
    with np.errstate(invalid="ignore", over="ignore"):
        for a in range(c.S):
            m = np.flatnonzero(c.tok == a)
            if not len(m):
                continue
            s = float(c.scale[a])
            U = dY[m] @ B[a]
            out[m] += s * (T[m] @ B[a].T)
            so[m] += s * (np.abs(T[m]) @ np.abs(B[a]).T)
            term, sterm = s * (U @ A[a]), s * (np.abs(U) @ np.abs(A[a]))
            if c.mask is not None:    # a dropped element has no gradient, whatever it would be
                term, sterm = (np.where(c.mask[m], v, 0.0) * c.keep for v in (term, sterm))
            dX[m] += term
            sx[m] += sterm
            dA[a], sa[a] = s * (U.T @ Xd[m]), s * (np.abs(U).T @ np.abs(Xd[m]))
            dB[a], sb[a] = s * (dY[m].T @ T[m]), s * (np.abs(dY[m]).T @ np.abs(T[m]))
    return (out, dX, dA, dB), (so, sx, sa, sb)


def check(c, T=None):
    out, Tg = c.fwd()
    if T is not None:
        Tg = dev_f32(np.asarray(T, np.float32))
    dX, dA, dB = c.bwd(Tg)
    t.cuda.synchronize()
    Th = host(Tg).astype(np.float64)
    want, sums = formulas(c, Th)
    got = (host_bf16_f64(out), host_bf16_f64(dX), host(dA), host(dB))
    for name, g, w, s in zip(("out", "dX", "dA", "dB"), got, want, sums):
        if name == "out" and T is not None:
            continue
        same(name, g, w, s)
    return want


RANKS = [8, 16, 24, 64, 72]     # one per form of the kernels
TOKENS = [3, 50]                # a narrow tile, a wide one


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("n", TOKENS)
def test_values_above_bf16s_largest(n, r):
    """A finite T or U whose rounding to bf16 would be infinite: the products
    with 2^-20 are finite."""
    log(f"[adapters] near the largest n={n} r={r}")
    M, K, N = n + 2, 64, 72
    c = Case([n], [0], M, K, N, r, 1)
    A, B = np.zeros((1, r, K)), np.full((1, N, r), 2.0 ** -20)
    X, dY = np.zeros((M, K)), np.zeros((M, N))
    # T[m, 1] and U[m, 1] between bf16's largest and fp32's largest
    X[:, 0], X[:, 1] = BF16_MAX, 1.5 * 2.0 ** 119
    A[0, 1, 0] = A[0, 1, 1] = 1.0
    A[0, :, 2] = 2.0 ** -20
    X[:, 2] = 2.0 ** -20
    dY[:, 0], dY[:, 1] = -BF16_MAX, -1.5 * 2.0 ** 119
    dY[:, 2] = 2.0 ** -20
    B[0, :2] = 0.0
    B[0, :2, 1] = 1.0
    B[0, 2:, 1] = 2.0 ** -20
    put(c, X=bits(X), dY=bits(dY), A=bits(A), B=bits(B), scale=np.ones(1, np.float32))
    # X and T so large times dY would leave fp32: the gradients of small X, T
    T = host(c.fwd()[1])
    assert np.all(np.isfinite(T)) and np.all(T[:n, 1] > BF16_MAX)
    out, _ = c.fwd()
    want, sums = formulas(c, T.astype(np.float64))
    o = host_bf16_f64(out)
    same("out", o[:, 2:], want[0][:, 2:], sums[0][:, 2:])
    X[:, :2] = 2.0 ** -20
    put(c, X=bits(X))
    check(c)
    small = np.full((M, r), 2.0 ** -20)
    dY[:] = 2.0 ** -20
    small[:, 1] = BF16_MAX + 2.0 ** 119 + 2.0 ** 118
    assert np.all(np.float32(small[:, 1]) < np.inf)
    put(c, dY=bits(dY))
    check(c, T=small)


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("n", TOKENS)
def test_infinite_operands(n, r, p):
    """Infinities in B, A, dY and X of tokens that also have ordinary values:
    each product with a term is infinite with the sign of T or U."""
    log(f"[adapters] infinite operands n={n} r={r} p={p}")
    M, K, N = n + 2, 72, 136
    e = np.random.default_rng([n, r])
    for which in ("B", "A", "dY", "X"):
        c = Case([n], [1], M, K, N, r, 2, p=p, seed=21)
        T = host(c.fwd()[1])
        v = getattr(c, which).copy()
        inf = np.array([0x7F80, 0xFF80], np.uint16)
        if which in ("A", "B"):
            at = (1, slice(0, None, 5), int(e.integers(r))) if which == "B" else \
                 (1, int(e.integers(r)), slice(0, None, 5))
        else:
            at = (int(e.integers(n)), slice(0, None, 5))
        v[at] = e.choice(inf, v[at].shape)
        put(c, **{which: v})
        check(c, T=None if which == "B" else T)


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("n", TOKENS)
def test_terms_that_would_be_zero(n, r):
    """T and U that bf16 holds exactly (whole numbers below 256, zeros among
    them) against infinities: infinite unless the number is zero, then NaN."""
    log(f"[adapters] exact T and U n={n} r={r}")
    M, K, N = n + 2, 64, 72
    e = np.random.default_rng([n, r, 2])
    inf = np.array([0x7F80, 0xFF80], np.uint16)
    c = Case([n], [0], M, K, N, r, 1)
    X, dY = np.zeros((M, K)), np.zeros((M, N))
    A, B = np.zeros((1, r, K)), np.zeros((1, N, r))
    for j in range(r):
        A[0, j, j % 8], B[0, j % 8, j] = 1 + j % 3, 1 + j % 3
    X[:, :8], dY[:, :8] = e.integers(-3, 4, (M, 8)), e.integers(-3, 4, (M, 8))
    put(c, X=bits(X), dY=bits(dY), A=bits(A), B=bits(B))
    T = host(c.fwd()[1])
    assert (T[:n] == 0).any() and (T[:n] != 0).any() and np.all(T == np.rint(T))
    check(c)
    for which, at in (("B", (0, slice(8, None, 3), int(e.integers(r)))),
                      ("A", (0, int(e.integers(r)), slice(8, None, 3))),
                      ("dY", (1, slice(8, None, 3))), ("X", (1, slice(8, None, 3)))):
        d = Case([n], [0], M, K, N, r, 1)
        put(d, X=c.X, dY=c.dY, A=c.A, B=c.B)
        v = getattr(d, which).copy()
        v[at] = e.choice(inf, v[at].shape)
        put(d, **{which: v})
        check(d, T=None if which == "B" else T)


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("n", TOKENS)
def test_infinite_T_and_U(n, r):
    """One infinity in a token's input: T and U are infinite, and their products
    with infinite, finite and zero values are the formulas'."""
    log(f"[adapters] infinite T and U n={n} r={r}")
    M, K, N = n + 2, 64, 72
    c = Case([n], [0], M, K, N, r, 1)
    # operands of one sign, so that infinities do not cancel
    A, B = np.abs(f64(c.A)) + 2.0 ** -6, np.abs(f64(c.B)) + 2.0 ** -6
    A[0, :, 7], B[0, 9] = 0.0, 0.0
    A[0, 1, 12], B[0, 14, 1] = np.inf, np.inf
    X, dY = f64(c.X).copy(), f64(c.dY).copy()
    X[0, 3], X[2, 5], dY[1, 4], dY[2, 6] = np.inf, -np.inf, np.inf, -np.inf
    put(c, X=bits(X), dY=bits(dY), A=bits(A), B=bits(B))
    check(c)
    A[0, 1, 12], B[0, 14, 1] = 0.5, 0.5
    put(c, A=bits(A), B=bits(B))
    T = host(c.fwd()[1])
    assert np.all(np.isposinf(T[0])) and np.all(np.isneginf(T[2]))
    check(c)


def test_nan_payloads_stay_nan():
    """A NaN whose payload lies in the low half of its bits alone (a T given by
    the caller) is no infinity."""
    c = Case([3], [0], 5, 64, 72, 8, 1)
    T = c.fwd()[1].clone()
    T.view(t.int32)[1, 2] = 0x7F800001
    _, _, dB = c.bwd(T)
    t.cuda.synchronize()
    assert np.all(np.isnan(host(dB)[0][:, 2]))
    assert np.all(np.isfinite(np.delete(host(dB)[0], 2, axis=1)))
