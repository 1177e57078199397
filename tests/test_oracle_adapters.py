"""Pins of the oracle's adapters of many requests: the plan's invariants, the
one-slot case against the single-adapter layer, every gradient against central
differences (exact here up to rounding: the outputs are linear in each
operand), the dropout mask held fixed."""
import numpy as np
import pytest

import oracle


def _case(seed, M, K, N, r, S):
    g = np.random.default_rng(seed)
    return (g.standard_normal((M, K)), g.standard_normal((M, N)), g.standard_normal((S, r, K)),
            g.standard_normal((S, N, r)), g.uniform(0.5, 2.0, S).astype(np.float32),
            g.integers(-1, S, M))


@pytest.mark.parametrize("lengths,slots,M,S", [
    ([1], [0], 1, 1), ([0, 3, 0, 70], [1, 0, 0, 1], 80, 2), ([5, 5], [7, -3], 10, 2),
    ([9, 9, 9], [0, 1, 0], 20, 3), ([-4, 6], [0, 0], 6, 1), ([], [], 5, 4)])
def test_plan_invariants(lengths, slots, M, S):
    tok, order, start, tiles = oracle.adapter_plan(lengths, slots, M, S)
    assert sorted(order.tolist()) == list(range(M))
    assert start[0] == 0 and start[-1] == M and len(start) == S + 2
    for a in range(S + 1):
        part = order[start[a]:start[a + 1]]
        assert np.all(tok[part] == (a if a < S else -1)) and np.all(np.diff(part) > 0)
    used = tiles[tiles[:, 2] > 0]
    covered = np.concatenate([np.arange(f, f + n) for _, f, n in used]) if len(used) else []
    assert np.array_equal(covered, np.arange(M))
    assert np.all(used[:, 2] <= 64)
    for a, f, n in used:
        assert np.all(tok[order[f:f + n]] == a)


def test_one_slot_is_the_single_adapter():
    X, dY, A, B, scale, _ = _case(1, 12, 32, 24, 4, 1)
    tok = np.zeros(12, int)
    out, T = oracle.adapters_forward(X, None, A, B, scale, tok)
    W = np.zeros((24, 32))
    alpha = float(scale[0]) * 4
    Y1, T1 = oracle.forward(X, W, A[0], B[0], alpha, 4)
    assert np.allclose(out, Y1, rtol=1e-12) and np.allclose(T, T1, rtol=1e-12)
    got = oracle.adapters_backward(dY, X, A, B, scale, tok)
    ref = oracle.backward(dY, X, W, A[0], B[0], alpha, 4)
    for a, b in zip(got, ref):
        assert np.allclose(a.reshape(b.shape), b, rtol=1e-12)


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_gradients_against_differences(p):
    M, K, N, r, S = 7, 16, 8, 3, 3
    X, dY, A, B, scale, tok = _case(2, M, K, N, r, S)
    mask = oracle.dropout_mask(M, K, p, 99) if p else None
    dX, dA, dB = oracle.adapters_backward(dY, X, A, B, scale, tok, mask=mask, p=p)

    def loss(X, A, B):
        out, _ = oracle.adapters_forward(X, None, A, B, scale, tok, mask=mask, p=p)
        return float((out * dY).sum())

    g = np.random.default_rng(3)
    for name, ops, grad, at in (("X", (X, A, B), dX, 0), ("A", (X, A, B), dA, 1),
                                ("B", (X, A, B), dB, 2)):
        d = g.standard_normal(ops[at].shape)
        plus, minus = list(ops), list(ops)
        plus[at], minus[at] = ops[at] + d, ops[at] - d
        diff = (loss(*plus) - loss(*minus)) / 2     # linear in each operand: exact
        assert abs(diff - float((grad * d).sum())) <= 1e-10 * max(1.0, abs(diff)), name


def test_no_adapter_leaves_the_base():
    X, dY, A, B, scale, _ = _case(4, 5, 16, 8, 2, 2)
    tok = np.full(5, -1)
    Y = np.ones((5, 8))
    out, T = oracle.adapters_forward(X, Y, A, B, scale, tok)
    assert np.array_equal(out, Y) and not T.any()
    dX, dA, dB = oracle.adapters_backward(dY, X, A, B, scale, tok, dX0=X)
    assert np.array_equal(dX, X) and not dA.any() and not dB.any()
