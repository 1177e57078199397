"""dX of the backward from kept 8-bit inputs, where the bounds can be tight: inputs
on which every rounding but the last is exact or is made in the reference as well."""
import numpy as np
import pytest

import gpu_helpers as h

pytestmark = pytest.mark.gpu

F32, BF = 2.0 ** -24, 2.0 ** -8


def _q():
    import bit_nf4_quantized_07_amd as q
    return q


def _no_base(kind, N, K):
    """A base of zeros."""
    q, t = _q(), h.torch()
    if kind == "int8":
        return q.Int8Tensor(t.zeros(N, K, dtype=t.int8, device="cuda"), t.zeros(N, device="cuda"))
    if kind == "bf16":
        return t.zeros(N, K, dtype=t.bfloat16, device="cuda")
    return q.quantize(t.zeros(N, K, device="cuda"))


@pytest.mark.parametrize("kind", ["int8", "nf4", "bf16"])
@pytest.mark.parametrize("M,K,N,r", [(3, 128, 72, 8), (40, 320, 512, 40), (200, 192, 264, 16), (200, 256, 512, 24),
                                     (600, 320, 264, 8), (600, 256, 512, 64), (700, 192, 768, 3)])
def test_adapter_term_is_rounded_once(kind, M, K, N, r):
    """With s = 1.5 and powers of two in U, s U is a bf16 value and 1.5 A is not: what
    is left is the sum in fp32 and dX's own rounding."""
    q, t = _q(), h.torch()
    g = np.random.default_rng([M, K, N, r])
    A = h.dev_f32(g.uniform(-1, 1, (r, K))).bfloat16()
    B = h.dev_f32(np.ldexp(g.choice([-1.0, 1.0], (N, r)), g.integers(-3, 4, (N, r)))).bfloat16()
    pick = g.integers(0, N, M)                        # a token's dY is 1 at one output
    dY = t.zeros(M, N, dtype=t.bfloat16, device="cuda")
    dY[t.arange(M), t.from_numpy(pick)] = 1.0
    X = q.int8_quantize(h.dev_f32(g.standard_normal((M, K))).bfloat16())
    dX = q.linear_bwd_int8(dY, X, _no_base(kind, N, K), A, B, 1.5 * r)[0].double()
    U = B.double()[t.from_numpy(pick).cuda()]
    ref, mag = 1.5 * U @ A.double(), 1.5 * U.abs() @ A.double().abs()
    # r products, exact in fp32, summed in up to two halves (a step may cut)
    err = (dX - ref).abs() - ref.abs() * BF - mag * (r + 2) * 2 * F32 * (1 + BF)
    assert float(err.max()) <= 0.0, float(err.max())
