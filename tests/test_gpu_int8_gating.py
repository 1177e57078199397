"""The gating in 8 bits where the sigmoid is near the smallest normal number."""
import numpy as np
import pytest

from oracle import int8 as o8

import gpu_helpers as h

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24
# the fast exponential: its argument's rounding (89 log2 e = 129 2^-24 of the result),
# v_exp_f32 within 2^-22; the sum, the reciprocal and the products three each
GATE = (129 + 4 + 9) * F32


@pytest.mark.parametrize("M,I", [(3, 64), (5, 1088), (2, 11008), (1, 65600)])
def test_rows_of_the_smallest_sigmoids(M, I):
    import bit_nf4_quantized_07_amd as q
    g = np.random.default_rng([M, I])
    G = h.dev_f32(g.uniform(-88.5, -87.5, (M, I))).bfloat16()
    U = h.dev_f32(g.uniform(-1, 1, (M, I)) * 2.0 ** 20).bfloat16()
    Gv, Uv = h.host_bf16_f64(G), h.host_bf16_f64(U)
    assert Gv.min() > -88.7 and Gv.max() < -87.4       # exp(-g) finite, the sigmoid subnormal
    H, _, _ = q.silu_mul_fwd_int8(G, U)
    ref = o8.silu(Gv) * Uv
    a = np.abs(ref).max(1)
    assert np.all(np.abs(h.host(H.scale) - a / 127.0) <= a / 127.0 * (GATE + F32))
    n = 127.0 * ref / a[:, None]
    # half a step, and up to 127 times the value's and the maximum's own error
    assert np.abs(h.host(H.codes) - n).max() <= 0.5 + 127 * (2 * GATE + 2 * F32)
