"""The layer on 8-bit rows just under its size limits, over whole numbers."""
import pytest

import gpu_helpers as h
from test_gpu_int8_whole import Whole, _check

pytestmark = pytest.mark.gpu


def _room():
    if h.torch().cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GiB of free memory")


FWD = [(9, 32768, 65528, 8), (40, 32768, 65528, 8),        # the weight's codes
       (65528, 32768, 8, 8),                               # X's codes
       (65528, 64, 16376, 8),                              # Y
       (2097151, 64, 8, 256),                              # T, and the operands made of it
       (3, 64, 4194296, 256), (20, 64, 4194296, 256)]      # B


@pytest.mark.parametrize("M,K,N,r", FWD)
def test_forward(M, K, N, r):
    _room()
    L = Whole(M, K, N, r)
    (Y, T), (low, high), refT = L.forward()
    assert L.t.equal(T, refT)
    assert bool(((low <= Y) & (Y <= high)).all())


@pytest.mark.parametrize("M", [3, 40])
def test_the_longest_whole_sums(M):
    """127^2 2^17, the largest sum of codes that 32 bits are to hold."""
    import bit_nf4_quantized_07_amd as q
    t = h.torch()
    K, N = 1 << 17, 136
    full = lambda n: q.Int8Tensor(t.full((n, K), 127, dtype=t.int8, device="cuda"), t.ones(n, device="cuda"))
    X, W = full(M), full(N)
    X.codes[1] = -127
    Y, _ = q.linear_fwd_int8(X, W)
    want = t.full((M, N), 127.0 * 127.0 * K, device="cuda")
    want[1] = -want[1]
    assert t.equal(Y, want.bfloat16())


BWD = [(32760, 32768, 8, 8, "int8"),                       # dX
       (65528, 64, 16376, 8, "bf16"),                      # dY
       (2097151, 64, 8, 256, "int8"),                      # U's and T's terms
       (3, 64, 4194296, 256, "nf4"), (20, 64, 4194296, 256, "bf16"),   # B and dB
       (9, 32768, 32760, 8, "bf16"), (200, 32768, 32760, 8, "bf16")]   # a bf16 base


@pytest.mark.parametrize("M,K,N,r,base", BWD)
def test_backward(M, K, N, r, base):
    _room()
    active = None if M < 300 else [0, 31, 32, M // 2, M - 33, M - 1] + list(range(65, M, M // 10))[:10]
    L = Whole(M, K, N, r, base, active)
    g = L.t.Generator("cuda")
    g.manual_seed(N)
    T = L.t.randint(-8, 9, (M, r), device="cuda", generator=g)
    T = T.to(L.t.float32 if base == "int8" else L.t.bfloat16)
    _check(L, L.q.linear_bwd_int8(L.dY, L.X, L.W, L.A, L.B, L.alpha, T=T), L.backward(T), "")
