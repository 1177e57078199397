"""The layer on 8-bit rows over whole numbers: every product and sum is exact in fp32
in any order, and what is rounded to bf16 on the way is rounded alike here.  T and dX
are equal to the reference, value by value; Y, dA and dB are but for what the terms
leave that T and U go in as.  A column, a row, a split or a rank that is left out,
taken twice or from another place shows as such.

What the terms leave: a term that would be zero is 2^-40 of the value, so that a
product is off by less than 2^-39 of itself, and a sum that takes it in may lose its
last place, 2^-23 of the magnitudes at most, once for each product of each term
(products with zero are zero and lose nothing).  For n products in k terms: (k n + 8)
2^-23 of the magnitudes' sum.  The rounding to bf16 is monotonic, so that Y lies
between the roundings of the exact value that much lower and higher.
"""
import pytest

import gpu_helpers as h

pytestmark = pytest.mark.gpu

S = 1.5                 # alpha / r
TOP = 2.0 ** 23         # what is below it stays exact times S in fp32


def left(terms, products):
    return (terms * products + 8) * 2.0 ** -23


class Whole:
    """Inputs of a layer: codes in [-3, 3] with scale 1, 2 or 1/2 per row, weights of
    -1, 0 and 1 (codes up to 3 on an 8-bit base), A and B of -1, 0 and 1."""

    def __init__(self, M, K, N, r, base="int8", active=None):
        import bit_nf4_quantized_07_amd as q
        t = h.torch()
        g = t.Generator("cuda")
        g.manual_seed(M * 31 + K * 7 + N * 3 + r)
        ints = lambda lo, hi, *s: t.randint(lo, hi + 1, s, device="cuda", generator=g)
        two = lambda n: t.pow(2.0, ints(-1, 1, n).float())
        self.t, self.q, self.alpha = t, q, S * max(r, 1)
        self.X = q.Int8Tensor(ints(-3, 3, M, K).to(t.int8), two(M))
        self.x = self.X.codes.double() * self.X.scale.double()[:, None]
        if base == "int8":
            self.W = q.Int8Tensor(ints(-3, 3, N, K).to(t.int8), two(N))
            self.w = self.W.codes.double() * self.W.scale.double()[:, None]
        elif base == "bf16":
            self.W = ints(-1, 1, N, K).bfloat16()
            self.w = self.W.double()
        else:           # levels 0, 7 and 15 are -1, 0 and 1; code 127 leaves a constant its mean
            nib = t.tensor([0, 7, 15], device="cuda", dtype=t.uint8)[ints(0, 2, N * K // 2, 2)]
            nb = N * K // 64
            self.W = q.QuantizedWeight((nib[:, 0] * 16 + nib[:, 1]).contiguous(),
                                       t.full((nb,), 127, dtype=t.uint8, device="cuda"),
                                       t.ones((nb + 255) // 256, device="cuda"),
                                       t.ones(1, device="cuda"), N, K)
            self.w = q.nf4_dequant(self.W).double()
            assert set(self.w.unique().tolist()) <= {-1.0, 0.0, 1.0}
        self.A, self.B = ints(-1, 1, r, K).bfloat16(), ints(-1, 1, N, r).bfloat16()
        self.dY = ints(-2, 2, M, N).bfloat16()
        if active is not None:          # tokens whose dY is not zero
            keep = t.zeros(M, 1, dtype=t.bfloat16, device="cuda")
            keep[active] = 1.0
            self.dY *= keep

    def small(self, *sums):
        for v in sums:
            assert float(v.max()) < TOP

    def forward(self):
        q, t = self.q, self.t
        if self.A.shape[0] == 0:
            ref = (self.x @ self.w.t()).bfloat16()
            return q.linear_fwd_int8(self.X, self.W), (ref, ref), None
        a, b = self.A.double(), self.B.double()
        T = self.x @ a.t()
        assert float(T.abs().max()) < 2.0 ** 14         # S T in two bf16 terms, quarters included
        self.small(self.x.abs() @ self.w.abs().t() + S * T.abs() @ b.abs().t(), self.x.abs() @ a.abs().t())
        mag = self.x.abs() @ self.w.abs().t() + S * T.abs() @ b.abs().t()
        ref, off = self.x @ self.w.t() + S * T @ b.t(), mag * left(2, self.A.shape[0])
        return (q.linear_fwd_int8(self.X, self.W, self.A, self.B, self.alpha),
                ((ref - off).float().bfloat16(), (ref + off).float().bfloat16()), T.float())

    def backward(self, T, dX0=None):
        """The reference: dX (from dX0 on), and dA and dB with how far they may be off."""
        t = self.t
        a, b, dY = self.A.double(), self.B.double(), self.dY.double()
        U = dY @ b
        sU = (S * U).float().bfloat16().double()
        self.small(dY.abs() @ self.w.abs() + sU.abs() @ a.abs(), S * U.abs().t() @ self.x.abs(),
                   S * dY.abs().t() @ T.double().abs())
        dX = dY @ self.w + sU @ a + (0.0 if dX0 is None else dX0.double())
        n = left(3, int((dY != 0).any(1).sum()))
        return (dX.float().bfloat16(), (S * U.t() @ self.x, S * U.abs().t() @ self.x.abs() * n),
                (S * dY.t() @ T.double(), S * dY.abs().t() @ T.double().abs() * n))


FWD = [(1, 64, 8, 8), (1, 512, 264, 32), (16, 640, 1000, 24), (7, 64, 40, 20), (16, 320, 4104, 17), (2, 8256, 72, 16),
       (16, 16448, 264, 8), (3, 2048, 136, 8), (5, 4160, 40, 256), (16, 832, 1000, 72), (1, 192, 33000, 3),
       (17, 64, 8, 8), (33, 448, 72, 24), (64, 1024, 520, 0), (70, 320, 264, 136), (100, 4096, 264, 12),
       (129, 512, 1032, 128), (257, 192, 776, 200), (300, 2048, 2056, 256), (40, 16448, 72, 32), (61, 8256, 200, 96),
       (647, 3264, 1096, 40), (700, 576, 1304, 40), (2048, 1024, 4096, 16), (4100, 448, 5000, 65), (1030, 1152, 2824, 8)]


@pytest.mark.parametrize("M,K,N,r", FWD)
def test_forward(M, K, N, r):
    L = Whole(M, K, N, r)
    (Y, T), (low, high), refT = L.forward()
    assert bool(((low <= Y) & (Y <= high)).all())
    assert (T is None) == (refT is None) and (T is None or L.t.equal(T, refT))


BWD = [(1, 64, 8, 8), (3, 4096, 4104, 16), (16, 8192, 1000, 8), (5, 192, 40, 3), (16, 256, 256, 8), (40, 320, 72, 40),
       (4, 128, 16648, 16), (4, 128, 22744, 24), (2, 576, 28576, 64), (70, 64, 8200, 24), (100, 2048, 2056, 72),
       (129, 512, 1032, 128), (130, 4160, 520, 8), (128, 64, 768, 136), (7, 1088, 4096, 16), (257, 1088, 4096, 32),
       (300, 4096, 1544, 256), (512, 11008, 264, 8), (511, 576, 8200, 16), (513, 320, 72, 200), (600, 256, 264, 17),
       (700, 2112, 776, 64), (1100, 4096, 1032, 8), (2100, 4160, 328, 96), (4100, 4096, 200, 12)]


def _check(L, got, ref, what):
    assert ref[0] is None and got[0] is None or L.t.equal(got[0], ref[0]), "dX" + what
    for v, (r, off), name in zip(got[1:], ref[1:], ("dA", "dB")):
        assert bool(((v.double() - r).abs() <= off).all()), name + what


@pytest.mark.parametrize("base", ["int8", "nf4", "bf16"])
@pytest.mark.parametrize("M,K,N,r", BWD)
def test_backward(M, K, N, r, base):
    L = Whole(M, K, N, r, base)
    q, t = L.q, L.t
    g = t.Generator("cuda")
    g.manual_seed(N)
    T = t.randint(-8, 9, (M, r), device="cuda", generator=g).to(t.float32 if base == "int8" else t.bfloat16)
    dX0 = t.randint(-100, 101, (M, K), device="cuda", generator=g).bfloat16()
    run = lambda **kw: q.linear_bwd_int8(L.dY, L.X, L.W, L.A, L.B, L.alpha, **kw)
    _check(L, run(T=T), L.backward(T), "")
    acc = dX0.clone()
    run(T=T, accumulate_into=acc)
    assert t.equal(acc, L.backward(T, dX0)[0]), "added to"
    again = L.x @ L.A.double().t()                     # T computed again from the codes
    _check(L, run(need_dX=False), (None, *L.backward(again)[1:]), ", T computed again")


@pytest.mark.parametrize("base", ["int8", "nf4", "bf16"])
@pytest.mark.parametrize("M,K,N,r", [c for c in BWD if c[0] > 64])
def test_backward_of_few_tokens_among_zeros(M, K, N, r, base):
    """dA and dB are sums over 16 tokens alone, so that one product more or less is
    far above what their terms leave."""
    edges = [0, 31, 32, M // 2, M - 1]
    active = edges + [m for m in range(7, M, M // 12) if m not in edges][:11]
    L = Whole(M, K, N, r, base, active)
    g = L.t.Generator("cuda")
    g.manual_seed(N)
    T = L.t.randint(-8, 9, (M, r), device="cuda", generator=g)
    T = T.to(L.t.float32 if base == "int8" else L.t.bfloat16)
    ref = L.backward(T)
    # the smallest product: 1.5 times a whole U and half a code, or a whole dY and T
    assert max(float(off.max()) for _, off in ref[1:]) < 0.75 / 4
    _check(L, L.q.linear_bwd_int8(L.dY, L.X, L.W, L.A, L.B, L.alpha, T=T), ref, "")
