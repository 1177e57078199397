"""Adapters of many requests beside one shared projection, on the GPU, against
the fp64 oracle.

Tolerances, element by element, from the roundings the calls may make.  With
g(n) = (n + 8) 2^-23 for an fp32 sum of n products (each addition off by at
most one unit in the last place, whatever its order), |.| taken elementwise:
  T, U    g(K) |X| |A|^T, g(N) |dY| |B|                      (exact products)
  out     E = c (errT |B|^T + (|T| + errT) |B|^T (2^-17 + g(2 r))), T entering
          as two bf16 terms; then one rounding to bf16, half a step:
          E + 2^-8 (|out| + E)
  dX      the same with U and A, times 1 / (1 - p)
  dA, dB  c (errU^T |X| + |U|^T |X| (2^-25 + g(3 n))) for the slot's n tokens,
          three bf16 terms of U (T, for dB, is given: errT = 0)
plus 2^-22 of the value for the factors c and 1 / (1 - p) in fp32.
The plan is compared bit for bit."""
import numpy as np
import pytest

import bit_nf4_quantized_07_amd as q
import oracle
import qlora_workloads as wl
from gpu_helpers import dev_bf16, dev_f32, f64, host, host_bf16_bits, host_bf16_f64, log

pytestmark = pytest.mark.gpu
t = pytest.importorskip("torch")


def g(n):
    return (n + 8) * 2.0 ** -23


def dev_i32(a):
    return t.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def make_plan(lengths, slots, M, S):
    return q.adapter_plan(dev_i32(slots), S, lengths=dev_i32(lengths), tokens=M)


def bits_of(x):
    return host_bf16_bits(x) if x.dtype == t.bfloat16 else host(x.view(t.int32))


# ---- the plan ---------------------------------------------------------------

def _random_requests(seed, Q, M, S, longest):
    r = np.random.default_rng(seed)
    return r.integers(0, longest + 1, Q), r.integers(-1, S + 1, Q)


PLANS = [
    ([1], [0], 1, 1), ([1], [-1], 1, 1), ([3], [0], 1, 1), ([], [], 7, 3),
    ([64], [0], 64, 1), ([65], [0], 65, 1), ([0, 0, 5, 0], [1, 0, 1, 2], 5, 3),
    ([10, 200, 64, 1], [1, 0, 1, 7], 300, 2), ([-3, 4], [0, 0], 10, 1),
    ([2 ** 31 - 1, 2 ** 31 - 1, 5], [0, 1, 0], 130, 2),      # sums past 32 bits, cut at M
    ([100] * 7, [5, 5, 5, 1023, 0, 1023, 5], 650, 1024),
    (*_random_requests(1, 70, 500, 9, 12), 500, 9),
    (*_random_requests(2, 1023, 9000, 64, 16), 9000, 64),
    (*_random_requests(3, 1024, 9000, 1000, 12), 9000, 1000),
    (*_random_requests(4, 1025, 9000, 3, 12), 9000, 3),
    (*_random_requests(5, 5000, 16500, 200, 6), 16500, 200),
]


@pytest.mark.parametrize("i", range(len(PLANS)))
def test_plan_is_the_oracles(i):
    lengths, slots, M, S = PLANS[i]
    log(f"[plan] case {i}: Q={len(lengths)} M={M} S={S}")
    pl = make_plan(lengths, slots, M, S)
    t.cuda.synchronize()
    ref = oracle.adapter_plan(lengths, slots, M, S)
    for name, a, b in zip(("token_slot", "order", "start", "tiles"), pl, ref):
        assert np.array_equal(host(a), b), name


@pytest.mark.parametrize("Q,S", [(1, 1), (64, 5), (256, 64), (1024, 1024), (3000, 17)])
def test_plan_of_single_tokens(Q, S):
    log(f"[plan] single tokens Q={Q} S={S}")
    slots = np.random.default_rng(Q).integers(-1, S, Q)
    pl = q.adapter_plan(dev_i32(slots), S)
    t.cuda.synchronize()
    for a, b in zip(pl, oracle.adapter_plan([1] * Q, slots, Q, S)):
        assert np.array_equal(host(a), b)
    padded = q.adapter_plan(dev_i32(slots), S, tokens=Q + 3)
    t.cuda.synchronize()
    for a, b in zip(padded, oracle.adapter_plan([1] * Q, slots, Q + 3, S)):
        assert np.array_equal(host(a), b)


# ---- the layer --------------------------------------------------------------

class Case:
    def __init__(self, lengths, slots, M, K, N, r, S, p=0.0, seed=11):
        self.M, self.K, self.N, self.r, self.S, self.p, self.seed = M, K, N, r, S, p, seed
        e = np.random.default_rng([seed, M, K, N, r, S])
        bf = lambda a: wl.round_to_bf16_bits(np.asarray(a, np.float32))
        self.X = bf(e.standard_normal((M, K)))
        self.Y = bf(e.standard_normal((M, N)))
        self.dY = bf(e.standard_normal((M, N)))
        self.dX0 = bf(e.standard_normal((M, K)))
        self.A = bf(e.uniform(-1, 1, (S, r, K)) / np.sqrt(K))
        self.B = bf(e.standard_normal((S, N, r)) * 0.05)
        self.scale = e.uniform(0.25, 3.0, S).astype(np.float32)
        self.tok = oracle.adapter_plan(lengths, slots, M, S)[0]
        self.plan = make_plan(lengths, slots, M, S)
        self.mask = oracle.dropout_mask(M, K, p, seed) if p else None
        self.drop = (p, seed) if p else None
        self.keep = 1.0 if not p else 1.0 / (1.0 - p)
        self.d = {k: dev_bf16(getattr(self, k)) for k in ("X", "Y", "dY", "dX0", "A", "B")}
        self.d["scale"] = dev_f32(self.scale)

    def fwd(self, Y=True, **kw):
        d = self.d
        return q.adapters_fwd(d["X"], d["Y"] if Y else None, d["A"], d["B"], d["scale"], self.plan,
                              dropout=self.drop, **kw)

    def bwd(self, T, dX0=True, **kw):
        d = self.d
        return q.adapters_bwd(d["dY"], d["X"], d["A"], d["B"], d["scale"], self.plan, T=T,
                              dX=d["dX0"] if dX0 else None, dropout=self.drop, **kw)

    def by_slot(self, f, shape):
        """sum over slots of f(slot, rows) placed at the slot's rows."""
        out = np.zeros(shape)
        for a in range(self.S):
            rows = np.flatnonzero(self.tok == a)
            if len(rows):
                out[rows] = f(a, rows)
        return out

    def tolerances(self, T, Tref, ref):
        """(T, out, dX, dA, dB) bounds; ref = oracle's (out, dX, dA, dB)."""
        X = np.abs(f64(self.X)) * self.keep
        if self.mask is not None:
            X = X * self.mask
        dY, A, B, c = np.abs(f64(self.dY)), np.abs(f64(self.A)), np.abs(f64(self.B)), self.scale
        M, K, N, r = self.M, self.K, self.N, self.r
        eT = self.by_slot(lambda a, m: X[m] @ A[a].T * (g(K) + 2.0 ** -22), (M, r))
        eU = self.by_slot(lambda a, m: dY[m] @ B[a] * g(N), (M, r))
        U = np.abs(self.by_slot(lambda a, m: f64(self.dY)[m] @ f64(self.B)[a], (M, r)))
        w = 2.0 ** -17 + g(2 * r) + 2.0 ** -22
        eo = self.by_slot(lambda a, m: c[a] * ((eT[m] + (np.abs(Tref[m]) + eT[m]) * w) @ B[a].T), (M, N))
        ex = self.keep * self.by_slot(lambda a, m: c[a] * ((eU[m] + (U[m] + eU[m]) * w) @ A[a]), (M, K))
        out, dX, dA, dB = ref
        tA, tB = np.zeros(dA.shape), np.zeros(dB.shape)
        for a in range(self.S):
            m = np.flatnonzero(self.tok == a)
            s = 2.0 ** -25 + g(3 * len(m)) + 2.0 ** -22
            tA[a] = c[a] * (eU[m].T @ X[m] + (U[m] + eU[m]).T @ X[m] * s)
            tB[a] = c[a] * (dY[m].T @ np.abs(T[m])) * s
        half = 2.0 ** -8
        return (eT, eo + half * (np.abs(out) + eo) + 2.0 ** -22 * np.abs(out),
                ex + half * (np.abs(dX) + ex) + 2.0 ** -22 * np.abs(dX), tA, tB)


def within(name, got, ref, tol):
    err = np.abs(np.asarray(got, np.float64) - ref)
    assert np.all(np.isfinite(got)), f"{name}: non-finite"
    bad = err > tol
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    log(f"  {name}: worst error / tolerance {worst:.3f}")
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} outside, worst {worst:.2f}"


def check(c: Case):
    out, T = c.fwd()
    dX, dA, dB = c.bwd(T)
    t.cuda.synchronize()
    Th = host(T).astype(np.float64)
    ro, rT = oracle.adapters_forward(f64(c.X), f64(c.Y), f64(c.A), f64(c.B), c.scale, c.tok,
                                     mask=c.mask, p=c.p)
    rx, ra, rb = oracle.adapters_backward(f64(c.dY), f64(c.X), f64(c.A), f64(c.B), c.scale, c.tok,
                                          dX0=f64(c.dX0), mask=c.mask, p=c.p, T=Th)
    tT, to, tx, ta, tb = c.tolerances(Th, rT, (ro, rx, ra, rb))
    within("T", Th, rT, tT)
    within("out", host_bf16_f64(out), ro, to)
    within("dX", host_bf16_f64(dX), rx, tx)
    within("dA", host(dA), ra, ta)
    within("dB", host(dB), rb, tb)
    bare = np.flatnonzero(c.tok < 0)
    assert np.array_equal(host_bf16_bits(out)[bare], c.Y[bare])
    assert np.array_equal(host_bf16_bits(dX)[bare], c.dX0[bare])
    if c.mask is not None:   # a dropped input has no gradient through the adapter
        assert np.array_equal(host_bf16_bits(dX)[~c.mask], c.dX0[~c.mask])
    idle = [a for a in range(c.S) if not (c.tok == a).any()]
    assert not host(dA)[idle].any() and not host(dB)[idle].any()
    return out, T, dX, dA, dB


CASES = [
    # lengths, slots, M, K, N, r, S
    ([1], [0], 1, 8, 8, 8, 1),
    ([1], [2], 1, 256, 1000, 16, 4),
    ([1] * 16, list(range(16)), 16, 512, 264, 16, 16),
    ([1] * 37, [i % 5 - 1 for i in range(37)], 40, 104, 72, 8, 4),
    ([16], [1], 16, 256, 256, 8, 4),
    ([63, 1, 64, 2], [0, 1, 0, 1], 130, 200, 88, 24, 2),
    ([65, 0, 130, 7], [2, 0, -1, 2], 220, 264, 312, 40, 3),
    ([100, 50], [0, 1], 150, 328, 520, 64, 2),
    ([33, 90], [1, 1], 128, 136, 264, 72, 2),
    ([70, 3], [0, 2], 80, 72, 40, 136, 3),
    ([20, 50], [0, 1], 70, 64, 280, 256, 2),
    ([300], [0], 300, 64, 64, 32, 1),
    ([9, 9], [-1, 77], 18, 64, 64, 8, 2),                    # nobody has an adapter
    ([5, 6, 7], [900, 3, 900], 20, 64, 48, 8, 1024),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_layer_against_the_oracle(i):
    log(f"[adapters] case {i}: {CASES[i][2:]}")
    check(Case(*CASES[i]))


# tiles of each number of token groups, contractions shorter than the waves'
# share, and the number of slots either side of a wave's lanes
EDGES = [
    ([17], [0], 17, 8, 8, 64, 1), ([33], [0], 33, 72, 8, 48, 1), ([49, 64], [0, 1], 113, 8, 136, 64, 2),
    ([31, 32, 33, 1], [0, 1, 2, 3], 97, 64, 72, 56, 4), ([1, 1, 1], [0, 1, 0], 3, 128, 8, 64, 2),
    ([257, 31], [1, 0], 290, 136, 200, 24, 2), ([600, 1], [0, 1], 601, 72, 264, 64, 2),
    ([2, 3, 40, 2], [63, 0, 31, 63], 47, 64, 72, 16, 64),
    ([2, 3, 40, 2], [64, 0, 31, 64], 47, 64, 72, 16, 65),
    ([90, 70], [1, 0], 160, 72, 136, 128, 2),
]


@pytest.mark.parametrize("i", range(len(EDGES)))
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_edges_against_the_oracle(i, p):
    log(f"[adapters] edge {i}: {EDGES[i][2:]} p={p}")
    check(Case(*EDGES[i], p=p))


@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 80])
def test_narrow_tiles_of_every_count(r):
    """Tiles of 1 .. 16 tokens in one batch, each of its own slot: the last
    token's columns of every block are its own."""
    log(f"[adapters] narrow tiles r={r}")
    check(Case(list(range(1, 17)), list(range(16)), 136, 64, 1160, r, 16))


@pytest.mark.parametrize("i,p,seed", [(1, 0.3, 1), (3, 0.05, 2), (5, 0.05, 2 ** 63 + 5), (6, 0.5, 4),
                                      (7, 0.1, 5), (10, 0.25, 6), (11, 0.9, 7), (12, 0.5, 8)])
def test_layer_with_dropout(i, p, seed):
    log(f"[adapters] dropout case {i}: {CASES[i][2:]} p={p}")
    check(Case(*CASES[i], p=p, seed=seed))


def test_the_mask_is_lora_dropouts():
    """With p a power of two 1 / (1 - p) = 2 is exact, and Xd of `dropout` fed
    without dropout gives the same T bits as the regenerated mask."""
    c = Case([40, 60], [0, 1], 100, 288, 64, 16, 2, p=0.5, seed=77)   # K a multiple of 32
    d = c.d
    Xd, _ = q.dropout(d["X"], 0.5, 77)
    _, T = c.fwd()
    _, T2 = q.adapters_fwd(Xd, None, d["A"], d["B"], d["scale"], c.plan)
    t.cuda.synchronize()
    assert np.array_equal(bits_of(T), bits_of(T2))


def test_repeats_and_variants_give_the_same_bits():
    c = Case([65, 0, 130, 7], [2, 0, -1, 2], 220, 264, 312, 40, 3, p=0.2)
    out, T = c.fwd()
    dX, dA, dB = c.bwd(T)
    ref = [bits_of(v) for v in (out, T, dX, dA, dB)]
    out2, T2 = c.fwd()
    for a, b in zip(ref, [out2, T2, *c.bwd(T2)]):
        assert np.array_equal(a, bits_of(b))
    # T not saved; T computed again in the backward
    out3, none = c.fwd(save_T=False)
    assert none is None and np.array_equal(ref[0], bits_of(out3))
    for a, b in zip(ref[2:], c.bwd(None)):
        assert np.array_equal(a, bits_of(b))
    # in place
    y, x0 = c.d["Y"].clone(), c.d["dX0"].clone()
    d = c.d
    q.adapters_fwd(d["X"], y, d["A"], d["B"], d["scale"], c.plan, dropout=c.drop, out=y)
    q.adapters_bwd(d["dY"], d["X"], d["A"], d["B"], d["scale"], c.plan, T=T, dX=x0, dX_out=x0,
                   dropout=c.drop)
    assert np.array_equal(ref[0], bits_of(y)) and np.array_equal(ref[2], bits_of(x0))
    # without dX
    none, a2, b2 = c.bwd(T, dX0=False, need_dX=False)
    assert none is None and np.array_equal(ref[3], bits_of(a2)) and np.array_equal(ref[4], bits_of(b2))


def test_without_a_base():
    c = Case([50, 20], [1, -1], 75, 136, 104, 16, 2)
    out, T = c.fwd(Y=False)
    dX, _, _ = c.bwd(T, dX0=False)
    t.cuda.synchronize()
    ro, rT = oracle.adapters_forward(f64(c.X), None, f64(c.A), f64(c.B), c.scale, c.tok)
    rx, ra, rb = oracle.adapters_backward(f64(c.dY), f64(c.X), f64(c.A), f64(c.B), c.scale, c.tok)
    _, to, tx, _, _ = c.tolerances(host(T).astype(np.float64), rT, (ro, rx, ra, rb))
    within("out", host_bf16_f64(out), ro, to)
    within("dX", host_bf16_f64(dX), rx, tx)
    assert not host_bf16_bits(out)[50:].any() and not host_bf16_bits(dX)[50:].any()


def test_nothing_leaks_from_other_rows_and_slots():
    """NaN and infinities in rows without an adapter, in unused slots, in rows
    of other slots and in dropped elements change nothing elsewhere."""
    M, K, N, r, S, p, seed = 120, 72, 88, 24, 4, 0.4, 5
    args = ([40, 30, 30], [2, -1, 0], M, K, N, r, S)
    clean, dirty = Case(*args, p=p, seed=seed), Case(*args, p=p, seed=seed)
    bad = np.array([0x7FC0, 0x7F80, 0xFF80], np.uint16)      # NaN, inf, -inf
    e = np.random.default_rng(1)
    dirty.X[40:70] = e.choice(bad, (30, K))
    dirty.dY[40:70] = e.choice(bad, (30, N))
    dirty.X[100:] = e.choice(bad, (20, K))
    dirty.A[[1, 3]] = e.choice(bad, (2, r, K))
    dirty.B[[1, 3]] = e.choice(bad, (2, N, r))
    dirty.scale[[1, 3]] = np.nan
    dirty.X[~dirty.mask] = e.choice(bad, int((~dirty.mask).sum()))
    dirty.X[70:100] = np.where(dirty.mask[70:100], dirty.X[70:100], 0x7F80)
    dirty.d.update({k: dev_bf16(getattr(dirty, k)) for k in ("X", "dY", "A", "B")})
    dirty.d["scale"] = dev_f32(dirty.scale)
    o1, T1 = clean.fwd()
    o2, T2 = dirty.fwd()
    r1, r2 = clean.bwd(T1), dirty.bwd(T2)
    t.cuda.synchronize()
    for name, a, b in zip(("out", "T", "dX", "dA", "dB"), (o1, T1, *r1), (o2, T2, *r2)):
        assert np.array_equal(bits_of(a), bits_of(b)), name


def test_infinities_of_a_token_stay_infinite():
    """A token whose own input is infinite gets what the formula gives, not NaN
    made by splitting T into terms."""
    c = Case([2], [0], 2, 64, 32, 8, 1)
    c.A[:] = wl.round_to_bf16_bits(np.full(c.A.shape, 0.25, np.float32))
    c.B[:] = wl.round_to_bf16_bits(np.full(c.B.shape, 0.5, np.float32))
    c.X[0, 3] = 0x7F80
    c.d.update({k: dev_bf16(getattr(c, k)) for k in ("X", "A", "B")})
    out, T = c.fwd()
    t.cuda.synchronize()
    assert np.all(np.isposinf(host(T)[0])) and np.all(np.isfinite(host(T)[1]))
    assert np.all(np.isposinf(host_bf16_f64(out)[0])) and np.all(np.isfinite(host_bf16_f64(out)[1]))


def test_differences_along_directions():
    """(loss(x + d) - loss(x - d)) / 2 of the GPU's forward against the GPU's
    gradients, for A, B and X; loss = sum(out dY).  Operands and steps are
    multiples of 2^-6 below 2, so x +- d are exact in bf16, and the loss is
    linear in each operand: what remains is the rounding of out, at most half a
    step (2^-8) of each value at either end, T's and the gradients' own, below
    2^-14 of the sums of absolute values, and dX's half step."""
    M, K, N, r, S = 48, 64, 40, 8, 2
    c = Case([20, 25], [1, 0], M, K, N, r, S, p=0.25, seed=3)
    e = np.random.default_rng(8)
    grid = lambda shape: e.integers(-31, 32, shape) / 64.0
    base = {"A": grid((S, r, K)), "B": grid((S, N, r)), "X": grid((M, K))}
    dev = lambda a: dev_bf16(wl.round_to_bf16_bits(a.astype(np.float32)))

    def forward(ops):
        out, T = q.adapters_fwd(dev(ops["X"]), None, dev(ops["A"]), dev(ops["B"]), c.d["scale"],
                                c.plan, dropout=c.drop)
        return host_bf16_f64(out), T

    out0, T = forward(base)
    dX, dA, dB = q.adapters_bwd(c.d["dY"], dev(base["X"]), dev(base["A"]), dev(base["B"]),
                                c.d["scale"], c.plan, T=T, dropout=c.drop)
    grads = {"A": host(dA).astype(np.float64), "B": host(dB).astype(np.float64),
             "X": host_bf16_f64(dX)}
    dY = f64(c.dY)
    for name in ("A", "B", "X"):
        d = grid(base[name].shape)
        ends = [forward({**base, name: base[name] + s * d})[0] for s in (1, -1)]
        diff = ((ends[0] - ends[1]) * dY).sum() / 2
        want = (grads[name] * d).sum()
        tol = (2.0 ** -8 + 2.0 ** -14) * ((np.abs(ends[0]) + np.abs(ends[1])) * np.abs(dY)).sum() / 2
        tol += (2.0 ** -8 if name == "X" else 2.0 ** -14) * (np.abs(grads[name]) * np.abs(d)).sum()
        log(f"  {name}: difference {diff:.4f}, gradient {want:.4f}, tolerance {tol:.4f}")
        assert abs(diff - want) <= tol, name


# ---- beside the shared projection, streams, graphs --------------------------

def test_beside_the_layer_of_this_library():
    """Plan, forward and backward beside the shared projection: with one slot
    and the same adapter the layer's own fused call is the reference."""
    M, N, K, r, alpha = 300, 512, 256, 16, 32.0
    case = wl.linear_case(5, M, N, K, r, alpha)
    qw = q.quantize(dev_f32(case["W"]))
    X, A, B, dY = (dev_bf16(case[k]) for k in ("X", "A", "B", "dY"))
    zero = t.zeros_like(B)
    plan = q.adapter_plan(dev_i32([0, 0]), 1, lengths=dev_i32([120, 180]), tokens=M)
    scale = dev_f32(np.array([alpha / r], np.float32))
    base, _ = q.linear_fwd(X, qw, A, zero, alpha)          # B = 0: the projection alone
    out, T = q.adapters_fwd(X, base, A[None], B[None], scale, plan)
    dX0, _, _ = q.linear_bwd(dY, X, qw, A, zero, alpha)
    dX, dA, dB = q.adapters_bwd(dY, X, A[None], B[None], scale, plan, T=T, dX=dX0)
    Y1, T1 = q.linear_fwd(X, qw, A, B, alpha)
    dX1, dA1, dB1 = q.linear_bwd(dY, X, qw, A, B, alpha, T=T1)
    t.cuda.synchronize()
    # two roundings to bf16 on one side, one on the other and a bf16 T, U:
    # 2^-8 of |Y| three times, 2^-8 of the adapter's own sums of absolute values
    sab = np.abs(f64(case["X"])) @ np.abs(f64(case["A"])).T @ np.abs(f64(case["B"])).T * alpha / r
    sxb = np.abs(f64(case["dY"])) @ np.abs(f64(case["B"])) @ np.abs(f64(case["A"])) * alpha / r
    for name, a, b, s in (("Y", out, Y1, sab), ("dX", dX, dX1, sxb)):
        a, b = host_bf16_f64(a), host_bf16_f64(b)
        within(name, a, b, 2.0 ** -8 * (3.1 * np.maximum(np.abs(a), np.abs(b)) + s) + 2.0 ** -8 * np.abs(b))
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)
    # the layer rounds U and T to bf16 (half a step, 2^-8, of each)
    assert rel(host(dA)[0], host(dA1)) <= 2.0 ** -8 and rel(host(dB)[0], host(dB1)) <= 2.0 ** -8


def test_two_streams_at_once():
    a = Case([65, 0, 130, 7], [2, 0, -1, 2], 220, 264, 312, 40, 3, p=0.2, seed=1)
    b = Case([100, 50], [0, 1], 150, 328, 520, 64, 2, seed=2)
    ref = []
    for c in (a, b):
        out, T = c.fwd()
        ref.append([bits_of(v) for v in (out, T, *c.bwd(T))])
    t.cuda.synchronize()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    got = [None, None]
    for rep in range(3):
        for j, c in enumerate((a, b)):
            with t.cuda.stream(streams[j]):
                out, T = c.fwd()
                got[j] = (out, T, *c.bwd(T))
        t.cuda.synchronize()
        for j in range(2):
            for x, y in zip(ref[j], got[j]):
                assert np.array_equal(x, bits_of(y)), (rep, j)


def test_captured_step_replays_the_eager_bits():
    """Plan, forward and backward in one graph, replayed with other requests in
    the same buffers: each replay against the eager result of those requests."""
    M, K, N, r, S = 130, 264, 200, 24, 3
    c = Case([60, 40, 20], [0, 2, -1], M, K, N, r, S, p=0.1, seed=9)
    d = c.d
    lengths, slots = dev_i32([60, 40, 20]), dev_i32([0, 2, -1])
    ws = q.Workspace("cuda")
    ws.get(q.load_library().lora_adapters_workspace_bytes(M, K, N, r, S, 1))
    keep = {}

    def step():
        plan = q.adapter_plan(slots, S, lengths=lengths, tokens=M)
        out, T = q.adapters_fwd(d["X"], d["Y"], d["A"], d["B"], d["scale"], plan, dropout=c.drop,
                                workspace=ws)
        return (plan.order, out, T, *q.adapters_bwd(d["dY"], d["X"], d["A"], d["B"], d["scale"],
                                                    plan, T=T, dX=d["dX0"], dropout=c.drop,
                                                    workspace=ws))

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        keep["outs"] = step()
    t.cuda.synchronize()
    for rep, (ln, sl) in enumerate([([60, 40, 20], [0, 2, -1]), ([1, 128, 1], [1, 1, 0]),
                                    ([0, 70, 30], [2, -1, 0]), ([60, 40, 20], [0, 2, -1])]):
        lengths.copy_(dev_i32(ln))
        slots.copy_(dev_i32(sl))
        eager = [bits_of(v) for v in step()]
        for v in keep["outs"]:
            v.fill_(-1)
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        for j, (x, y) in enumerate(zip(eager, keep["outs"])):
            assert np.array_equal(x, bits_of(y)), (rep, j)


def test_two_graphs_with_their_own_scratch():
    """Without a Workspace each graph holds its scratch memory: two captured
    steps replayed in turn, with eager calls and other allocations between
    them, keep the eager bits."""
    cases = [Case([60, 40, 20], [0, 2, -1], 130, 264, 200, 24, 3, p=0.1, seed=9),
             Case([100, 50], [0, 1], 150, 328, 520, 64, 2, seed=2)]
    step = lambda c: (lambda o: (*o, *c.bwd(o[1])))(c.fwd())
    eager = [[bits_of(v) for v in step(c)] for c in cases]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        for c in cases:
            step(c)
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        graphs.append(t.cuda.CUDAGraph())
        with t.cuda.graph(graphs[-1]):
            outs.append(step(c))
    t.cuda.synchronize()
    for rep in range(3):
        for g_, o in zip(graphs, outs):
            for v in o:
                v.fill_(-1)
            g_.replay()
        junk = t.full((1 << 20,), float("nan"), device="cuda")
        again = step(cases[rep % 2])
        t.cuda.synchronize()
        del junk
        for j in range(2):
            for x, y in zip(eager[j], outs[j]):
                assert np.array_equal(x, bits_of(y)), (rep, j)
        for x, y in zip(eager[rep % 2], again):
            assert np.array_equal(x, bits_of(y)), rep


@pytest.mark.parametrize("M,K,N,r,S,Q,p", [
    (2048, 4096, 4096, 16, 4, 9, 0.05), (1500, 2048, 5504, 64, 8, 11, 0.0),
    (256, 4096, 11008, 16, 64, 256, 0.0), (16, 8192, 28672, 16, 16, 16, 0.0),
    # more than 32768 tiles; X, then Y and dY, just under 2 GiB
    (2112000, 8, 8, 8, 2, 9, 0.0), (130000, 8192, 8, 8, 2, 9, 0.0), (130000, 8, 8192, 8, 2, 9, 0.0)])
def test_large_shapes_against_64_bits(M, K, N, r, S, Q, p):
    """Whole-tensor errors at real sizes against fp64 on the GPU: bf16 outputs
    within one rounding (2-norm: half a step, 2^-8, at most, plus 2^-12 for the
    sums), fp32 outputs within 2^-18 (sums of up to 28672 products with random
    signs; 2^-18 is a sixteenth of a bf16 term lost).  A gradient of n tokens is
    made of J = 3 n / 128 additions (three terms, 32 tokens at a time, four
    waves) of at most 2^-23 of a partial sum each, which after k of them is in
    the root mean square sqrt(k / J) of the result; errors of independent signs
    add in squares, to 2^-23 sqrt(J / 2): below 2^-18 up to 87000 tokens, the
    tolerance beyond."""
    log(f"[adapters] large M={M} K={K} N={N} r={r} S={S} p={p}")
    e = np.random.default_rng(M)
    lengths = np.ones(Q, int) if Q == M else np.diff(np.concatenate(
        [[0], np.sort(e.integers(0, M + 1, Q - 1)), [M]]))
    slots = e.integers(-1, S, Q)
    gen = t.Generator("cuda")
    gen.manual_seed(M)
    rnd = lambda *s: t.randn(*s, device="cuda", generator=gen)
    X, Y, dY, dX0 = (v.bfloat16() for v in (rnd(M, K), rnd(M, N), rnd(M, N), rnd(M, K)))
    A, B = (rnd(S, r, K) / K ** 0.5).bfloat16(), (rnd(S, N, r) * 0.05).bfloat16()
    scale = 0.5 + t.rand(S, device="cuda", generator=gen)
    plan = make_plan(lengths, slots, M, S)
    drop = (p, 31) if p else None
    out, T = q.adapters_fwd(X, Y, A, B, scale, plan, dropout=drop)
    dX, dA, dB = q.adapters_bwd(dY, X, A, B, scale, plan, T=T, dX=dX0, dropout=drop)
    keep = 1.0
    if p:
        keep = t.from_numpy(oracle.dropout_mask(M, K, p, 31)).cuda().double() / (1 - p)
    tok = np.repeat(slots, lengths)
    Xd, dYd = X.double() * keep, dY.double()
    rT, ro, rx = t.zeros(M, r).cuda().double(), Y.double(), t.zeros(M, K).cuda().double()
    ra, rb = t.zeros(S, r, K).cuda().double(), t.zeros(S, N, r).cuda().double()
    for a in range(S):
        m = t.from_numpy(np.flatnonzero(tok == a)).cuda()
        if len(m) == 0:
            continue
        c = float(scale[a])
        rT[m] = Xd[m] @ A[a].double().t()
        ro[m] += c * (rT[m] @ B[a].double().t())
        U = dYd[m] @ B[a].double()
        rx[m] = c * (U @ A[a].double())
        ra[a] = c * (U.t() @ Xd[m])
        rb[a] = c * (dYd[m].t() @ T[m].double())
    rx = rx * keep + dX0.double()
    longest = max((tok == a).sum() for a in range(S))
    sums = max(2.0 ** -18, 2.0 ** -23 * (3 * longest / 128 / 2) ** 0.5)
    for name, x, y, tol in (("T", T, rT, 2.0 ** -18), ("out", out, ro, 2.0 ** -8 + 2.0 ** -12),
                            ("dX", dX, rx, 2.0 ** -8 + 2.0 ** -12), ("dA", dA, ra, sums),
                            ("dB", dB, rb, sums)):
        rel = float((x.double() - y).norm() / y.norm())
        log(f"  {name}: relative error {rel:.2e}")
        assert rel <= tol, name
