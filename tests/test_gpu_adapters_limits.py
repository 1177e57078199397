"""The batched adapters at the ends of their ranges, on the GPU."""
import numpy as np
import pytest

import bit_nf4_quantized_07_amd as q
from gpu_helpers import host, log
from test_gpu_adapters import dev_i32, make_plan

pytestmark = pytest.mark.gpu
t = pytest.importorskip("torch")

TOP = 1 << 30      # the most rows a plan takes


@pytest.mark.parametrize("lengths,slots,S", [
    ([TOP, TOP], [1, 0], 2),                 # sums of 2^31, cut at M
    ([TOP - 7, 2 ** 31 - 1], [0, 2], 2),     # the rows behind the first without an adapter
    ([5, TOP - 9, TOP], [1, 1, 0], 2)])
def test_plan_of_the_largest_batch(lengths, slots, S):
    """2^30 rows: every request's share of them, bit for bit."""
    log(f"[plan] {TOP} rows, lengths {lengths}")
    pl = make_plan(lengths, slots, TOP, S)
    t.cuda.synchronize()
    ends = np.minimum(TOP, np.cumsum(lengths))            # 64 bits
    begins = np.concatenate([[0], ends[:-1]])
    cls = [s if 0 <= s < S else S for s in slots]
    rows, tiles, start = [], [], [0]
    for c in range(S + 1):
        rows += [(int(b), int(e), c) for b, e, k in zip(begins, ends, cls) if k == c and e > b]
        start.append(sum(e - b for b, e, _ in rows))
    assert host(pl.start).tolist() == start
    at = 0
    for b, e, c in rows:
        part = pl.order[at:at + e - b]
        assert bool((part == t.arange(b, e, dtype=t.int32, device="cuda")).all()), (b, e)
        del part
        assert bool((pl.token_slot[b:e] == (c if c < S else -1)).all()), (b, e)
        at += e - b
    assert at == TOP
    for c in range(S + 1):
        first, count = start[c], start[c + 1] - start[c]
        tiles += [(c if c < S else -1, first, count)] if count else []
    got, n = host(pl.tiles), 0
    for c, first, count in tiles:
        k = -(-count // 64)
        f = 64 * np.arange(k, dtype=np.int64)
        assert np.all(got[n:n + k, 0] == c)
        assert np.array_equal(got[n:n + k, 1], first + f)
        assert np.array_equal(got[n:n + k, 2], np.minimum(64, count - f))
        n += k
    assert np.all(got[n:] == np.array([-1, 0, 0]))


def test_outputs_that_overlap_are_refused():
    """An output given by the caller may be the base it is added to, and may
    otherwise share no byte with an input or another output."""
    M, K, r, S = 32, 64, 8, 2
    bf, f32 = t.bfloat16, t.float32
    plan = make_plan([20, 12], [0, 1], M, S)
    X, Y, dY = (t.randn(M, K, device="cuda").to(bf) for _ in range(3))
    A, B = t.randn(S, r, K, device="cuda").to(bf), t.randn(S, K, r, device="cuda").to(bf)
    c = t.ones(S, device="cuda")
    long = t.randn(M + 8, K, device="cuda").to(bf)
    two = t.empty(2 * S * r * K, device="cuda")
    dA, dB = two[:S * r * K].view(S, r, K), two[S * r * K:].view(S, K, r)
    T = q.adapters_fwd(X, Y, A, B, c, plan)[1]
    fwd = lambda X=X, Y=Y, **kw: q.adapters_fwd(X, Y, A, B, c, plan, **kw)
    bwd = lambda dY=dY, X=X, **kw: q.adapters_bwd(dY, X, A, B, c, plan, T=T, **kw)
    for match, call in (
            ("out: overlaps X", lambda: fwd(out=X)),
            ("out: overlaps X", lambda: fwd(X=long[8:], Y=None, out=long[:M])),
            ("out: overlaps Y", lambda: fwd(Y=long[8:], out=long[:M])),
            ("T_out: overlaps scale", lambda: q.adapters_fwd(
                X, Y, A, B, two[:S], plan, T_out=two[:M * r].view(M, r))),
            ("dX_out: overlaps X", lambda: bwd(dX_out=X)),
            ("dX_out: overlaps dY", lambda: bwd(dX_out=dY)),
            ("dX_out: overlaps dX", lambda: bwd(dX=long[8:], dX_out=long[:M])),
            ("dB: overlaps dA", lambda: bwd(dA_out=dA, dB_out=dA.view(S, K, r))),
            ("dA: overlaps T", lambda: q.adapters_bwd(
                dY, X, A, B, c, plan, T=two[:M * r].view(M, r), dA_out=dA))):
        with pytest.raises(ValueError, match=match):
            call()
    # beside each other, and the base itself
    y, x0 = Y.clone(), X.clone()
    fwd(Y=y, out=y, T_out=t.empty(M, r, device="cuda"))
    bwd(dX=x0, dX_out=x0, dA_out=dA, dB_out=dB)
    ref = bwd(dX=X)
    t.cuda.synchronize()
    for a, b in zip((x0, dA, dB), ref):
        assert t.equal(a, b)
