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
