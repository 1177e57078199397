"""Operators for adapters of many requests beside one shared projection: what
is measured, on which cases, and their plain forms.

Three operators share these cases.  S adapters (slots) stand beside a
projection of K inputs and N outputs: A [S, r, K] and B [S, N, r] in bf16, one
scale per slot.  A batch of M tokens packs the tokens of its requests one
after the other; a request names the slot of its adapter, or none.

  plan  from the requests' lengths and slots: the slot of every token, the
        tokens ordered by slot, where each slot starts in that order, and
        tiles of up to 64 ordered tokens of one slot
  fwd   T = drop(X) A^T, out = Y + scale T B^T, each token with its own slot
  bwd   dX = dX0 + drop(scale (dY B) A), dA and dB of every slot

drop() keeps an element where the word of a counter-based generator
(Philox4x32-10, counter = element index div 4, key = the seed) is at least
floor(p 2^32) and multiplies it by 1 / (1 - p); p = 0 leaves everything.
"""
import math

import numpy as np
import torch

own = False

TILE = 64     # ordered tokens of one slot in a tile of the plan


# ---- cases ------------------------------------------------------------------

def _plan(name, requests, tokens, S, used, bare, pad):
    return dict(name=name, op="plan", requests=requests, tokens=tokens, S=S, used=used, bare=bare,
                pad=pad)


def _layer(name, op, requests, tokens, K, N, r, S, used, bare=0, pad=0, p=0.0):
    return dict(name=name, op=op, requests=requests, tokens=tokens, K=K, N=N, r=r, S=S, used=used,
                bare=bare, pad=pad, p=p)


def listed():
    return [
        # 256 running requests, one token each: the plan of a serving step
        _plan("plan_step_256", 256, 256, 64, 48, 9, 0),
        # prompts of 53 requests admitted together, in a buffer padded to 16384 tokens
        _plan("plan_prompts_16k", 53, 16384, 128, 37, 5, 211),
        # a single token of a single request: latency
        _layer("fwd_token", "fwd", 1, 1, 4096, 4096, 16, 8, 1),
        # the small-batch step of a wide projection, every request its own adapter
        _layer("fwd_step_16", "fwd", 16, 16, 8192, 28672, 16, 16, 16),
        # a full serving step: 256 requests over 64 adapters, some on the bare base
        _layer("fwd_step_256", "fwd", 256, 256, 4096, 11008, 16, 64, 64, bare=11),
        # ragged prompts of seven requests in one pass
        _layer("fwd_prompts_2048", "fwd", 7, 2048, 4096, 4096, 16, 8, 5, bare=1, pad=37),
        # the same kind of pass at a high rank on an MLP projection
        _layer("fwd_prompts_r64", "fwd", 13, 4096, 4096, 11008, 64, 16, 9, bare=2, pad=3),
        # training four adapters at once over one base, with LoRA dropout
        _layer("fwd_drop_2048", "fwd", 8, 2048, 4096, 4096, 16, 4, 4, p=0.05),
        # a tiny layer's backward: latency
        _layer("bwd_tiny", "bwd", 3, 16, 256, 256, 8, 4, 2),
        # the backward of several adapters trained together, ragged sequences
        _layer("bwd_train_2048", "bwd", 9, 2048, 4096, 4096, 16, 4, 3, bare=1, pad=21),
        # the same with dropout
        _layer("bwd_drop_2048", "bwd", 8, 2048, 4096, 4096, 16, 4, 4, p=0.05),
        # a high rank on an MLP projection, with dropout
        _layer("bwd_drop_r64", "bwd", 11, 4096, 4096, 11008, 64, 8, 7, pad=5, p=0.1),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("plan", "fwd", "fwd", "bwd", "bwd"))
    step = rng.random() < 0.35                       # one token per request
    if op == "plan":
        requests = _log_int(rng, 1, 2048 if step else 512)
        tokens = requests if step else requests + _log_int(rng, 1, 14000)
        S = _log_int(rng, 1, 512)
    else:
        step = step and op == "fwd"
        requests = _log_int(rng, 1, 256 if step else 24)
        tokens = requests if step else requests + _log_int(rng, 1, 2000)
        S = _log_int(rng, 1, 64 if step else 16)
    pad = 0 if rng.random() < 0.5 else _log_int(rng, 1, 40)
    bare = 0 if rng.random() < 0.5 else rng.randint(0, requests // 4)
    used = rng.randint(1, S)
    if op == "plan":
        case = _plan("", requests, tokens + pad, S, used, bare, pad)
    else:
        K = 64 * _log_int(rng, 4, 128)
        N = 8 * _log_int(rng, 32, 1400)
        r = rng.choice((8, 16, 24, 32, 64))
        p = 0.0 if step or rng.random() < 0.5 else round(rng.uniform(0.01, 0.5), 3)
        case = _layer("", op, requests, tokens + pad, K, N, r, S, used, bare, pad, p)
    del case["name"]
    return case


def _used(case):
    return max(0, min(case["used"], case["requests"] - case["bare"], case["S"]))


def work(case):
    M, S, Q = case["tokens"], case["S"], case["requests"]
    if case["op"] == "plan":
        # lengths and slots in; token slots, order, starts and tiles out
        return {"bytes": 4 * (2 * Q + 2 * M + S + 2 + 3 * _tiles(M, S)), "flops": 2 * M}
    K, N, r = case["K"], case["N"], case["r"]
    a = M - case["pad"]
    if case["bare"]:
        a = a * (Q - case["bare"]) // Q              # tokens with an adapter, on average
    adapters = 2 * _used(case) * r * (K + N)
    if case["op"] == "fwd":
        # X, the used A and B, Y in; out and T out
        return {"bytes": 2 * a * K + adapters + 2 * 2 * M * N + 4 * M * r,
                "flops": 2 * a * r * (K + N)}
    # dY, X, T, the used A and B, dX0 in; dX and all slots' dA and dB out
    return {"bytes": 2 * a * (K + N) + 4 * a * r + adapters + 2 * 2 * M * K + 4 * S * r * (K + N),
            "flops": 4 * a * r * (K + N)}


# ---- inputs -----------------------------------------------------------------

def _requests(case, seed):
    """Lengths and slots of the requests (host): every used slot at least once,
    `bare` requests without one, the lengths a random split of the tokens."""
    g = np.random.default_rng([seed, 17])
    Q, total = case["requests"], case["tokens"] - case["pad"]
    if total == Q:
        lengths = np.ones(Q, np.int64)
    else:
        cuts = np.sort(g.integers(0, total + 1, Q - 1))
        lengths = np.diff(np.concatenate([[0], cuts, [total]]))
    used = _used(case)
    slots = np.full(Q, -1, np.int64)
    if used:
        pool = g.permutation(case["S"])[:used]
        n = Q - case["bare"]
        slots[:n] = np.concatenate([pool, g.choice(pool, n - used)])
        slots = g.permutation(slots)
    return lengths.astype(np.int32), slots.astype(np.int32)


def prepare(case, seed):
    """A program's inputs on the GPU and, for fwd and bwd, the plan that it
    keeps for all projections of the batch; bwd has the forward's T."""
    lengths, slots = (torch.from_numpy(v).cuda() for v in _requests(case, seed))
    s = dict(case, lengths=lengths, slots=slots)
    if case["op"] == "plan":
        return s
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    M, K, N, r, S = (case[k] for k in ("tokens", "K", "N", "r", "S"))

    def normal(*shape, std):
        return (torch.randn(*shape, device="cuda", generator=g) * std).bfloat16()

    s["X"] = normal(M, K, std=1.0)
    s["A"] = ((torch.rand(S, r, K, device="cuda", generator=g) * 2 - 1) / math.sqrt(K)).bfloat16()
    s["B"] = normal(S, N, r, std=0.05)
    s["scale"] = 0.5 + 2.0 * torch.rand(S, device="cuda", generator=g)
    s["seed"] = seed * 0x9E3779B97F4A7C15 % (1 << 64)
    s["plan"] = _plan_plain(s)
    if case["op"] == "fwd":
        s["Y"] = normal(M, N, std=1.3)
    else:
        s["dY"] = normal(M, N, std=1.0)
        s["dX0"] = normal(M, K, std=1.0)
        s["T"] = _down(_drop(s["X"].float(), s), s)
    return s


# ---- plain forms ------------------------------------------------------------

def _tiles(M, S):
    return M // TILE + min(S + 1, M)


def _plan_plain(s):
    """Slots without an adapter (and rows behind the last request) come last
    in the order, as class S; unused rows of the tiles are (-1, 0, 0)."""
    M, S, dev = s["tokens"], s["S"], s["slots"].device
    ends = torch.cumsum(s["lengths"].long(), 0)
    owner = torch.cat([s["slots"].long(), torch.full((1,), -1, device=dev)])
    token_slot = owner[torch.searchsorted(ends, torch.arange(M, device=dev), right=True)]
    cls = torch.where(token_slot < 0, S, token_slot)
    order = torch.sort(cls, stable=True).indices
    count = torch.zeros(S + 1, dtype=torch.long, device=dev).index_add_(0, cls, torch.ones_like(cls))
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), torch.cumsum(count, 0)])
    last = torch.cumsum((count + TILE - 1) // TILE, 0)
    i = torch.arange(_tiles(M, S), device=dev)
    c = torch.searchsorted(last, i, right=True)
    real = c <= S
    c = torch.clamp(c, max=S)
    first = start[c] + TILE * (i - last[c] + (count[c] + TILE - 1) // TILE)
    n = torch.clamp(start[c + 1] - first, max=TILE)
    tiles = torch.stack([torch.where(c < S, c, -1), first, n], 1)
    tiles = torch.where(real[:, None], tiles, torch.tensor([-1, 0, 0], device=dev))
    return {k: v.int().contiguous() for k, v in
            dict(token_slot=token_slot, order=order, start=start, tiles=tiles).items()}


def _philox_round(c, i, seed):
    m = 0xFFFFFFFF
    k0 = ((seed & m) + i * 0x9E3779B9) & m
    k1 = ((seed >> 32) + i * 0xBB67AE85) & m
    p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57     # 64-bit products, wrapped
    return ((p1 >> 32) & m) ^ c[1] ^ k0, p1 & m, ((p0 >> 32) & m) ^ c[3] ^ k1, p0 & m


def _drop(x, s):
    """drop() of an fp32 [M, K]."""
    if not s["p"]:
        return x
    i = torch.arange(x.numel() // 4, device=x.device)
    c = (i & 0xFFFFFFFF, i >> 32, torch.zeros_like(i), torch.zeros_like(i))
    for rnd in range(10):
        c = _philox_round(c, rnd, s["seed"])
    keep = (torch.stack(c, 1) >= math.floor(s["p"] * 2.0 ** 32)).reshape(x.shape)
    return x * keep * (1.0 / (1.0 - s["p"]))


def _own_columns(x, s):
    """[M, S r] -> [M, r]: each token's columns of its slot (zeros without one)."""
    slot = s["plan"]["token_slot"].long()
    at = torch.clamp(slot, min=0)[:, None] * s["r"] + torch.arange(s["r"], device=x.device)
    return torch.gather(x, 1, at) * (slot >= 0)[:, None]


def _spread(t, s):
    """[M, r] -> [M, S r], scaled: zeros in the columns of other slots."""
    slot = s["plan"]["token_slot"][:, None]
    mine = slot == torch.arange(s["S"], device=t.device, dtype=torch.int32)
    return (t[:, None, :] * (mine * s["scale"])[:, :, None]).reshape(t.shape[0], -1)


def _down(x, s):
    """Each token's r products with the rows of its slot's A."""
    return _own_columns(x @ s["A"].float().reshape(-1, s["K"]).t(), s)


def _fwd_plain(s):
    T = _down(_drop(s["X"].float(), s), s)
    Bt = s["B"].float().permute(0, 2, 1).reshape(-1, s["N"])
    return {"out": (s["Y"].float() + _spread(T, s) @ Bt).bfloat16(), "T": T}


def _bwd_plain(s):
    dY, S, r = s["dY"].float(), s["S"], s["r"]
    U = _own_columns(dY @ s["B"].float().permute(1, 0, 2).reshape(s["N"], -1), s)
    Us = _spread(U, s)
    dX = s["dX0"].float() + _drop(Us @ s["A"].float().reshape(-1, s["K"]), s)
    dA = (Us.t() @ _drop(s["X"].float(), s)).reshape(S, r, s["K"])
    dB = (dY.t() @ _spread(s["T"], s)).reshape(s["N"], S, r).permute(1, 0, 2).contiguous()
    return {"dX": dX.bfloat16(), "dA": dA, "dB": dB}


def run(s):
    if own:
        import bit_nf4_quantized_07_amd as q
        if s["op"] == "plan":
            pl = q.adapter_plan(s["slots"], s["S"], lengths=s["lengths"], tokens=s["tokens"])
            return {"token_slot": pl.token_slot, "order": pl.order, "start": pl.start,
                    "tiles": pl.tiles}
        plan = q.AdapterPlan(S=s["S"], **s["plan"])
        drop = (s["p"], s["seed"]) if s["p"] else None
        if s["op"] == "fwd":
            out, T = q.adapters_fwd(s["X"], s["Y"], s["A"], s["B"], s["scale"], plan, dropout=drop)
            return {"out": out, "T": T}
        dX, dA, dB = q.adapters_bwd(s["dY"], s["X"], s["A"], s["B"], s["scale"], plan, T=s["T"],
                                    dX=s["dX0"], dropout=drop)
        return {"dX": dX, "dA": dA, "dB": dB}
    if s["op"] == "plan":
        return _plan_plain(s)
    return _fwd_plain(s) if s["op"] == "fwd" else _bwd_plain(s)


# ---- 64 bits ----------------------------------------------------------------

def _kept(case, seed):
    """drop()'s factors, [M, K] in 64 bits, from 32-bit words on the host."""
    M, K, p = case["tokens"], case["K"], case["p"]
    g = np.arange(M * K // 4, dtype=np.uint64)
    x = [g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), np.zeros_like(g), np.zeros_like(g)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        lo = np.uint64(0xFFFFFFFF)
        x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64(key[0]), b & lo,
             (a >> np.uint64(32)) ^ x[3] ^ np.uint64(key[1]), a & lo]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    words = np.stack(x, 1).reshape(M, K)
    return torch.from_numpy((words >= np.uint64(int(p * 4294967296))) / (1.0 - p)).cuda()


def exact(case, seed):
    """Slot by slot, in 64 bits."""
    if case["op"] == "plan":
        lengths, slots = _requests(case, seed)
        M, S = case["tokens"], case["S"]
        tok = np.concatenate([np.repeat(slots, lengths), np.full(case["pad"], -1)])
        groups = [np.flatnonzero(tok == c) for c in range(S)] + [np.flatnonzero(tok < 0)]
        start = np.concatenate([[0], np.cumsum([len(x) for x in groups])])
        tiles = np.tile([-1, 0, 0], (_tiles(M, S), 1))
        n = 0
        for c in range(S + 1):
            for f in range(int(start[c]), int(start[c + 1]), TILE):
                tiles[n] = c if c < S else -1, f, min(TILE, start[c + 1] - f)
                n += 1
        as_int = lambda v: torch.from_numpy(np.asarray(v, np.int32))
        return {"token_slot": as_int(tok), "order": as_int(np.concatenate(groups)),
                "start": as_int(start), "tiles": as_int(tiles)}
    s = prepare(case, seed)
    lengths, slots = _requests(case, seed)
    tok = np.concatenate([np.repeat(slots, lengths), np.full(case["pad"], -1)])
    keep = _kept(case, s["seed"]) if case["p"] else 1.0
    Xd = s["X"].double() * keep
    M, K, N, r, S = (case[k] for k in ("tokens", "K", "N", "r", "S"))
    f64 = dict(dtype=torch.float64, device="cuda")
    T = torch.zeros(M, r, **f64)
    if case["op"] == "fwd":
        out = s["Y"].double()
    else:
        out, dY = torch.zeros(M, K, **f64), s["dY"].double()
        dA, dB = torch.zeros(S, r, K, **f64), torch.zeros(S, N, r, **f64)
    for c in sorted(set(tok.tolist()) - {-1}):
        rows = torch.from_numpy(np.flatnonzero(tok == c)).cuda()
        A, B, sc = s["A"][c].double(), s["B"][c].double(), float(s["scale"][c])
        if case["op"] == "fwd":
            T[rows] = Xd[rows] @ A.t()
            out[rows] += sc * (T[rows] @ B.t())
        else:
            U = dY[rows] @ B
            out[rows] = sc * (U @ A)
            dA[c] = sc * (U.t() @ Xd[rows])
            dB[c] = sc * (dY[rows].t() @ s["T"][rows].double())
    if case["op"] == "fwd":
        return {"out": out, "T": T}
    return {"dX": s["dX0"].double() + out * keep, "dA": dA, "dB": dB}
