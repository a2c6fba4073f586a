"""Cases of several continuations verified side by side over one paged cache:
attention of groups of sequences that share a prefix, the resampling of
continuations (losers release their pages, winners are forked), the accepted
path of a token tree moved to the front, and the log probabilities of the
emitted tokens with the entropy and the top alternatives.

Each operator has its plain form (elementary torch operations in 32 bits), the
library's call, and its definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
DEV = "cuda"
D = 128


# ------------------------------------------------------------------ cases

def listed():
    return [
        # four continuations of one short prompt, a token each: latency
        dict(name="shared-decode-short", op="shared", cache="bf16", groups=1, n=4, k=1, Hq=32,
             Hkv=8, P=16, slo=448, shi=448, olo=20, ohi=120, tree=False),
        # best of 32 on one prompt, a mid-size target with four drafts
        dict(name="shared-8b-best-of-32", op="shared", cache="bf16", groups=1, n=32, k=4, Hq=32,
             Hkv=8, P=16, slo=6000, shi=6000, olo=100, ohi=900, tree=False),
        # four prompts of 32 rollouts each, a large target's layer, 8-bit floating cache
        dict(name="shared-70b-rollouts", op="shared", cache="e4m3", groups=4, n=32, k=4, Hq=64,
             Hkv=8, P=16, slo=2000, shi=8000, olo=100, ohi=1500, tree=False),
        # token trees behind one long document, INT8 cache, 112 query rows a sequence
        dict(name="shared-long-trees", op="shared", cache="i8", groups=1, n=16, k=16, Hq=28,
             Hkv=4, P=32, slo=32768, shi=32768, olo=50, ohi=400, tree=True),
        # the best of four continuations goes on three times
        dict(name="fork-best-of-4", op="fork", cache="bf16", parents=1, n=3, Hkv=8, P=16, lo=905,
             hi=905, room=5),
        # beams of eight prompts resampled, 8-bit floating cache
        dict(name="fork-beams", op="fork", cache="e4m3", parents=8, n=7, Hkv=8, P=16, lo=1024,
             hi=8192, room=16),
        # sixteen long contexts, fifteen rollouts each, INT8 cache
        dict(name="fork-long", op="fork", cache="i8", parents=16, n=15, Hkv=8, P=16, lo=16384,
             hi=32768, room=16),
        # the accepted path of one small tree: latency
        dict(name="compact-single", op="compact", cache="bf16", B=1, k=8, Hkv=8, P=16, lo=777,
             hi=777),
        # trees of 64 nodes of many sequences, pages of 16, 8-bit floating cache
        dict(name="compact-trees", op="compact", cache="e4m3", B=64, k=64, Hkv=8, P=16, lo=500,
             hi=4000),
        # five rows of a small vocabulary: latency
        dict(name="logprob-tiny", op="logprob", dtype="f32", B=1, n=5, V=1000, K=5, T=1.0,
             ragged=False, masked=False),
        # the emitted tokens of the ragged step, twenty alternatives
        dict(name="logprob-8b-step", op="logprob", dtype="bf16", B=32, n=5, V=128256, K=20, T=0.7,
             ragged=True, masked=False),
        # a prompt scored: every position of two thousand
        dict(name="logprob-prompt", op="logprob", dtype="bf16", B=1, n=2048, V=152064, K=5, T=1.0,
             ragged=False, masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "fork", "compact", "logprob", "logprob"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (28, 4), (32, 32), (12, 2), (16, 1)])
    P = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["bf16", "e4m3", "i8"])
    if op == "shared":
        G = Hq // Hkv
        k = rng.randint(1, min(16, 128 // G))
        groups = _log(rng, 1, 8)
        n = max(2, min(_log(rng, 2, 64), 160 // groups))
        # keys times query heads, so that no case costs more than the largest
        most = max(200, min(32768, 200_000_000 // (groups * n * k * Hq)))
        shi = _log(rng, 40, most)
        ohi = max(2, min(_log(rng, 2, 2048), most, 40_000_000 // (groups * n * Hkv * D)))
        return dict(op=op, cache=cache, groups=groups, n=n, k=k, Hq=Hq, Hkv=Hkv, P=P,
                    slo=int(shi * rng.uniform(0.2, 1.0)), shi=shi,
                    olo=int(ohi * rng.uniform(0.0, 1.0)), ohi=ohi, tree=rng.random() < 0.3)
    if op == "fork":
        parents, n = _log(rng, 1, 16), _log(rng, 1, 15)
        hi = max(20, min(_log(rng, 20, 32768), 4_000_000 // (parents * Hkv)))
        return dict(op=op, cache=cache, parents=parents, n=n, Hkv=Hkv, P=P,
                    lo=int(hi * rng.uniform(0.1, 1.0)), hi=hi, room=rng.choice([0, 1, 5, 16, 100]))
    if op == "compact":
        hi = _log(rng, 10, 4000)
        return dict(op=op, cache=cache, B=_log(rng, 1, 64), k=rng.randint(2, 64), Hkv=Hkv, P=P,
                    lo=int(hi * rng.uniform(0.0, 1.0)), hi=hi)
    V = rng.choice([32000, 128256, 152064, _log(rng, 40, 150000), 2 * _log(rng, 500, 70000) + 1])
    B = _log(rng, 1, 64)
    n = max(1, min(_log(rng, 1, 2048), 280_000_000 // (B * V)))
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), B=B, n=n, V=V,
                K=rng.choice([0, 1, 5, 20, 32]), T=rng.choice([0.5, 0.7, 1.0, 1.3]),
                ragged=rng.random() < 0.5, masked=rng.random() < 0.3)


def _spread(lo, hi, count):
    """Lengths spread evenly over [lo, hi], odd ones among them (the work does
    not depend on the seed; their order does)."""
    return [lo + (hi - lo) * (2 * i + 1) // (2 * count) for i in range(count)]


def _shared(case):
    """Keys that each group shares: whole pages, as a fork leaves them."""
    return [s // case["P"] * case["P"] for s in _spread(case["slo"], case["shi"], case["groups"])]


def _kept(case):
    """Nodes of each sequence's tree that were accepted: at most half."""
    return [(7 * b + 3) % (case["k"] // 2 + 1) for b in range(case["B"])]


def _rows(case):
    """Rows of each sequence whose token was emitted."""
    B, n = case["B"], case["n"]
    if not case["ragged"]:
        return [n] * B
    return [1 + (3 * b + n // 2) % n for b in range(B)]


def _elem(case):
    return 2 if case["cache"] == "bf16" else 1


def _scale_bytes(case, keys, pages):
    """Scales of one kv-head, k and v: INT8 two bytes a key, e4m3 four a page."""
    return {"bf16": 0, "i8": 4 * keys, "e4m3": 8 * pages}[case["cache"]]


def work(case):
    op = case["op"]
    if op == "shared":
        B, k, Hq, Hkv, P = case["groups"] * case["n"], case["k"], case["Hq"], case["Hkv"], case["P"]
        own_keys = _spread(case["olo"], case["ohi"], B)
        shared = _shared(case)
        distinct = sum(shared) + sum(o + k for o in own_keys)
        pages = sum(s // P for s in shared) + sum(-(-(o + k) // P) for o in own_keys)
        seen = case["n"] * sum(shared) + sum(o + k for o in own_keys)
        nbytes = Hkv * (2 * distinct * D * _elem(case) + _scale_bytes(case, distinct, pages))
        nbytes += 4 * pages + 4 * B + B * k * Hq * (2 * 2 * D + 4) + (8 * B * k if case["tree"] else 0)
        return {"bytes": nbytes, "flops": 4 * k * Hq * D * seen}
    if op == "fork":
        P, Hkv, n = case["P"], case["Hkv"], case["n"]
        lens = _spread(case["lo"], case["hi"], case["parents"])
        part = sum(c % P for c in lens) * n  # rows copied, read and written
        whole = sum(c // P for c in lens)
        copied = Hkv * (2 * part * D * _elem(case) + _scale_bytes(case, part, len(lens) * n))
        # tables and counts of holders: entries released and written, counts down and up
        ints = 4 * (whole * (1 + 2 * n) + 4 * whole * n)
        return {"bytes": 2 * copied + ints, "flops": 2 * whole * n}
    if op == "compact":
        rows = sum(_kept(case))
        return {"bytes": 2 * case["Hkv"] * 2 * rows * D * _elem(case) + 4 * case["B"] * case["k"],
                "flops": 2 * case["Hkv"] * rows * D}
    rows = sum(_rows(case))
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": rows * (case["V"] * size + 12 + 8 * case["K"]), "flops": 6 * rows * case["V"]}


# ------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pool(case, gen, NP, pages=None):
    """A pool of rows whose magnitude differs from page to page (or as `pages`
    [NP] gives it): cache and scales."""
    x = torch.randn((NP, case["Hkv"], case["P"], D), generator=gen, device=DEV)
    if pages is None:
        x *= torch.exp(0.3 * torch.randn(NP, case["Hkv"], 1, 1, generator=gen, device=DEV))
    else:
        x = x.clamp(-4.0, 4.0) * pages[:, None, None, None]
    if case["cache"] == "bf16":
        return x.bfloat16(), None
    if case["cache"] == "i8":
        s = (x.abs().amax(-1) / 127).half()
        return torch.round(x / s.float()[..., None]).clamp(-127, 127).to(torch.int8), s
    s = x.abs().amax((2, 3)) / E4M3_MAX
    if pages is not None:  # one scale for pages of one magnitude
        s = (pages * (4.0 / E4M3_MAX))[:, None].expand_as(s).contiguous()
    return (x / s[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s


def _caches(s, case, gen, NP, pages=None):
    s["k_cache"], s["k_scale"] = _pool(case, gen, NP, pages)
    s["v_cache"], s["v_scale"] = _pool(case, gen, NP, pages)


def _tree(B, k, r):
    """Ancestor masks of random trees (bit t of row i: node i sees node t)."""
    mask = np.zeros((B, k), np.int64)
    for b in range(B):
        for i in range(k):
            p = r.randint(-1, i) if i else -1
            mask[b, i] = (1 << i) | (int(mask[b, p]) if p >= 0 else 0)
    return mask


def _prepare_shared(case, gen, r):
    P, k, Hq, n = case["P"], case["k"], case["Hq"], case["n"]
    B = case["groups"] * n
    shared = [_shared(case)[i] for i in r.permutation(case["groups"])]
    own_keys = [_spread(case["olo"], case["ohi"], B)[i] for i in r.permutation(B)]
    ctx = [shared[b // n] + own_keys[b] for b in range(B)]
    need = [-(-(own_keys[b] + k) // P) for b in range(B)]
    NP = sum(s // P for s in shared) + sum(need) + 3
    perm = torch.randperm(NP, generator=gen, device=DEV).int()
    table = torch.zeros(B, max(-(-(c + k) // P) for c in ctx), dtype=torch.int32, device=DEV)
    at = 0
    for g, length in enumerate(shared):
        m = length // P
        table[g * n:(g + 1) * n, :m] = perm[at:at + m]
        at += m
        for b in range(g * n, (g + 1) * n):
            table[b, m:m + need[b]] = perm[at:at + need[b]]
            at += need[b]
    s = {"case": case, "table": table, "ctx": _ints(ctx), "shared": _ints(shared),
         "starts": _ints([g * n for g in range(case["groups"] + 1)])}
    s["own_max"] = max(own_keys) + k
    s["shared_max"] = max(shared)
    _caches(s, case, gen, NP)
    # queries a little longer than unit length: some keys stand out
    s["q"] = (1.5 * torch.randn(B, k, Hq, D, generator=gen, device=DEV)).bfloat16()
    s["mask"] = torch.from_numpy(_tree(B, k, r)).to(DEV) if case["tree"] else None
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, k, Hq, device=DEV)
    return s


def _prepare_fork(case, gen, r):
    """Rows of parents, then of their children, which hold a short continuation
    of their own before they are resampled."""
    P, parents, n = case["P"], case["parents"], case["n"]
    rows = parents * (1 + n)
    lens = [_spread(case["lo"], case["hi"], parents)[i] for i in r.permutation(parents)]
    short = _spread(1, 6 * P, rows - parents)
    ctx = lens + [short[i] for i in r.permutation(rows - parents)]
    held = [-(-c // P) for c in ctx]
    spare = 3 + (rows - parents) * (2 + case["room"] // P)
    NP = sum(held) + spare
    table = torch.full((rows, max(held) + 2 + case["room"] // P), -1, dtype=torch.int32, device=DEV)
    refs = torch.zeros(NP, dtype=torch.int32, device=DEV)
    perm = torch.randperm(NP, generator=gen, device=DEV).int()
    at = 0
    for b, m in enumerate(held):
        table[b, :m] = perm[at:at + m]
        at += m
    refs[perm[:at].long()] = 1
    s = {"case": case, "table": table, "ctx": _ints(ctx), "refs": refs}
    s["children"] = _ints(list(range(parents, rows)))
    s["parents"] = _ints([j // n for j in range(parents * n)])
    _caches(s, case, gen, NP)
    return s


def _prepare_compact(case, gen, r):
    B, k, P = case["B"], case["k"], case["P"]
    ctx = [_spread(case["lo"], case["hi"], B)[i] for i in r.permutation(B)]
    need = [-(-(c + k) // P) for c in ctx]
    NP = sum(need) + 3
    perm = torch.randperm(NP, generator=gen, device=DEV).int()
    table = torch.zeros(B, max(need), dtype=torch.int32, device=DEV)
    # rows of a sequence's pages after the first that holds drafts are larger
    # than before it, and alike among themselves: a moved row may raise the
    # scale of an e4m3 page
    size = torch.ones(NP, device=DEV)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        size[table[b, :ctx[b] // P + 1].long()] = 0.25 + 0.5 * float(r.rand())
        at += m
    # the kept nodes: the first few are in their place, the rest come from
    # behind the places that are filled
    kept = _kept(case)
    path = np.full((B, k), -1, np.int32)
    for b, m in enumerate(kept):
        stay = r.randint(0, m + 1)
        path[b, :stay] = np.arange(stay)
        path[b, stay:m] = np.sort(r.permutation(np.arange(m, k))[:m - stay])
    s = {"case": case, "table": table, "ctx": _ints(ctx), "accepted": _ints(kept),
         "path": torch.from_numpy(path).to(DEV)}
    _caches(s, case, gen, NP, size)
    return s


def _prepare_logprob(case, gen, r):
    B, n, V, K = case["B"], case["n"], case["V"], case["K"]
    x = torch.empty(B, n, V, dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16,
                    device=DEV)
    x.normal_(0.0, 2.0, generator=gen)
    if case["masked"]:  # a grammar allows part of the vocabulary
        closed = torch.rand(V, generator=gen, device=DEV) < 0.5
        closed[0] = False
        x.masked_fill_(closed, -math.inf)
    # likely tokens for the most part: the largest of a few candidates
    pick = torch.randint(0, V, (B, n, 64), generator=gen, device=DEV)
    pick[..., 0] = 0
    best = x.gather(2, pick).argmax(-1, keepdim=True)
    s = {"case": case, "logits": x, "tokens": pick.gather(2, best)[..., 0].int()}
    rows = [_rows(case)[i] for i in r.permutation(B)]
    s["lens"] = _ints(rows) if case["ragged"] else None
    s["logprob"] = torch.zeros(B, n, device=DEV)
    s["entropy"] = torch.zeros(B, n, device=DEV)
    s["top_ids"] = torch.zeros(B, n, K, dtype=torch.int32, device=DEV) if K else None
    s["top_logprobs"] = torch.zeros(B, n, K, device=DEV) if K else None
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    make = {"shared": _prepare_shared, "fork": _prepare_fork, "compact": _prepare_compact,
            "logprob": _prepare_logprob}[case["op"]]
    return make(case, gen, np.random.RandomState(seed % (1 << 31)))


# ------------------------------------------------------------------ plain forms

def _bytes(t):
    """A cache as bytes where torch cannot index its type."""
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def _values(cache, scale, page, slot):
    """Rows at (page, slot) in fp32: [..., Hkv, D]."""
    x = _bytes(cache)[page, :, slot].view(cache.dtype).float()
    if scale is None:
        return x
    return x * (scale[page] if scale.dim() == 2 else scale[page, :, slot].float())[..., None]


def _partial(q, kd, vd, see):
    """Unnormalised attention of q [.., R, D] over kd, vd [.., J, D] where `see`
    allows: maximum, sum and output."""
    sc = (q @ kd.transpose(-1, -2)) * (D ** -0.5)
    sc = torch.where(see, sc, torch.full((), -math.inf, device=DEV))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.clamp_min(-3e38))
    return m, p.sum(-1, keepdim=True), p @ vd


def _plain_shared(s):
    case, q, ctx = s["case"], s["q"], s["ctx"].long()
    B, k, Hq, _ = q.shape
    Hkv, P, n, Gp = case["Hkv"], case["P"], case["n"], case["groups"]
    G = Hq // Hkv
    table, shared = s["table"].long(), s["shared"].long()
    # the prefixes, once for a group: [Gp, Hkv, n * k * G, D] over [Gp, Hkv, J, D]
    j = torch.arange(s["shared_max"], device=DEV)
    page = table[::n].gather(1, (j // P).clamp_max(table.shape[1] - 1).expand(Gp, -1))
    qd = q.float().view(Gp, n, k, Hkv, G, D).permute(0, 3, 1, 2, 4, 5)
    kd = _values(s["k_cache"], s["k_scale"], page, j % P).transpose(1, 2)
    vd = _values(s["v_cache"], s["v_scale"], page, j % P).transpose(1, 2)
    see = (j[None, :] < shared[:, None])[:, None, None, :]
    m1, l1, o1 = _partial(qd.reshape(Gp, Hkv, n * k * G, D), kd, vd, see)

    def split(x):  # [Gp, Hkv, n * k * G, c] -> [B, Hkv, k * G, c]
        c = x.shape[-1]
        return x.view(Gp, Hkv, n, k * G, c).transpose(1, 2).reshape(B, Hkv, k * G, c)

    # what each sequence has of its own
    first = shared.repeat_interleave(n)
    pos = first[:, None] + torch.arange(s["own_max"], device=DEV)
    last = (ctx + k - 1)[:, None]
    page = table.gather(1, torch.minimum(pos, last) // P)
    kd = _values(s["k_cache"], s["k_scale"], page, pos % P).transpose(1, 2)
    vd = _values(s["v_cache"], s["v_scale"], page, pos % P).transpose(1, 2)
    t = (pos - ctx[:, None])[:, None, :]  # draft index of a key, negative in the context
    i = torch.arange(k, device=DEV)[None, :, None]
    if s["mask"] is None:
        see = t <= i
    else:
        see = (t < 0) | ((((s["mask"][:, :, None] >> t.clamp(0, 63)) & 1) == 1) & (t < k))
    see = see[:, None, :, None, :].expand(B, 1, k, G, -1).reshape(B, 1, k * G, -1)
    qd = q.float().view(B, k, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, k * G, D)
    vd = torch.where((t < k).transpose(1, 2)[:, None], vd, torch.zeros((), device=DEV))
    m2, l2, o2 = _partial(qd, kd, vd, see)
    m1, l1, o1 = split(m1), split(l1), split(o1)
    m = torch.maximum(m1, m2)
    w1, w2 = torch.exp(m1 - m), torch.exp(m2 - m)
    l = w1 * l1 + w2 * l2
    o = (w1 * o1 + w2 * o2) / l
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.view(B, Hkv, k, G, D).transpose(1, 2).reshape(B, k, Hq, D)
    return [o.bfloat16(), lse.view(B, Hkv, k, G).transpose(1, 2).reshape(B, k, Hq)]


def _outputs(s, extra=()):
    out = [s["k_cache"], s["v_cache"], *extra]
    return out if s["k_scale"] is None else out + [s["k_scale"], s["v_scale"]]


def _plain_fork(s):
    case = s["case"]
    P, room = case["P"], case["room"]
    table, refs, ctx = s["table"], s["refs"], s["ctx"]
    kids, par = s["children"].long(), s["parents"].long()
    MP = table.shape[1]
    # the children's pages lose a holder
    old = table[kids]
    ones = (old >= 0).int()
    refs.index_add_(0, old.clamp_min(0).reshape(-1).long(), -ones.reshape(-1))
    # whole pages are shared; the page in use and those for `room` tokens are fresh
    c = ctx[par].long()
    whole, need = c // P, -(-(c + room) // P) - c // P
    at = torch.arange(MP, device=DEV)[None, :]
    keep = at < whole[:, None]
    source = table[par]
    ones = keep.int()
    refs.index_add_(0, torch.where(keep, source, 0).reshape(-1).long(), ones.reshape(-1))
    free = torch.nonzero(refs == 0)[:, 0]
    before = torch.cumsum(need, 0) - need
    rank = before[:, None] + at - whole[:, None]
    fresh = (at >= whole[:, None]) & (at < (whole + need)[:, None])
    pages = free[torch.where(fresh, rank, 0)]
    refs[pages[fresh]] = 1
    table[kids] = torch.where(keep, source, torch.where(fresh, pages.int(), -1))
    ctx[kids] = c.int()
    # the rows of the page in use
    part = c % P
    slot = torch.arange(P, device=DEV)
    mine = (slot[None, :] < part[:, None])
    src = source.gather(1, whole.clamp_max(MP - 1)[:, None])[:, 0].clamp_min(0).long()
    dst = torch.where(part > 0, pages.gather(1, whole.clamp_max(MP - 1)[:, None])[:, 0], -1)
    j, p = torch.nonzero(mine, as_tuple=True)
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        b = _bytes(cache)
        b[dst[j], :, p] = b[src[j], :, p]
        if scale is not None and scale.dim() == 3:
            scale[dst[j], :, p] = scale[src[j], :, p]
        elif scale is not None:
            used = dst >= 0
            scale[dst[used]] = scale[src[used]]
    return _outputs(s, (table, ctx, refs))


def _plain_compact(s):
    case, path = s["case"], s["path"].long()
    B, k, P = case["B"], case["k"], case["P"]
    ctx, n = s["ctx"].long()[:, None], s["accepted"].long()[:, None]
    i = torch.arange(k, device=DEV)[None, :]
    moved = (i < n) & (path != i)
    table = s["table"].long()
    here, there = ctx + i, ctx + torch.where(moved, path, i)
    dst, src = table.gather(1, here // P), table.gather(1, there // P)
    b, t = torch.nonzero(moved, as_tuple=True)
    d, u, ds, us = dst[b, t], src[b, t], (here % P)[b, t], (there % P)[b, t]
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        if scale is None or scale.dim() == 3:
            cache[d, :, ds] = cache[u, :, us]
            if scale is not None:
                scale[d, :, ds] = scale[u, :, us]
            continue
        rows = _values(cache, scale, u, us)  # [rows, Hkv, D]
        top = torch.where((d != u)[:, None], rows.abs().amax(-1) / E4M3_MAX, 0.0)
        grown = scale.clone()
        grown.scatter_reduce_(0, d[:, None].expand_as(top), top, "amax")
        # every row of a grown page keeps its value: slots below ctx + k
        pg = torch.arange(table.shape[1], device=DEV)[None, :]
        some = (pg >= ctx // P) & (pg <= (ctx + k - 1) // P)
        bb, pp = torch.nonzero(some, as_tuple=True)
        ids = table[bb, pp]
        mine = torch.arange(P, device=DEV)[None, :] < (ctx[bb, 0] + k - pp * P)[:, None]
        pick = mine[:, None, :, None] & (grown[ids] > scale[ids])[:, :, None, None]
        codes = _bytes(cache)[ids].view(E4M3)
        again = (codes.float() * scale[ids][..., None, None] / grown[ids][..., None, None])
        again = again.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        _bytes(cache)[ids] = torch.where(pick, _bytes(again), _bytes(codes))
        # an arriving row is rounded once more only where the scales differ
        x = (rows / grown[d][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
        _bytes(cache)[d, :, ds] = _bytes(x)
        scale.copy_(grown)
    return _outputs(s)


def _plain_logprob(s):
    case, x = s["case"], s["logits"]
    V, K = case["V"], case["K"]
    z = x.float() / case["T"]
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    lse = m + torch.log(l)
    lp = z.gather(2, s["tokens"].long()[..., None]) - lse
    ent = torch.log(l) - torch.where(e > 0, e * (z - m), 0.0).sum(-1, keepdim=True) / l
    rows = torch.arange(case["n"], device=DEV)[None, :]
    ok = rows < (s["lens"][:, None] if s["lens"] is not None else case["n"])
    out = [torch.where(ok, lp[..., 0], s["logprob"]), torch.where(ok, ent[..., 0], s["entropy"])]
    if K:
        # unique keys: the value's bits in the order of the values, then the lower index
        kk = min(K, V)
        bits = (x.float() + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = bits * (1 << 31) + (V - 1 - torch.arange(V, device=DEV))
        ids = torch.topk(key, kk, dim=-1).indices
        top = z.gather(2, ids) - lse
        ids = torch.where(top > -math.inf, ids, -1)  # a masked token is no alternative
        ids = torch.nn.functional.pad(ids, (0, K - kk), value=-1)
        top = torch.nn.functional.pad(top, (0, K - kk), value=-math.inf)
        out += [torch.where(ok[..., None], ids.int(), s["top_ids"]),
                torch.where(ok[..., None], top, s["top_logprobs"])]
    return out


# ------------------------------------------------------------------ the library's calls

def _own_run(s):
    from speculative_decoding_verification_attn_gb300 import binding
    case = s["case"]
    op = case["op"]
    if op == "shared":
        binding.spec_verify_attn_shared(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"],
                                        s["starts"], s["shared"], case["k"], D ** -0.5, s["out"],
                                        s["lse"], s["k_scale"], s["v_scale"], tree_mask=s["mask"])
        return [s["out"], s["lse"]]
    if op == "fork":
        binding.spec_kv_release(s["table"], s["ctx"], s["refs"], s["children"], case["P"])
        binding.spec_kv_fork(s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["refs"],
                             s["parents"], s["children"], case["room"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"])
        return _outputs(s, (s["table"], s["ctx"], s["refs"]))
    if op == "compact":
        binding.spec_kv_compact(s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["path"],
                                s["accepted"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        return _outputs(s)
    binding.spec_token_logprobs(s["logits"], s["tokens"], s["logprob"], entropy=s["entropy"],
                                top_ids=s["top_ids"], top_logprobs=s["top_logprobs"],
                                lens=s["lens"], temperature=case["T"])
    out = [s["logprob"], s["entropy"]]
    return out + [s["top_ids"], s["top_logprobs"]] if case["K"] else out


def run(state):
    if own:
        return _own_run(state)
    return {"shared": _plain_shared, "fork": _plain_fork, "compact": _plain_compact,
            "logprob": _plain_logprob}[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits

def _rows64(s, which, b, count):
    """Rows 0 .. count - 1 of sequence b, [count, Hkv, D] in fp64."""
    P = s["case"]["P"]
    ids = s["table"][b, :-(-count // P)].long()
    x = _bytes(s[which + "_cache"])[ids].view(s[which + "_cache"].dtype).double()
    scale = s[which + "_scale"]
    if scale is not None:
        x = x * scale[ids].double().view(len(ids), s["case"]["Hkv"], -1, 1)
    return x.permute(0, 2, 1, 3).reshape(-1, s["case"]["Hkv"], D)[:count]


def _exact_shared(s):
    case = s["case"]
    k, Hq, Hkv = case["k"], case["Hq"], case["Hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(out.shape[:3], dtype=torch.float64, device=DEV)
    masks = s["mask"].tolist() if s["mask"] is not None else None
    for b, ctx in enumerate(s["ctx"].tolist()):
        K, V = _rows64(s, "k", b, ctx + k), _rows64(s, "v", b, ctx + k)
        hidden = torch.zeros(k, ctx + k, dtype=torch.bool, device=DEV)
        for i in range(k):
            row = masks[b][i] if masks else (1 << (i + 1)) - 1
            hidden[i, ctx:] = torch.tensor([not (row >> t) & 1 for t in range(k)], device=DEV)
        q = s["q"][b].double().view(k, Hkv, Hq // Hkv, D)
        z = torch.einsum("ihgd,jhd->ihgj", q, K) / math.sqrt(D)
        z.masked_fill_(hidden[:, None, None, :], -math.inf)
        lse[b] = torch.logsumexp(z, -1).reshape(k, Hq)
        out[b] = torch.einsum("ihgj,jhd->ihgd", torch.softmax(z, -1), V).reshape(k, Hq, D)
    return [out, lse]


def _exact_fork(s):
    case = s["case"]
    P, room = case["P"], case["room"]
    table, refs = s["table"].cpu().numpy(), s["refs"].cpu().numpy()
    ctx = s["ctx"].cpu().numpy()
    kids, par = s["children"].tolist(), s["parents"].tolist()
    for c in kids:
        held = table[c][table[c] >= 0]
        refs[held] -= 1
        table[c] = -1
        ctx[c] = 0
    shares = np.zeros_like(refs)
    free = [int(p) for p in np.nonzero(refs == 0)[0]]
    moves = []
    for p, c in zip(par, kids):
        length = int(ctx[p])
        whole, total = length // P, -(-(length + room) // P)
        table[c, :whole] = table[p, :whole]
        shares[table[p, :whole]] += 1
        for at in range(whole, total):
            table[c, at] = free.pop(0)
            shares[table[c, at]] += 1
        if length % P:
            moves.append((int(table[p, whole]), int(table[c, whole]), length % P))
        ctx[c] = length
    out = []
    for w in "kv":
        cache, scale = s[w + "_cache"], s[w + "_scale"]
        for a, b, m in moves:
            _bytes(cache)[b, :, :m] = _bytes(cache)[a, :, :m]
            if scale is not None and scale.dim() == 3:
                scale[b, :, :m] = scale[a, :, :m]
            elif scale is not None:
                scale[b] = scale[a]
    out = [s["k_cache"], s["v_cache"], torch.from_numpy(table), torch.from_numpy(ctx),
           torch.from_numpy(refs + shares)]
    return out if s["k_scale"] is None else out + [s["k_scale"], s["v_scale"]]


def _exact_compact(s):
    case = s["case"]
    k, P = case["k"], case["P"]
    table, ctx = s["table"].tolist(), s["ctx"].tolist()
    path, kept = s["path"].tolist(), s["accepted"].tolist()
    new = {}
    for w in "kv":
        cache, scale = s[w + "_cache"].double(), s[w + "_scale"]
        paged = scale is not None and scale.dim() == 2
        wide = None if scale is None else scale.double()
        before, sizes = cache.clone(), None if wide is None else wide.clone()
        for b, n in enumerate(kept):
            go = [(ctx[b] + i, ctx[b] + path[b][i]) for i in range(n) if path[b][i] != i]
            if paged:
                for to, of in go:
                    d, u = table[b][to // P], table[b][of // P]
                    if d != u:
                        top = (before[u, :, of % P] * sizes[u][:, None]).abs().amax(-1) / E4M3_MAX
                        wide[d] = torch.maximum(wide[d], top)
                for g in range(ctx[b] // P, (ctx[b] + k - 1) // P + 1):
                    p, m = table[b][g], min(P, ctx[b] + k - g * P)
                    up = (wide[p] > sizes[p])[:, None, None]
                    again = before[p, :, :m] * (sizes[p] / wide[p])[:, None, None]
                    cache[p, :, :m] = torch.where(up, again.float().to(E4M3).double(),
                                                  before[p, :, :m])
            for to, of in go:
                d, u = table[b][to // P], table[b][of // P]
                row = before[u, :, of % P]
                if paged:
                    row = (row * (sizes[u] / wide[d])[:, None]).float().to(E4M3).double()
                elif wide is not None:
                    wide[d, :, to % P] = sizes[u, :, of % P]
                cache[d, :, to % P] = row
        new[w] = (cache, wide)
    out = [new["k"][0], new["v"][0]]
    return out if new["k"][1] is None else out + [new["k"][1], new["v"][1]]


def _exact_logprob(s):
    case, x = s["case"], s["logits"]
    V, K = case["V"], case["K"]
    lens = _rows(case) if s["lens"] is None else s["lens"].tolist()
    out = [s["logprob"].double(), s["entropy"].double()]
    if K:
        out += [s["top_ids"].clone(), s["top_logprobs"].double()]
    for b, n in enumerate(lens):
        for a in range(0, n, 64):
            e = min(n, a + 64)
            raw = x[b, a:e].double()
            logp = torch.log_softmax(raw / case["T"], -1)
            out[0][b, a:e] = logp.gather(1, s["tokens"][b, a:e].long()[:, None])[:, 0]
            out[1][b, a:e] = -torch.nan_to_num(torch.exp(logp) * logp, nan=0.0).sum(-1)
            if K:
                kk = min(K, V)
                ids = torch.sort(raw, dim=-1, descending=True, stable=True).indices[:, :kk]
                out[3][b, a:e, :kk] = logp.gather(1, ids)
                out[2][b, a:e, :kk] = torch.where(torch.isinf(raw.gather(1, ids)), -1, ids).int()
                out[2][b, a:e, kk:] = -1
                out[3][b, a:e, kk:] = -math.inf
    return out


def exact(case, seed):
    return {"shared": _exact_shared, "fork": _exact_fork, "compact": _exact_compact,
            "logprob": _exact_logprob}[case["op"]](prepare(case, seed))
