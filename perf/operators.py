"""Cases of the verification step over an 8-bit paged cache: attention over an
e4m3 cache with one scale per (page, kv-head), attention with a sliding window
and sinks, rotary positions with the append, and the cache read back.

Each operator has its plain form (elementary torch operations in 32 bits,
angles in 64), the library's call, and its definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one short conversation: latency
        dict(name="e4m3-decode-short", op="attn", cache="e4m3", B=1, k=1, Hq=32, Hkv=8, P=16,
             lo=100, hi=100, tree=False, window=0, sinks=0),
        # the ragged grouped-query step of a mid-size target
        dict(name="e4m3-8b-ragged", op="attn", cache="e4m3", B=32, k=4, Hq=32, Hkv=8, P=16,
             lo=1024, hi=8192, tree=False, window=0, sinks=0),
        # a large target's layer: eight drafts, 64 query rows per kv-head
        dict(name="e4m3-70b-layer", op="attn", cache="e4m3", B=32, k=8, Hq=64, Hkv=8, P=16,
             lo=2048, hi=2048, tree=False, window=0, sinks=0),
        # long contexts, a token tree of sixteen nodes, 112 query rows
        dict(name="e4m3-long-tree", op="attn", cache="e4m3", B=4, k=16, Hq=28, Hkv=4, P=32,
             lo=32768, hi=32768, tree=True, window=0, sinks=0),
        # single tokens of two short sequences in a sliding-window layer
        dict(name="window-decode-short", op="window", cache="bf16", B=2, k=1, Hq=28, Hkv=4, P=16,
             lo=301, hi=555, tree=False, window=128, sinks=4),
        # a sliding-window layer of the ragged step, bf16 cache
        dict(name="window-bf16-8b", op="window", cache="bf16", B=32, k=4, Hq=32, Hkv=8, P=16,
             lo=1024, hi=8192, tree=False, window=2048, sinks=4),
        # a streaming window over long contexts, 8-bit cache
        dict(name="window-e4m3-long", op="window", cache="e4m3", B=16, k=16, Hq=28, Hkv=4, P=32,
             lo=16384, hi=32768, tree=False, window=4096, sinks=16),
        # one token of one sequence: latency of rotation, quantisation and append
        dict(name="rope-append-single", op="rope", cache="e4m3", B=1, n=1, Hq=32, Hkv=8, P=16,
             lo=777, hi=777, rot=128, inter=False, scaling="none", factor=1.0, ragged=False),
        # the drafts of the ragged step into pages that are partly full
        dict(name="rope-append-8b-step", op="rope", cache="e4m3", B=32, n=4, Hq=32, Hkv=8, P=16,
             lo=1024, hi=8192, rot=128, inter=False, scaling="yarn", factor=4.0, ragged=False),
        # prompts of unequal lengths after long prefixes, half of the head rotated
        dict(name="rope-append-prompts", op="rope", cache="bf16", B=8, n=2048, Hq=32, Hkv=8, P=16,
             lo=0, hi=65536, rot=64, inter=True, scaling="linear", factor=8.0, ragged=True),
        # a short prefix read back for another consumer
        dict(name="gather-short", op="gather", cache="e4m3", B=1, Hkv=8, P=16, lo=203, hi=203,
             start=5),
        # every sequence of the ragged step read back to bf16
        dict(name="gather-8b-ragged", op="gather", cache="e4m3", B=32, Hkv=8, P=16, lo=1024,
             hi=8192, start=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "window", "rope", "gather"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (28, 4), (32, 32), (12, 2), (16, 1)])
    P = rng.choice([16, 32, 64, 128])
    cache = rng.choice(["e4m3", "bf16"]) if op in ("window", "rope") else "e4m3"
    if op in ("attn", "window"):
        G = Hq // Hkv
        k = rng.randint(1, min(16, 128 // G))
        B = _log(rng, 1, 32)
        room = 64_000_000 // (B * max(256, Hkv * 128))  # keys of a sequence
        hi = max(40, min(32768, _log(rng, 40, 32768), room))
        lo = max(0, int(hi * rng.uniform(0.1, 1.0)))
        case = dict(op=op, cache=cache, B=B, k=k, Hq=Hq, Hkv=Hkv, P=P, lo=lo, hi=hi,
                    tree=rng.random() < 0.3, window=0, sinks=0)
        if op == "window":
            case["window"] = max(k, _log(rng, 17, 8192))
            case["sinks"] = rng.choice([0, 1, 4, 16, 130])
        return case
    if op == "rope":
        B = _log(rng, 1, 32)
        n = max(1, min(_log(rng, 1, 2048), 12000 // B))
        hi = min(_log(rng, 10, 65536), 4_000_000 // (B * Hkv))  # positions before the append
        return dict(op=op, cache=cache, B=B, n=n, Hq=Hq, Hkv=Hkv, P=P, lo=0, hi=hi,
                    rot=rng.choice([32, 64, 96, 128]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), ragged=rng.random() < 0.5)
    B = _log(rng, 1, 32)
    hi = max(2, min(_log(rng, 2, 32768), 64_000_000 // (B * Hkv * 128 * 2)))
    return dict(op=op, cache=cache, B=B, Hkv=Hkv, P=P, lo=max(1, int(hi * rng.uniform(0.1, 1.0))),
                hi=hi, start=rng.choice([0, 0, 1, 17, 100]))


D = 128
THETA = 500000.0
ORIGINAL = 8192  # positions the frequencies were trained on (yarn)
FAST, SLOW = 32.0, 1.0


def _spread(case, count):
    """Lengths spread evenly over [lo, hi], odd ones among them (the work does
    not depend on the seed; their order does)."""
    lo, hi = case["lo"], case["hi"]
    return [lo + (hi - lo) * (2 * i + 1) // (2 * count) for i in range(count)]


def _news(case):
    """Tokens each sequence appends."""
    B, n = case["B"], case["n"]
    if not case["ragged"]:
        return [n] * B
    return [max(1, n - (n * ((5 * b) % B)) // (2 * B)) for b in range(B)]


def work(case):
    B, Hkv, P = case["B"], case["Hkv"], case["P"]
    cb = 1 if case["cache"] == "e4m3" else 2
    lens = _spread(case, B)
    if case["op"] in ("attn", "window"):
        k, Hq = case["k"], case["Hq"]
        tot = [c + k for c in lens]
        seen = [min(L, case["sinks"] + case["window"] + k - 1) if case["window"] else L
                for L in tot]
        pages = sum(-(-s // P) for s in seen)
        nbytes = 2 * sum(seen) * Hkv * D * cb + 4 * pages + 4 * B
        nbytes += 2 * 4 * pages * Hkv if cb == 1 else 0
        nbytes += B * k * Hq * (2 * 2 * D + 4) + (8 * B * k if case["tree"] else 0)
        return {"bytes": nbytes, "flops": 4 * k * Hq * D * sum(seen)}
    if case["op"] == "rope":
        Hq = case["Hq"]
        rows = sum(_news(case))
        nbytes = rows * D * (2 * 2 * Hq + 2 * Hkv * (2 + cb))
        nbytes += 16 * B * Hkv if cb == 1 else 0  # a scale in and out (k and v)
        return {"bytes": nbytes, "flops": 6 * rows * (Hq + Hkv) * case["rot"] // 2}
    n = sum(lens)
    return {"bytes": 2 * n * Hkv * D * (cb + 2), "flops": 2 * n * Hkv * D}


# ------------------------------------------------------------------ inputs

def _pages(case, gen, tot):
    """Block table over a shuffled pool, one entry per page of each sequence."""
    P = case["P"]
    need = [-(-t // P) for t in tot]
    NP, MP = sum(need) + 3, max(need)
    perm = torch.randperm(NP, generator=gen, device=DEV).int()
    table = torch.zeros(len(tot), MP, dtype=torch.int32, device=DEV)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, NP


def _fill(case, gen, NP):
    """A pool of rows whose magnitude differs from page to page."""
    shape = (NP, case["Hkv"], case["P"], D)
    x = torch.randn(shape, generator=gen, device=DEV)
    x *= torch.exp(0.3 * torch.randn(NP, case["Hkv"], 1, 1, generator=gen, device=DEV))
    if case["cache"] == "bf16":
        return x.bfloat16(), None
    s = x.abs().amax((2, 3)) / E4M3_MAX
    return (x / s[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s


def _tree(case, seed):
    """Ancestor masks of random trees (bit t of row i: node i sees node t)."""
    r = np.random.RandomState(seed % (1 << 31))
    B, k = case["B"], case["k"]
    mask = np.zeros((B, k), np.int64)
    for b in range(B):
        for i in range(k):
            p = r.randint(-1, i) if i else -1
            mask[b, i] = (1 << i) | (int(mask[b, p]) if p >= 0 else 0)
    return mask


def _freqs(case):
    """Radians per position of each rotated pair (float64) and the amplitude."""
    rot, how, f = case["rot"], case["scaling"], case["factor"]
    j = np.arange(0, rot, 2, dtype=np.float64)
    theta = THETA * f ** (rot / (rot - 2)) if how == "ntk" else THETA
    w = theta ** (-j / rot)
    if how == "linear":
        return w / f, 1.0
    if how == "yarn":
        g = np.clip((ORIGINAL * w / (2 * np.pi) - SLOW) / (FAST - SLOW), 0.0, 1.0)
        return g * w + (1 - g) * w / f, 0.1 * math.log(f) + 1.0
    return w, 1.0


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    B, Hkv = case["B"], case["Hkv"]
    order = np.random.RandomState(seed % (1 << 31)).permutation(B)
    lens = [_spread(case, B)[i] for i in order]
    s = {"case": case}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    if case["op"] in ("attn", "window"):
        k, Hq = case["k"], case["Hq"]
        s["ctx"] = ints(lens)
        s["table"], NP = _pages(case, gen, [c + k for c in lens])
        s["k_cache"], s["k_scale"] = _fill(case, gen, NP)
        s["v_cache"], s["v_scale"] = _fill(case, gen, NP)
        # queries a little longer than unit length: some keys stand out
        s["q"] = (1.5 * torch.randn(B, k, Hq, D, generator=gen, device=DEV)).bfloat16()
        s["mask"] = torch.from_numpy(_tree(case, seed)).to(DEV) if case["tree"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, k, Hq, device=DEV)
        return s
    if case["op"] == "rope":
        n, Hq = case["n"], case["Hq"]
        news = [_news(case)[i] for i in order]
        s["ctx"] = ints(lens)
        s["news"] = ints(news) if case["ragged"] else None
        s["table"], NP = _pages(case, gen, [c + n for c in lens])
        s["k_cache"], s["k_scale"] = _fill(case, gen, NP)
        s["v_cache"], s["v_scale"] = _fill(case, gen, NP)
        # the projection's output: q, k and v of a token side by side
        qkv = torch.randn(B, n, Hq + 2 * Hkv, D, generator=gen, device=DEV).bfloat16()
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["q_out"] = torch.zeros(B, n, Hq, D, dtype=torch.bfloat16, device=DEV)
        w, amp = _freqs(case)
        turns = [int(x) for x in (w / (2 * np.pi) * 2.0 ** 64)]
        turns = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]
        s["turns"] = torch.tensor(turns, dtype=torch.int64, device=DEV)
        s["freqs"], s["amp"] = torch.from_numpy(w).to(DEV), amp
        return s
    s["start"] = ints([case["start"]] * B)
    s["lens"] = ints(lens)
    s["table"], NP = _pages(case, gen, [case["start"] + t for t in lens])
    s["k_cache"], s["k_scale"] = _fill(case, gen, NP)
    s["v_cache"], s["v_scale"] = _fill(case, gen, NP)
    s["k_out"] = torch.zeros(B, max(lens), Hkv, D, dtype=torch.bfloat16, device=DEV)
    s["v_out"] = torch.zeros_like(s["k_out"])
    return s


# ------------------------------------------------------------------ plain forms

def _take(cache, pages):
    """Pages of a cache (e4m3 codes are moved as bytes)."""
    if cache.dtype == E4M3:
        return cache.view(torch.uint8)[pages].view(E4M3)
    return cache[pages]


def _dense(cache, scale, table):
    """[B, Hkv, keys, D] in fp32, gathered through the block table."""
    x = _take(cache, table.long()).float()  # [B, MP, Hkv, P, D]
    if scale is not None:
        x = x * scale[table.long()][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    case, q, ctx = s["case"], s["q"], s["ctx"].long()
    B, k, Hq, _ = q.shape
    Hkv = case["Hkv"]
    G = Hq // Hkv
    kd = _dense(s["k_cache"], s["k_scale"], s["table"])
    vd = _dense(s["v_cache"], s["v_scale"], s["table"])
    # [B, Hkv, k * G, D]
    qd = q.float().view(B, k, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, k * G, D)
    sc = (qd @ kd.transpose(2, 3)) * (D ** -0.5)
    j = torch.arange(kd.shape[2], device=DEV)
    i = torch.arange(k, device=DEV)
    t = j[None, None, :] - ctx[:, None, None]  # draft index of a key, negative in the context
    if s["mask"] is None:
        draft = t <= i[None, :, None]
        pos = (ctx[:, None] + i[None, :])[:, :, None]
    else:
        bit = (s["mask"][:, :, None] >> t.clamp(0, 63)) & 1
        draft = (bit == 1) & (t < k)
        depth = ((s["mask"][:, :, None] >> torch.arange(k, device=DEV)) & 1).sum(-1) - 1
        pos = (ctx[:, None] + depth)[:, :, None]
    see = (t < 0) | ((t >= 0) & draft)
    if case["window"]:
        j = j[None, None, :]
        see = see & ((j > pos - case["window"]) | (j < case["sinks"]))
    see = see[:, None, :, None, :].expand(B, 1, k, G, -1).reshape(B, 1, k * G, -1)
    sc = torch.where(see, sc, torch.full((), -math.inf, device=DEV))
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    o = (p @ vd) / l
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.view(B, Hkv, k, G, D).permute(0, 2, 1, 3, 4).reshape(B, k, Hq, D)
    lse = lse.view(B, Hkv, k, G).permute(0, 2, 1, 3).reshape(B, k, Hq)
    return [o.bfloat16(), lse]


def _rotate(x, c, s, rot, inter):
    """Rotated pairs of the first `rot` elements (fp32; c, s: [B, n, 1, rot / 2])."""
    head = x[..., :rot]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_write(case, x, cache, scale, page, slot, ctx, first):
    """x [B, n, Hkv, D] (fp32) into the cache at (page, slot) [B, n]; an e4m3
    page's scale covers its kept rows and the new ones."""
    if scale is None:
        cache[page, :, slot] = x.bfloat16()
        return
    P = case["P"]
    top = x.abs().amax(-1) / E4M3_MAX  # [B, n, Hkv]
    fresh = torch.zeros_like(scale)
    fresh.scatter_reduce_(0, page.reshape(-1, 1).expand(-1, scale.shape[1]),
                          top.reshape(-1, scale.shape[1]), "amax")
    kept = (ctx % P)[:, None]  # rows already in the first page
    old = scale[first]
    both = torch.where(kept > 0, torch.maximum(old, fresh[first]), fresh[first])
    fresh[first] = both
    grown = ((both > old) & (kept > 0))[..., None, None]
    mine = torch.arange(P, device=DEV)[None, None, :, None] < kept[..., None, None]
    codes = _take(cache, first)
    moved = (codes.float() * old[..., None, None] / both[..., None, None])
    moved = moved.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    pick = torch.where(grown & mine, moved.view(torch.uint8), codes.view(torch.uint8))
    cache.view(torch.uint8)[first] = pick
    scale[page] = fresh[page]
    s = fresh[page][..., None]
    c = torch.where(s > 0, x / s, torch.zeros((), device=DEV))
    c = c.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)
    cache.view(torch.uint8)[page, :, slot] = c.view(torch.uint8)


def _plain_rope(s):
    case = s["case"]
    B, n, P, rot = case["B"], case["n"], case["P"], case["rot"]
    ctx = s["ctx"].long()
    t = torch.arange(n, device=DEV)[None, :].expand(B, n)
    valid = t < (s["news"].long()[:, None] if s["news"] is not None else n)
    ang = ((ctx[:, None] + t).double()[..., None] * s["freqs"])[:, :, None, :]
    c, sn = (torch.cos(ang) * s["amp"]).float(), (torch.sin(ang) * s["amp"]).float()
    q = _rotate(s["q"].float(), c, sn, rot, case["inter"]).bfloat16()
    q_out = torch.where(valid[..., None, None], q, s["q_out"])
    kr = _rotate(s["k"].float(), c, sn, rot, case["inter"])
    v = s["v"].float()
    if s["news"] is not None:  # a padded row repeats its sequence's last one
        t = torch.minimum(t, s["news"].long()[:, None] - 1)
        at = torch.arange(B, device=DEV)[:, None]
        kr, v = kr[at, t], v[at, t]
    pos = ctx[:, None] + t
    page = s["table"].long().gather(1, pos // P)
    first = s["table"].long().gather(1, ctx[:, None] // P)[:, 0]
    _plain_write(case, kr, s["k_cache"], s["k_scale"], page, pos % P, ctx, first)
    _plain_write(case, v, s["v_cache"], s["v_scale"], page, pos % P, ctx, first)
    out = [q_out, s["k_cache"], s["v_cache"]]
    return out if s["k_scale"] is None else out + [s["k_scale"], s["v_scale"]]


def _plain_gather(s):
    P = s["case"]["P"]
    n = s["k_out"].shape[1]
    t = torch.arange(n, device=DEV)[None, :]
    valid = (t < s["lens"].long()[:, None])[..., None, None]
    pos = torch.minimum(t, s["lens"].long()[:, None] - 1) + s["start"].long()[:, None]
    page = s["table"].long().gather(1, pos // P)

    def read(cache, scale, out):
        x = cache.view(torch.uint8)[page, :, pos % P].view(E4M3).float() * scale[page][..., None]
        return torch.where(valid, x.bfloat16(), out)

    return [read(s["k_cache"], s["k_scale"], s["k_out"]),
            read(s["v_cache"], s["v_scale"], s["v_out"])]


# ------------------------------------------------------------------ the library's calls

def _own_run(s):
    from speculative_decoding_verification_attn_gb300 import binding
    case = s["case"]
    op = case["op"]
    if op == "window":
        binding.spec_verify_attn_window(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], case["k"], D ** -0.5,
            case["window"], case["sinks"], s["out"], s["lse"], s["k_scale"], s["v_scale"],
            tree_mask=s["mask"])
        return [s["out"], s["lse"]]
    if op == "attn" and s["mask"] is not None:
        binding.spec_verify_attn_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"],
                                      s["mask"], case["k"], D ** -0.5, s["out"], s["lse"],
                                      s["k_scale"], s["v_scale"])
        return [s["out"], s["lse"]]
    if op == "attn":
        binding.spec_verify_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"],
                                 case["k"], D ** -0.5, s["out"], s["lse"], s["k_scale"],
                                 s["v_scale"])
        return [s["out"], s["lse"]]
    if op == "rope":
        binding.spec_rope_append(s["q"], s["k"], s["v"], s["q_out"], s["k_cache"], s["v_cache"],
                                 s["table"], s["ctx"], s["turns"], interleaved=case["inter"],
                                 amplitude=s["amp"], new_lens=s["news"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"])
        out = [s["q_out"], s["k_cache"], s["v_cache"]]
        return out if s["k_scale"] is None else out + [s["k_scale"], s["v_scale"]]
    binding.spec_kv_gather(s["k_cache"], s["v_cache"], s["table"], s["lens"], s["k_out"],
                           s["v_out"], starts=s["start"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
    return [s["k_out"], s["v_out"]]


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "rope":
        return _plain_rope(state)
    return _plain_gather(state) if op == "gather" else _plain_attn(state)


# ------------------------------------------------------------------ in 64 bits

def _rows64(s, which, b, count):
    """Rows 0 .. count - 1 of sequence b, [count, Hkv, D] in fp64."""
    P = s["case"]["P"]
    ids = s["table"][b, :-(-count // P)].long()
    x = _take(s[which + "_cache"], ids).double()
    if s[which + "_scale"] is not None:
        x = x * s[which + "_scale"][ids].double()[:, :, None, None]
    return x.permute(0, 2, 1, 3).reshape(-1, s["case"]["Hkv"], D)[:count]


def _exact_attn(s):
    case = s["case"]
    k, Hq, Hkv = case["k"], case["Hq"], case["Hkv"]
    out = torch.empty(case["B"], k, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(case["B"], k, Hq, dtype=torch.float64, device=DEV)
    masks = s["mask"].tolist() if s["mask"] is not None else None
    for b, ctx in enumerate(s["ctx"].tolist()):
        K, V = _rows64(s, "k", b, ctx + k), _rows64(s, "v", b, ctx + k)
        for i in range(k):
            row = masks[b][i] if masks else (1 << (i + 1)) - 1
            far = ctx + bin(row).count("1") - 1  # the query's position
            keys = torch.arange(ctx + k, device=DEV)
            ok = keys < ctx
            for t in range(k):
                if (row >> t) & 1:
                    ok[ctx + t] = True
            if case["window"]:
                ok &= (far - keys < case["window"]) | (keys < case["sinks"])
            at = ok.nonzero()[:, 0]
            q = s["q"][b, i].double().view(Hkv, Hq // Hkv, D)
            z = torch.einsum("hgd,jhd->hgj", q, K[at]) / math.sqrt(D)
            lse[b, i] = torch.logsumexp(z, -1).reshape(-1)
            out[b, i] = torch.einsum("hgj,jhd->hgd", torch.softmax(z, -1), V[at]).reshape(Hq, D)
    return [out, lse]


def _exact_rope(s):
    case = s["case"]
    P, rot = case["P"], case["rot"]
    q_out = s["q_out"].double()
    caches = {w: s[w + "_cache"].double() for w in "kv"}
    scales = {w: None if s[w + "_scale"] is None else s[w + "_scale"].double() for w in "kv"}
    news = s["news"].tolist() if s["news"] is not None else [case["n"]] * case["B"]
    w = s["freqs"].double()
    first = torch.arange(0, rot, 2) if case["inter"] else torch.arange(rot // 2)
    second = first + (1 if case["inter"] else rot // 2)
    for b, (ctx, n) in enumerate(zip(s["ctx"].tolist(), news)):
        pos = torch.arange(ctx, ctx + n, device=DEV, dtype=torch.float64)
        turn = torch.polar(torch.full((n, rot // 2), s["amp"], dtype=torch.float64, device=DEV),
                           pos[:, None] * w)[:, None, :]

        def spin(x):
            y = x.double().clone()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        q_out[b, :n] = spin(s["q"][b, :n])
        rows = {"k": spin(s["k"][b, :n]), "v": s["v"][b, :n].double()}
        for which, x in rows.items():
            cache, scale = caches[which], scales[which]
            for g in range(ctx // P, (ctx + n - 1) // P + 1):
                page = int(s["table"][b, g])
                lo, hi = max(ctx, g * P), min(ctx + n, (g + 1) * P)
                part = x[lo - ctx:hi - ctx].transpose(0, 1)  # [Hkv, rows, D]
                at = slice(lo - g * P, hi - g * P)
                if scale is None:
                    cache[page, :, at] = part
                    continue
                top = part.abs().amax((1, 2)) / E4M3_MAX
                kept = lo - g * P
                if kept:
                    top = torch.maximum(top, scale[page])
                    moved = cache[page, :, :kept] * (scale[page] / top)[:, None, None]
                    cache[page, :, :kept] = moved.float().to(E4M3).double()
                scale[page] = top
                cache[page, :, at] = (part / top[:, None, None]).float().to(E4M3).double()
    out = [q_out, caches["k"], caches["v"]]
    return out if scales["k"] is None else out + [scales["k"], scales["v"]]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s) if sum(_news(case)) <= 20000 else None
    if case["op"] in ("attn", "window"):
        return _exact_attn(s)
    outs = []
    for which in "kv":
        out = s[which + "_out"].double()
        for b, n in enumerate(s["lens"].tolist()):
            a = case["start"]
            out[b, :n] = _rows64(s, which, b, a + n)[a:]
        outs.append(out)
    return outs
