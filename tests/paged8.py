"""Plain implementations in 64 bits of the e4m3 cache, the windowed attention,
the rotary append and the cache read-back, and seeded inputs for their tests.
Everything here runs on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn
BF16_HALF_STEP = 2.0 ** -8  # relative, finfo(bfloat16).eps / 2


def pool(rng, B, lens, Hkv, D, P, spare=3, canary=True):
    """Block table over a shuffled pool; entries past a sequence are -1."""
    need = [max(1, -(-n // P)) for n in lens]
    NP, MP = sum(need) + spare, max(need)
    ids = rng.permutation(NP)
    table = np.full((B, MP), -1 if canary else 0, np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    return torch.from_numpy(table), NP


def fill_cache(gen, kind, NP, Hkv, P, D):
    """(cache, scale) of random rows; every page has a magnitude of its own."""
    x = torch.randn(NP, Hkv, P, D, generator=gen)
    x *= torch.exp(0.5 * torch.randn(NP, Hkv, 1, 1, generator=gen))
    if kind == "f32":
        return x, None
    if kind == "bf16":
        return x.bfloat16(), None
    if kind == "i8":
        s = (x.abs().amax(-1) / 127).half()
        c = torch.round(x / s.float()[..., None]).clamp(-127, 127).to(torch.int8)
        return c, s
    s = x.abs().amax((2, 3)) / 448.0
    return (x / s[:, :, None, None]).to(E4M3), s


def value64(cache, scale):
    """Element values of a cache in fp64, [NP, Hkv, P, D]."""
    x = cache.double()
    if scale is None:
        return x
    s = scale.double()
    return x * (s[:, :, None, None] if s.dim() == 2 else s[..., None])


def dense64(cache, scale, table, b, n):
    """Rows 0 .. n - 1 of sequence b, [n, Hkv, D] in fp64."""
    P = cache.shape[2]
    rows = []
    for j in range(n):
        page = int(table[b, j // P])
        rows.append(value64(cache[page:page + 1, :, j % P:j % P + 1],
                            None if scale is None else
                            scale[page:page + 1] if scale.dim() == 2 else
                            scale[page:page + 1, :, j % P:j % P + 1])[0, :, 0])
    return torch.stack(rows) if rows else torch.zeros(0, cache.shape[1], cache.shape[3],
                                                      dtype=torch.float64)


def visible(ctx, k, i, mask_row, window, sinks):
    """Cache positions query i sees."""
    bits = (1 << (i + 1)) - 1 if mask_row is None else int(mask_row) & ((1 << 64) - 1)
    depth = i if mask_row is None else max(0, bin(bits).count("1") - 1)
    keys = list(range(ctx)) + [ctx + t for t in range(k) if (bits >> t) & 1]
    if window:
        keys = [j for j in keys if j < sinks or ctx + depth - j < window]
    return keys


def attn64(q, kc, vc, ks, vs, table, ctx, scale, mask=None, window=0, sinks=0):
    """out, lse, and what the tolerances need: A = sum p |v| / l per output (over
    an e4m3 cache with the step of its P, see attn_bounds) and the largest
    sum_d |k_d| a row of queries meets."""
    B, k, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    out = torch.zeros(B, k, Hq, D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((B, k, Hq), -math.inf, dtype=torch.float64)
    knorm = torch.zeros(B, k, Hq, dtype=torch.float64)
    for b in range(B):
        c = int(ctx[b])
        seen = [visible(c, k, i, None if mask is None else mask[b, i], window, sinks)
                for i in range(k)]
        need = sorted(set().union(*map(set, seen)))
        if not need:
            continue
        P = kc.shape[2]
        pages = torch.tensor([int(table[b, j // P]) for j in need])
        slots = torch.tensor([j % P for j in need])

        def rows(cache, sc):
            x = cache.view(torch.uint8)[pages, :, slots].view(E4M3).double() \
                if cache.dtype == E4M3 else cache[pages, :, slots].double()
            if sc is None:
                return x
            return x * (sc[pages] if sc.dim() == 2 else sc[pages, :, slots]).double()[..., None]

        K, V = rows(kc, ks), rows(vc, vs)
        where = {j: n for n, j in enumerate(need)}
        for i in range(k):
            if not seen[i]:
                continue
            at = torch.tensor([where[j] for j in seen[i]])
            z = torch.einsum("hgd,jhd->hgj", q[b, i].double().view(Hkv, G, D), K[at]) * scale
            p = torch.softmax(z, -1)
            lse[b, i] = torch.logsumexp(z, -1).reshape(Hq)
            out[b, i] = torch.einsum("hgj,jhd->hgd", p, V[at]).reshape(Hq, D)
            mag[b, i] = torch.einsum("hgj,jhd->hgd", p, V[at].abs()).reshape(Hq, D)
            if kc.dtype == E4M3:
                top = p.amax(-1)[..., None] * V[at].abs().sum(0)[:, None]
                mag[b, i] += 2.0 ** -9 * top.reshape(Hq, D)
            if kc.dtype == torch.int8:
                mag[b, i] += 2.0 ** -17 * rows(vc, None)[at].abs().sum(0).repeat_interleave(G, 0)
            knorm[b, i] = K[at].abs().sum(-1).amax(0).repeat_interleave(G)
    return out, lse, mag, knorm


def attn_bounds(q, out, mag, knorm, scale, f32=False):
    """Largest errors (out, lse) of a kernel that keeps scores, maxima, sums and
    accumulators in fp32, holds a bf16 q to 2^-18 of its row's largest element
    or better, rounds P to 8 significant bits (half a step: 2^-8) and the
    output once.  f32: fp32 throughout (128 products of 2^-24 and expf).

    Over an e4m3 cache P is a sum of two e4m3 values under a power of two per
    32 keys that puts the largest of them in [128, 256).  Half of e4m3's
    smallest step, 2^-10, is then at most 2^-17 of the block's largest p, and so
    of the row's: each key adds up to 2^-17 max(p) |v| beside its half step of
    2^-8 p |v|.  attn64 counts that into A as 2^-9 max(p) sum |v|, of which a
    half step is 2^-17.  Over an i8 cache P is p times the key's scale in fp16,
    half of whose smallest step is 2^-25: each key adds up to 2^-25 |code| / l,
    with l >= 1 (a term of the row's maximum is at least 1); attn64 counts
    2^-17 sum |code| into A."""
    top = q.double().abs().amax(-1)
    z = (2.0 ** -18 * top + 256 * 2.0 ** -24 * top) * knorm * abs(scale)
    if f32:
        z = 256 * 2.0 ** -24 * top * knorm * abs(scale)
        return (2 * z[..., None] + 1e-5) * mag + 1e-7, z + 1e-5
    rnd = BF16_HALF_STEP * 1.01
    return rnd * out.abs() + (rnd + 2 * z[..., None] + 1e-5) * mag + 1e-6, z + 1e-5


def freqs64(rot, theta=10000.0, scaling="none", factor=1.0, original=0.0, fast=32.0, slow=1.0):
    d = rot
    f = [theta ** (-2 * j / d) for j in range(d // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "ntk":
        f = [(theta * factor ** (d / (d - 2))) ** (-2 * j / d) for j in range(d // 2)]
    if scaling == "yarn":
        g = [min(1.0, max(0.0, (original * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
        f = [a * x + (1 - a) * x / factor for a, x in zip(g, f)]
    return torch.tensor(f, dtype=torch.float64), (0.1 * math.log(factor) + 1
                                                  if scaling == "yarn" else 1.0)


def rotate64(x, pos, f, amp, interleaved):
    """x [n, H, D] at positions pos [n]."""
    y = x.double().clone()
    rot = 2 * len(f)
    a = pos.double()[:, None] * f
    c, s = (torch.cos(a) * amp)[:, None], (torch.sin(a) * amp)[:, None]
    i = torch.arange(rot // 2)
    u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    xu, xv = y[..., u].clone(), y[..., v].clone()
    y[..., u], y[..., v] = xu * c - xv * s, xu * s + xv * c
    return y
