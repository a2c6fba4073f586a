"""Plain implementations, in 64 bits or of exact integers, of forking, releasing
and compacting a paged cache and of token log probabilities, and seeded inputs
for their tests.  Everything here runs on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch

import paged8
from paged8 import E4M3

POOL, CTX, PAGE, TREE, TOKEN, GROUP = 64, 2, 1, 16, 8, 128


def raw(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def copy_row(kc, ks, src, dst):
    """Row (page, slot) src to dst, every head, with an int8 row's scale."""
    raw(kc)[dst[0], :, dst[1]] = raw(kc)[src[0], :, src[1]].clone()
    if ks is not None and ks.dim() == 3:
        ks[dst[0], :, dst[1]] = ks[src[0], :, src[1]]


def fork(s, parents, children, room):
    """The state after spec_kv_fork (s is changed) and the error bits."""
    table, ctx, refs = s["table"], s["ctx"], s["refs"]
    rows, MP = table.shape
    P, NP = s["kc"].shape[2], s["kc"].shape[0]
    t0, r0, c0 = table.clone(), refs.clone(), ctx.clone()
    free = [i for i in range(NP) if int(r0[i]) == 0]
    flags, spent = 0, 0
    jobs = []
    for j, (p, c) in enumerate(zip(parents, children)):
        if not (0 <= p < rows and 0 <= c < rows):
            flags |= POOL
            continue
        n = int(c0[p])
        total = -(-(n + room) // P)
        bad = 0
        if n < 0 or total > MP:
            bad |= CTX
        if any(children[i] == c for i in range(j)):
            bad |= POOL
        if c != p and any(parents[i] == c for i in range(len(parents)) if i != j):
            bad |= POOL
        if c != p and int(t0[c, 0]) >= 0:
            bad |= POOL
        whole, part = n // P if n >= 0 else 0, n % P if n >= 0 else 0
        if not bad & CTX:
            used = [int(x) for x in t0[p, :whole + (part > 0)]]
            if any(x < 0 or x >= NP for x in used):
                bad |= PAGE
        flags |= bad
        if bad:
            continue
        places = []
        for i in range(whole, total):
            e = int(t0[p, i]) if c == p else -1
            if e < 0 or int(r0[e]) != 1:
                places.append((i, e))
        if places and spent + len(places) > len(free):
            flags |= POOL
            spent += len(places)
            continue
        jobs.append((p, c, n, whole, total, part, [(i, e, free[spent + m])
                                                   for m, (i, e) in enumerate(places)]))
        spent += len(places)
    for p, c, n, whole, total, part, places in jobs:
        if c != p:
            table[c] = -1
            table[c, :whole] = t0[p, :whole]
            for i in range(whole):
                refs[int(t0[p, i])] += 1
            ctx[c] = n
        for i, e, page in places:
            table[c, i] = page
            refs[page] = 1
            if e >= 0:
                refs[e] -= 1
            if i == whole and part:
                src = int(t0[p, whole])
                for w in ("k", "v"):
                    for slot in range(part):
                        copy_row(s[w + "c"], s[w + "s"], (src, slot), (page, slot))
                    if s[w + "s"] is not None and s[w + "s"].dim() == 2:
                        s[w + "s"][page] = s[w + "s"][src]
    return flags


def release(s, rows, keep=None):
    table, ctx, refs = s["table"], s["ctx"], s["refs"]
    P, NP = s["kc"].shape[2], s["kc"].shape[0]
    flags = 0
    for j, r in enumerate(rows):
        if not 0 <= r < table.shape[0]:
            flags |= POOL
            continue
        k = 0 if keep is None else max(0, keep[j])
        ctx[r] = min(int(ctx[r]), k)
        for i in range(-(-k // P), table.shape[1]):
            page = int(table[r, i])
            if page < 0:
                continue
            table[r, i] = -1
            if page >= NP:
                flags |= PAGE
            elif int(refs[page]) <= 0:
                flags |= POOL
            else:
                refs[page] -= 1
    return flags


def compact(s, path, accepted):
    """The caches after spec_kv_compact (s is changed) and the error bits."""
    table, ctx = s["table"], s["ctx"]
    B, MP = table.shape
    P, NP, k = s["kc"].shape[2], s["kc"].shape[0], path.shape[1]
    flags = 0
    for b in range(B):
        n, moves = min(max(int(accepted[b]), 0), k), []
        for i in range(n):
            f = int(path[b, i])
            if not i <= f < k:
                flags |= TREE
                continue
            if int(ctx[b]) < 0:
                flags |= CTX
                continue
            if f == i:
                continue
            at = []
            for pos in (int(ctx[b]) + i, int(ctx[b]) + f):
                if pos // P >= MP:
                    flags |= CTX
                    at.append(None)
                    continue
                page = int(table[b, pos // P])
                if not 0 <= page < NP:
                    flags |= PAGE
                    at.append(None)
                    continue
                at.append((page, pos % P))
            if None not in at:
                moves.append((at[0], at[1]))
        for w in ("k", "v"):
            cache, scale = s[w + "c"], s[w + "s"]
            if scale is None or scale.dim() == 3:
                old = raw(cache).clone()
                olds = None if scale is None else scale.clone()
                for d, u in moves:
                    raw(cache)[d[0], :, d[1]] = old[u[0], :, u[1]]
                    if scale is not None:
                        scale[d[0], :, d[1]] = olds[u[0], :, u[1]]
                continue
            old, olds = raw(cache).clone().view(E4M3), scale.clone()
            for d, u in moves:
                if d[0] != u[0]:
                    x = (raw(old)[u[0], :, u[1]].view(E4M3).float().abs().amax(-1) * olds[u[0]])
                    scale[d[0]] = torch.maximum(scale[d[0]], x / 448.0)

            def code(x, sc):
                y = torch.where(sc[:, None] > 0, x / sc[:, None], torch.zeros(()))
                return y.clamp(-448, 448).to(E4M3)

            if int(ctx[b]) >= 0:
                for pos in range(int(ctx[b]) // P * P, int(ctx[b]) + k):
                    if pos // P >= MP or not 0 <= int(table[b, pos // P]) < NP:
                        continue
                    p = int(table[b, pos // P])
                    x = raw(old)[p, :, pos % P].view(E4M3).float() * olds[p][:, None]
                    c = code(x, scale[p])
                    grown = (scale[p] > olds[p])[:, None]
                    raw(cache)[p, :, pos % P] = torch.where(grown, raw(c), raw(old)[p, :, pos % P])
            for d, u in moves:
                x = raw(old)[u[0], :, u[1]].view(E4M3).float() * olds[u[0]][:, None]
                c = raw(code(x, scale[d[0]]))
                if d[0] == u[0]:
                    c = torch.where((scale[d[0]] > olds[d[0]])[:, None], c, raw(old)[u[0], :, u[1]])
                raw(cache)[d[0], :, d[1]] = c
    return flags


def pool_state(seed, kind, ctx, Hkv=2, D=64, P=16, MP=None, spare=6, hold_more=0):
    """Rows that hold their own pages, and a few free ones."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    need = [-(-(max(c, 0) + hold_more) // P) if c > 0 or hold_more else 0 for c in ctx]
    NP = sum(need) + spare
    MP = MP or max(need) + 3
    ids = rng.permutation(NP)
    table = torch.full((len(ctx), MP), -1, dtype=torch.int32)
    refs = torch.zeros(NP, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.from_numpy(ids[at:at + m].astype(np.int32))
        at += m
    refs[torch.from_numpy(ids[:at])] = 1
    kc, ks = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    vc, vs = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    return dict(table=table, ctx=torch.tensor(ctx, dtype=torch.int32), refs=refs, kc=kc, ks=ks,
                vc=vc, vs=vs)


def to_gpu(s):
    return {n: None if v is None else v.cuda() for n, v in s.items()}


def same_state(got, want):
    for n, v in want.items():
        if v is None:
            continue
        g = got[n].cpu()
        assert torch.equal(raw(g), raw(v)), n


def logprob64(x, tokens, K, T):
    """logprob, entropy, ids, their log probabilities, and the errors that fp32
    sums and a hardware 2^y allow, for rows x [rows, V].

    With d = m / T - z >= 0, a weight e^-d carries 2^-22 (ex2) and the rounding
    of y = (x - m) log2(e) / T, three half steps: 3 * 2^-24 d.  A thread's sum has at
    most V / 512 + 1 terms per accumulator (two of them), merged over 13 levels and up to 32
    parts: r = 2^-22 + (V / 512 + 64) 2^-24, of l and of a = sum e^-d d alike, l
    further off by 3 * 2^-24 sum p d and a / l by the same with d^2.  The entropy is
    ln l + a / l: the error of a / l is r sum p d for each of its two parts."""
    x = x.double()
    rows, V = x.shape
    none = (x == -math.inf).all(-1)
    z = x / T
    lse = torch.logsumexp(z, -1)
    lp = torch.full((rows,), -math.inf, dtype=torch.float64)
    ok = (tokens >= 0) & (tokens < V) & ~none
    lp[ok] = z[ok, tokens[ok].long()] - lse[ok]
    logp = z - lse[:, None]
    p = torch.exp(logp)
    ent = -torch.where(p > 0, p * logp, torch.zeros((), dtype=torch.float64)).sum(-1)
    ent[none] = 0.0
    d = z.amax(-1, keepdim=True) - z
    pd = torch.where(p > 0, p * d, torch.zeros((), dtype=torch.float64)).sum(-1)
    pd2 = torch.where(p > 0, p * d * d, torch.zeros((), dtype=torch.float64)).sum(-1)
    r = 2.0 ** -22 + (V / 512 + 64) * 2.0 ** -24 + 3 * 2.0 ** -24 * pd
    lp_tol = 1.01 * (r + 2.0 ** -24 * lp.abs()) + 1e-12
    ent_tol = 1.01 * (r + 2 * r * pd + 3 * 2.0 ** -24 * pd2 + 2.0 ** -24 * ent.abs()) + 1e-12
    ids = torch.full((rows, K), -1, dtype=torch.int64)
    top = torch.full((rows, K), -math.inf, dtype=torch.float64)
    kk = min(K, V)
    if kk:
        order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :kk]
        v = x.gather(1, order)
        ids[:, :kk] = torch.where(v > -math.inf, order, -1)
        top[:, :kk] = torch.where(v > -math.inf, logp.gather(1, order), -math.inf)
    top_tol = 1.01 * (r[:, None] + 2.0 ** -24 * top.abs()) + 1e-12
    return lp, ent, ids, top, lp_tol, ent_tol, top_tol
