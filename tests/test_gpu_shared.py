"""GPU parity of the verification attention over shared prefixes against a plain
64-bit implementation, and a run of sampled continuations with the operators
around it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged8
import rollouts
from paged8 import E4M3
from rollouts import GROUP
from test_gpu_paged8 import cuda, poison, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture()
def binding():
    from speculative_decoding_verification_attn_gb300 import binding as m
    m.spec_set_option(m.SPEC_OPT_ATTN_PATH, 5)  # the groups' kernel, whatever it saves
    m.spec_device_error()
    yield m
    for opt in (m.SPEC_OPT_ATTN_PATH, m.SPEC_OPT_NUM_CTAS, m.SPEC_OPT_SPLIT_WEIGHT,
                m.SPEC_OPT_VALIDATE):
        m.spec_set_option(opt, 0)
    assert m.spec_device_error() == 0


def case(seed, kind, sizes, shared, own, k, Hq, Hkv, P, D=128, tree=False, lead=0, tail=0,
         qdt=torch.bfloat16, qscale=1.5):
    """Groups of `sizes` sequences with `shared` keys in the same pages, then
    own[b] keys and the drafts; `lead` / `tail` sequences before and behind them
    in no group."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    starts = [lead]
    first = [0] * lead
    of = [-1] * lead
    for g, n in enumerate(sizes):
        starts.append(starts[-1] + n)
        first += [shared[g]] * n
        of += [g] * n
    first += [0] * tail
    of += [-1] * tail
    B = len(first)
    ctx = [first[b] + own[b % len(own)] for b in range(B)]
    need = [-(-(c + k) // P) for c in ctx]
    common = [-(-s // P) for s in shared]  # a page that is shared in part is the same page too
    NP = sum(need) + 3
    ids = iter(rng.permutation(NP))
    prefix = [[int(next(ids)) for _ in range(m)] for m in common]
    table = np.full((B, max(need)), -1, np.int32)
    for b in range(B):
        have = prefix[of[b]][:need[b]] if of[b] >= 0 else []
        table[b, :len(have)] = have
        for i in range(len(have), need[b]):
            table[b, i] = next(ids)
    table = torch.from_numpy(table)
    kc, ks = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    vc, vs = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    q = (qscale * torch.randn(B, k, Hq, D, generator=gen)).to(qdt)
    mask = torch.from_numpy(random_tree(rng, B, k)) if tree else None
    safe = table.clamp(min=0)
    poison(kc, safe, ctx, k, 0, 0)
    poison(vc, safe, ctx, k, 0, 0)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, ctx=torch.tensor(ctx).int(),
                mask=mask, k=k, scale=D ** -0.5, starts=torch.tensor(starts).int(),
                shared=torch.tensor(shared).int().reshape(-1))


def call(m, c, g=None, stream=None):
    g = g or {n: cuda(v) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    out = torch.full_like(g["q"], float("nan"))
    lse = torch.full(c["q"].shape[:3], float("nan"), device="cuda")
    m.spec_verify_attn_shared(g["q"], g["kc"], g["vc"], g["table"], g["ctx"], g["starts"],
                              g["shared"], c["k"], c["scale"], out, lse, g["ks"], g["vs"],
                              tree_mask=g["mask"], stream=stream)
    return out, lse


def reference(c):
    return paged8.attn64(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["ctx"],
                         c["scale"], c["mask"])


def check(c, out, lse, ref=None, f32=False):
    o64, l64, mag, kn = ref or reference(c)
    ob, lb = paged8.attn_bounds(c["q"], o64, mag, kn, c["scale"], f32)
    err = (out.double().cpu() - o64).abs()
    assert bool((err <= ob).all()), float((err / ob).max())
    lerr = (lse.double().cpu() - l64).abs()
    assert bool((lerr <= lb).all()), float((lerr / lb).max())


SHAPES = [
    # sizes, shared, own, k, Hq, Hkv, P
    ([2], [128], [0, 5], 1, 4, 2, 16),
    ([4], [256], [1, 40, 130, 300], 4, 8, 2, 16),
    ([3, 2], [384, 130], [17, 0, 200], 3, 28, 4, 32),
    ([12], [512], [9, 33], 8, 16, 1, 64),            # 1536 rows of one kv-head
    ([20, 1, 6], [257, 640, 131], [3, 60], 16, 8, 1, 128),
    ([5], [768], [250, 700], 2, 2, 2, 256),
    ([7], [300], [11], 18, 7, 1, 16),                # 126 of 128 rows
    ([3], [400], [29], 64, 2, 1, 16),                # more drafts than a Q tile has tokens
    ([4], [140], [2], 1, 128, 1, 16),                # a token fills a Q tile
]


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[0])) + "x%d" % s[3])
def test_shared(binding, kind, shape):
    c = case(len(kind), kind, *shape)
    check(c, *call(binding, c))


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_shared_tree_and_ungrouped(binding, kind):
    c = case(5, kind, [4, 3], [300, 260], [0, 70, 129, 3], 12, 16, 2, 16, tree=True, lead=2, tail=3)
    check(c, *call(binding, c))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_shared_splits(binding, kind):
    """The same call over few and many CTAs, with and without a charge for a piece."""
    c = case(6, kind, [9, 2], [700, 300], [5, 200, 64], 5, 12, 2, 16, lead=1)
    g = {n: cuda(v) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    ref = reference(c)
    for ctas in (1, 2, 3, 7, 20, 61, 152, 400):
        for alpha in (0, 1, 6, 31):
            binding.spec_set_option(binding.SPEC_OPT_NUM_CTAS, ctas)
            binding.spec_set_option(binding.SPEC_OPT_SPLIT_WEIGHT, alpha)
            check(c, *call(binding, c, g), ref=ref)


def test_shared_scores_over_the_exponent_range(binding):
    """Prefixes that outweigh the sequences' own keys and the other way round."""
    for seed, s in ((1, 12.0), (2, 0.001), (3, 40.0)):
        c = case(seed, "bf16", [6], [290], [1, 77], 4, 8, 2, 16, qscale=s)
        check(c, *call(binding, c))


@pytest.mark.parametrize("kind,D,P,qdt", [
    ("f32", 64, 16, torch.float32), ("bf16", 64, 16, torch.bfloat16), ("bf16", 128, 8, torch.bfloat16),
    ("i8", 96, 5, torch.bfloat16), ("e4m3", 256, 16, torch.float32), ("f32", 128, 16, torch.bfloat16)])
def test_shared_other_shapes(binding, kind, D, P, qdt):
    """Shapes that each sequence reads by itself."""
    binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, 0)
    c = case(7, kind, [3, 2], [140, 50], [4, 30], 3, 4, 2, P, D=D, qdt=qdt, tail=1)
    check(c, *call(binding, c), f32=True if qdt == torch.float32 else False)


def test_shared_forced_paths_and_no_groups(binding):
    """Kernels that know no groups, and a call without any."""
    c = case(8, "bf16", [4], [256], [30, 90], 4, 8, 2, 16)
    ref = reference(c)
    for path in (1, 2, 3, 5):
        binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, path)
        check(c, *call(binding, c), ref=ref)
    binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, 0)
    binding.spec_set_option(binding.SPEC_OPT_VALIDATE, 1)
    check(c, *call(binding, c), ref=ref)
    c["starts"], c["shared"] = torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    check(c, *call(binding, c), ref=ref)


@pytest.mark.parametrize("n,P,taken", [(40, 16, True), (40, 8, False), (4, 16, False)])
def test_shared_rule(binding, n, P, taken):
    """Automatic: the groups are read (and a bad one is seen) where that saves enough."""
    binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, 0)
    c = case(12, "i8", [n], [256], [0, 30, 110], 1, 8, 4, P)
    check(c, *call(binding, c))
    assert binding.spec_device_error() == 0
    c["shared"] = torch.tensor([-1]).int()
    check(c, *call(binding, c))
    assert binding.spec_device_error() == (GROUP if taken else 0)


@pytest.mark.parametrize("starts,shared", [
    ([0, 2, 4], [900, 256]),       # longer than the contexts
    ([0, 2, 4], [-3, 256]),
    ([0, 9], [256]),               # a start behind the last sequence
    ([-1, 4], [256]),
    ([0, 3, 2, 4], [256] * 3),     # a start before the one before it
])
def test_shared_bad_groups(binding, starts, shared):
    """Clamped and flagged; the tables agree, so the answer stands."""
    c = case(9, "bf16", [4], [256], [0], 3, 8, 2, 16)
    c["starts"], c["shared"] = torch.tensor(starts).int(), torch.tensor(shared).int()
    check(c, *call(binding, c))
    assert binding.spec_device_error() == GROUP


def test_shared_bad_tables(binding):
    """A page id that is none, a context past the table: flagged, no fault; the other
    sequences' answers stand."""
    c = case(10, "bf16", [3], [256], [20], 3, 8, 2, 16, tail=2)
    ref = reference(c)
    c["table"][3, 1] = 10 ** 8
    c["ctx"][4] = 10 ** 8
    out, lse = call(binding, c)
    flags = binding.spec_device_error()
    assert flags == 3
    some = {n: v[:3] if n in ("q",) else v for n, v in c.items()}
    check(some, out[:3], lse[:3], ref=[r[:3] for r in ref])


def test_shared_captured_and_other_stream(binding):
    c = case(11, "e4m3", [5], [384], [20, 150], 4, 8, 2, 16)
    g = {n: cuda(v) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out, lse = call(binding, c, g)
    side.synchronize()
    check(c, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = call(binding, c, g)
    for seed in (1, 2):
        d = dict(c, q=1.5 * torch.randn(c["q"].shape, generator=torch.Generator().manual_seed(seed)))
        d["q"] = d["q"].bfloat16()
        d["ctx"] = c["ctx"] - seed  # other lengths, the same prefix or less of it
        d["shared"] = c["shared"] - 128 * seed
        g["q"].copy_(d["q"])
        g["ctx"].copy_(d["ctx"])
        g["shared"].copy_(d["shared"])
        graph.replay()
        torch.cuda.synchronize()
        check(d, out, lse)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_rollouts_together(binding, kind):
    """Continuations of two prompts: the prompts are appended once and forked, two steps
    of tree verification run over the shared prefixes, the accepted paths are
    kept, the tokens scored, and the worse continuation is replaced by the better one's fork."""
    m, P, Hkv, Hq, D, k, V, n = binding, 16, 2, 8, 128, 6, 3001, 3
    rows, NP = 2 * n, 140
    gen = torch.Generator().manual_seed(21)
    rng = np.random.default_rng(21)
    prompts = [200, 167]
    ref = dict(table=torch.full((rows, 24), -1, dtype=torch.int32), ctx=torch.zeros(rows).int(),
               refs=torch.zeros(NP, dtype=torch.int32))
    kc, ks = paged8.fill_cache(gen, kind, NP, Hkv, P, D)
    ref.update(kc=kc, ks=ks, vc=kc.clone(), vs=None if ks is None else ks.clone())
    g = rollouts.to_gpu(ref)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32).cuda()

    def fork(p, c, room):
        assert rollouts.fork(ref, p, c, room) == 0
        m.spec_kv_fork(g["kc"], g["vc"], g["table"], g["ctx"], g["refs"], ints(p), ints(c), room,
                       g["ks"], g["vs"])
        for name in ("table", "ctx", "refs"):
            assert torch.equal(g[name].cpu(), ref[name])

    def pull():  # the caches as they are now (appends round; the plain forms go on from there)
        for name in ("kc", "vc", "ks", "vs"):
            if ref[name] is not None:
                ref[name] = g[name].cpu()

    def append(lens):  # rows of the given lengths behind every context
        most = max(lens)
        new = [torch.randn(rows, most, Hkv, D, generator=gen).bfloat16().cuda() for _ in range(2)]
        m.spec_rope_append(None, new[0], new[1], None, g["kc"], g["vc"], g["table"], g["ctx"], None,
                           new_lens=ints(lens), k_scale=g["ks"], v_scale=g["vs"])
        pull()

    # the prompts, into rows 0 and n, then a fork to the others with room for the drafts
    fork([0, n], [0, n], 200)
    append([prompts[0] if b == 0 else prompts[1] if b == n else 0 for b in range(rows)])
    g["ctx"][0], g["ctx"][n] = prompts
    ref["ctx"][0], ref["ctx"][n] = prompts
    others = [b for b in range(rows) if b % n]
    fork([b // n * n for b in others] + [0, n], others + [0, n], 2 * (k + 1))
    starts, shared = ints([0, n, rows]), ints([p // P * P for p in prompts])
    score = torch.zeros(rows, dtype=torch.float64)
    for step in range(2):
        append([k] * rows)
        q = (1.5 * torch.randn(rows, k, Hq, D, generator=gen)).bfloat16()
        mask = torch.from_numpy(random_tree(rng, rows, k))
        parents = torch.full((rows, k), -1, dtype=torch.int32)
        for b in range(rows):
            for i in range(k):
                above = int(mask[b, i]) & ~(1 << i)
                parents[b, i] = above.bit_length() - 1
        c = dict(q=q, kc=ref["kc"], vc=ref["vc"], ks=ref["ks"], vs=ref["vs"], table=ref["table"],
                 ctx=ref["ctx"], mask=mask, k=k, scale=D ** -0.5, starts=starts.cpu(),
                 shared=shared.cpu())
        gg = dict(g, q=q.cuda(), mask=mask.cuda(), starts=starts, shared=shared)
        check(c, *call(m, c, gg))
        # acceptance: drafts that follow the target's argmax along some path
        x = (2.0 * torch.randn(rows, k + 1, V, generator=gen)).bfloat16()
        best = x.float().argmax(-1)
        drafts = torch.randint(0, V, (rows, k), generator=gen).int()
        for b in range(rows):
            for i in range(k):
                if rng.random() < 0.8:
                    drafts[b, i] = int(best[b, int(parents[b, i]) + 1])
        xg = x.cuda()
        acc, nxt = ints([0] * rows), ints([0] * rows)
        path = torch.zeros(rows, k, dtype=torch.int32).cuda()
        m.spec_accept_tree(xg, drafts.cuda(), parents.cuda(), k, acc, nxt, path)
        m.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path, acc, g["ks"], g["vs"])
        assert rollouts.compact(ref, path.cpu(), acc.cpu()) == 0
        rollouts.same_state({n_: g[n_] for n_ in ("kc", "vc", "ks", "vs")},
                            {n_: ref[n_] for n_ in ("kc", "vc", "ks", "vs")})
        # the emitted tokens' log probabilities: rows of the kept nodes and the last one's
        emitted = torch.zeros(rows, k + 1, dtype=torch.int32)
        picked = torch.zeros(rows, k + 1, V, dtype=torch.bfloat16)
        for b in range(rows):
            at = 0
            for i in range(int(acc[b]) + 1):
                node = int(path[b, i]) if i < int(acc[b]) else -1
                emitted[b, i] = drafts[b, node] if i < int(acc[b]) else nxt[b]
                picked[b, i] = x[b, at]
                at = node + 1
        lp, ent = torch.zeros(rows, k + 1).cuda(), torch.zeros(rows, k + 1).cuda()
        m.spec_token_logprobs(picked.cuda(), emitted.cuda(), lp, ent, lens=acc + 1)
        want = rollouts.logprob64(picked.reshape(-1, V).float(), emitted.reshape(-1), 0, 1.0)
        live = torch.arange(k + 1)[None] < acc.cpu()[:, None] + 1
        err = (lp.cpu().double() - want[0].reshape(rows, -1)).abs()[live]
        assert bool((err <= want[4].reshape(rows, -1)[live]).all())
        score += torch.where(live, lp.cpu().double(), torch.zeros((), dtype=torch.float64)).sum(1)
        m.spec_commit(g["ctx"], acc, 0)
        ref["ctx"] += acc.cpu()
        assert torch.equal(g["ctx"].cpu(), ref["ctx"])
        # of each prompt's continuations the last is replaced by the best of the others
        lose = [n - 1, 2 * n - 1]
        win = [int(score[:n - 1].argmax()), n + int(score[n:2 * n - 1].argmax())]
        rollouts.release(ref, lose)
        m.spec_kv_release(g["table"], g["ctx"], g["refs"], ints(lose), P)
        fork(win + list(range(rows))[:n - 1] + list(range(n, 2 * n - 1)),
             lose + list(range(rows))[:n - 1] + list(range(n, 2 * n - 1)), 2 * (k + 1))
        rollouts.same_state({n_: g[n_] for n_ in ("kc", "vc", "ks", "vs")},
                            {n_: ref[n_] for n_ in ("kc", "vc", "ks", "vs")})
    held = torch.zeros_like(ref["refs"])
    for e in ref["table"].reshape(-1).tolist():
        if e >= 0:
            held[e] += 1
    assert torch.equal(held, ref["refs"])
