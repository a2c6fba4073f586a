"""GPU parity at the edges of the operators of several continuations, against
plain implementations in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

import paged8
import rollouts
from paged8 import E4M3
from test_gpu_paged8 import cuda
from test_gpu_rollouts import binding, check_logprobs, logits, run_logprobs  # noqa: F401
from test_gpu_shared import call, case, check, reference

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ log probabilities

def staircase(seed, B, V, dtype, step, per):
    """Rows of noise far down in which every `step` elements hold `per` that beat all
    before them: each round of loads adds a few candidates, so that the list crosses the
    length that cuts it between any two looks at it."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(B, 1, V, generator=gen) - 200.0
    at = 0
    for r in range(-(-V // step)):
        for u in range(per[r % len(per)]):
            where = r * step + torch.randint(0, step, (B,), generator=gen)
            ok = where < V
            x[torch.arange(B)[ok], 0, where[ok]] = at * 0.5 - 100.0
            at += 1
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("per", [[1], [3, 0, 5], [0, 2, 0, 13, 1]])
@pytest.mark.parametrize("B,V,K", [(1300, 4001, 1), (1300, 4090, 5), (1300, 30001, 5), (1300, 20003, 20),
                                   (700, 40001, 2), (700, 60007, 20), (3, 152064, 5), (1, 300007, 32)])
def test_logprobs_list_across_looks(binding, dtype, per, B, V, K):
    """CTAs of 64, 128 and 256 threads, rows whole and in parts: the list grows in every
    round, is looked at every few, and is cut at some of the looks."""
    threads = 64 if B >= 1216 and V <= 4096 else 128 if B >= 1216 else 256
    step = threads * 64 // (4 if dtype == torch.float32 else 2)
    x = staircase(V + K, B, V, dtype, step, per)
    tokens = torch.randint(0, V, (B, 1), generator=torch.Generator().manual_seed(K)).int().cuda()
    g = run_logprobs(binding, x, tokens, K, 1.0)
    some = torch.arange(0, B, 60)
    check_logprobs({k: v[some] for k, v in g.items()}, x[some.cuda()], tokens[some.cuda()], K, 1.0)
    for _ in range(3):  # the other rows too: a call repeats itself
        again = run_logprobs(binding, x, tokens, K, 1.0)
        assert all(torch.equal(again[n], g[n]) for n in g)


def logprob_errors(x, T, threads, rounds):
    """What fp32 sums allow a row x [rows, V] in the form that runs: CTAs of `threads` (a warp
    where rounds is 0) in `rounds` rounds, each of 64 bytes a thread in two accumulators.

    A weight carries 2^-22 (2^y by the unit) and the rounding of its exponent, three half
    steps, 3 * 2^-24 d with d = m / T - z.  An accumulator takes rounds * 32 / size terms (16
    in a warp's registers), each a rounding of 2^-24 of the sum; halves, lanes, warps and parts
    are merged over 1 + 5 + 3 + 5 levels.  A sum is moved to a new maximum once a round at
    most, and at two of the merges: each time a factor 2^d with 2^-22, its exponent's two half
    steps (2^d |d| <= 0.54) and two roundings, 2^-21 together.  The logarithm, z's two
    roundings and the last difference are within 2^-22 of ln V and of the result."""
    x = x.double()
    z = x / T
    p = torch.softmax(z, -1)
    d = z.amax(-1, keepdim=True) - z
    d = torch.where(p > 0, d, torch.zeros((), dtype=torch.float64))
    pd, pd2 = (p * d).sum(-1), (p * d * d).sum(-1)
    terms = max(16, rounds * 16)
    r = 2.0 ** -22 + (terms + 14) * 2.0 ** -24 + (rounds + 2) * 2.0 ** -21 + 3 * 2.0 ** -24 * pd
    last = 2.0 ** -22 * math.log(x.shape[-1] + 1)
    return (lambda v: r + last + 2.0 ** -22 * v.abs(),
            lambda v: r + 2 * r * pd + 3 * 2.0 ** -24 * pd2 + last + 2.0 ** -22 * v.abs())


@pytest.mark.parametrize("how", ["normal", "rising", "falling", "peaked", "far"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V,threads", [(70, 1013, 0), (1300, 4001, 64), (1300, 30001, 128),
                                         (700, 33001, 256), (2, 152064, 256)])
def test_logprobs_within_the_form_s_own_errors(binding, how, dtype, B, V, threads):
    T, K = 0.9, 3
    x = logits(V + B, B, 1, V, dtype, how)
    tokens = torch.randint(0, V, (B, 1), generator=torch.Generator().manual_seed(K)).int().cuda()
    g = run_logprobs(binding, x, tokens, K, T)
    some = torch.arange(0, B, 70)
    rows = x[some.cuda(), 0].cpu().float()
    size = x.element_size()
    rounds = -(-(V + 8) * size // (64 * threads)) if threads else 0
    lp, ent, ids, top = rollouts.logprob64(rows, tokens[some.cuda(), 0].cpu(), K, T)[:4]
    lt, et = logprob_errors(rows, T, threads, rounds)
    got = {n: v[some.cuda(), 0].double().cpu() for n, v in g.items()}
    assert torch.equal(got["ids"].long(), ids)
    assert bool(((got["lp"] - lp).abs() <= lt(lp)).all())
    assert bool(((got["ent"] - ent).abs() <= et(ent)).all())
    assert bool(((got["top"] - top).abs().T <= torch.stack([lt(t) for t in top.T])).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1.0, 2.0])
@pytest.mark.parametrize("B,V,K", [(3, 900, 20), (3, 152064, 20), (1300, 4001, 5), (700, 20011, 32)])
def test_logprobs_masked_with_the_lowest_value(binding, dtype, T, B, V, K):
    """Masks of the type's lowest value, which is finite: such tokens have a probability of 0,
    are alternatives where no others are left, and rows of them alone are uniform.  (The 64-bit
    form takes rows less their maximum: a log-sum of -3e38 + ln V has no ln V left in 64 bits.)"""
    x = logits(V, B, 1, V, dtype)
    gen = torch.Generator().manual_seed(V)
    x[(torch.rand(B, 1, V, generator=gen) < 0.999).cuda()] = torch.finfo(dtype).min
    x[0] = torch.finfo(dtype).min
    tokens = torch.randint(0, V, (B, 1), generator=gen).int().cuda()
    g = run_logprobs(binding, x, tokens, K, T)
    some = torch.arange(0, B, 70).cuda()
    rows = x[some, 0].double().cpu()
    rows -= rows.amax(-1, keepdim=True)
    lp, ent, ids, top, lt, et, tt = rollouts.logprob64(rows, tokens[some, 0].cpu(), K, T)
    got = {n: v[some, 0].cpu() for n, v in g.items()}
    assert torch.equal(got["ids"].long(), ids)
    for name, want, tol in (("lp", lp, lt), ("ent", ent, et), ("top", top, tt)):
        far = want < -torch.finfo(torch.float32).max  # (past fp32: -inf)
        assert bool((got[name][far] == -math.inf).all())
        assert bool(((got[name].double() - want).abs() <= tol)[~far].all())


# ------------------------------------------------------------------ pages

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("ctx", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 60, 2 ** 31 - 65])
def test_compact_context_at_the_end_of_its_type(binding, kind, ctx):
    """Pages of one token and a context far past the table: flagged, nothing moves, and
    the other sequence's rows do."""
    s = rollouts.pool_state(13, kind, [9, 70], 2, 64, 1, hold_more=64)
    s["ctx"][0] = ctx
    path = torch.full((2, 64), -1, dtype=torch.int32)
    path[:, :8] = torch.arange(1, 16, 2)
    n = torch.tensor([8, 8], dtype=torch.int32)
    g = rollouts.to_gpu(s)
    assert rollouts.compact(s, path, n) == rollouts.CTX
    binding.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path.cuda(), n.cuda(), g["ks"],
                            g["vs"])
    rollouts.same_state(g, s)
    assert binding.spec_device_error() == rollouts.CTX


@pytest.mark.parametrize("P", [1, 2, 16])
@pytest.mark.parametrize("keep", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 300, 70, 1])
def test_release_that_keeps_all(binding, P, keep):
    """As many tokens kept as a number holds: the row stays as it is."""
    s = rollouts.pool_state(17, "bf16", [60, 33, 0], 1, 32, P, MP=300, hold_more=9)
    s["ctx"][1] = 60  # behind its pages
    g = rollouts.to_gpu(s)
    for rows, keeps in (([0, 1], [keep, keep]), ([1, 2, 1], [2 ** 31 - 1, keep, keep])):
        assert rollouts.release(s, rows, keeps) == 0
        binding.spec_kv_release(g["table"], g["ctx"], g["refs"], torch.tensor(rows).int().cuda(), P,
                                torch.tensor(keeps).int().cuda())
        rollouts.same_state(g, s)


def test_compact_e4m3_nan_row_into_a_page_of_zeros(binding):
    """A NaN code stays one where the page that it comes into has scale 0."""
    P, D = 8, 64
    s = rollouts.pool_state(19, "e4m3", [13], 2, D, P, hold_more=8)
    for t in (s["ks"], s["vs"]):
        t.zero_()
    for t in (s["kc"], s["vc"]):
        rollouts.raw(t).zero_()
    page, to = int(s["table"][0, 18 // P]), int(s["table"][0, 14 // P])
    assert page != to
    rollouts.raw(s["kc"])[page, 0, 18 % P, 3] = 0x7f  # node 5, which becomes node 1
    rollouts.raw(s["vc"])[page, 1, 18 % P, 60] = 0xff
    s["vs"][page] = 2.0
    path, n = torch.tensor([[0, 5] + [-1] * 6], dtype=torch.int32), torch.tensor([2]).int()
    g = rollouts.to_gpu(s)
    binding.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path.cuda(), n.cuda(), g["ks"],
                            g["vs"])
    assert torch.equal(g["ks"].cpu(), s["ks"]) and torch.equal(g["vs"].cpu(), s["vs"])
    for name, h, d in (("kc", 0, 3), ("vc", 1, 60)):
        got, want = rollouts.raw(g[name]).cpu(), rollouts.raw(s[name]).clone()
        assert int(got[to, h, 14 % P, d]) & 0x7f == 0x7f
        want[to, h, 14 % P, d] = got[to, h, 14 % P, d]
        assert torch.equal(got, want)


def test_fork_copies_a_page_past_31_bits_of_bytes(binding):
    """The page in use of an fp32 cache holds more than 2^31 bytes a head."""
    P, D = 2 ** 22 + 64, 128
    part = P - 3
    assert part * D * 4 > 2 ** 31
    cache = [torch.empty(2, 1, P, D, device="cuda") for _ in range(2)]
    for i, c in enumerate(cache):
        c[1].zero_()
        c[0] = (torch.arange(P, device="cuda") * (i + 1)).float()[:, None]
        c[0, 0, :, 1:].add_(torch.arange(1, D, device="cuda"))
    table = torch.tensor([[0, -1], [-1, -1]]).int().cuda()
    ctx, refs = torch.tensor([part, 0]).int().cuda(), torch.tensor([1, 0]).int().cuda()
    binding.spec_kv_fork(*cache, table, ctx, refs, torch.tensor([0]).int().cuda(),
                         torch.tensor([1]).int().cuda())
    assert table.tolist() == [[0, -1], [1, -1]] and refs.tolist() == [1, 1]
    assert ctx.tolist() == [part, part]
    for c in cache:
        assert torch.equal(c[1, 0, :part], c[0, 0, :part])
        assert not bool(c[1, 0, part:].any())


# ------------------------------------------------------------------ shared prefixes

@pytest.fixture()
def grouped(binding):  # noqa: F811
    binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, 5)  # the groups' kernel, whatever it saves
    yield binding
    binding.spec_set_option(binding.SPEC_OPT_ATTN_PATH, 0)


@pytest.mark.parametrize("entries,taken", [(64, True), (2 ** 27 - 32, True), (2 ** 27, False)])
def test_shared_tables_of_2_31_keys(grouped, entries, taken):
    """Keys are counted in 32 bits: a table of more goes to the kernels that read each
    sequence by itself (the groups are not read, and a bad one is not seen)."""
    c = case(41, "bf16", [2], [256], [30, 45], 3, 8, 2, 16)
    table = torch.full((2, entries), -1, dtype=torch.int32, device="cuda")
    table[:, :c["table"].shape[1]] = c["table"].cuda()
    g = {n: cuda(v) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    g["table"] = table
    check(c, *call(grouped, c, g))
    g["shared"] = torch.tensor([-1]).int().cuda()
    check(c, *call(grouped, c, g))
    assert grouped.spec_device_error() == (rollouts.GROUP if taken else 0)


def spoil(c, what, b, key):
    """A NaN in the K or V row of a key of sequence b, in every head."""
    P = c["kc"].shape[2]
    page, slot = int(c["table"][b, key // P]), key % P
    if c["kc"].dtype == torch.int8:
        c[what + "s"][page, :, slot] = math.nan
    else:
        rollouts.raw(c[what + "c"])[page, :, slot, 7] = 0x7f if c["kc"].dtype == E4M3 else math.nan


@pytest.mark.parametrize("ctas", [0, 1, 7, 61])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("where", ["prefix", "own"])
@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("sizes", [[3], [40]])
def test_shared_nan_rows(grouped, kind, sizes, what, where, ctas):
    """A NaN in a cached row that a query sees is one in its output (of K: in its log-sum
    too), whichever of its pieces holds the row; other queries have their answers."""
    k, Hq, Hkv = (4, 8, 2) if sizes == [3] else (8, 16, 1)
    c = case(43, kind, sizes, [300], [20, 150], k, Hq, Hkv, 16, tail=2)
    ref = reference(c)
    n, B = sizes[0], sizes[0] + 2
    hit = torch.zeros(B, dtype=torch.bool)
    if where == "prefix":
        spoil(c, what, 0, 70)
        hit[:n] = True
    else:
        spoil(c, what, 1, int(c["ctx"][1]) - 3)
        hit[1] = True
    grouped.spec_set_option(grouped.SPEC_OPT_NUM_CTAS, ctas)
    out, lse = call(grouped, c)
    grouped.spec_set_option(grouped.SPEC_OPT_NUM_CTAS, 0)
    some = dict(c, q=c["q"][~hit])
    check(some, out[~hit.cuda()], lse[~hit.cuda()], ref=[r[~hit] for r in ref])
    nan = torch.isnan(out[hit.cuda()]).reshape(-1, 128)
    if what == "k":
        assert bool(nan.all()) and bool(torch.isnan(lse[hit.cuda()]).all())
    else:  # the spoiled column (an int8 row's scale: all of them)
        assert bool((nan if kind == "i8" else nan[:, 7]).all())
        assert not bool(torch.isnan(lse[hit.cuda()]).any())


def int8_bounds(c, ref):
    """Largest error of an output over an INT8 cache: weights times V's scales in fp16 (half a
    step: 2^-11, at least 2^-25), codes exact, scores and sums in fp32, one rounding to bf16.

    The weights' common factor puts the largest product of a weight and the largest V scale of
    its 64 keys at 2^-1 or more, so that 2^-25 is at most 2^-24 max(v_scale) of a weight's sum:
    each key adds up to 2^-24 max(v_scale) |code| beside 2^-11 p |v|.  q is bf16 and exact; a
    score's error z is that of attn_bounds (128 products and sums of 2^-24, and the scales')."""
    o64, l64, _, kn = ref
    q, k, P = c["q"], c["k"], c["kc"].shape[2]
    Hq, Hkv = q.shape[2], c["kc"].shape[1]
    z = (256 * 2.0 ** -24 * q.double().abs().amax(-1)) * kn * abs(c["scale"])
    bound = torch.zeros_like(o64)
    mag = paged8.attn64(q, c["kc"], c["vc"].abs(), c["ks"], c["vs"].abs(), c["table"], c["ctx"],
                        c["scale"], c["mask"])[0]
    for b in range(q.shape[0]):
        n = int(c["ctx"][b]) + k
        at = [(int(c["table"][b, j // P]), j % P) for j in range(n)]
        pages, slots = torch.tensor(at).T
        codes = c["vc"][pages, :, slots].double().abs().sum(0)          # [Hkv, D]
        top = c["vs"][pages, :, slots].double().abs().amax(0)           # [Hkv]
        bound[b] = (2.0 ** -24 * top[:, None] * codes).repeat_interleave(Hq // Hkv, 0)
    half_step = torch.exp2(torch.floor(torch.log2(o64.abs().clamp(min=2.0 ** -120))) - 8)
    return half_step * 1.01 + bound + (2.0 ** -11 * 1.01 + 2 * z[..., None] + 1e-5) * mag + 1e-9


def check_int8(c, out, lse):
    ref = reference(c)
    bound = int8_bounds(c, ref)
    err = (out.double().cpu() - ref[0]).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    check(c, out, lse, ref=ref)


@pytest.mark.parametrize("sizes,k,Hq,Hkv", [([3], 4, 8, 2), ([40], 8, 16, 1), ([2, 30], 3, 24, 4)])
@pytest.mark.parametrize("how", ["uniform", "spread", "peaked", "signs", "long"])
def test_shared_int8_weights_in_11_bits(grouped, sizes, k, Hq, Hkv, how):
    """Weights over an INT8 cache have fp16's bits, as in the kernels of single sequences."""
    shared, own_keys = [300, 270][:len(sizes)], [20, 150]
    if how == "long":
        shared, own_keys = [1800, 1500][:len(sizes)], [3, 700]
    c = case(45, "i8", sizes, shared, own_keys, k, Hq, Hkv, 16, tail=1,
             qscale={"uniform": 0.0, "peaked": 6.0}.get(how, 1.5))
    gen = torch.Generator().manual_seed(45)
    if how == "uniform":  # every weight rounds alike: nothing cancels
        c["vs"] = (0.01 + torch.rand(1, Hkv, 1, generator=gen)).half().expand_as(c["vs"]).contiguous()
        c["vc"] = torch.randint(-127, 128, (1, Hkv, 1, 128), generator=gen).to(torch.int8).expand_as(
            c["vc"]).contiguous()
    if how == "spread":  # V's scales 2^-20 .. 2^4, zeros among them; K's a factor of 16 apart
        c["vs"] = torch.exp2(torch.randint(-20, 5, c["vs"].shape, generator=gen).float()).half()
        c["vs"][torch.rand(c["vs"].shape, generator=gen) < 0.1] = 0
        c["ks"] = (c["ks"].float() * torch.exp2(-4 * torch.rand(c["ks"].shape, generator=gen))).half()
    if how == "signs":
        c["ks"] *= torch.where(torch.rand(c["ks"].shape, generator=gen) < 0.5, 1, -1).half()
        c["vs"] *= torch.where(torch.rand(c["vs"].shape, generator=gen) < 0.5, 1, -1).half()
    check_int8(c, *call(grouped, c))


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
@pytest.mark.parametrize("sizes,shared", [([40], [300]), ([30, 9], [1300, 150]), ([3], [260])])
def test_shared_tables_wider_than_the_contexts(grouped, kind, sizes, shared):
    """A captured step has one table width for all its lengths: the same bits behind a wide
    table, and where it is too wide for prefixes to be widened ahead."""
    c = case(46, kind, sizes, shared, [20, 150, 0], 8, 16, 1, 16, tail=1)
    g = {n: cuda(v) if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    first = call(grouped, c, g)
    check(c, *first)
    width = c["table"].shape[1]
    for wide in (width + 1, 4 * width, 40000, 140000):
        g["table"] = torch.full((c["q"].shape[0], wide), -1, dtype=torch.int32, device="cuda")
        g["table"][:, :width] = c["table"].cuda()
        again = call(grouped, c, g)
        assert all(torch.equal(a, b) for a, b in zip(again, first))
    grouped.spec_set_option(grouped.SPEC_OPT_ATTN_PATH, 0)  # by the rule
    check(c, *call(grouped, c, g))


def test_calls_repeat_themselves(grouped):
    """The same call over the same inputs, other calls between them: the same bits."""
    cases = [case(s, kind, [20, 3], [700, 200], [90, 0, 31], 4, 8, 2, 16, tree=s == 51)
             for s, kind in ((50, "bf16"), (51, "i8"), (52, "e4m3"))]
    gs = [{n: cuda(v) if isinstance(v, torch.Tensor) else v for n, v in c.items()} for c in cases]
    first = [call(grouped, c, g) for c, g in zip(cases, gs)]
    for _ in range(20):
        for c, g, f in zip(cases, gs, first):
            assert all(torch.equal(a, b) for a, b in zip(call(grouped, c, g), f))


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_shared_rows_that_see_nothing(grouped, kind):
    """Rows whose mask is empty: behind a prefix they see it alone, without a context
    nothing (0 and -inf)."""
    c = case(47, kind, [4], [300], [0, 40, 0, 9], 5, 8, 2, 16, tree=True, lead=2, tail=1)
    c["mask"][:, 1] = 0
    c["mask"][0] = 0
    out, lse = call(grouped, c)
    o64, l64, mag, kn = ref = reference(c)
    none = torch.isinf(l64)
    assert bool(none[0].all()) and not bool(none[2:6].any())
    assert not bool(out.cpu()[none].any()) and torch.equal(lse.cpu()[none].double(), l64[none])
    ob, lb = paged8.attn_bounds(c["q"], *ref[:1], mag, kn, c["scale"])
    assert bool(((out.double().cpu() - o64).abs() <= ob).all())
    assert bool(((lse.double().cpu() - l64).abs() <= lb)[~none].all())
