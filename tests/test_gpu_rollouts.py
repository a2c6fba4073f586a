"""GPU parity of forking, releasing and compacting a paged cache and of token log
probabilities against plain implementations."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged8
import rollouts
from paged8 import E4M3
from rollouts import CTX, PAGE, POOL, TOKEN, TREE, pool_state, same_state, to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture()
def binding():
    from speculative_decoding_verification_attn_gb300 import binding as m
    m.spec_device_error()
    yield m
    assert m.spec_device_error() == 0


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def clone(s):
    return {n: None if v is None else v.clone() for n, v in s.items()}


def gpu_fork(m, g, parents, children, room, stream=None):
    m.spec_kv_fork(g["kc"], g["vc"], g["table"], g["ctx"], g["refs"], ints(parents),
                   ints(children), room, g["ks"], g["vs"], stream=stream)


# ------------------------------------------------------------------ fork

@pytest.mark.parametrize("kind", ["f32", "bf16", "i8", "e4m3"])
@pytest.mark.parametrize("P,D,Hkv", [(16, 128, 2), (1, 32, 3), (7, 64, 1), (64, 256, 5)])
def test_fork(binding, kind, P, D, Hkv):
    ctx = [5 * P + P // 2, 0, 3 * P, 0, 0, 0, 1, 0]
    s = pool_state(P + D, kind, ctx, Hkv, D, P, MP=12, spare=40)
    g = to_gpu(s)
    pairs = [(0, 1), (2, 3), (0, 4), (6, 5), (0, 7)]
    for room in (0, P + 3):
        w, h = clone(s), clone(g)
        p, c = zip(*pairs)
        assert rollouts.fork(w, p, c, room) == 0
        gpu_fork(binding, h, p, c, room)
        same_state(h, w)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_fork_own_room_and_copy_on_write(binding, kind):
    """A row that is its own parent: fresh pages for its room, and sole pages in
    the place of those that another row holds."""
    P = 16
    s = pool_state(3, kind, [41, 0, 0, 32, 0], 2, 64, P, MP=9, spare=30)
    g = to_gpu(s)
    for p, c, room in [([0, 0, 0], [1, 0, 2], 20), ([3], [4], 0)]:
        assert rollouts.fork(s, p, c, room) == 0
        gpu_fork(binding, g, p, c, room)
        same_state(g, s)
    # rows 3 and 4 share two pages; both fall back into the second and go on
    for w, f in ((s, lambda *a: rollouts.release(s, *a)),):
        f([3, 4], [20, 25])
    binding.spec_kv_release(g["table"], g["ctx"], g["refs"], ints([3, 4]), P, ints([20, 25]))
    same_state(g, s)
    assert rollouts.fork(s, [3, 4], [3, 4], 40) == 0
    gpu_fork(binding, g, [3, 4], [3, 4], 40)
    same_state(g, s)
    assert int(s["refs"].min()) >= 0


def test_fork_skips_and_flags(binding):
    P = 16
    s = pool_state(5, "bf16", [40, 0, 20, 0, -1, 33], 2, 64, P, MP=4, spare=4)
    s["table"][5, 1] = 10 ** 6
    cases = [
        ([0, 7], [1, 3], 0, POOL),             # no such row
        ([0], [2], 0, POOL),                   # the child holds pages
        ([0, 2], [1, 1], 0, POOL),             # one child of two parents
        ([0, 1], [1, 3], 0, POOL),             # a child that is a parent
        ([4], [1], 0, CTX),                    # a negative context
        ([0], [1], 30, CTX),                   # more room than the table has
        ([0], [1], 2 ** 31 - 1, CTX),
        ([5], [1], 0, PAGE),                   # a page that is none
        ([0, 2, 0], [1, 3, 0], 24, POOL),      # fewer free pages than asked for
    ]
    for p, c, room, flag in cases:
        w = clone(s)
        g = to_gpu(s)
        assert rollouts.fork(w, p, c, room) == flag
        gpu_fork(binding, g, p, c, room)
        same_state(g, w)
        assert binding.spec_device_error() == flag


def test_fork_large_pool(binding):
    """Free pages far apart, over several blocks of the scan."""
    NP, P = 70001, 2
    gen = torch.Generator().manual_seed(1)
    s = dict(table=torch.full((300, 9), -1, dtype=torch.int32), ctx=torch.zeros(300).int(),
             refs=torch.ones(NP, dtype=torch.int32),
             kc=torch.randn(NP, 1, P, 32, generator=gen).bfloat16(), ks=None,
             vc=torch.randn(NP, 1, P, 32, generator=gen).bfloat16(), vs=None)
    free = torch.randperm(NP, generator=gen)[:900]
    s["refs"][free] = 0
    held = [i for i in range(NP) if int(s["refs"][i])][:4]
    s["table"][0, :4] = torch.tensor(held).int()
    s["ctx"][0] = 7
    g = to_gpu(s)
    p, c = [0] * 299, list(range(1, 300))
    assert rollouts.fork(s, p, c, 4) == 0
    gpu_fork(binding, g, p, c, 4)
    same_state(g, s)
    # all rows go; only the pages held elsewhere stay
    rollouts.release(s, list(range(300)))
    binding.spec_kv_release(g["table"], g["ctx"], g["refs"], ints(list(range(300))), P)
    same_state(g, s)

def test_fork_needs_past_32_bits(binding):
    """Pairs that together ask for more than 2^31 pages: the first has them, no other."""
    n, room = 4099, 1 << 19
    NP = room + 5
    cache = [torch.zeros(NP, 1, 1, 32, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.full((n + 1, room), -1, dtype=torch.int32, device="cuda")
    ctx, refs = torch.zeros(n + 1).int().cuda(), torch.zeros(NP).int().cuda()
    binding.spec_kv_fork(*cache, table, ctx, refs, torch.zeros(n).int().cuda(),
                         torch.arange(1, n + 1).int().cuda(), room)
    assert binding.spec_device_error() == POOL
    assert torch.equal(table[1], torch.arange(room).int().cuda())
    assert bool((refs[:room] == 1).all()) and not bool(refs[room:].any())
    table[1] = -1
    assert bool((table == -1).all())


# ------------------------------------------------------------------ release

def test_release(binding):
    P = 16
    s = pool_state(9, "bf16", [100, 16, 0, 33, 64], 1, 32, P, spare=3, hold_more=20)
    g = to_gpu(s)
    for rows, keep in [([0, 3], [50, 33]), ([1, 1], [0, 0]), ([4], [1000]), ([0, 2, 4], None),
                       ([3], [-5])]:
        assert rollouts.release(s, rows, keep) == 0
        binding.spec_kv_release(g["table"], g["ctx"], g["refs"], ints(rows), P,
                                None if keep is None else ints(keep))
        same_state(g, s)
    assert int(s["refs"].sum()) == 0


def test_release_flags(binding):
    s = pool_state(9, "bf16", [40, 20], 1, 32, 16)
    s["refs"][int(s["table"][0, 0])] = 0     # a page that nobody holds
    s["table"][1, 1] = 10 ** 6
    g = to_gpu(s)
    flags = rollouts.release(s, [0, 5, 1, -1])
    binding.spec_kv_release(g["table"], g["ctx"], g["refs"], ints([0, 5, 1, -1]), 16)
    same_state(g, s)
    assert flags == POOL | PAGE and binding.spec_device_error() == flags


# ------------------------------------------------------------------ compaction

def random_paths(rng, B, k):
    path = np.full((B, k), -1, np.int32)
    n = rng.integers(0, k + 1, B)
    for b in range(B):
        path[b, :n[b]] = np.sort(rng.permutation(k)[:n[b]])
    return torch.from_numpy(path), torch.from_numpy(n.astype(np.int32))


@pytest.mark.parametrize("kind", ["f32", "bf16", "i8", "e4m3"])
@pytest.mark.parametrize("B,k,P,D,Hkv", [
    (1, 1, 16, 128, 2), (3, 8, 16, 128, 4), (5, 64, 16, 64, 1), (2, 64, 1, 32, 2),
    (2, 33, 7, 256, 1), (4, 64, 128, 256, 3), (70, 5, 4, 32, 1)])
def test_compact(binding, kind, B, k, P, D, Hkv):
    rng = np.random.default_rng(B * k + P)
    ctx = [int(c) for c in rng.integers(0, 70, B)]
    s = pool_state(B + k, kind, ctx, Hkv, D, P, hold_more=k)
    path, n = random_paths(rng, B, k)
    g = to_gpu(s)
    assert rollouts.compact(s, path, n) == 0
    binding.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path.cuda(), n.cuda(), g["ks"],
                            g["vs"])
    same_state(g, s)


def test_compact_e4m3_zero_scales_and_extremes(binding):
    """Pages whose scale is 0, whose rows are all zero, and scales 2^60 apart."""
    s = pool_state(4, "e4m3", [10, 3], 2, 64, 8, hold_more=40)
    NP = s["kc"].shape[0]
    f = torch.tensor([0.0, 1.0, 2.0 ** 60, 2.0 ** -60])
    s["ks"] *= f[torch.arange(NP) % 4][:, None]
    rollouts.raw(s["vc"])[::2] = 0x80  # -0
    path = torch.full((2, 40), -1, dtype=torch.int32)
    path[0, :20] = torch.arange(0, 40, 2)
    path[1, :3] = torch.tensor([7, 20, 39])
    n = torch.tensor([20, 3], dtype=torch.int32)
    g = to_gpu(s)
    rollouts.compact(s, path, n)
    binding.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path.cuda(), n.cuda(), g["ks"],
                            g["vs"])
    same_state(g, s)


def test_compact_e4m3_nan_row(binding):
    """A NaN in a row that comes into a page costs the page's other rows nothing."""
    s = pool_state(5, "e4m3", [13], 2, 64, 8, hold_more=8)
    path, n = torch.tensor([[4, 5, 6, 7, -1, -1, -1, -1]], dtype=torch.int32), torch.tensor([3]).int()
    clean = clone(s)
    page = int(s["table"][0, 18 // 8])
    rollouts.raw(s["kc"])[page, :, 18 % 8, 3] = 0x7f  # node 5, behind the page's end
    rollouts.raw(clean["kc"])[page, :, 18 % 8, 3] = 0
    g = to_gpu(s)
    rollouts.compact(clean, path, n)
    binding.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path.cuda(), n.cuda(), g["ks"],
                            g["vs"])
    to = int(clean["table"][0, 14 // 8])
    assert to != page and torch.equal(g["ks"].cpu(), clean["ks"])
    got, want = rollouts.raw(g["kc"]).cpu(), rollouts.raw(clean["kc"])
    assert bool((got[to, :, 14 % 8, 3] & 0x7f == 0x7f).all())
    got[to, :, 14 % 8, 3] = want[to, :, 14 % 8, 3]
    got[page, :, 18 % 8, 3] = want[page, :, 18 % 8, 3]
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", ["bf16", "i8", "e4m3"])
def test_compact_flags(binding, kind):
    s = pool_state(6, kind, [10, -3, 30, 12], 1, 32, 8, MP=5, hold_more=10)
    s["table"][3, 2] = -7
    path = torch.tensor([[0, 2, 1, 9], [1, 2, 3, 3], [3, 3, 3, 3], [0, 3, 2, 3]], dtype=torch.int32)
    path = torch.nn.functional.pad(path, (0, 6), value=-1)
    n = torch.tensor([4, 99, 4, 4], dtype=torch.int32)
    s["ctx"][2] = 38
    g = to_gpu(s)
    flags = rollouts.compact(s, path, n)
    binding.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path.cuda(), n.cuda(), g["ks"],
                            g["vs"])
    same_state(g, s)
    assert flags & TREE and flags & CTX
    assert binding.spec_device_error() == flags


# ------------------------------------------------------------------ log probabilities

def run_logprobs(m, x, tokens, K, T, lens=None, stream=None, entropy=True):
    B, n, V = x.shape
    g = dict(lp=torch.full((B, n), 7.0).cuda(), ent=torch.full((B, n), 7.0).cuda(),
             ids=torch.full((B, n, K), 7, dtype=torch.int32).cuda(),
             top=torch.full((B, n, K), 7.0).cuda())
    m.spec_token_logprobs(x, tokens, g["lp"], g["ent"] if entropy else None,
                          g["ids"] if K else None, g["top"] if K else None, lens, T, stream=stream)
    return g


def check_logprobs(g, x, tokens, K, T, lens=None):
    B, n, V = x.shape
    live = torch.ones(B, n, dtype=torch.bool)
    if lens is not None:
        live = torch.arange(n)[None] < lens.cpu()[:, None]
    want = rollouts.logprob64(x.cpu().reshape(B * n, V).float(), tokens.cpu().reshape(-1), K, T)
    lp, ent, ids, top, lt, et, tt = [w.reshape((B, n) + w.shape[1:]) for w in want]
    got = {k: v.cpu() for k, v in g.items()}
    assert torch.equal(got["ids"].long()[live], ids[live])

    def close(a, b, tol):
        a, b, tol = a.double()[live], b[live], tol[live]
        inf = torch.isinf(b)
        assert torch.equal(a[inf], b[inf])
        assert bool(((a - b).abs()[~inf] <= tol[~inf]).all()), (a - b).abs()[~inf].max()

    close(got["lp"], lp, lt)
    close(got["ent"], ent, et)
    close(got["top"], top, tt)
    for v in got.values():
        assert bool((v[~live] == 7).all())


def logits(seed, B, n, V, dtype, how="normal"):
    gen = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(B, n, V, generator=gen)
    if how == "coarse":      # many equal values, both zeros among them
        x = torch.round(x) * torch.where(torch.rand(B, n, V, generator=gen) < 0.5, 1.0, -1.0)
    if how == "constant":
        x = torch.full((B, n, V), -3.25)
    if how == "rising":      # every element beats all before it
        x = torch.linspace(-20, 20, V).expand(B, n, V).contiguous()
    if how == "falling":
        x = torch.linspace(20, -20, V).expand(B, n, V).contiguous()
    if how == "peaked":
        x[..., V // 2] = 90.0
    if how == "masked":
        x[torch.rand(B, n, V, generator=gen) < 0.97] = -math.inf
    if how == "far":
        x = x * 1e4
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,n,V,K,T", [
    (1, 1, 1, 1, 1.0), (1, 3, 2, 5, 0.5), (2, 2, 7, 7, 1.0), (1, 2, 33, 32, 2.0),
    (3, 5, 1000, 20, 0.7), (1, 1, 8191, 32, 1.0), (1, 2, 8193, 3, 1.3), (2, 3, 32000, 0, 1.0),
    (1, 1, 128257, 32, 0.9), (2, 2, 152064, 1, 1.0), (40, 5, 20001, 20, 1.0), (700, 1, 5000, 5, 1.0),
    (7, 5, 1017, 32, 1.0), (5, 3, 1021, 20, 1.0), (3, 3, 1022, 5, 1.0), (9, 4, 250, 32, 1.0),
    (11, 3, 466, 0, 0.5), (60, 35, 4096, 7, 1.0), (65, 65, 4099, 20, 1.0), (5, 250, 8193, 32, 1.0)])
def test_logprobs(binding, dtype, B, n, V, K, T):
    x = logits(V + K, B, n, V, dtype)
    tokens = torch.randint(0, V, (B, n), generator=torch.Generator().manual_seed(V)).int().cuda()
    check_logprobs(run_logprobs(binding, x, tokens, K, T), x, tokens, K, T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("how", ["coarse", "constant", "rising", "falling", "peaked", "masked", "far"])
@pytest.mark.parametrize("B,V,K", [(1, 40000, 32), (700, 33001, 20), (71, 1013, 32), (71, 130, 20),
                                   (1050, 3001, 32), (4130, 6001, 5), (1230, 3001, 20), (1250, 9001, 32)])
def test_logprobs_shapes_of_rows(binding, dtype, how, B, V, K):
    """Values that fill the list of candidates, tie, or leave few of them: rows
    split over CTAs and whole rows."""
    n, T = 1, 1.0
    x = logits(V, B, n, V, dtype, how)
    tokens = torch.randint(0, V, (B, n), generator=torch.Generator().manual_seed(K)).int().cuda()
    if B == 1:
        check_logprobs(run_logprobs(binding, x, tokens, K, T), x, tokens, K, T)
        return
    g = run_logprobs(binding, x, tokens, K, T)
    some = torch.arange(0, B, 70)
    check_logprobs({k: v[some] for k, v in g.items()}, x[some.cuda()], tokens[some.cuda()], K, T)


@pytest.mark.parametrize("lens", [[0, 3, 5, 9, -4], [5] * 5, [0] * 5])
@pytest.mark.parametrize("V", [999, 50000])
def test_logprobs_ragged(binding, lens, V):
    B, n, K, T = 5, 5, 4, 0.8
    x = logits(2, B, n, V, torch.bfloat16)
    tokens = torch.randint(0, V, (B, n), generator=torch.Generator().manual_seed(1)).int().cuda()
    ln = ints(lens)
    check_logprobs(run_logprobs(binding, x, tokens, K, T, ln), x, tokens, K, T, ln)


@pytest.mark.parametrize("V", [500, 40000])
def test_logprobs_extreme_rows(binding, V):
    """Rows of -inf, with a NaN, with +inf; a masked token; tokens that are none."""
    x = logits(3, 1, 6, V, torch.float32)
    x[0, 0] = -math.inf
    x[0, 1, V // 3] = math.nan
    x[0, 2, V // 2] = math.inf
    x[0, 3, 17] = -math.inf
    tokens = ints([[4, 4, 4, 17, V, -1]])
    g = {k: v.cpu() for k, v in run_logprobs(binding, x, tokens, 3, 1.0).items()}
    assert binding.spec_device_error() == TOKEN
    assert g["lp"][0, 0] == -math.inf and g["ent"][0, 0] == 0
    assert g["ids"][0, 0].tolist() == [-1] * 3 and bool((g["top"][0, 0] == -math.inf).all())
    assert math.isnan(g["lp"][0, 1]) and math.isnan(g["ent"][0, 1])
    assert math.isnan(g["lp"][0, 2]) and math.isnan(g["ent"][0, 2])
    assert bool((g["lp"][0, 3:] == -math.inf).all())
    part = {k: v[:, 3:].cuda() for k, v in g.items()}
    check_logprobs(part, x[:, 3:], tokens[:, 3:], 3, 1.0)


def test_logprobs_many_rows_and_optional_outputs(binding):
    """More rows than the split form has tickets for; entropy and one of the
    alternatives' outputs left out."""
    B, n, V = 20000, 1, 70
    x = logits(4, B, n, V, torch.bfloat16)
    tokens = torch.randint(0, V, (B, n), generator=torch.Generator().manual_seed(1)).int().cuda()
    lp = torch.zeros(B, n).cuda()
    ids = torch.zeros(B, n, 2, dtype=torch.int32).cuda()
    binding.spec_token_logprobs(x, tokens, lp, top_ids=ids)
    g = run_logprobs(binding, x, tokens, 2, 1.0)
    assert torch.equal(lp, g["lp"]) and torch.equal(ids, g["ids"])
    check_logprobs(g, x, tokens, 2, 1.0)
    top = torch.zeros(B, n, 2).cuda()
    binding.spec_token_logprobs(x, tokens, lp, top_logprobs=top)
    assert torch.equal(top, g["top"])


def test_other_stream_and_captured(binding):
    """The calls on a stream of their own and replayed from a graph, over inputs
    that change between the replays."""
    P = 16
    s = pool_state(11, "bf16", [90, 0, 0, 40], 2, 64, P, MP=9, spare=20, hold_more=0)
    g = to_gpu(s)
    x = logits(5, 2, 3, 30001, torch.bfloat16)
    tokens = torch.randint(0, 30001, (2, 3), generator=torch.Generator().manual_seed(1)).int().cuda()
    path, n = ints([[0, 2, 3, -1]] * 4), ints([3, 0, 0, 2])
    out = dict(lp=torch.zeros(2, 3).cuda(), ent=torch.zeros(2, 3).cuda(),
               ids=torch.zeros(2, 3, 6, dtype=torch.int32).cuda(), top=torch.zeros(2, 3, 6).cuda())
    par, kid, both = ints([0, 0, 0, 3]), ints([1, 2, 0, 3]), ints([1, 2])

    def step():
        binding.spec_kv_release(g["table"], g["ctx"], g["refs"], both, P)
        binding.spec_kv_fork(g["kc"], g["vc"], g["table"], g["ctx"], g["refs"], par, kid, 8)
        binding.spec_kv_compact(g["kc"], g["vc"], g["table"], g["ctx"], path, n)
        binding.spec_token_logprobs(x, tokens, out["lp"], out["ent"], out["ids"], out["top"],
                                    temperature=0.9)

    def expect():
        rollouts.release(s, [1, 2])
        rollouts.fork(s, [0, 0, 0, 3], [1, 2, 0, 3], 8)
        rollouts.compact(s, path.cpu(), n.cpu())

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    expect()
    same_state(g, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (6, 7):
        x.copy_(logits(seed, 2, 3, 30001, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        expect()
        same_state(g, s)
        check_logprobs(out, x, tokens, 6, 0.9)
