"""Attention over the paged 8-bit cache for sequences that share prefixes: the plan against a model of it,
the attention against each sequence's definition alone (tests/kv8_ref.py), with the tolerances of the
other forwards (tests/helpers.py): scores of exact keys, softmax terms in fp16 (2^-11 of themselves), sums
and the merge of prefix and rest in fp32, as there."""
import random

import pytest
import torch

from tests import helpers, kv8_ref
from tiled_memory_efficient_gb300 import _lib
from tiled_memory_efficient_gb300.kvcache import PagedKVCache
from tiled_memory_efficient_gb300.rope import Rope

F16, BF16, F8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
P = 256  # a fake, 16-byte-aligned "device" address: validation fails before any use
RUN = 128    # positions that are shared or not together


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


CALL = dict(q=P, kp=P, vp=P, ks=P, vs=P, table=P, lens=P, n_new=P, granted=P, plan=P, out=P, lse=P, ws=P, n=1 << 40, B=2,
            Hq=4, Hkv=2, Nq=1, D=64, page=64, n_pages=10, max_pages=5, scale=0.1, dtype=0)


@pytest.mark.parametrize("change,code", [
    ({"q": 0}, 1), ({"plan": 0}, 1), ({"ws": 0}, 1), ({"Hq": 3}, 1), ({"B": 0}, 1), ({"scale": 0.0}, 1), ({"dtype": 3}, 1),
    ({"D": 96}, 2), ({"page": 48}, 2), ({"B": 1025}, 2), ({"kp": P + 8}, 3), ({"plan": P + 2}, 3), ({"n_new": P + 1}, 3),
    ({"n": 16}, 6),
])
def test_attention_refusals(lib, change, code):
    assert lib.kv8_attn_shared(*{**CALL, **change}.values(), None) == code


FIND = dict(table=P, lens=P, n=4, max_pages=5, page=64, least=0, plan=P)


@pytest.mark.parametrize("change,code", [
    ({"table": 0}, 1), ({"plan": 0}, 1), ({"n": 0}, 1), ({"least": -2}, 1), ({"max_pages": 0}, 1), ({"n": 1025}, 2),
    ({"page": 20}, 2), ({"lens": P + 2}, 3), ({"max_pages": 1 << 28}, 2),
])
def test_plan_refusals(lib, change, code):
    assert lib.kvp_find_shared(*{**FIND, **change}.values(), None) == code


def test_plan_sizes(lib):
    assert lib.kvp_plan_words(0) == 0 and lib.kvp_plan_words(1025) == 0 and lib.kvp_plan_words(3) >= 4 + 3 * 7
    assert lib.kv8_attn_shared_workspace_size(2, 4, 2, 1, 96) == 0
    assert lib.kv8_attn_shared_workspace_size(2, 4, 2, 1, 64) > lib.kv8_attn_workspace_size(2, 4, 2, 1, 64)


# ------------------------------------------------------------------ the plan

def _plan_model(table, lens, page, least):
    """{first sequence: (members, runs)} of the groups that are kept."""
    B, cols = len(lens), RUN // page
    full = [min(max(n, 0), len(table[0]) * page) // RUN for n in lens]
    depth = []
    for b in range(B):
        best = (0.0, 0)
        for i in range(full[b]):
            c = (i + 1) * cols - 1
            r = sum(table[k][c] == table[b][c] and full[k] > i for k in range(B)) if table[b][c] >= 0 else 0
            if r > 1:
                best = max(best, ((i + 1) * (r - 1) / r, i + 1))
        depth.append(best[1])
    groups = {}
    for b in range(B):
        d = depth[b]
        if d == 0:
            continue
        key = (d, table[b][d * cols - 1])
        first = next(k for k in range(B) if depth[k] == d and table[k][d * cols - 1] == key[1])
        if table[first][:d * cols] == table[b][:d * cols]:
            groups.setdefault(first, ([], d))[0].append(b)
    return {f: (m, d) for f, (m, d) in groups.items() if len(m) > 1 and (len(m) - 1) * d * RUN >= least}


def _read_plan(plan, B):
    w = plan.tolist()
    at = lambda a: w[4 + a * B: 4 + (a + 1) * B]
    groups = {}
    for g in range(w[1]):
        m = at(3)[at(0)[g]: at(0)[g] + at(1)[g]]
        groups[m[0]] = (m, at(2)[g])
        for rank, b in enumerate(m):
            assert at(4)[b] == g and at(5)[b] == rank and at(6)[b] == at(2)[g] * RUN
    held = {b for m, _ in groups.values() for b in m}
    assert all(at(4)[b] == -1 and at(6)[b] == 0 for b in range(B) if b not in held)
    return groups


def _i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(8))
def test_plans_match_the_model(cuda_lib, seed):
    """Random forks of forks: nested prefixes, lengths inside them, empty sequences."""
    rng = random.Random(seed)
    page, B = rng.choice([16, 32, 64, 128]), rng.choice([2, 7, 33, 60])
    most = rng.choice([4, 20]) * RUN // page
    ids = iter(range(1, 10 ** 6))
    rows, lens = [], []
    for b in range(B):
        if rows and rng.random() < 0.8:
            k = rng.randrange(len(rows))
            keep = rng.randint(0, lens[k] // page)
            row = rows[k][:keep]
        else:
            row = []
        n = rng.choice([0, len(row) * page + rng.randint(0, most * page)]) if rng.random() < 0.15 else \
            min(len(row) * page + rng.randint(1, most * page // 2), most * page)
        while len(row) * page < n:
            row.append(next(ids))
        rows.append(row[: -(-n // page)])
        lens.append(n)
    width = max(max(map(len, rows)), 1)
    table = [r + [-1] * (width - len(r)) for r in rows]
    lens = [min(n, width * page) for n in lens]
    for least in (0, 600):
        plan = _lib.kvp_find_shared(_i32(table), _i32(lens), page, least)
        assert _read_plan(plan, B) == _plan_model(table, lens, page, least)
    again = _lib.kvp_find_shared(_i32(table), _i32(lens), page, least, plan=torch.zeros_like(plan))
    assert torch.equal(plan, again)


@pytest.mark.gpu
def test_pages_in_another_order_are_not_a_prefix(cuda_lib):
    """Tables that meet in a page without the same beginning share nothing."""
    table = [[5, 6, 7, 8], [6, 5, 7, 8], [5, 6, 7, 9]]
    plan = _lib.kvp_find_shared(_i32(table), _i32([512, 512, 512]), 128, 0)
    assert _read_plan(plan, 3) == _plan_model(table, [512] * 3, 128, 0)
    for m, d in _read_plan(plan, 3).values():
        assert all(table[b][:d] == table[m[0]][:d] for b in m)


@pytest.mark.gpu
def test_the_largest_plan(cuda_lib):
    """1024 sequences in 300 groups."""
    g = torch.Generator().manual_seed(1)
    of = torch.randint(0, 300, (1024,), generator=g)
    table = torch.stack([of * 2, of * 2 + 1, 1000 + torch.arange(1024)], 1).int()
    lens = torch.full((1024,), 300, dtype=torch.int32)
    plan = _lib.kvp_find_shared(table.cuda(), lens.cuda(), 128, 0)
    assert _read_plan(plan, 1024) == _plan_model(table.tolist(), lens.tolist(), 128, 0)


# ------------------------------------------------------------------ the attention

def _batch(groups, tails, alone, Hkv, D, page, seed, spread=3):
    """A cache of sequences that share: groups = [(positions, members)], members interleaved; tails: own
    positions of each member in turn; alone: lengths of sequences that share nothing.  Scales of
    2^-spread .. 2^spread."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    order = [i for i, (_, m) in enumerate(groups) for _ in range(m)] + [-1] * len(alone)
    rng.shuffle(order)
    heads = [-(-n // page) for n, _ in groups]
    lens, rows, next_page, alone, tails = [], [], 0, list(alone), list(tails)
    shared = []
    for h in heads:
        shared.append(list(range(next_page, next_page + h)))
        next_page += h
    k = 0
    for i in order:
        if i < 0:
            n, row = alone.pop(), []
        else:
            t = tails[k % len(tails)]
            k += 1
            # a member's own positions begin on a page of its own
            row, n = list(shared[i]), len(shared[i]) * page + t
        while len(row) * page < n:
            row.append(next_page)
            next_page += 1
        rows.append(row)
        lens.append(n)
    width = max(map(len, rows)) + 1
    n_pages = next_page + 2
    perm = torch.randperm(n_pages, generator=g).tolist()
    table = torch.tensor([[perm[i] for i in r] + [-1] * (width - len(r)) for r in rows], dtype=torch.int32)
    pools = []
    for amp in (0.5, 1.0):
        x = torch.randn(n_pages, Hkv, page, D, generator=g)
        e = torch.randint(-spread, spread + 1, (n_pages, Hkv), generator=g)
        s = torch.ldexp(torch.ones(n_pages, Hkv), e)
        pools += [(x * amp / s[:, :, None, None]).clamp(-448, 448).to(F8), s]
    return pools[0], pools[2], pools[1], pools[3], table, torch.tensor(lens, dtype=torch.int32)


def _check(q, cache, n_new, out, lse, what, some=None):
    out, lse = out.double().cpu(), lse.double().cpu()
    for b in range(q.shape[0]) if some is None else some:
        n = q.shape[2] if n_new is None else n_new[b]
        assert bool((out[b, :, n:] == 0).all()) and bool((lse[b, :, n:] == float("-inf")).all()), (what, b)
        if n:
            one = cache[:4] + (cache[4][b:b + 1], cache[5][b:b + 1])
            ro, rl = kv8_ref.attention(q[b:b + 1, :, :n], *one)
            helpers.assert_fwd_close(out[b, :, :n].numpy(), lse[b, :, :n].numpy(), ro[0].numpy(), rl[0].numpy(), q.dtype,
                                     f"{what} sequence {b}")


CASES = [
    # Hq, Hkv, Nq, D, page, groups, tails, alone, dtype
    (1, 1, 1, 64, 64, [(128, 2)], [1, 1], [], F16),
    (1, 1, 1, 128, 128, [(128, 2)], [1, 5], [], BF16),
    (4, 2, 1, 64, 16, [(300, 3)], [7, 130, 64], [50], F16),             # 256 of 304 positions are shared
    (14, 2, 1, 64, 32, [(1000, 5)], [1, 40, 300], [], BF16),
    (8, 2, 1, 128, 64, [(640, 9), (128, 2)], [3, 99, 0], [1, 700], F16),  # members without own positions
    (16, 4, 3, 128, 16, [(500, 6), (260, 4)], [3, 50, 2, 1], [9], BF16),  # queries that stand in the prefix
    (8, 1, 1, 64, 64, [(2048, 20)], [10, 60], [], F16),                 # 160 rows: a second Q tile
    (8, 1, 2, 128, 128, [(1408, 21)], [2, 77], [300], BF16),            # 336 rows: a second row block
    (32, 8, 1, 128, 32, [(384, 40)], [20, 33], [], F16),
    (7, 1, 5, 64, 16, [(256, 4), (384, 4), (128, 3)], [5, 6, 40], [], BF16),
    (2, 2, 1, 64, 128, [(12800, 3)], [4000, 1], [], F16),               # own positions over many CTAs
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention_matches_the_definition(cuda_lib, case):
    Hq, Hkv, Nq, D, page, groups, tails, alone, dtype = case
    cache = _batch(groups, tails, alone, Hkv, D, page, seed=Hq + D)
    B = cache[5].numel()
    q = torch.randn(B, Hq, Nq, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dev = [t.cuda() for t in cache]
    plan = _lib.kvp_find_shared(dev[4], dev[5], page, 0)
    found = _read_plan(plan, B)
    assert sorted((d * RUN, len(m)) for m, d in found.values()) == sorted(
        (-(-n // page) * page // RUN * RUN, m) for n, m in groups)
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan)
    assert _lib.sync_status() == _lib.ATTN_OK
    _check(q, cache, None, out, lse, f"shared {case}")
    again = _lib.kv8_attn_shared(q.cuda(), *dev, plan)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    # without groups every sequence reads for itself
    none = _lib.kvp_find_shared(dev[4], dev[5], page, (1 << 31) - 1)
    assert _read_plan(none, B) == {}
    _check(q, cache, None, *_lib.kv8_attn_shared(q.cuda(), *dev, none), f"shared without groups {case}")
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,Nq,D,page,dtype", [(8, 2, 4, 64, 16, F16), (6, 1, 3, 128, 64, BF16)])
def test_ragged_steps(cuda_lib, Hq, Hkv, Nq, D, page, dtype):
    """Counts of 0 to Nq, more queries than own positions, and a step without room."""
    cache = _batch([(700, 6), (256, 3)], [Nq, 40, 1, 100], [5, 0], Hkv, D, page, seed=3)
    B, rng = cache[5].numel(), random.Random(5)
    n_new = [min(rng.randint(0, Nq), int(n)) for n in cache[5]]
    q = torch.randn(B, Hq, Nq, D, generator=torch.Generator().manual_seed(2)).to(dtype)
    dev = [t.cuda() for t in cache]
    plan = _lib.kvp_find_shared(dev[4], dev[5], page, 0)
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(n_new), granted=_i32([1]))
    assert _lib.sync_status() == _lib.ATTN_OK
    _check(q, cache, n_new, out, lse, f"shared ragged D={D}")
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(n_new), granted=_i32([0]))
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all()) and _lib.sync_status() == _lib.ATTN_OK
    # a count that does not fit: that sequence sees nothing, the others what they saw
    good = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(n_new))
    victim = _read_plan(plan, B).popitem()[1][0][1]
    bad = [Nq + 1 if b == victim else n for b, n in enumerate(n_new)]
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(bad))
    assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
    assert bool((out[victim] == 0).all()) and bool((lse[victim] == float("-inf")).all())
    for b in range(B):
        if b != victim and n_new[b]:
            helpers.assert_fwd_close(*(x[b, :, :n_new[b]].double().cpu().numpy() for x in (out, lse, *good)), q.dtype,
                                     "shared, bad count")


@pytest.mark.gpu
@pytest.mark.parametrize("D,page,dtype", [(64, 16, F16), (128, 32, BF16)])
def test_pages_of_very_different_scales(cuda_lib, D, page, dtype):
    """Scales of 2^-9 to 2^9 beside each other, and positions far apart in size."""
    cache = _batch([(1200, 5)], [30, 200], [], 2, D, page, seed=9, spread=9)
    q = torch.randn(5, 8, 1, D, generator=torch.Generator().manual_seed(4)).to(dtype)
    dev = [t.cuda() for t in cache]
    plan = _lib.kvp_find_shared(dev[4], dev[5], page, 0)
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan)
    _check(q, cache, None, out, lse, f"shared, scales D={D}")
    # queries whose largest value is far from 1 (bf16 reaches further than the fp16 products)
    q = q * 2.0 ** (-10 if dtype is F16 else 30)
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan, scale=D ** -0.5 * 2.0 ** (10 if dtype is F16 else -30))
    _check_scaled(q, cache, out, lse, D, dtype)
    assert _lib.sync_status() == _lib.ATTN_OK


def _check_scaled(q, cache, out, lse, D, dtype):
    scale = D ** -0.5 * 2.0 ** (10 if dtype is F16 else -30)
    ro, rl = kv8_ref.attention(q, *cache, scale=scale)
    helpers.assert_fwd_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), ro.numpy(), rl.numpy(), dtype,
                             f"shared, scaled queries D={D}")


@pytest.mark.gpu
def test_bad_pages_and_plans_are_recorded(cuda_lib):
    cache = _batch([(512, 4)], [20, 60], [77], 2, 64, 32, seed=11)
    q = torch.randn(5, 4, 1, 64, generator=torch.Generator().manual_seed(2)).to(F16)
    dev = [t.cuda() for t in cache]
    plan = _lib.kvp_find_shared(dev[4], dev[5], 32, 0)
    first = _read_plan(plan, 5).popitem()[1][0][0]
    # pages of the prefix outside the pool: their positions are not seen
    table = cache[4].clone()
    for col, pid in ((3, -1), (9, 10 ** 6)):
        table[first, col] = pid
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev[:4], table.cuda(), dev[5], plan)
    assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
    for b in range(5):
        if int(cache[5][b]) < 512:
            keep = list(range(int(cache[5][b])))
        else:
            keep = [t for t in range(int(cache[5][b])) if t // 32 not in (3, 9)]
        k, v = (kv8_ref.dense(p, s, cache[4][b], int(cache[5][b]))[:, keep] for p, s in ((cache[0], cache[2]), (cache[1], cache[3])))
        s = (q[b].double().view(2, 2, 64) @ k.transpose(1, 2)) / 8.0
        ref = torch.softmax(s, -1) @ v
        helpers.assert_fwd_close(out[b].double().cpu().numpy(), lse[b].double().cpu().numpy(), ref.view(4, 1, 64).numpy(),
                                 torch.logsumexp(s, -1).view(4, 1).numpy(), F16, f"bad pages, sequence {b}")
    # what is not a plan: recorded, and every sequence reads for itself
    none = _lib.kvp_find_shared(dev[4], dev[5], 32, (1 << 31) - 1)
    want = _lib.kv8_attn_shared(q.cuda(), *dev, none)
    other = _lib.kvp_find_shared(dev[4][:4].contiguous(), dev[5][:4].contiguous(), 32, 0)
    for junk in (torch.zeros_like(plan), torch.full_like(plan, 10 ** 9), torch.cat([other, other])[: plan.numel()]):
        out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, junk)
        assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(ValueError, match="plan"):
        _lib.kv8_attn_shared(q.cuda(), *dev, plan[:-1])
    with pytest.raises(ValueError, match="plan"):
        _lib.kv8_attn_shared(q.cuda(), *dev, None)
    with pytest.raises(ValueError, match="lens"):
        _lib.kvp_find_shared(dev[4], dev[5].long(), 32)
    with pytest.raises(_lib.AttnError):
        _lib.kvp_find_shared(dev[4], dev[5], 48)
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_special_values(cuda_lib):
    """A NaN key or value of the prefix reaches the group's rows; one behind every row's end does not."""
    cache = _batch([(256, 3)], [10, 20], [64], 1, 64, 32, seed=13)
    q = torch.randn(4, 2, 1, 64, generator=torch.Generator().manual_seed(2)).to(F16)
    plan = _lib.kvp_find_shared(cache[4].cuda(), cache[5].cuda(), 32, 0)
    group = _read_plan(plan, 4).popitem()[1][0]
    alone = [b for b in range(4) if b not in group]
    clean = _lib.kv8_attn_shared(q.cuda(), *(t.cuda() for t in cache), plan)
    for w in (0, 1):
        pools = [t.clone() for t in cache]
        pools[w].view(torch.uint8)[int(cache[4][group[0], 2]), 0, 5, 7] = 0x7F
        out, lse = _lib.kv8_attn_shared(q.cuda(), *(t.cuda() for t in pools), plan)
        assert bool(torch.isnan(out[group, :, :, 7]).all()) and torch.equal(out[alone], clean[0][alone])
        assert bool(torch.isnan(lse[group]).all() if w == 0 else torch.isfinite(lse[group]).all())
    # garbage past the ends
    pools = [t.clone() for t in cache]
    for b in range(4):
        n = int(cache[5][b])
        if n % 32:
            for w in (0, 1):
                pools[w].view(torch.uint8)[int(cache[4][b, n // 32]), :, n % 32:] = 0x7F
    out, lse = _lib.kv8_attn_shared(q.cuda(), *(t.cuda() for t in pools), plan)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.gpu
def test_captured_and_side_by_side(cuda_lib):
    """Replayed on other queries and lengths, the workspace kept; two calls on two streams at once."""
    cache = _batch([(1024, 7)], [40, 90], [10], 2, 128, 64, seed=17)
    dev = [t.cuda() for t in cache]
    g = torch.Generator().manual_seed(3)
    qs = [torch.randn(8, 8, 1, 128, generator=g).to(BF16).cuda() for _ in range(4)]
    plan = _lib.kvp_find_shared(dev[4], dev[5], 64, 0)
    want = [_lib.kv8_attn_shared(q, *dev, plan) for q in qs]
    ws = torch.empty(_lib.load().kv8_attn_shared_workspace_size(8, 8, 2, 1, 128), dtype=torch.uint8, device="cuda")
    buf = qs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = _lib.kv8_attn_shared(buf, *dev, plan, workspace=ws)
        second = _lib.kv8_attn_shared(buf, *dev, plan, workspace=ws)
    for q, (o, l) in zip(qs, want):
        buf.copy_(q)
        graph.replay()
        for x in (held, second):
            assert torch.equal(x[0], o) and torch.equal(x[1], l)
    dev[5] -= 3
    graph.replay()
    short = _lib.kv8_attn_shared(buf, *dev, plan)
    assert torch.equal(held[0], short[0]) and not torch.equal(held[0], want[3][0])
    dev[5] += 3
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            got.append(_lib.kv8_attn_shared(qs[i % 4], *dev, plan))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 4][0]) and torch.equal(l, want[i % 4][1])
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,Nq,dtype", [(64, 3, 1, F16), (128, 1, 2, BF16)])
def test_the_largest_batch(cuda_lib, D, G, Nq, dtype):
    """1024 sequences: one large group, many small ones, some alone."""
    cache = _batch([(384, 500)] + [(128, 2)] * 200, [5, 17, 40], [30] * 124, 1, D, 128, seed=19)
    q = torch.randn(1024, G, Nq, D, generator=torch.Generator().manual_seed(4)).to(dtype)
    dev = [t.cuda() for t in cache]
    plan = _lib.kvp_find_shared(dev[4], dev[5], 128, 0)
    assert len(_read_plan(plan, 1024)) == 201
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan)
    assert _lib.sync_status() == _lib.ATTN_OK
    _check(q, cache, None, out, lse, f"shared, 1024 sequences D={D}", some=range(0, 1024, 41))
    a, b = _lib.kv8_attn(q.cuda(), *dev)
    helpers.assert_fwd_close(*(x.double().cpu().numpy() for x in (out, lse, a, b)), dtype, f"shared against plain D={D}")


@pytest.mark.gpu
@pytest.mark.parametrize("members,worth", [(32, False), (34, True)])
def test_the_attention_decides(cuda_lib, members, worth):
    """A plan that leaves the choice is followed from 128 MB of keys and values saved on: 32 or 34
    sequences with 2048 positions of 2 KB in common."""
    Hkv, D, page = 8, 128, 64
    cache = [t.cuda() for t in _batch([(2048, members)], [70, 3], [300], Hkv, D, page, seed=5)]
    B = cache[5].numel()
    q = torch.randn(B, 2 * Hkv, 1, D, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    by = {least: _lib.kvp_find_shared(cache[4], cache[5], page, least) for least in (-1, 0, (1 << 31) - 1)}
    assert by[-1].tolist()[:4] == [by[0].tolist()[0], 1, B, (members - 1) * 2048 // RUN]
    assert _read_plan(by[-1], B) == _read_plan(by[0], B) and len(_read_plan(by[0], B)) == 1
    res = {least: _lib.kv8_attn_shared(q, *cache, plan) for least, plan in by.items()}
    same = {least: all(torch.equal(a, b) for a, b in zip(res[least], res[-1])) for least in by}
    assert same == {-1: True, 0: worth, (1 << 31) - 1: not worth}
    assert (members - 1) * 2048 * 2 * Hkv * D // (128 << 20) == int(worth) and _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_small_groups_are_left_alone(cuda_lib):
    """A plan that leaves the choice: no group of fewer than 8192 positions saved."""
    _, _, _, _, table, lens = _batch([(1024, 9), (1024, 8), (4096, 3)], [5], [], 1, 64, 64, seed=2)
    plan = _lib.kvp_find_shared(table.cuda(), lens.cuda(), 64)
    assert sorted((d * RUN, len(m)) for m, d in _read_plan(plan, 20).values()) == [(1024, 9), (4096, 3)]
    assert plan[3].item() == (8 * 1024 + 2 * 4096) // RUN


@pytest.mark.gpu
def test_pools_past_32_bits(cuda_lib):
    """Pages whose bytes start past 2^32: rotated prompts and steps, the plan and the attention against a
    small pool that holds the same pages, byte for byte and bit for bit."""
    Hkv, page, D, n_pages = 8, 64, 128, 70000
    ids = [69999, 1, 68000, 69000, 20000, 69998, 5, 67777]
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(2, Hkv, 300, D, generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn(2, 32, 3, D, generator=g).to(BF16).cuda()
    rope, res = Rope(D), []
    for n, at in ((n_pages, ids), (len(ids), list(range(len(ids))))):
        pools = [torch.zeros(n, Hkv, page, D, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
        scales = [torch.ones(n, Hkv, device="cuda") for _ in range(2)]
        # the second sequence's first four pages are the first one's, which has 297 positions of its own
        table = _i32([*at[:6], *at[:4], *at[6:8]]).view(2, 6)
        _lib.kv8_append(k, v, *pools, *scales, table, _i32([297, 0]), n_new=_i32([297, 0]), rope=rope)
        _lib.kv8_append(k[:, :, :44].contiguous(), v[:, :, :44].contiguous(), *pools, *scales, table, _i32([297, 300]),
                        n_new=_i32([0, 44]), rope=rope)
        turned = _lib.kv8_append(k[:, :, :3], v[:, :, :3], *pools, *scales, table, _i32([300, 301]),
                                 n_new=_i32([3, 1]), rope=rope, q=q)
        plan = _lib.kvp_find_shared(table, _i32([300, 301]), page, 0)
        assert _read_plan(plan, 2) == {0: ([0, 1], 2)}
        out = _lib.kv8_attn_shared(turned, *pools, *scales, table, _i32([300, 301]), plan, n_new=_i32([3, 1]))
        assert _lib.sync_status() == _lib.ATTN_OK
        res.append([turned, *out, *(p.view(torch.uint8)[at].clone() for p in pools), *(s[at].clone() for s in scales)])
        del pools, scales
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert bool(res[0][1][1, :, 0].any()) and bool(res[0][3].any())


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,Nq,D,page,dtype", [(4, 2, 1, 64, 16, F16), (3, 3, 2, 128, 32, BF16), (20, 1, 1, 64, 64, F16)])
def test_many_short_ends(cuda_lib, Hq, Hkv, Nq, D, page, dtype):
    """Dozens of sequences with no, one or a few positions of their own, where a warp's share begins, ends and
    lies inside the steps that a unit starts with."""
    for seed, tails in enumerate(([0, 1, 33, 0, 64, 2, 129], [0] * 20 + [700], [1], [31, 0, 0, 0, 32])):
        cache = _batch([(256, 50), (128, 21)], tails, [0, 5, 0, 300], Hkv, D, page, seed=seed)
        B = cache[5].numel()
        q = torch.randn(B, Hq, Nq, D, generator=torch.Generator().manual_seed(seed)).to(dtype)
        n_new = [min(Nq, int(n)) for n in cache[5]]
        dev = [t.cuda() for t in cache]
        plan = _lib.kvp_find_shared(dev[4], dev[5], page, 0)
        out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(n_new))
        assert _lib.sync_status() == _lib.ATTN_OK
        _check(q, cache, n_new, out, lse, f"short ends {seed} D={D}")


# ------------------------------------------------------------------ the cache that shares

def test_a_cache_with_a_window_does_not_share():
    with pytest.raises(ValueError, match="window"):
        PagedKVCache(1, 2, 1, 64, n_pages=4, window=8, share=True, device="cpu")


@pytest.mark.gpu
def test_only_a_sharing_cache_looks_for_prefixes(cuda_lib):
    with pytest.raises(ValueError, match="share"):
        PagedKVCache(1, 2, 1, 64, n_pages=4).find_shared()


@pytest.mark.gpu
@pytest.mark.parametrize("D,page,rot,inter,dtype", [(64, 32, 64, False, F16), (128, 64, 32, True, BF16)])
def test_a_run_of_samples(cuda_lib, D, page, rot, inter, dtype):
    """A prompt with rotated keys, its fork into samples, steps that are captured as one graph, a second
    fork (beams change, one ends, another prompt comes in) that the same graph follows, and a
    compaction: each step's attention against the definition over the cache's own content, the rotated
    rows against the rotation alone."""
    S, Hq, Hkv, L, prompt, T = 10, 4, 2, 2, 1100, 2
    rope, g, rng = Rope(D, rot, interleaved=inter), torch.Generator().manual_seed(D), random.Random(7)
    cache = PagedKVCache(L, S, Hkv, D, n_pages=3 * prompt // page + 8 * S, page_size=page, max_pages=prompt // page + 8,
                         share=True, min_saved=8192)

    def rows(h, n):
        return torch.randn(S, h, n, D, generator=g).to(dtype).cuda()

    def step(x, n):
        cache.reserve(n)
        res = []
        for i in range(L):
            q = cache.append(i, x[i][1], x[i][2], n, rope=rope, q=x[i][0])
            res.append((q,) + cache.attend(i, q, n_new=n))
        return res

    def check(x, n, res, what):
        assert _lib.sync_status() == _lib.ATTN_OK
        n_new, lens = n.tolist(), cache.lens.tolist()
        at = (cache.lens - n)[:, None] + torch.arange(x[0][0].shape[2], dtype=torch.int32, device="cuda")[None]
        for i in range(L):
            q, out, lse = res[i]
            want = rope(x[i][0], positions=at)
            held = [t[i].cpu() for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
            for b, k in enumerate(n_new):
                assert torch.equal(q[b, :, :k], want[b, :, :k]) and not q[b, :, k:].any()
            _check(q.cpu(), (*held, cache.table.cpu(), cache.lens.cpu()), n_new, out, lse, f"{what} layer {i}", some=(
                0, 3, 4, 9))

    def fork(parents):
        cache.reassign(_i32(parents))
        assert _lib.sync_status() == _lib.ATTN_OK
        return sorted((d * RUN, len(m)) for m, d in _read_plan(cache.plan, S).values())

    assert _read_plan(cache.plan, S) == {}
    first = [(rows(Hq, prompt), rows(Hkv, prompt), rows(Hkv, prompt)) for _ in range(L)]
    n = _i32([prompt] + [0] * (S - 1))
    cache.reserve(n)
    for i, (q, k, v) in enumerate(first):
        cache.append(i, k, v, n, rope=rope)
    assert fork([0] * S) == [(prompt // RUN * RUN, S)]
    bufs = [(rows(Hq, T), rows(Hkv, T), rows(Hkv, T)) for _ in range(L)]
    counts = _i32([1, 2] * (S // 2))
    check(bufs, counts, step(bufs, counts), "eager")
    book = [t.clone() for t in (cache.table, cache.lens, cache.refs, cache.info, cache.granted)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(bufs, counts)

    def replay(what):
        for x in bufs:
            for t in x:
                t.copy_(torch.randn(t.shape, generator=g).to(dtype))
        counts.copy_(torch.tensor([rng.randint(0, T) for _ in range(S)]))
        graph.replay()
        check(bufs, counts, res, what)

    assert all(torch.equal(a, b) for a, b in zip(book, (cache.table, cache.lens, cache.refs, cache.info, cache.granted)))
    for k in range(3):
        replay(f"replay {k}")
    assert fork([0, 0, 0, 3, 3, 3, 3, 3, 3, -1]) == [(prompt // RUN * RUN, S - 1)]
    replay("second fork")
    n = _i32([0] * (S - 1) + [prompt])
    cache.reserve(n)
    for i, (q, k, v) in enumerate(first):
        cache.append(i, k, v, n, rope=rope)
    replay("another prompt beside the group")
    cache.compact()
    replay("compacted")
    assert fork([0] * 5 + [9] * 5) == []                # 4 * 1024 positions saved by each: too few
    replay("no group")
    fork([-1] * S)
    assert not cache.refs.any() and _read_plan(cache.plan, S) == {}


@pytest.mark.gpu
def test_a_captured_fork(cuda_lib):
    """reassign with its search for prefixes captured, and steps without counts behind it; a cache of one
    sequence shares with nobody."""
    S, Hq, Hkv, D, page, prompt = 9, 3, 1, 64, 16, 1050
    g = torch.Generator().manual_seed(2)
    cache = PagedKVCache(1, S, Hkv, D, n_pages=3 * prompt // page + 2 * S, page_size=page, max_pages=prompt // page + 3,
                         share=True, min_saved=1024)
    k, v = (torch.randn(S, Hkv, prompt, D, generator=g).to(F16).cuda() for _ in range(2))
    q = torch.randn(S, Hq, 1, D, generator=g).to(F16).cuda()
    n, parents = _i32([prompt, prompt] + [0] * (S - 2)), _i32(range(S))
    cache.reserve(n)
    cache.append(0, k, v, n)
    cache.reassign(parents)                     # (the calls' first use is not captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.reassign(parents)
    for fork, want in (([0] * 4 + [1] * 5, [(1024, 4), (1024, 5)]), ([0] * 2 + [8] * 7, [(1024, 2), (1024, 7)]),
                       ([8] * S, [(1024, S)])):
        parents.copy_(torch.tensor(fork))
        graph.replay()
        assert sorted((d * RUN, len(m)) for m, d in _read_plan(cache.plan, S).values()) == want
        cache.reserve(1)
        cache.append(0, k[:, :, :1].contiguous(), v[:, :, :1].contiguous())
        out, lse = cache.attend(0, q)
        assert _lib.sync_status() == _lib.ATTN_OK
        held = [t[0].cpu() for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
        _check(q.cpu(), (*held, cache.table.cpu(), cache.lens.cpu()), None, out, lse, f"fork {fork}", some=(0, 4, 8))
    alone = PagedKVCache(1, 1, Hkv, D, n_pages=70, page_size=page, share=True, min_saved=0)
    alone.reserve(prompt)
    alone.append(0, k[:1], v[:1])
    alone.find_shared()
    assert _read_plan(alone.plan, 1) == {}
    out, lse = alone.attend(0, q[:1])
    want = _lib.kv8_attn(q[:1], alone.k_pages[0], alone.v_pages[0], alone.k_scale[0], alone.v_scale[0], alone.table,
                         alone.lens)
    helpers.assert_fwd_close(*(t.double().cpu().numpy() for t in (out, lse, *want)), F16, "one sequence")
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("D,page,dtype,size,scale", [(64, 16, BF16, 2.0 ** -9, None), (128, 64, BF16, 2.0 ** -9, None),
                                                     (64, 32, F16, 1.0, 1e-8), (128, 128, F16, 2.0 ** -14, 1e-20)])
def test_keys_of_zeros_under_tiny_queries(cuda_lib, D, page, dtype, size, scale):
    """A tile whose keys are all 0 has the smallest scale: its scores' factor is below fp32's range, and what
    the queries that stand in it do not see is hidden all the same."""
    cache = _batch([(256, 3)], [0, 2, 40], [], 1, D, page, seed=3)
    zeros = sorted({int(r[c]) for r in cache[4] for c in range(RUN // page, 2 * RUN // page)})
    cache[0].view(torch.uint8)[zeros] = 0
    cache[2][zeros] = 2.0 ** -126
    q = (torch.randn(3, 2, 4, D, generator=torch.Generator().manual_seed(1)) * size).to(dtype)
    dev = [t.cuda() for t in cache]
    plan = _lib.kvp_find_shared(dev[4], dev[5], page, 0)
    assert len(_read_plan(plan, 3)) == 1
    ref = kv8_ref.attention(q, *cache, scale=scale)
    for out, lse in (_lib.kv8_attn_shared(q.cuda(), *dev, plan, scale=scale), _lib.kv8_attn(q.cuda(), *dev, scale=scale)):
        assert _lib.sync_status() == _lib.ATTN_OK
        helpers.assert_fwd_close(*(t.double().cpu().numpy() for t in (out, lse, *ref)), dtype, f"zero keys D={D}")
    # pages of the tile that hold nothing readable, for rows of which some see nothing at all
    bad = dev[4].clone()
    bad[:, RUN // page] = -1
    n_new = _i32([4, 0, 1])
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev[:4], bad, dev[5], plan, scale=scale, n_new=n_new)
    assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
    want = _lib.kv8_attn(q.cuda(), *dev[:4], bad, dev[5], scale=scale, n_new=n_new)
    assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
    for b, n in enumerate((4, 0, 1)):
        assert not out[b, :, n:].any() and bool((lse[b, :, n:] == float("-inf")).all())
        if n:
            helpers.assert_fwd_close(*(t[b, :, :n].double().cpu().numpy() for t in (out, lse, *want)), dtype,
                                     f"zero keys, bad page D={D}")


@pytest.mark.gpu
def test_more_rows_than_the_shared_attention_takes(cuda_lib, monkeypatch):
    """Prompts past its rows, or past the workspace it may ask for, are read by every sequence for itself."""
    from tiled_memory_efficient_gb300 import kvcache
    Hq, n = 64, 16400                         # 1.05 million rows of the one KV head
    cache = PagedKVCache(1, 1, 1, 64, n_pages=-(-n // 128), page_size=128, share=True, min_saved=0)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(1, 1, n, 64, generator=g, device="cuda").to(BF16) for _ in range(2))
    cache.reserve(n)
    cache.append(0, k, v)
    pools = [t[0] for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)] + [cache.table, cache.lens]
    q = torch.randn(1, Hq, n, 64, generator=g, device="cuda").to(BF16)
    want = _lib.kv8_attn(q, *pools)
    for n_new in (None, n):
        assert all(torch.equal(a, b) for a, b in zip(cache.attend(0, q, n_new=n_new), want))
    assert _lib.sync_status() == _lib.ATTN_OK
    # the workspace: rows in fp32 twice, as long as they fit the limit
    q = q[:, :, -64:].contiguous()
    sizes = []
    for limit in (8 * q.numel(), 8 * q.numel() - 1):
        monkeypatch.setattr(kvcache, "_SHARED_BYTES", limit)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        out, lse = cache.attend(0, q)
        sizes.append(torch.cuda.max_memory_allocated() - before - out.numel() * 2 - lse.numel() * 4)
        helpers.assert_fwd_close(*(t.double().cpu().numpy() for t in (out, lse, want[0][:, :, -64:], want[1][:, :, -64:])),
                                 BF16, "a prompt's last queries")
    # what either call's own workspace takes, in the allocator's steps (512 bytes, 2 MB for larger blocks)
    most = [f(1, Hq, 1, 64, 64) for f in (cuda_lib.kv8_attn_shared_workspace_size, cuda_lib.kv8_attn_workspace_size)]
    assert 8 * q.numel() <= sizes[0] and all(a <= b + (2 << 20) for a, b in zip(sizes, most))
    assert most[1] + (2 << 20) < most[0] and _lib.sync_status() == _lib.ATTN_OK


QUESTIONS = [
    # Hq, Hkv, Nq, D, page, groups, tails, alone, dtype: queries in several tiles of the prefix, members' rows over
    # several blocks of 256, sequences shorter than their queries
    (4, 2, 70, 64, 32, [(256, 3)], [3, 90, 200], [100], F16),
    (7, 1, 40, 128, 16, [(384, 5), (128, 2)], [0, 41, 7], [39], BF16),
    (2, 1, 300, 128, 64, [(512, 4)], [10, 310, 0], [400, 120], BF16),
    (14, 2, 129, 64, 64, [(256, 2), (1024, 3)], [1, 150], [], F16),
    (1, 1, 700, 64, 128, [(640, 3)], [0, 300], [], F16),
    (8, 2, 17, 128, 128, [(1280, 30)], [17, 20, 300], [5], BF16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", QUESTIONS, ids=str)
def test_questions_behind_a_prefix(cuda_lib, case):
    """Many queries a sequence: all of them, and a number for each sequence."""
    Hq, Hkv, Nq, D, page, groups, tails, alone, dtype = case
    cache = _batch(groups, tails, alone, Hkv, D, page, seed=Nq)
    B, rng = cache[5].numel(), random.Random(Nq)
    q = torch.randn(B, Hq, Nq, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dev = [t.cuda() for t in cache]
    plan = _lib.kvp_find_shared(dev[4], dev[5], page, 0)
    assert len(_read_plan(plan, B)) == len(groups)
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan)
    assert _lib.sync_status() == _lib.ATTN_OK
    for b in range(B):   # all Nq rows: those before a sequence's first position see nothing
        n = min(Nq, int(cache[5][b]))
        assert not out[b, :, : Nq - n].any() and bool((lse[b, :, : Nq - n] == float("-inf")).all())
        one = cache[:4] + (cache[4][b:b + 1], cache[5][b:b + 1])
        ref = kv8_ref.attention(q[b:b + 1, :, Nq - n:], *one)
        helpers.assert_fwd_close(*(t[b, :, Nq - n:].double().cpu().numpy() for t in (out, lse)), *(t[0].numpy() for t in ref),
                                 dtype, f"questions {case} sequence {b}")
    n_new = [min(rng.choice([0, 1, rng.randint(1, Nq), Nq]), int(n)) for n in cache[5]]
    held = q.cuda()
    held[0, :, n_new[0]:] = float("nan")         # rows past a count may hold anything
    res = [_lib.kv8_attn_shared(held, *dev, plan, n_new=_i32(n_new)) for _ in range(2)]
    assert _lib.sync_status() == _lib.ATTN_OK and all(torch.equal(a, b) for a, b in zip(*res))
    _check(q, cache, n_new, *res[0], f"questions, counts {case}")


@pytest.mark.gpu
@pytest.mark.parametrize("D,page,dtype", [(64, 16, F16), (128, 64, BF16)])
def test_questions_about_one_text(cuda_lib, D, page, dtype):
    """A sharing cache from its first prompt on: the text attends before any fork, each sequence's question of its own
    length behind it, then drafts."""
    S, Hq, Hkv, text = 6, 4, 2, 900
    rope, g = Rope(D), torch.Generator().manual_seed(D)
    cache = PagedKVCache(1, S, Hkv, D, n_pages=S * 300 // page + 2 * text // page, page_size=page, max_pages=1400 // page,
                         share=True, min_saved=0)

    def turn(counts, T):
        q, k, v = (torch.randn(S, h, T, D, generator=g).to(dtype).cuda() for h in (Hq, Hkv, Hkv))
        n = _i32(counts)
        cache.reserve(n)
        q = cache.append(0, k, v, n, rope=rope, q=q)
        out, lse = cache.attend(0, q, n_new=n)
        assert _lib.sync_status() == _lib.ATTN_OK
        held = [t[0].cpu() for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
        _check(q.cpu(), (*held, cache.table.cpu(), cache.lens.cpu()), counts, out, lse, f"questions D={D} T={T}")

    turn([text] + [0] * (S - 1), text)
    cache.reassign(_i32([0] * S))
    assert sorted((d * RUN, len(m)) for m, d in _read_plan(cache.plan, S).values()) == [(text // RUN * RUN, S)]
    turn([200, 1, 77, 130, 0, 199], 200)
    turn([1, 5, 0, 3, 2, 4], 5)
    turn([0, 0, 0, 0, 90, 20], 90)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,Nq,members,followed", [
    (8, 8, 64, 1, 7, False), (8, 8, 64, 1, 8, True), (16, 8, 64, 5, 5, False), (16, 8, 64, 5, 6, True), (32, 8, 64, 5, 2, True),
    (8, 8, 128, 1, 2, False), (8, 8, 128, 1, 3, True), (24, 8, 128, 6, 2, True)])
def test_groups_too_small_to_follow(cuda_lib, Hq, Hkv, D, Nq, members, followed):
    """A plan that leaves the choice: groups whose rows cost more together than apart are read apart, beside a large one
    that is followed; a plan made by hand follows all of them."""
    page, big, small, n = 128, 40, 2, 4096 * 1024 // (Hkv * D)
    cache = [t.cuda() for t in _batch([(n, big)] + [(8192, members)] * small, [70, 3, 200], [300], Hkv, D, page, seed=members)]
    B = cache[5].numel()
    q = torch.randn(B, Hq, Nq, D, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    by = {least: _lib.kvp_find_shared(cache[4], cache[5], page, least) for least in (-1, 0, (members - 1) * 8192 + 1, (1 << 31) - 1)}
    assert [len(_read_plan(p, B)) for p in by.values()] == [1 + small, 1 + small, 1, 0]
    assert _read_plan(by[-1], B) == _read_plan(by[0], B) and (big - 1) * n * 2 * Hkv * D > 128 << 20
    own, hand, large, none = (_lib.kv8_attn_shared(q, *cache, plan) for plan in by.values())
    assert all(torch.equal(a, b) for a, b in zip(own, hand if followed else large))
    assert not all(torch.equal(a, b) for a, b in zip(own, large if followed else hand))
    for res in (hand, large, none):
        helpers.assert_fwd_close(*(x.double().cpu().numpy() for x in (*own, *res)), BF16, f"small groups D={D} Nq={Nq}")
    assert _lib.sync_status() == _lib.ATTN_OK
    # nothing but small ones
    cache = [t.cuda() for t in _batch([(8192, members)] * small, [70, 3, 200], [300], Hkv, D, page, seed=members)]
    q = q[: cache[5].numel()].contiguous()
    own = _lib.kv8_attn_shared(q, *cache, _lib.kvp_find_shared(cache[4], cache[5], page))
    helpers.assert_fwd_close(*(x.double().cpu().numpy() for x in (*own, *_lib.kv8_attn(q, *cache))), BF16, "small groups alone")
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,Nq,D,page,dtype", [(20, 1, 1, 64, 16, F16), (8, 1, 5, 64, 64, BF16), (8, 2, 6, 128, 32, F16),
                                                    (34, 2, 1, 128, 128, BF16), (6, 2, 23, 64, 32, F16)])
def test_short_ends_of_many_rows(cuda_lib, Hq, Hkv, Nq, D, page, dtype):
    """More than 16 rows a KV head: runs of short ends beside long sequences that share nothing, where a CTA's share begins,
    ends and lies inside the steps that a unit starts with; empty sequences first, last and between."""
    for seed, (tails, alone) in enumerate(([[1, 33, 0, 64, 129], [0, 5, 0, 3000, 2500]], [[0] * 9 + [700], [0, 0, 0]],
                                           [[1], [4100]], [[31, 0, 0, 0, 200], [17, 1900, 0, 40]])):
        cache = _batch([(256, 30), (128, 11)], tails, alone, Hkv, D, page, seed=seed + Nq)
        B = cache[5].numel()
        q = torch.randn(B, Hq, Nq, D, generator=torch.Generator().manual_seed(seed)).to(dtype)
        n_new = [min(Nq, int(n)) for n in cache[5]]
        dev = [t.cuda() for t in cache]
        plan = _lib.kvp_find_shared(dev[4], dev[5], page, 0)
        out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(n_new))
        assert _lib.sync_status() == _lib.ATTN_OK
        _check(q, cache, n_new, out, lse, f"short ends, many rows {seed} D={D}")
        again = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(n_new))
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
def test_the_largest_batch_of_many_rows(cuda_lib):
    """1024 sequences of 24 rows: the count of sequences before and the queries share a word."""
    cache = _batch([(128, 700), (256, 200)], [0, 5, 40], [30, 0, 200, 0] * 31, 1, 64, 128, seed=23)
    q = torch.randn(1024, 8, 3, 64, generator=torch.Generator().manual_seed(4)).to(F16)
    dev = [t.cuda() for t in cache]
    n_new = [min(3, int(n)) for n in cache[5]]
    plan = _lib.kvp_find_shared(dev[4], dev[5], 128, 0)
    out, lse = _lib.kv8_attn_shared(q.cuda(), *dev, plan, n_new=_i32(n_new))
    assert _lib.sync_status() == _lib.ATTN_OK
    _check(q, cache, n_new, out, lse, "shared, 1024 sequences of many rows", some=range(0, 1024, 41))
    a, b = _lib.kv8_attn(q.cuda(), *dev, n_new=_i32(n_new))
    for i, n in enumerate(n_new):
        if n:
            helpers.assert_fwd_close(*(x[i, :, :n].double().cpu().numpy() for x in (out, lse, a, b)), F16, "shared against plain")


@pytest.mark.gpu
def test_a_cache_too_small_to_share(cuda_lib):
    """Where no plan can be followed, attention is the plain one and a fork looks for no prefixes; a number of positions
    asks for them all the same, and so does a larger table."""
    S, Hkv, D, page = 8, 2, 64, 32
    g = torch.Generator().manual_seed(5)
    k = torch.randn(S, Hkv, 520, D, generator=g).to(F16).cuda()
    q = torch.randn(S, 4, 1, D, generator=g).to(F16).cuda()
    per_page = (S - 1) * page * 2 * Hkv * D
    for max_pages, least, shares in ((20, -1, False), (20, 0, True), (-(-(128 << 20) // per_page), -1, True),
                                     (-(-(128 << 20) // per_page) - 1, -1, False)):
        cache = PagedKVCache(1, S, Hkv, D, n_pages=200, page_size=page, max_pages=max_pages, share=True, min_saved=least)
        n = _i32([512] + [0] * (S - 1))
        cache.reserve(n)
        cache.append(0, k, k, n)
        cache.reassign(_i32([0] * S))
        assert len(_read_plan(cache.plan, S)) == (1 if least == 0 else 0)   # (7 * 512 positions are too few by itself)
        cache.plan.fill_(7)                    # no plan: a call that reads it says so
        cache.reserve(3)
        cache.append(0, k[:, :, 512:515].contiguous(), k[:, :, 512:515].contiguous())
        out, lse = cache.attend(0, q)
        assert _lib.sync_status() == (_lib.ATTN_ERR_PAGE if shares else _lib.ATTN_OK)
        pools = [t[0] for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)] + [cache.table, cache.lens]
        want = _lib.kv8_attn(q, *pools)
        if not shares:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        cache.find_shared()
        assert _lib.sync_status() == _lib.ATTN_OK and cache.plan[0] != 7
