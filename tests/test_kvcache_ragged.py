"""Attention over the paged 8-bit KV cache when sequences take different numbers of
tokens in one step: the first n_new rows of a sequence are its newest
positions, the others see nothing.

Rows that see something are held to the tolerances of the other forwards
(tests/helpers.py) against the CPU definition of each sequence alone; the others are
0 and -inf exactly."""
import random

import pytest
import torch

from tests import helpers, kv8_ref
from tests.test_kvcache import _cache
from tiled_memory_efficient_gb300 import _lib
from tiled_memory_efficient_gb300.kvcache import PagedKVCache

F16, BF16, F8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
P = 256  # a fake, 16-byte-aligned "device" address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


STEP = dict(q=P, kp=P, vp=P, ks=P, vs=P, table=P, lens=P, n_new=P, granted=P, out=P, lse=P, ws=P, n=1 << 40, B=2,
            Hq=4, Hkv=2, Nq=1, D=64, page=64, n_pages=10, max_pages=5, scale=0.1, window=0, sinks=0, dtype=0)


@pytest.mark.parametrize("change,code", [
    ({"q": 0}, 1), ({"ws": 0}, 1), ({"Hq": 3}, 1), ({"D": 96}, 2), ({"page": 48}, 2), ({"scale": 0.0}, 1),
    ({"window": -1}, 1), ({"kp": P + 8}, 3), ({"n_new": P + 2}, 3), ({"granted": P + 1}, 3), ({"n": 16}, 6),
    ({"B": 1025}, 2),
])
def test_step_refusals(lib, change, code):
    assert lib.kv8_attn_step(*{**STEP, **change}.values(), None) == code


def _i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _hide(cache, n_new, page, window, sinks):
    """Takes from the table what the n_new newest positions do not see."""
    table = cache[4]
    for b, n in enumerate(n_new):
        length = int(cache[5][b])
        for j in range(table.shape[1]):
            if window and j * page >= sinks and (j + 1) * page <= length - n - window + 1:
                table[b, j] = -1


def _check(q, cache, n_new, window, sinks, out, lse, what):
    out, lse = out.double().cpu(), lse.double().cpu()
    for b, n in enumerate(n_new):
        assert bool((out[b, :, n:] == 0).all()) and bool((lse[b, :, n:] == float("-inf")).all()), (what, b)
        if n:
            one = cache[:4] + (cache[4][b:b + 1], cache[5][b:b + 1])
            ro, rl = kv8_ref.attention(q[b:b + 1, :, :n], *one, window=window, sinks=sinks)
            helpers.assert_fwd_close(out[b, :, :n].numpy(), lse[b, :, :n].numpy(), ro[0].numpy(), rl[0].numpy(),
                                     q.dtype, what)


CASES = [
    # Hq, Hkv, Nq, D, page, lens, n_new, window, sinks, dtype
    (8, 2, 4, 64, 16, [100, 57, 300, 4, 33], [4, 1, 0, 2, 3], 0, 0, F16),
    (8, 2, 4, 64, 16, [100, 57, 300, 41, 136], [4, 1, 0, 2, 1], 40, 5, BF16),   # older queries want a page given back
    (4, 4, 2, 128, 64, [9000, 700], [1, 2], 0, 0, BF16),                        # one unit over many CTAs
    (14, 2, 5, 64, 64, [4100, 65, 1], [2, 5, 1], 1000, 70, F16),                # 35 rows: two row blocks
    (5, 1, 3, 128, 16, [95, 33, 0], [1, 3, 0], 16, 0, BF16),
    (32, 8, 4, 128, 32, [515, 64], [3, 1], 0, 0, F16),
    (2, 2, 64, 64, 32, [70, 64, 200], [64, 1, 13], 33, 1, F16),                 # a chunk
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_ragged_steps_match_the_definition(cuda_lib, case):
    Hq, Hkv, Nq, D, page, lens, n_new, window, sinks, dtype = case
    cache = _cache(lens, Hkv, D, page, window, sinks, Nq, seed=sum(lens))
    _hide(cache, n_new, page, window, sinks)
    q = torch.randn(len(lens), Hq, Nq, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dev = [t.cuda() for t in cache]
    out, lse = _lib.kv8_attn(q.cuda(), *dev, window=window, sinks=sinks, n_new=_i32(*n_new))
    assert _lib.sync_status() == _lib.ATTN_OK
    _check(q, cache, n_new, window, sinks, out, lse, f"ragged {case}")
    again = _lib.kv8_attn(q.cuda(), *dev, window=window, sinks=sinks, n_new=_i32(*n_new))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
def test_all_rows_equal_the_plain_call(cuda_lib):
    """n_new = Nq everywhere is the call without it, bit for bit."""
    cache = [t.cuda() for t in _cache([500, 70, 9], 2, 64, 16, 100, 3, 3, seed=1)]
    q = torch.randn(3, 4, 3, 64, generator=torch.Generator().manual_seed(2)).to(F16).cuda()
    a = _lib.kv8_attn(q, *cache, window=100, sinks=3)
    b = _lib.kv8_attn(q, *cache, window=100, sinks=3, n_new=_i32(3, 3, 3), granted=_i32(1))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_counts_that_do_not_fit_are_recorded(cuda_lib):
    cache = [t.cuda() for t in _cache([50, 2, 40], 2, 64, 16, 0, 0, 4, seed=1)]
    q = torch.randn(3, 4, 4, 64, generator=torch.Generator().manual_seed(2)).to(F16).cuda()
    good = _lib.kv8_attn(q, *cache, n_new=_i32(2, 2, 1))
    assert _lib.sync_status() == _lib.ATTN_OK
    for bad in ((2, 3, 1), (2, -1, 1), (2, 5, 1)):      # past the length, negative, past Nq
        out, lse = _lib.kv8_attn(q, *cache, n_new=_i32(*bad))
        assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
        assert bool((out[1] == 0).all()) and bool((lse[1] == float("-inf")).all())
        for c in (0, 2):
            assert torch.equal(out[c], good[0][c]) and torch.equal(lse[c], good[1][c])


@pytest.mark.gpu
def test_a_step_without_room_attends_to_nothing(cuda_lib):
    cache = [t.cuda() for t in _cache([500, 70], 2, 128, 64, 0, 0, 2, seed=1)]
    q = torch.randn(2, 4, 2, 128, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    out, lse = _lib.kv8_attn(q, *cache, n_new=_i32(2, 1), granted=_i32(0))
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    assert _lib.sync_status() == _lib.ATTN_OK
    full = PagedKVCache(1, 1, 2, 64, n_pages=1, page_size=16)
    full.reserve(16)
    k = torch.randn(1, 2, 16, 64, generator=torch.Generator().manual_seed(3)).to(F16).cuda()
    full.append(0, k, k)
    full.reserve(1)
    out, lse = full.attend(0, k[:, :, :1].contiguous(), n_new=1)
    assert bool((out == 0).all()) and bool((lse == float("-inf")).all())
    assert _lib.sync_status() == _lib.ATTN_ERR_POOL


@pytest.mark.gpu
def test_rows_that_see_nothing_are_zero_beside_a_nan(cuda_lib):
    """A NaN among the values that the step's rows see does not reach its other rows."""
    cache = _cache([300, 20], 2, 64, 64, 0, 0, 4, seed=1)
    cache[1].view(torch.uint8)[cache[4][0, 2], :, 5] = 0x7F
    q = torch.randn(2, 4, 4, 64, generator=torch.Generator().manual_seed(2)).to(F16).cuda()
    out, lse = _lib.kv8_attn(q, *(t.cuda() for t in cache), n_new=_i32(2, 4))
    assert bool(torch.isnan(out[0, :, :2]).all()) and bool(torch.isfinite(lse[0, :, :2]).all())
    assert bool((out[0, :, 2:] == 0).all()) and bool(torch.isfinite(out[1]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [lambda: torch.ones(2, device="cuda"), lambda: _i32(1, 1, 1)])
def test_counts_of_the_wrong_kind_are_refused(cuda_lib, bad):
    cache = [t.cuda() for t in _cache([50, 2], 2, 64, 16, 0, 0, 1, seed=1)]
    q = torch.zeros(2, 4, 1, 64, dtype=F16, device="cuda")
    with pytest.raises(ValueError, match="n_new"):
        _lib.kv8_attn(q, *cache, n_new=bad())
    with pytest.raises(ValueError, match="granted"):
        _lib.kv8_attn(q, *cache, granted=bad())


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks,page,dtype", [(40, 5, 16, F16), (70, 0, 16, BF16), (0, 0, 32, F16)])
def test_a_ragged_run(cuda_lib, window, sinks, page, dtype):
    """Drafts of 0 to 3 tokens a sequence until the window has left many pages behind:
    every step against the definition over what the sequence holds, and nothing
    recorded."""
    S, Hq, Hkv, D, T = 3, 4, 2, 64, 3
    cache = PagedKVCache(1, S, Hkv, D, n_pages=40, page_size=page, max_pages=16, window=window, sinks=sinks)
    g, rng = torch.Generator().manual_seed(9), random.Random(page + window)
    rows = [[], [], []]      # (k, v) of each call
    given_back = 0
    for step in range(70):
        n_new = [rng.randint(0, 3) for _ in range(S)]
        k, v, q = (torch.randn(S, h, T, D, generator=g).to(dtype) for h in (Hkv, Hkv, Hq))
        n = _i32(*n_new)
        cache.reserve(n)
        given_back += cache.info[2].item()
        cache.append(0, k.cuda(), v.cuda(), n)
        out, lse = (t.double().cpu() for t in cache.attend(0, q.cuda(), n_new=n))
        assert _lib.sync_status() == _lib.ATTN_OK, step
        lens = cache.lens.tolist()
        for c in range(S):
            if n_new[c]:
                rows[c].append((k[c, :, :n_new[c]], v[c, :, :n_new[c]]))
            assert bool((out[c, :, n_new[c]:] == 0).all()) and bool((lse[c, :, n_new[c]:] == float("-inf")).all())
            if n_new[c] == 0 or step % 5:
                continue
            n_pages = -(-lens[c] // page)
            kv = []
            for w in range(2):
                pool, sc = torch.zeros(n_pages, Hkv, page, D).to(F8), torch.ones(n_pages, Hkv)
                at = 0
                for call in rows[c]:
                    at += call[w].shape[1]
                    pool, sc = kv8_ref.append(call[w][None], pool, sc, torch.arange(n_pages)[None], [at],
                                              [call[w].shape[1]])
                kv += [pool, sc]
            ro, rl = kv8_ref.attention(q[c:c + 1, :, :n_new[c]], kv[0], kv[2], kv[1], kv[3],
                                       torch.arange(n_pages)[None], torch.tensor([lens[c]]), window, sinks)
            helpers.assert_fwd_close(out[c, :, :n_new[c]].numpy(), lse[c, :, :n_new[c]].numpy(), ro[0].numpy(),
                                     rl[0].numpy(), dtype, f"ragged run {window}+{sinks} sequence {c}")
    assert min(lens) > 71 and (given_back > 5 if window else given_back == 0)


@pytest.mark.gpu
def test_a_captured_step_follows_the_counts(cuda_lib):
    """A step captured once, with counts, lengths and tables read on the device."""
    make = lambda: PagedKVCache(1, 3, 2, 64, n_pages=30, page_size=16, max_pages=8, window=20, sinks=2)
    g = torch.Generator().manual_seed(3)
    steps = [[torch.randn(3, h, 2, 64, generator=g).to(F16).cuda() for h in (2, 2, 8)] for _ in range(30)]
    counts = [_i32(*(random.Random(i * 7 + c).randint(0, 2) for c in range(3))) for i in range(30)]

    def step(c, k, v, q, n):
        c.reserve(n)
        c.append(0, k, v, n)
        return c.attend(0, q, n_new=n)
    eager, held = make(), make()
    want = [step(eager, *s, n) for s, n in zip(steps, counts)]
    bufs, n = [t.clone() for t in steps[0]], counts[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(make(), *bufs, n)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(held, *bufs, n)
    for s, c, (wo, wl) in zip(steps, counts, want):
        for t, x in zip(bufs, s):
            t.copy_(x)
        n.copy_(c)
        graph.replay()
        assert torch.equal(out, wo) and torch.equal(lse, wl)
    assert _lib.sync_status() == _lib.ATTN_OK
    assert torch.equal(held.table, eager.table) and torch.equal(held.lens, eager.lens)


@pytest.mark.gpu
@pytest.mark.parametrize("D,G,Nq,dtype", [(64, 1, 1, F16), (64, 3, 5, BF16), (64, 7, 4, F16), (128, 1, 1, BF16),
                                          (128, 3, 4, F16), (128, 8, 4, BF16)])
def test_the_largest_batch(cuda_lib, D, G, Nq, dtype):
    """1024 sequences, whose lengths and counts live in shared memory."""
    g = torch.Generator().manual_seed(D + G)
    lens = torch.randint(0, 60, (1024,), generator=g).tolist()
    n_new = [min(n, int(torch.randint(0, Nq + 1, (1,), generator=g))) for n in lens]
    cache = _cache(lens, 1, D, 16, 20, 2, Nq, seed=5)
    _hide(cache, n_new, 16, 20, 2)
    q = torch.randn(1024, G, Nq, D, generator=g).to(dtype)
    out, lse = _lib.kv8_attn(q.cuda(), *(t.cuda() for t in cache), window=20, sinks=2, n_new=_i32(*n_new))
    assert _lib.sync_status() == _lib.ATTN_OK
    out, lse = out.cpu(), lse.cpu()
    some = [c for c in range(1024) if c % 37 == 0 or c > 1015]
    pick = torch.tensor(some)
    _check(q[pick], cache[:4] + (cache[4][pick], cache[5][pick]), [n_new[c] for c in some], 20, 2, out[pick], lse[pick],
           f"1024 sequences D={D}")
    for c in range(1024):
        assert bool((out[c, :, n_new[c]:] == 0).all()) and bool((lse[c, :, n_new[c]:] == float("-inf")).all())


@pytest.mark.gpu
def test_pools_past_32_bits(cuda_lib):
    """Pages whose bytes start past 2^31: append, attention and copies against a small pool
    that holds the same pages, byte for byte and bit for bit."""
    Hkv, page, D, n_pages = 8, 64, 128, 40000
    ids = [39999, 1, 38000, 39000, 20000, 39998, 5, 37777]
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(2, Hkv, 300, D, generator=g).to(BF16).cuda() for _ in range(2))
    q = torch.randn(2, 32, 3, D, generator=g).to(BF16).cuda()
    res = []
    for n, at in ((n_pages, ids), (len(ids), list(range(len(ids))))):
        pools = [torch.zeros(n, Hkv, page, D, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2)]
        scales = [torch.ones(n, Hkv, device="cuda") for _ in range(2)]
        table = _i32(*at[:3], -1, -1, *at[3:]).view(2, 5)
        _lib.kv8_append(k, v, *pools, *scales, table, _i32(130, 300), n_new=_i32(130, 300))
        out = _lib.kv8_attn(q, *pools, *scales, table, _i32(130, 300), n_new=_i32(3, 1))
        _lib.kv8_copy_pages(*pools, *scales, _i32(at[0]), _i32(at[2]), _i32(1))
        assert _lib.sync_status() == _lib.ATTN_OK
        res.append([*out, *(p.view(torch.uint8)[at].clone() for p in pools), *(s[at].clone() for s in scales)])
        del pools, scales
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert bool(res[0][2][0].any()) and torch.equal(res[0][2][0], res[0][2][2])
