"""Steps of a decoding loop that no host looks at: a pool that runs out, and
sequences that take different numbers of tokens.

A refused step is compared for equality: nothing of the cache may change."""
import pytest
import torch

from tiled_memory_efficient_gb300 import _lib
from tiled_memory_efficient_gb300.kvcache import PagedKVCache

F16, BF16 = torch.float16, torch.bfloat16
P = 256  # a fake, 16-byte-aligned "device" address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


def _i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ CPU: refusals

APPEND = dict(k=P, v=P, kp=P, vp=P, ks=P, vs=P, table=P, lens=P, n_new=0, granted=0, B=2, Hkv=2, T=3, D=64,
              page=16, n_pages=10, max_pages=5, sb=384, sh=192, st=64, dtype=1)


@pytest.mark.parametrize("change,code", [
    ({"k": 0}, 1), ({"lens": 0}, 1), ({"T": 0}, 1), ({"D": 32}, 2), ({"page": 24}, 2), ({"st": 60}, 3),
    ({"granted": P + 2}, 3), ({"n_new": P + 1}, 3),
])
def test_append_step_refusals(lib, change, code):
    assert lib.kv8_append_step(*{**APPEND, **change}.values(), None) == code


@pytest.mark.parametrize("change,code", [
    ({"table": 0}, 1), ({"n_new": 0}, 1), ({"window": -1}, 1), ({"page": 20}, 2), ({"ws": 0}, 1),
    ({"bytes": 8}, 6), ({"granted": P + 1}, 3), ({"info": P + 2}, 3),
])
def test_reserve_step_refusals(lib, change, code):
    args = dict(table=P, lens=P, refs=P, n_new=P, n_seqs=4, max_pages=5, n_pages=20, page=64, window=0, sinks=0,
                info=P, granted=0, ws=P, bytes=1 << 40)
    assert lib.kvp_reserve_step(*{**args, **change}.values(), None) == code


# ------------------------------------------------------------------ GPU: a pool that runs out

def _state(cache):
    """Everything a step may change, as bytes and numbers."""
    return [t.clone() for t in (cache.k_pages.view(torch.uint8), cache.v_pages.view(torch.uint8), cache.k_scale,
                                cache.v_scale, cache.table, cache.lens, cache.refs)]


def _assert_same(cache, want):
    for name, a, b in zip(("keys", "values", "key scales", "value scales", "table", "lens", "refs"), _state(cache), want):
        assert torch.equal(a, b), name


def _tokens(g, T, amp=1.0, layers=2, seqs=3, heads=2, D=64, dtype=F16):
    return [[(amp * torch.randn(seqs, heads, T, D, generator=g)).to(dtype).cuda() for _ in "kv"]
            for _ in range(layers)]


def _forked_cache(g):
    """Three sequences that share two full pages each, in a pool of three."""
    cache = PagedKVCache(2, 3, 2, 64, n_pages=3, page_size=16, max_pages=4)
    cache.reserve(_i32(32, 0, 0))
    for i, (k, v) in enumerate(_tokens(g, 32)):
        cache.append(i, k, v, _i32(32, 0, 0))
    cache.reassign(_i32(0, 0, 0))
    assert _lib.sync_status() == _lib.ATTN_OK and cache.granted.item() == 1
    assert cache.refs.tolist() == [3, 3, 0] and cache.lens.tolist() == [32, 32, 32]
    return cache


@pytest.mark.gpu
@pytest.mark.parametrize("as_int", [True, False])
def test_a_step_without_room_changes_nothing(cuda_lib, as_int):
    """reserve, append, attend on a full pool: no byte, scale, length or table entry of
    any sequence moves, until pages are free again."""
    g = torch.Generator().manual_seed(1)
    cache = _forked_cache(g)
    want = _state(cache)
    big = _tokens(g, 1, amp=100.0)      # larger than what the pages hold: their scales would grow
    q = torch.randn(3, 4, 1, 64, generator=g).to(F16).cuda()
    before = cache.attend(0, q)
    n = 1 if as_int else _i32(1, 1, 1)
    for _ in range(2):                  # three pages are needed, one is free
        cache.reserve(n)
        for i, (k, v) in enumerate(big):
            cache.append(i, k, v, n)
        assert cache.info.tolist() == [0, 0, 0, 1] and cache.granted.item() == 0
        after = cache.attend(0, q)
        assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
        assert _lib.sync_status() == _lib.ATTN_ERR_POOL
        _assert_same(cache, want)
    cache.compact()                     # neither of these gives the step its room
    cache.reassign(_i32(0, 1, 2))
    for i, (k, v) in enumerate(big):
        cache.append(i, k, v)
    _assert_same(cache, want)
    cache.reassign(_i32(0, -1, -1))     # two sequences end: the step fits now
    cache.reserve(_i32(1, 0, 0))
    for i, (k, v) in enumerate(big):
        cache.append(i, k, v, _i32(1, 0, 0))
    assert _lib.sync_status() == _lib.ATTN_OK and cache.granted.item() == 1
    assert cache.lens.tolist() == [33, 0, 0] and cache.refs.tolist() == [1, 1, 1]
    for i, (k, _) in enumerate(big):
        page = cache.k_pages[i, 2, :, 0].float() * cache.k_scale[i, 2, :, None]
        # e4m3's half step of 2^-4 of each value
        assert bool(((page - k[0, :, 0].float()).abs() <= 2.0 ** -4 * k[0, :, 0].float().abs() + 1e-2).all())
    a, b = _state(cache)[:2], want[:2]
    assert all(torch.equal(x[:, :2], y[:, :2]) for x, y in zip(a, b))


@pytest.mark.gpu
def test_a_full_table_row_changes_nothing(cuda_lib):
    """One sequence at the end of its table row refuses the step of all of them."""
    g = torch.Generator().manual_seed(2)
    cache = PagedKVCache(1, 2, 2, 64, n_pages=20, page_size=16, max_pages=2)
    cache.reserve(_i32(32, 5))
    k, v = _tokens(g, 32, layers=1, seqs=2)[0]
    cache.append(0, k, v, _i32(32, 5))
    assert _lib.sync_status() == _lib.ATTN_OK
    want = _state(cache)
    k, v = _tokens(g, 3, amp=50.0, layers=1, seqs=2)[0]
    cache.reserve(_i32(1, 3))
    cache.append(0, k, v, _i32(1, 3))
    assert _lib.sync_status() == _lib.ATTN_ERR_POOL
    _assert_same(cache, want)
    cache.reserve(_i32(0, 3))
    cache.append(0, k, v, _i32(0, 3))
    assert _lib.sync_status() == _lib.ATTN_OK and cache.lens.tolist() == [32, 8]


@pytest.mark.gpu
def test_a_captured_step_stops_at_a_full_pool(cuda_lib):
    """A captured step replayed past the pool's end leaves the cache as the last step
    with room left it."""
    g = torch.Generator().manual_seed(3)
    make = lambda: PagedKVCache(1, 2, 2, 64, n_pages=4, page_size=16, max_pages=8)
    k, v = _tokens(g, 1, layers=1, seqs=2)[0]

    def step(c):
        c.reserve(1)
        c.append(0, k, v, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(make())
    torch.cuda.current_stream().wait_stream(side)
    cache = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache)
    for _ in range(32):
        graph.replay()
    assert _lib.sync_status() == _lib.ATTN_OK and cache.lens.tolist() == [32, 32]
    want = _state(cache)
    k *= 64.0
    for _ in range(3):
        graph.replay()
    assert _lib.sync_status() == _lib.ATTN_ERR_POOL
    _assert_same(cache, want)


@pytest.mark.gpu
def test_granted_of_the_wrong_kind_is_refused(cuda_lib):
    cache = PagedKVCache(1, 2, 2, 64, n_pages=4)
    k, v = _tokens(torch.Generator().manual_seed(4), 1, layers=1, seqs=2)[0]
    pools = (cache.k_pages[0], cache.v_pages[0], cache.k_scale[0], cache.v_scale[0])
    for bad in (torch.ones(1, device="cuda"), _i32(1, 1), torch.ones(1, dtype=torch.int32)):
        with pytest.raises(ValueError, match="granted"):
            _lib.kvp_reserve(cache.table, cache.lens, cache.refs, _i32(1, 1), 64, cache.info, granted=bad)
        with pytest.raises(ValueError, match="granted"):
            _lib.kv8_append(k, v, *pools, cache.table, cache.lens, granted=bad)
    assert cache.lens.tolist() == [0, 0]


# ------------------------------------------------------------------ GPU: the status word

@pytest.mark.gpu
def test_one_kind_of_error_does_not_hide_another(cuda_lib):
    """A time-out, a bad length and a full pool in one go are returned one by one."""
    assert _lib.sync_status() == _lib.ATTN_OK
    cache = PagedKVCache(1, 1, 2, 64, n_pages=1, page_size=16)
    k = torch.ones(1, 2, 20, 64, dtype=F16, device="cuda")
    for timeout in (False, True):
        cache.reserve(17)                                       # one page of 16
        assert cache.granted.item() == 0
        _lib.kv8_append(k, k, cache.k_pages[0], cache.v_pages[0], cache.k_scale[0], cache.v_scale[0], cache.table,
                        cache.lens)                             # 20 tokens of a length of 0
        if timeout:
            stream = torch.cuda.current_stream().cuda_stream
            assert cuda_lib.attn_selftest_timeout(1_000_000, stream) == _lib.ATTN_OK   # 1 ms
            assert _lib.sync_status() == _lib.ATTN_ERR_TIMEOUT
        assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
        assert _lib.sync_status() == _lib.ATTN_ERR_POOL
        assert _lib.sync_status() == _lib.ATTN_OK
