"""The cache's append that turns its keys (kv8_append with rope), against its definition:
keys turned in 64 bits (tests/rope_ref.py), then quantised as kv8_append does (tests/kv8_ref.py).

A turned key is off by ARITH (|a| + |b|) A and, from one of a thread's tokens to its next, by two
products and a sum (2^-22.4 of the pair's length) seven times at most: under 2^-18 together.  It
is then rounded to e4m3, half a step off: 2^-4 of itself, 2^-10 of the scale near zero.  The scale
is that of the definition unless the largest magnitude lies so near a power of two times 448, which
the inputs are checked for.  Values and tokens that were there are compared for equality."""
import random

import pytest
import torch

from tests import kv8_ref, rope_ref
from tests.test_rope import _rows, _strides
from tiled_memory_efficient_gb300 import _lib
from tiled_memory_efficient_gb300.kvcache import PagedKVCache
from tiled_memory_efficient_gb300.rope import Rope

F16, BF16, F8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
P = 256  # a fake, 16-byte-aligned "device" address: validation fails before any use
OFF = 2.0 ** -18


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


ROWS = (512, 256, 64)
CALL = dict(k=P, v=P, kp=P, vp=P, ks=P, vs=P, table=P, lens=P, n_new=P, granted=P, q=P, qo=2 * P, turns=P, rot=64, inter=0,
            amp=1.0, B=2, Hq=4, Hkv=2, T=3, D=64, page=16, n_pages=10, max_pages=5, st=_strides(*ROWS, *ROWS, *ROWS),
            dtype=1)


@pytest.mark.parametrize("change,code", [
    ({"k": 0}, 1), ({"table": 0}, 1), ({"qo": 0}, 1), ({"q": 0}, 1), ({"Hq": 0}, 1), ({"turns": 0}, 1), ({"T": 0}, 1),
    ({"st": None}, 1), ({"rot": 65}, 1), ({"rot": 66}, 1), ({"inter": -1}, 1), ({"amp": -1.0}, 1), ({"dtype": 7}, 1),
    ({"D": 96}, 2), ({"page": 24}, 2), ({"B": 1 << 14, "T": 1 << 14, "page": 128, "max_pages": 1 << 10}, 2),
    ({"T": (1 << 31) - 100}, 2), ({"q": P + 8}, 3), ({"granted": P + 2}, 3), ({"turns": P + 4}, 3), ({"vp": P + 4}, 3),
    ({"st": _strides(512, 256, 68, *ROWS, *ROWS)}, 3), ({"st": _strides(*ROWS, *ROWS, 512, 256, -64)}, 1),
    ({"qo": P, "st": _strides(*ROWS, *ROWS, 512, 128, 64)}, 1),
])
def test_c_refusals(lib, change, code):
    assert lib.kv8_append_rope(*{**CALL, **change}.values(), None) == code


def _cache(lens, extra, Hkv, D, page, seed):
    """Pools with tokens of random scales, a table with pages for `extra` more tokens each."""
    g = torch.Generator().manual_seed(seed)
    cols = max(-(-(n + e) // page) for n, e in zip(lens, extra)) + 1
    n_pages = len(lens) * cols + 2
    pools = []
    for _ in range(2):
        x = torch.randn(n_pages, Hkv, page, D, generator=g) * 3
        e = torch.randint(-8, 3, (n_pages, Hkv), generator=g)
        pools += [(x * 20).clamp(-448, 448).to(F8), torch.ldexp(torch.ones(n_pages, Hkv), e)]
    ids = torch.randperm(n_pages, generator=g)[: len(lens) * cols].to(torch.int32).view(len(lens), cols)
    return pools, ids


CASES = [
    # D, rot, interleaved, B's old lengths, n_new, Hq, Hkv, T, page, layout, dtype
    (64, 64, False, [0, 5, 100], [1, 1, 1], 2, 1, 1, 16, "bhnd", F16),
    (128, 128, False, [70000, 64, 63], [1, 0, 1], 8, 2, 1, 64, "bhnd", BF16),
    (128, 128, False, [13, 0], [300, 257], 4, 2, 300, 64, "bnhd", BF16),
    (128, 128, True, [1, 90], [130, 77], 2, 2, 130, 128, "bhnd", F16),
    (128, 64, False, [40], [200], 2, 1, 200, 128, "bnhd", BF16),
    (64, 32, True, [7, 1000], [50, 3], 7, 1, 50, 32, "bhnd", F16),
    (64, 20, False, [30, 2], [100, 99], 3, 1, 100, 64, "bnhd", F16),      # pairs that no vector holds whole
    (64, 14, True, [30, 0], [33, 20], 1, 1, 33, 128, "bhnd", BF16),
    (128, 126, False, [500], [17], 2, 1, 17, 16, "bhnd", BF16),
    (128, 2, False, [9], [40], 1, 1, 40, 32, "bhnd", F16),
    (64, 16, False, [3, 3, 3, 3], [4, 0, 2, 5], 4, 2, 5, 16, "bhnd", F16),
    (64, 64, False, [120], [140], 2, 2, 140, 128, "bhnd", F16),
    # prompts long enough for a CTA to take several of a page's heads, the last one fewer
    (64, 64, False, [3, 0], [1290, 1300], 7, 7, 1300, 16, "bnhd", BF16),
    (128, 40, True, [17, 5], [700, 690], 7, 7, 700, 16, "bhnd", F16),
    (64, 20, False, [9, 1], [1300, 1], 3, 3, 1300, 16, "bnhd", F16),
    (128, 128, False, [1000, 60], [2600, 2590], 2, 5, 2600, 64, "bnhd", F16),
]


def _check_keys(got, scales, want, want_s, exact, table, lens, n_new, page, amp, old):
    """Keys of the cache against the definition; exact: the turned keys [B, H, T, D] in 64 bits."""
    assert torch.equal(scales, want_s)
    got, want = got.double(), want.double()
    seen = torch.zeros_like(got, dtype=torch.bool)
    for b, n in enumerate(n_new):
        for t in range(n):
            pos = lens[b] - n + t
            pid, r = int(table[b, pos // page]), pos % page
            s = want_s[pid].double()[:, None]
            x = exact[b, :, t]
            over = ((got[pid, :, r] * s - x).abs() - old[b, :, t] * OFF * amp) / torch.maximum(
                x.abs() * 2.0 ** -4 * (1 + OFF), 2.0 ** -10 * s)
            assert float(over.max()) <= 1, (b, t, float(over.max()))
            seen[pid, :, r] = True
    assert torch.equal(torch.where(seen, 0.0, got), torch.where(seen, 0.0, want))


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_appends_match_the_definition(cuda_lib, case):
    D, rot, inter, old, n_new, Hq, Hkv, T, page, layout, dtype = case
    B, amp = len(old), 1.5
    rope = Rope(D, rot, interleaved=inter, base=5000.0, amplitude=amp)
    q, k, v = (_rows((B, h, T, D), dtype, s, layout) for h, s in ((Hq, 1), (Hkv, 2), (Hkv, 3)))
    pools, table = _cache(old, n_new, Hkv, D, page, seed=len(old) + T)
    lens = [a + n for a, n in zip(old, n_new)]
    positions = torch.tensor(old)[:, None] + torch.arange(T)[None]
    exact = rope_ref.rotate(k.cpu(), rope.inv_freq, positions, amp, inter)
    size = rope_ref.partner(k.cpu(), rot, inter)
    want = kv8_ref.append(exact, pools[0], pools[1], table, lens, n_new)
    # no page's largest new magnitude so near a border that the arithmetic decides its scale
    for b, n in enumerate(n_new):
        for t0 in range(lens[b] - n, lens[b]):
            if t0 == lens[b] - n or t0 % page == 0:
                a, e = t0 - lens[b] + n, min(n, (t0 // page + 1) * page - lens[b] + n)
                m, _ = torch.frexp(exact[b, :, a:e].abs().amax((1, 2)) / 448.0)
                assert float((m - 0.5).abs().min()) > 4 * OFF and float((m - 1.0).abs().min()) > 4 * OFF
    dev = [t.cuda() for t in pools]
    args = (table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    n_dev = torch.tensor(n_new, dtype=torch.int32).cuda()
    out = _lib.kv8_append(k, v, dev[0], dev[2], dev[1], dev[3], *args, n_new=n_dev, rope=rope, q=q)
    assert _lib.sync_status() == _lib.ATTN_OK
    _check_keys(dev[0].cpu(), dev[1].cpu(), *want, exact, table, lens, n_new, page, amp, size)
    # values as the plain append writes them, byte for byte
    plain = [t.cuda() for t in pools]
    _lib.kv8_append(k, v, plain[0], plain[2], plain[1], plain[3], *args, n_new=n_dev)
    assert torch.equal(dev[2].view(torch.uint8), plain[2].view(torch.uint8)) and torch.equal(dev[3], plain[3])
    # queries as the rotation alone gives them, bit for bit; 0 past the counts
    alone = _lib.rope(q, None, rope, positions.int().cuda())
    for b, n in enumerate(n_new):
        alone[b, :, n:] = 0
    assert out.is_contiguous() and torch.equal(out, alone)
    # once more gives the same cache; without queries and in place, too
    again = [t.cuda() for t in pools]
    assert _lib.kv8_append(k, v, again[0], again[2], again[1], again[3], *args, n_new=n_dev, rope=rope) is None
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again, dev))
    spare = _rows((B, Hq, T, D), dtype, 1, layout)
    got = _lib.kv8_append(k, v, *(again[i] for i in (0, 2, 1, 3)), *args, n_new=n_dev, rope=rope, q=spare, q_out=spare)
    assert got.data_ptr() == spare.data_ptr() and torch.equal(spare, alone)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again, dev))
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_without_room_nothing_is_written(cuda_lib):
    rope, (pools, table) = Rope(64), _cache([20, 3], [2, 2], 2, 64, 16, seed=1)
    dev = [t.cuda() for t in pools]
    q, k = _rows((2, 4, 2, 64), F16, 1), _rows((2, 2, 2, 64), F16, 2)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = _lib.kv8_append(k, k, dev[0], dev[2], dev[1], dev[3], table.cuda(),
                          torch.tensor([22, 5], dtype=torch.int32).cuda(), granted=zero, rope=rope, q=q)
    assert bool((out == 0).all()) and _lib.sync_status() == _lib.ATTN_OK
    assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(dev, pools))


@pytest.mark.gpu
def test_what_does_not_fit_is_recorded(cuda_lib):
    """Counts and pages that do not fit: recorded, the sequence's queries 0, the others as they would be."""
    rope, (pools, table) = Rope(64), _cache([20, 3, 40], [2, 2, 2], 2, 64, 16, seed=2)
    q, k = _rows((3, 4, 2, 64), F16, 1), _rows((3, 2, 2, 64), F16, 2)

    def run(lens, n_new, table):
        dev = [t.cuda() for t in pools]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
        out = _lib.kv8_append(k, k, dev[0], dev[2], dev[1], dev[3], table.cuda(), i32(lens), n_new=i32(n_new), rope=rope,
                              q=q)
        return [t.cpu() for t in dev] + [out.cpu()], _lib.sync_status()
    good, rc = run([22, 5, 42], [2, 2, 2], table)
    assert rc == _lib.ATTN_OK
    for lens, n_new in (([22, 1, 42], [2, 2, 2]), ([22, 5, 42], [2, -1, 2]), ([22, 5, 42], [2, 3, 2]),
                        ([22, 10 ** 6, 42], [2, 2, 2])):
        got, rc = run(lens, n_new, table)
        assert rc == _lib.ATTN_ERR_PAGE
        assert bool((got[4][1] == 0).all()) and torch.equal(got[4][::2], good[4][::2])
        for b in (0, 2):
            pid = int(table[b, lens[b] // 16])
            assert torch.equal(got[0][pid].view(torch.uint8), good[0][pid].view(torch.uint8))
        pid = int(table[1, 0])
        assert torch.equal(got[0][pid].view(torch.uint8), pools[0][pid].view(torch.uint8))
    bad = table.clone()
    bad[1, 0] = pools[0].shape[0]
    got, rc = run([22, 5, 42], [2, 2, 2], bad)
    assert rc == _lib.ATTN_ERR_PAGE and torch.equal(got[4], good[4])   # its queries still have positions
    with pytest.raises(ValueError, match="only turned with rope"):
        _lib.kv8_append(k, k, *(t.cuda() for t in (pools[0], pools[2], pools[1], pools[3])), table.cuda(),
                        torch.tensor([22, 5, 42], dtype=torch.int32).cuda(), q=q)
    dev = [t.cuda() for t in (pools[0], pools[2], pools[1], pools[3])]
    lens = torch.tensor([22, 5, 42], dtype=torch.int32).cuda()
    for wrong in (q[:, :, :1], q.to(BF16), q[:2], q.cpu()):
        with pytest.raises(ValueError, match="q "):
            _lib.kv8_append(k, k, *dev, table.cuda(), lens, rope=rope, q=wrong)
    with pytest.raises(ValueError, match="head dim"):
        _lib.kv8_append(k, k, *dev, table.cuda(), lens, rope=Rope(128), q=q)
    with pytest.raises(ValueError, match="q_out"):
        _lib.kv8_append(k, k, *dev, table.cuda(), lens, rope=rope, q=q, q_out=k)
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_special_keys(cuda_lib):
    """Infinities and NaN of dimensions that stay: stored as the largest magnitude and as NaN, and left
    out of the scale."""
    rope = Rope(64, 32)
    k = _rows((1, 1, 20, 64), F16, 5)
    k[0, 0, 3, 40], k[0, 0, 4, 50], k[0, 0, 17, 63] = float("inf"), float("nan"), float("-inf")
    clean = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
    res = []
    for x in (k, clean):
        cache = PagedKVCache(1, 1, 1, 64, n_pages=2, page_size=16)
        cache.reserve(20)
        cache.append(0, x, x, rope=rope)
        res.append((cache.k_pages[0].float().cpu(), cache.k_scale[0].cpu()))
    (a, sa), (b, sb) = res
    assert torch.equal(sa, sb)
    assert a[0, 0, 3, 40] == 448 and bool(torch.isnan(a[0, 0, 4, 50])) and a[1, 0, 1, 63] == -448
    for p, t, d in ((0, 3, 40), (0, 4, 50), (1, 1, 63)):
        a[p, 0, t, d] = b[p, 0, t, d]
    assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_decoding_loop(cuda_lib):
    """Prompt, drafts and single tokens through reserve, append and attend, captured as a graph from the
    second kind of step on; the attention against its definition over the rotated rows, to what e4m3
    and the type leave of them."""
    S, Hq, Hkv, D, page = 3, 4, 2, 64, 16
    rope, rng, g = Rope(D, base=200.0), random.Random(4), torch.Generator().manual_seed(8)
    cache = PagedKVCache(1, S, Hkv, D, n_pages=40, page_size=page, max_pages=12)
    keys, values = [[] for _ in range(S)], [[] for _ in range(S)]
    bufs = None
    for step in range(25):
        T = 40 if step == 0 else 3
        n_new = [rng.randint(1 if step == 0 else 0, T) for _ in range(S)]
        q, k, v = (torch.randn(S, h, T, D, generator=g).to(F16) for h in (Hq, Hkv, Hkv))
        n = torch.tensor(n_new, dtype=torch.int32)
        if step == 0:
            x = [t.cuda() for t in (q, k, v, n)]
        elif bufs is None:
            bufs = x = [t.cuda() for t in (q, k, v, n)]
        else:
            for b, t in zip(bufs, (q, k, v, n)):
                b.copy_(t)
            x = bufs

        def one():
            cache.reserve(x[3])
            rq = cache.append(0, x[1], x[2], x[3], rope=rope, q=x[0])
            return rq, cache.attend(0, rq, n_new=x[3])[0]
        if step == 0:
            rq, out = one()
        elif step == 1:
            held = [t.clone() for t in (cache.table, cache.lens, cache.refs, cache.info, cache.granted)]
            pools = [t.clone() for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                one()
            torch.cuda.current_stream().wait_stream(side)
            for a, b in zip((cache.table, cache.lens, cache.refs, cache.info, cache.granted), held):
                a.copy_(b)
            for a, b in zip((cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale), pools):
                a.copy_(b)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                rq, out = one()
            graph.replay()
        else:
            graph.replay()
        assert _lib.sync_status() == _lib.ATTN_OK
        lens = cache.lens.tolist()
        got = out.double().cpu()
        for c in range(S):
            at = torch.arange(lens[c] - n_new[c], lens[c])
            if n_new[c]:
                keys[c].append(rope_ref.rotate(k[c:c + 1, :, :n_new[c]], rope.inv_freq, at)[0])
                values[c].append(v[c, :, :n_new[c]].double())
            if not n_new[c]:
                assert bool((got[c] == 0).all())
                continue
            kk, vv = torch.cat(keys[c], 1), torch.cat(values[c], 1)
            qq = rope_ref.rotate(q[c:c + 1, :, :n_new[c]], rope.inv_freq, at)[0]
            s = (qq.view(Hkv, Hq // Hkv * n_new[c], D) @ kk.transpose(1, 2)) / 8.0
            hide = torch.arange(lens[c])[None] > at[:, None]
            s = s.masked_fill(hide.repeat(Hq // Hkv, 1), float("-inf"))
            ref = (torch.softmax(s, -1) @ vv).view(Hq, n_new[c], D)
            # e4m3: each key and value off by up to 2^-4 of itself (rms 2^-5.2): 4% on either side
            rel = (got[c, :, : n_new[c]] - ref).norm() / ref.norm()
            assert float(rel) < 0.12, (step, c, float(rel))


@pytest.mark.gpu
def test_queries_that_autograd_follows_are_refused(cuda_lib):
    """Turned queries have no gradient: a q with one is refused, and nothing is appended; under no_grad it is
    taken, and keys and values may require gradients."""
    from torch.autograd import forward_ad
    rope, q, k = Rope(64), _rows((1, 4, 3, 64), F16, 1), _rows((1, 2, 3, 64), F16, 2)
    cache = PagedKVCache(1, 1, 2, 64, n_pages=1, page_size=16)
    cache.reserve(3)
    leaf = q.clone().requires_grad_(True)
    for out in (None, torch.empty_like(q)):
        args = (k, k, cache.k_pages[0], cache.v_pages[0], cache.k_scale[0], cache.v_scale[0], cache.table, cache.lens)
        with pytest.raises(ValueError, match="autograd"):
            _lib.kv8_append(*args, rope=rope, q=leaf, q_out=out)
        with forward_ad.dual_level(), torch.no_grad(), pytest.raises(ValueError, match="autograd"):
            _lib.kv8_append(*args, rope=rope, q=forward_ad.make_dual(q, q), q_out=out)
    with pytest.raises(ValueError, match="autograd"):
        cache.append(0, k, k, rope=rope, q=leaf)
    assert not cache.k_pages.view(torch.uint8).any() and not cache.v_pages.view(torch.uint8).any()
    with torch.no_grad():
        got = cache.append(0, k, k, rope=rope, q=leaf)
    assert torch.equal(got, rope(q)) and cache.k_pages.view(torch.uint8).any()
    other = k.clone().requires_grad_(True)
    assert torch.equal(cache.append(0, other, other, rope=rope, q=q), got)
    assert _lib.sync_status() == _lib.ATTN_OK


# What the sines and the arithmetic leave of a turned key: a sine made for its position is off by 2^-23.3 (its angle) and
# 2^-23 (rope_ref.ARITH); a prompt's are one turn of such a pair by another, so twice that and the products' 2^-23, 2^-20.5
# in all; amplitude, products and sum of the key 4 units of 2^-24 more: 2^-20 of A (|a| + |b|).
EXACT = 2.0 ** -20


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot,inter,T,page,dtype", [
    (128, 128, False, 600, 64, BF16), (128, 128, False, 600, 128, F16), (64, 64, False, 900, 16, F16), (64, 64, True, 500, 32, BF16),
    (128, 32, True, 300, 64, F16), (128, 126, False, 400, 128, F16), (64, 20, False, 500, 16, BF16), (128, 40, False, 200, 16, F16),
    (128, 128, False, 8, 64, F16), (64, 64, True, 16, 16, F16)])
def test_codes_of_turned_keys(cuda_lib, D, rot, inter, T, page, dtype):
    """Every key's code lies between those of the exact key less and plus what the arithmetic may add: prompts from far
    positions on and steps, each page's tokens."""
    rope, H, old = Rope(D, rot, interleaved=inter, base=300.0, amplitude=1.25), 3, [70003, 0]
    k = _rows((2, H, T, D), dtype, T + D)
    pools, table = _cache(old, [T, T], H, D, page, seed=T)
    lens = [n + T for n in old]
    dev = [t.cuda() for t in pools]
    _lib.kv8_append(k, k, dev[0], dev[2], dev[1], dev[3], table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), rope=rope)
    assert _lib.sync_status() == _lib.ATTN_OK
    positions = torch.tensor(old)[:, None] + torch.arange(T)[None]
    x = rope_ref.rotate(k.cpu(), rope.inv_freq, positions, rope.amplitude, inter)
    off = rope.amplitude * EXACT * rope_ref.partner(k.cpu(), rot, inter)
    pid = table.long().gather(1, positions // page)                      # [2, T]
    s = dev[1].cpu().double()[pid].transpose(1, 2)[..., None]           # [2, H, T, 1]
    got = dev[0].cpu().double()[pid[:, :, None], torch.arange(H)[None, None], (positions % page)[:, :, None]].transpose(1, 2)
    code = lambda y: y.clamp(-448, 448).float().to(F8).double()
    # (fp64 to fp32 rounds once more, by 2^-24 of the value: the bounds are moved by as much; what stays is exact,
    # 16 bits that often lie between two codes)
    lo, hi = ((x + sign * torch.where(off > 0, off + x.abs() * 2.0 ** -23, 0.0)) / s for sign in (-1, 1))
    assert bool((code(lo) <= got).all()) and bool((got <= code(hi)).all())
    assert float((code(lo) != code(hi)).double().mean()) < 1e-3   # (the bounds are sharp)
