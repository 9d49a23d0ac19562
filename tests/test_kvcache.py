"""The paged 8-bit KV cache: append, attention, page bookkeeping and copies,
against the CPU definition (tests/kv8_ref.py), their refusals, and a decoding
loop that uses them together.

Appended bytes, scales and all bookkeeping are compared for equality.  The
attention's tolerances are those of the other forwards (tests/helpers.py): the
scores' keys are exact, the softmax terms fp16 (2^-11 of themselves) and the sums
fp32, as there; its reference reads the same quantised values."""
import numpy as np
import pytest
import torch

from tests import helpers, kv8_ref
from tiled_memory_efficient_gb300 import _lib
from tiled_memory_efficient_gb300.kvcache import PagedKVCache

F16, BF16, F8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
P = 256  # a fake, 16-byte-aligned "device" address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


# ------------------------------------------------------------------ CPU: refusals

ATTN = dict(q=P, kp=P, vp=P, ks=P, vs=P, table=P, lens=P, out=P, lse=P, ws=P, n=1 << 40, B=2, Hq=4,
            Hkv=2, Nq=1, D=64, page=64, n_pages=10, max_pages=5, scale=0.1, window=0, sinks=0, dtype=0)


@pytest.mark.parametrize("change,code", [
    ({"q": 0}, 1), ({"vs": 0}, 1), ({"ws": 0}, 1), ({"B": 0}, 1), ({"Hq": 3}, 1), ({"Nq": 0}, 1),
    ({"D": 96}, 2), ({"page": 48}, 2), ({"page": 0}, 1), ({"n_pages": 0}, 1), ({"max_pages": 0}, 1),
    ({"scale": 0.0}, 1), ({"scale": float("inf")}, 1), ({"window": -1}, 1), ({"sinks": -1}, 1),
    ({"dtype": 3}, 1), ({"kp": P + 8}, 3), ({"lens": P + 2}, 3), ({"n": 16}, 6), ({"B": 1025}, 2),
    ({"max_pages": 1 << 25}, 2), ({"n_pages": 1 << 30}, 2),
])
def test_attention_refusals(lib, change, code):
    assert lib.kv8_attn(*{**ATTN, **change}.values(), None) == code


APPEND = dict(k=P, v=P, kp=P, vp=P, ks=P, vs=P, table=P, lens=P, n_new=0, B=2, Hkv=2, T=3, D=64, page=16,
              n_pages=10, max_pages=5, sb=384, sh=192, st=64, dtype=1)


@pytest.mark.parametrize("change,code", [
    ({"k": 0}, 1), ({"table": 0}, 1), ({"T": 0}, 1), ({"D": 32}, 2), ({"page": 24}, 2), ({"dtype": 2}, 1),
    ({"st": 60}, 3), ({"sb": -8}, 1), ({"v": P + 8}, 3), ({"n_new": P + 1}, 3), ({"ks": P + 2}, 3),
])
def test_append_refusals(lib, change, code):
    assert lib.kv8_append(*{**APPEND, **change}.values(), None) == code


def test_page_call_refusals(lib):
    ws = lib.kvp_workspace_size(4, 5, 20)
    assert ws > 0 and ws % 256 == 0
    assert lib.kvp_workspace_size(0, 5, 20) == 0
    res = lambda **c: lib.kvp_reserve(*{**dict(t=P, l=P, r=P, n=P, n_seqs=4, mp=5, np=20, page=64, w=0, s=0,
                                               info=P, ws=P, b=ws), **c}.values(), None)
    assert [res(t=0), res(w=-1), res(page=20), res(ws=0), res(ws=P + 8), res(b=ws - 1), res(r=P + 2),
            res(n_seqs=0)] == [1, 1, 2, 1, 3, 6, 3, 1]
    rea = lambda **c: lib.kvp_reassign(*{**dict(t=P, l=P, r=P, p=P, n_seqs=4, mp=5, np=20, page=64, cs=P, cd=P,
                                                info=P, ws=P, b=ws), **c}.values(), None)
    assert [rea(p=0), rea(page=0), rea(b=0), rea(cd=P + 1)] == [1, 1, 6, 3]
    com = lambda **c: lib.kvp_compact(*{**dict(t=P, r=P, to=P, ro=P, n_seqs=4, mp=5, np=20, s=P, d=P, info=P,
                                               ws=P, b=ws), **c}.values(), None)
    assert [com(to=0), com(np=-1), com(b=8)] == [1, 1, 6]
    cop = lambda **c: lib.kv8_copy_pages(*{**dict(k=P, v=P, ks=P, vs=P, s=P, d=P, c=P, m=3, L=2, H=2, page=64, D=64,
                                                  np=20), **c}.values(), None)
    assert [cop(s=0), cop(m=-1), cop(L=0), cop(page=8), cop(k=P + 4), cop(m=0)] == [1, 1, 1, 2, 3, 0]


def test_python_refusals():
    z = torch.zeros(3, 2, 16, 64, dtype=F8)
    s = torch.zeros(3, 2)
    with pytest.raises(ValueError):      # CPU tensors: no CPU fallback
        _lib.kv8_attn(torch.zeros(1, 2, 1, 64, dtype=F16), z, z, s, s, torch.zeros(1, 2, dtype=torch.int32),
                      torch.zeros(1, dtype=torch.int32))
    for bad in ({"head_dim": 96}, {"page_size": 20}):
        with pytest.raises(NotImplementedError):
            PagedKVCache(**{**dict(n_layers=1, n_seqs=1, n_kv_heads=1, head_dim=64, n_pages=4, device="cpu"), **bad})
    with pytest.raises(ValueError):
        PagedKVCache(1, 1, 1, 64, 0, device="cpu")


def test_reference_scale_is_the_smallest_that_fits():
    for amax, e in ((448.0, 0), (448.5, 1), (224.0, -1), (1.75, -8), (1.76, -7), (0.0, -126), (1e-45, -126)):
        assert kv8_ref.page_exp(amax) == e


# ------------------------------------------------------------------ GPU: attention

CASES = [
    # Hq, Hkv, Nq, D, page, lens, window, sinks, dtype
    (14, 2, 1, 64, 16, [1, 100, 777], 0, 0, F16),
    (8, 8, 1, 128, 64, [0, 515], 0, 0, BF16),                  # one row a head; an empty sequence
    (32, 4, 4, 128, 32, [3, 1000, 4], 0, 0, F16),              # 32 rows; fewer positions than queries
    (16, 2, 2, 64, 128, [2049, 1], 100, 5, BF16),              # 16 rows, window and sinks
    (40, 1, 2, 64, 64, [300], 0, 0, F16),                      # 80 rows: three row blocks
    (7, 1, 3, 64, 16, [333, 64, 20], 37, 20, F16),             # small pages, their ends inside a tile
    (5, 1, 3, 128, 16, [95, 33], 16, 0, BF16),
    (2, 2, 1, 128, 64, [9000], 0, 0, F16),                     # one sequence over many CTAs
    (4, 2, 1, 128, 128, [5000, 40], 1, 0, BF16),               # a query sees itself alone
    (4, 1, 1, 64, 64, [4100], 1000, 300, F16),                 # sinks over many tiles
    (14, 2, 1, 64, 64, [64, 32, 65, 31, 96, 0, 0, 128, 1, 5, 200], 64, 4, BF16),
]


def _cache(lens, Hkv, D, page, window, sinks, Nq, seed):
    """Pools, scales, table and lens on the CPU; what no query may read holds NaN."""
    g = torch.Generator().manual_seed(seed)
    mp = max(1, -(-max(lens) // page)) + 1
    B = len(lens)
    n_pages = B * mp + 2
    pools = []
    for amp in (1.0, 1.0):
        x = amp * torch.randn(n_pages, Hkv, page, D, generator=g)
        # pages of different sizes have different scales
        x = x * torch.exp2(torch.randint(-3, 3, (n_pages, Hkv, 1, 1), generator=g).float()) / 4
        s = torch.tensor([[2.0 ** kv8_ref.page_exp(float(x[i, h].abs().max())) for h in range(Hkv)]
                          for i in range(n_pages)])
        pools += [(x / s[:, :, None, None]).to(F8), s]
    kp, ks, vp, vs = pools
    perm = torch.randperm(n_pages, generator=g)
    table = torch.full((B, mp), 10 ** 6, dtype=torch.int32)   # never needed: never read
    used = set()
    raw = [kp.view(torch.uint8), vp.view(torch.uint8)]
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            lo = n - Nq - window + 1
            if window and j * page >= sinks and (j + 1) * page <= lo:
                table[b, j] = -1                               # given back
                continue
            pid = int(perm[b * mp + j])
            table[b, j] = pid
            used.add(pid)
            for r in raw:
                r[pid, :, max(0, min(page, n - j * page)):] = 0x7F   # rows behind the last token
    for i in range(n_pages):
        if i not in used:
            for r, s in zip(raw, (ks, vs)):
                r[i] = 0x7F
                s[i] = float("nan")
    return kp, vp, ks, vs, table, torch.tensor(lens, dtype=torch.int32)


def _check(q, cache, window, sinks, out, lse, what, scale=None):
    ro, rl = kv8_ref.attention(q, *cache, window=window, sinks=sinks, scale=scale)
    out, lse = out.double().cpu(), lse.double().cpu()
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    assert bool((out[empty] == 0).all())
    helpers.assert_fwd_close(out[~empty].numpy(), lse[~empty].numpy(), ro[~empty].numpy(), rl[~empty].numpy(),
                             q.dtype, what)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention_matches_the_definition(cuda_lib, case):
    Hq, Hkv, Nq, D, page, lens, window, sinks, dtype = case
    cache = _cache(lens, Hkv, D, page, window, sinks, Nq, seed=sum(lens))
    q = torch.randn(len(lens), Hq, Nq, D, generator=torch.Generator().manual_seed(1)).to(dtype)
    dev = [t.cuda() for t in cache]
    out, lse = _lib.kv8_attn(q.cuda(), *dev, window=window, sinks=sinks)
    assert _lib.sync_status() == _lib.ATTN_OK
    _check(q, cache, window, sinks, out, lse, f"kv8 {case}")
    again = _lib.kv8_attn(q.cuda(), *dev, window=window, sinks=sinks)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
def test_attention_of_many_short_sequences(cuda_lib):
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    cache = _cache(lens, 2, 64, 32, 0, 0, 1, seed=8)
    q = torch.randn(300, 4, 1, 64, generator=g).to(F16)
    out, lse = _lib.kv8_attn(q.cuda(), *(t.cuda() for t in cache))
    assert _lib.sync_status() == _lib.ATTN_OK
    _check(q, cache, 0, 0, out, lse, "kv8 300 sequences")


@pytest.mark.gpu
def test_pages_of_very_different_scales(cuda_lib):
    """Values of 2^-60, 1 and 2^60 in different pages, a page of zeros, large and
    tiny queries: every row is compared relative to its own size."""
    lens, page, D = [256], 64, 64
    cache = _cache(lens, 1, D, page, 0, 0, 1, seed=3)
    kp, vp, ks, vs, table, ln = cache
    for j, f in enumerate((2.0 ** -60, 1.0, 2.0 ** 60)):
        vs[table[0, j]] *= f
    vp.view(torch.uint8)[table[0, 3]] = 0
    vs[table[0, 3]] = 2.0 ** -126
    q = torch.randn(1, 4, 1, D, generator=torch.Generator().manual_seed(2))
    q[0, 1] *= 2.0 ** -70       # every key alike
    q[0, 2] *= 8.0              # one key dominates
    k3 = kv8_ref.dense(kp, ks, table[0], 256)[0, 200]
    q[0, 3] = 60.0 * k3 / k3.norm() ** 2 * D ** 0.5    # the key in the page of zeros
    q = q.to(BF16)
    out, lse = _lib.kv8_attn(q.cuda(), *(t.cuda() for t in cache))
    assert _lib.sync_status() == _lib.ATTN_OK
    ro, rl = kv8_ref.attention(q, *cache)
    out, lse = out.double().cpu(), lse.double().cpu()
    assert float((lse - rl).abs().max()) <= helpers.TOL_LSE
    # terms rounded by 2^-11, the output by 2^-8, of the largest value a row could have:
    # sum of weight * |value| is at most the weighted sum below
    for h in range(4):
        k, v = kv8_ref.dense(kp, ks, table[0], 256)[0], kv8_ref.dense(vp, vs, table[0], 256)[0]
        w = torch.softmax(k @ q[0, h, 0].double() * D ** -0.5, 0)
        size = (w[:, None] * v.abs()).sum(0)
        # fp32 scores: |s| up to 60 with relative 2^-20 leaves the weights 2^-13 off, at most
        bound = size * (2.0 ** -11 + 2.0 ** -8 + 2 * 2.0 ** -13) + float(size.max()) * 2.0 ** -24
        assert bool(((out[0, h, 0] - ro[0, h, 0]).abs() <= bound).all()), h


@pytest.mark.gpu
def test_hidden_values_do_not_matter(cuda_lib):
    """Keys and values outside the window or in rows behind the last token may be NaN."""
    lens = [500]
    cache = _cache(lens, 2, 128, 64, 0, 0, 1, seed=4)
    kp, vp, ks, vs, table, ln = cache
    q = torch.randn(1, 4, 1, 128, generator=torch.Generator().manual_seed(2)).to(F16).cuda()
    a = _lib.kv8_attn(q, *(t.cuda() for t in cache), window=100, sinks=3)
    for pos in range(3, 400):       # the query at 499 sees 400 on
        for pool in (kp, vp):
            pool.view(torch.uint8)[table[0, pos // 64], :, pos % 64] = 0x7F
    b = _lib.kv8_attn(q, *(t.cuda() for t in cache), window=100, sinks=3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and bool(torch.isfinite(a[0]).all())


@pytest.mark.gpu
def test_bad_pages_and_lengths_are_skipped_and_recorded(cuda_lib):
    """A page id outside the pool hides its tokens; a length past the table is cut."""
    cache = _cache([300, 200], 2, 64, 64, 0, 0, 1, seed=5)
    kp, vp, ks, vs, table, lens = cache
    q = torch.randn(2, 4, 1, 64, generator=torch.Generator().manual_seed(2)).to(F16)
    for bad in (-1, 10 ** 9, kp.shape[0]):
        t2 = table.clone()
        t2[0, 1] = bad
        out, lse = _lib.kv8_attn(q.cuda(), *(t.cuda() for t in (kp, vp, ks, vs, t2, lens)))
        assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
        assert _lib.sync_status() == _lib.ATTN_OK      # cleared
        # the sequence without positions 64 .. 127: drop them and attend over the rest
        row = torch.cat([table[0, :1], table[0, 2:], table[0, :1]])
        ref = kv8_ref.attention(q, kp, vp, ks, vs, torch.stack([row, table[1]]),
                                torch.tensor([236, 200]))
        helpers.assert_fwd_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref[0].numpy(),
                                 ref[1].numpy(), F16, f"bad page {bad}")
    cut = torch.tensor([table.shape[1] * 64 + 5, -3], dtype=torch.int32)
    t2 = table.clone()
    t2[0] = t2[0].clamp(max=kp.shape[0] - 1)
    out, lse = _lib.kv8_attn(q.cuda(), *(t.cuda() for t in (kp, vp, ks, vs, t2, cut)))
    assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
    assert bool((out[1] == 0).all()) and bool((lse[1] == float("-inf")).all())


# ------------------------------------------------------------------ GPU: append

@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,D,page,T,old,n_new,dtype", [
    (2, 64, 16, 1, [0, 5, 16, 31], None, F16),
    (1, 128, 64, 200, [0, 63, 10], [200, 0, 117], BF16),
    (3, 64, 128, 130, [127, 1], [130, 2], F16),
    (2, 128, 32, 33, [0, 31, 95], [33, 1, 32], BF16),
    (1, 64, 64, 70, [3], [64], BF16),
    (2, 128, 128, 129, [200], None, F16),
    (1, 128, 16, 40, [9, 16], [40, 17], F16),
    (1, 64, 32, 65, [0], None, BF16),
], ids=str)
def test_append_matches_the_definition(cuda_lib, Hkv, D, page, T, old, n_new, dtype):
    B = len(old)
    counts = torch.tensor([T] * B if n_new is None else n_new, dtype=torch.int32)
    lens = torch.tensor(old, dtype=torch.int32) + counts
    mp = int(-(-lens.max() // page))
    g = torch.Generator().manual_seed(T + page)
    n_pages = B * mp + 1
    table = torch.randperm(n_pages, generator=g)[:B * mp].to(torch.int32).reshape(B, mp)
    pools = [torch.randint(0, 0x7F, (n_pages, Hkv, page, D), generator=g, dtype=torch.uint8).view(F8)
             for _ in range(2)]
    scales = [torch.exp2(torch.randint(-12, 1, (n_pages, Hkv), generator=g).float()) for _ in range(2)]
    new = []
    for _ in range(2):
        x = torch.randn(B, Hkv, T, D, generator=g) * torch.exp2(
            torch.randint(-6, 7, (B, Hkv, T, 1), generator=g).float())
        x[0, 0, 0, :5] = torch.tensor([float("inf"), -float("inf"), 0.0, 1e-7, 448.0])
        x[-1, 0, -1, 3] = float("nan")
        new.append(x.to(dtype))
    dev = [t.cuda() for t in (*pools, *scales, table, lens, counts)]
    # [B, T, H, D] memory: strided views, as a projection leaves them
    kd, vd = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in new)
    for _ in range(2):      # the second time changes nothing
        _lib.kv8_append(kd, vd, *dev[:6], n_new=None if n_new is None else dev[6])
        assert _lib.sync_status() == _lib.ATTN_OK
        for i in range(2):
            rp, rs = kv8_ref.append(new[i], pools[i], scales[i], table, lens, counts)
            gp, gs = dev[i].cpu(), dev[2 + i].cpu()
            assert torch.equal(gs, rs)
            a, b = gp.double(), rp.double()
            assert torch.equal(torch.isnan(a), torch.isnan(b))
            assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
            same = torch.ones(n_pages, page, dtype=torch.bool)   # rows the call may change
            for s in range(B):
                if counts[s]:
                    first = (int(lens[s]) - int(counts[s])) // page * page
                    for pos in range(first, int(lens[s])):
                        same[table[s, pos // page], pos % page] = False
            x, y = gp.view(torch.uint8).transpose(1, 2)[same], pools[i].view(torch.uint8).transpose(1, 2)[same]
            assert torch.equal(x, y)


@pytest.mark.gpu
def test_append_skips_what_does_not_fit(cuda_lib):
    """Bad counts, lengths and page ids write nothing and are recorded."""
    kp = torch.zeros(4, 1, 16, 64, dtype=F8, device="cuda")
    vp, ks = torch.zeros_like(kp), torch.ones(4, 1, device="cuda")
    vs = torch.ones_like(ks)
    x = torch.ones(1, 1, 20, 64, dtype=F16, device="cuda")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    table = i32([0, 1])
    for lens, n, t in ((20, 21, table), (20, -1, table), (10, 20, table), (40, 20, table), (20, 20, i32([-1, 4]))):
        _lib.kv8_append(x, x, kp, vp, ks, vs, t, i32(lens), n_new=i32(n))
        assert _lib.sync_status() == _lib.ATTN_ERR_PAGE, (lens, n)
        assert not bool(kp.view(torch.uint8).any()) and bool((ks == 1).all())
    _lib.kv8_append(x, x, kp, vp, ks, vs, table, i32(0), n_new=i32(0))
    assert _lib.sync_status() == _lib.ATTN_OK and not bool(kp.view(torch.uint8).any())


# ------------------------------------------------------------------ GPU: pages

def _state(n_seqs, max_pages, n_pages):
    i32 = dict(dtype=torch.int32, device="cuda")
    return (torch.full((n_seqs, max_pages), -1, **i32), torch.zeros(n_seqs, **i32), torch.zeros(n_pages, **i32),
            torch.zeros(4, **i32))


def _same(ref, table, lens, refs):
    assert refs.tolist() == ref.refs
    assert lens.tolist() == ref.lens
    assert table.tolist() == ref.table


@pytest.mark.gpu
@pytest.mark.parametrize("n_seqs,max_pages,n_pages,page,window,sinks", [
    (5, 9, 30, 16, 0, 0),
    (3, 40, 25, 16, 50, 20),
    (40, 6, 120, 64, 0, 0),
    (1, 1, 1, 128, 0, 0),
    (1100, 3, 2500, 32, 40, 1),     # more sequences and pages than threads of the planning CTA
    (90, 200, 30000, 16, 400, 3),   # plans that outgrow shared memory, a table of two compaction CTAs
    (700, 30, 9000, 16, 0, 0),
], ids=str)
def test_bookkeeping_matches_lists(cuda_lib, n_seqs, max_pages, n_pages, page, window, sinks):
    """A random run of reserve, reassign and compact against Python lists; calls that
    find no room change nothing."""
    import random
    rng = random.Random(n_seqs)
    table, lens, refs, info = _state(n_seqs, max_pages, n_pages)
    pairs = max(n_seqs, n_pages // 2, 1)
    src, dst = (torch.zeros(pairs, dtype=torch.int32, device="cuda") for _ in range(2))
    ref = kv8_ref.Pages(table, lens, refs, page)
    full = 0
    for step in range(25):
        do = rng.choice(["reserve", "reserve", "reassign", "compact"])
        if do == "reserve":
            most = rng.choice([1, page, 2 * page])
            n = [rng.choice([0, rng.randint(0, most)]) for _ in range(n_seqs)]
            _lib.kvp_reserve(table, lens, refs, torch.tensor(n, dtype=torch.int32, device="cuda"), page, info,
                             window=window, sinks=sinks)
            want, moves = ref.reserve(n, window, sinks), []
        elif do == "reassign":
            par = [rng.choice([c, c, c, -1, rng.randrange(n_seqs)]) for c in range(n_seqs)]
            _lib.kvp_reassign(table, lens, refs, torch.tensor(par, dtype=torch.int32, device="cuda"), page, src,
                              dst, info)
            want, moves = ref.reassign(par)
        else:
            _lib.kvp_compact(table, refs, src, dst, info)
            want, moves = ref.compact()
        assert info.tolist() == want, (step, do)
        assert list(zip(src.tolist(), dst.tolist()))[:len(moves)] == moves
        _same(ref, table, lens, refs)
        ok = _lib.sync_status()
        assert ok == (_lib.ATTN_OK if want[0] else _lib.ATTN_ERR_POOL)
        full += want[0] == 0
    assert n_pages != 30 or full < 25


@pytest.mark.gpu
def test_bad_parents_keep_their_sequences(cuda_lib):
    table, lens, refs, info = _state(3, 2, 6)
    _lib.kvp_reserve(table, lens, refs, torch.tensor([5, 20, 0], dtype=torch.int32, device="cuda"), 16, info)
    before = [t.clone() for t in (table, lens, refs)]
    src, dst = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    _lib.kvp_reassign(table, lens, refs, torch.tensor([3, -2, 2], dtype=torch.int32, device="cuda"), 16, src, dst, info)
    assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
    for a, b in zip(before, (table, lens, refs)):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("L,Hkv,page,D", [(1, 1, 16, 64), (3, 2, 64, 128), (2, 7, 32, 64)])
def test_copies_move_bytes_and_scales(cuda_lib, L, Hkv, page, D):
    g = torch.Generator().manual_seed(L)
    pools = [torch.randint(0, 256, (L, 9, Hkv, page, D), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = [torch.rand(L, 9, Hkv, generator=g).cuda() for _ in range(2)]
    src = torch.tensor([1, 8, 1, 5, 0], dtype=torch.int32, device="cuda")
    dst = torch.tensor([0, 2, 3, 9, 4], dtype=torch.int32, device="cuda")   # 9 is outside the pool
    ref = [t.clone() for t in pools + scales]
    for t in ref:
        for a, b in ((1, 0), (8, 2), (1, 3)):
            t[:, b] = t[:, a]
    _lib.kv8_copy_pages(*pools, *scales, src, dst, torch.tensor([4], dtype=torch.int32, device="cuda"))
    assert _lib.sync_status() == _lib.ATTN_ERR_PAGE
    for a, b in zip(pools + scales, ref):
        assert torch.equal(a, b)
    _lib.kv8_copy_pages(*pools, *scales, src, dst, torch.tensor([0], dtype=torch.int32, device="cuda"))
    _lib.kv8_copy_pages(*pools, *scales, src, dst, torch.tensor([9], dtype=torch.int32, device="cuda"), max_count=2)
    assert _lib.sync_status() == _lib.ATTN_OK
    for t in ref:
        t[:, 0] = t[:, 1]
        t[:, 2] = t[:, 8]
    for a, b in zip(pools + scales, ref):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        _lib.kv8_copy_pages(*pools, *scales, src, dst, torch.tensor([0], dtype=torch.int32, device="cuda"), max_count=6)


# ------------------------------------------------------------------ GPU: together

def _step(cache, layers, k, v, q, n_new):
    cache.reserve(n_new)
    res = []
    for i in range(layers):
        cache.append(i, k[i], v[i], n_new)
        res.append(cache.attend(i, q[i]))
    return res


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks,dtype", [(0, 0, F16), (40, 5, BF16)])
def test_a_decoding_run(cuda_lib, window, sinks, dtype):
    """Prompts, decoding steps, forks, a freed sequence and a compaction over two
    layers: after each step every row against the definition over what each
    sequence should hold, quantised by the definition page by page."""
    L, S, Hq, Hkv, D, page, T = 2, 4, 6, 2, 64, 16, 37
    cache = PagedKVCache(L, S, Hkv, D, n_pages=40, page_size=page, max_pages=12, window=window, sinks=sinks)
    g = torch.Generator().manual_seed(9)
    hist = [[[] for _ in range(S)] for _ in range(L)]      # (k, v) appended in one call, in order
    n_prompt = [37, 20, 0, 16]

    def rand(n, h):
        return torch.randn(S, h, n, D, generator=g).to(dtype)

    def check(res, q, Nq):
        lens = cache.lens.tolist()
        for i in range(L):
            out, lse = (t.double().cpu() for t in res[i])
            for c in range(S):
                rows = min(Nq, lens[c])
                if rows == 0:
                    assert bool((out[c] == 0).all())
                    continue
                # what the sequence holds: its calls replayed into a cache of its own
                n_pages = -(-lens[c] // page)
                kv = []
                for w in range(2):
                    pool = torch.zeros(n_pages, Hkv, page, D).to(F8)
                    sc = torch.ones(n_pages, Hkv)
                    row, at = torch.arange(n_pages)[None], 0
                    for call in hist[i][c]:
                        at += call[w].shape[1]
                        pool, sc = kv8_ref.append(call[w][None], pool, sc, row, [at], [call[w].shape[1]])
                    kv += [pool, sc]
                ref = kv8_ref.attention(q[i][c:c + 1], kv[0], kv[2], kv[1], kv[3], torch.arange(n_pages)[None],
                                        torch.tensor([lens[c]]), window, sinks)
                helpers.assert_fwd_close(out[c, :, Nq - rows:].numpy(), lse[c, :, Nq - rows:].numpy(),
                                         ref[0][0, :, Nq - rows:].numpy(), ref[1][0, :, Nq - rows:].numpy(), dtype,
                                         f"run layer {i} sequence {c}")

    def take(n_new, T):
        k, v, q = ([rand(T, h) for _ in range(L)] for h in (Hkv, Hkv, Hq))
        for i in range(L):
            for c in range(S):
                if n_new[c]:
                    hist[i][c].append((k[i][c, :, :n_new[c]], v[i][c, :, :n_new[c]]))
        dev = [[t.cuda() for t in x] for x in (k, v, q)]
        res = _step(cache, L, *dev, torch.tensor(n_new, dtype=torch.int32, device="cuda"))
        assert _lib.sync_status() == _lib.ATTN_OK
        return res, q

    def become(parents):
        cache.reassign(torch.tensor(parents, dtype=torch.int32, device="cuda"))
        assert _lib.sync_status() == _lib.ATTN_OK
        for i in range(L):
            old = [h[:] for h in hist[i]]
            hist[i] = [old[p][:] if p >= 0 else [] for p in parents]

    take(n_prompt, T)                       # the prompt's own attention is the dense kernels' work
    for _ in range(3):
        check(*take([1, 1, 0, 1], 1), 1)
    become([0, 0, 1, -1])                   # 1 becomes a child of 0, 2 takes over 1, 3 is freed
    check(*take([1, 1, 1, 0], 1), 1)
    become([1, 1, 2, 2])                    # the first child inherits: nobody keeps 0
    cache.compact()
    for _ in range(2):
        check(*take([2, 2, 2, 2], 2), 2)    # two drafted tokens each
    for _ in range(18):
        res, q = take([1, 1, 1, 1], 1)
    check(res, q, 1)
    become([-1] * S)
    assert cache.refs.tolist() == [0] * 40 and cache.lens.tolist() == [0] * S
    assert bool((cache.table == -1).all())


@pytest.mark.gpu
def test_two_caches_on_two_streams(cuda_lib):
    """Two decoding runs side by side give what each gives alone."""
    g = torch.Generator().manual_seed(6)
    data = [[[torch.randn(5, h, n, 64, generator=g).to(dt).cuda() for h in (2, 2, 8)] for n in (70, 1, 1, 2)]
            for dt in (F16, BF16)]

    def run(x, cache):
        res = []
        for k, v, q in x:
            res += _step(cache, 1, [k], [v], [q[:, :, -2:].contiguous()], k.shape[2])[0]
        cache.reassign(torch.tensor([1, 1, 0, -1, 4], dtype=torch.int32, device="cuda"))
        cache.compact()
        return res + [cache.table.clone(), cache.lens.clone(), cache.k_pages.view(torch.uint8)[:, :10].clone()]
    make = lambda: PagedKVCache(1, 5, 2, 64, n_pages=60, page_size=16, max_pages=9)
    want = [run(x, make()) for x in data]
    caches = [make() for _ in data]
    streams = [torch.cuda.Stream() for _ in data]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for s, x, c in zip(streams, data, caches):
        with torch.cuda.stream(s):
            got.append(run(x, c))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(t, u) for t, u in zip(a, b))
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_a_captured_step_follows_the_lengths(cuda_lib):
    """A decoding step captured once and replayed while the sequences grow past page
    ends gives what eager steps give."""
    def make():
        c = PagedKVCache(1, 3, 2, 64, n_pages=30, page_size=16, max_pages=8)
        c.reserve(14)
        g = torch.Generator().manual_seed(2)
        x = torch.randn(2, 3, 2, 14, 64, generator=g).to(F16).cuda()
        c.append(0, x[0], x[1])
        return c
    g = torch.Generator().manual_seed(3)
    steps = [[torch.randn(3, h, 1, 64, generator=g).to(F16).cuda() for h in (2, 2, 8)] for _ in range(5)]
    eager, held = make(), make()
    want = [_step(eager, 1, [k], [v], [q], 1)[0] for k, v, q in steps]
    k, v, q = (t.clone() for t in steps[0])
    warm = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(warm, 1, [k], [v], [q], 1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = _step(held, 1, [k], [v], [q], 1)[0]
    for i, s in enumerate(steps):
        for t, x in zip((k, v, q), s):
            t.copy_(x)
        graph.replay()
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    assert _lib.sync_status() == _lib.ATTN_OK
    assert torch.equal(held.table, eager.table) and torch.equal(held.lens, eager.lens)
