"""Pages that a window leaves behind, and forks that find no room: the bookkeeping against
Python lists (tests/kv8_ref.py, for equality) on runs that are long enough for both,
and a decoding run through them."""
import random

import pytest
import torch

from tests import helpers, kv8_ref
from tiled_memory_efficient_gb300 import _lib
from tiled_memory_efficient_gb300.kvcache import PagedKVCache

F16, BF16, F8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn

RUNS = [
    # name, n_seqs, max_pages, n_pages, page, window, sinks, prompts, steps, seed
    ("many columns at once", 4, 200, 260, 16, 50, 20, [1500, 700, 40, 0], 40, 0),
    ("no sinks", 3, 130, 160, 16, 1, 0, [2000, 33, 16], 30, 0),
    ("in small steps", 5, 60, 90, 16, 70, 5, [10, 20, 0, 5, 90], 80, 1),
    ("sinks over many pages", 4, 100, 150, 32, 100, 200, [900, 700, 100, 300], 40, 0),
    ("a pool that is often full", 6, 12, 9, 16, 40, 5, [60, 10, 0, 0, 0, 30], 120, 12),
    ("full, no window", 6, 6, 7, 16, 0, 0, [40, 10, 0, 0, 0, 20], 80, 0),
    ("plans that outgrow shared memory", 40, 120, 30000, 16, 90, 3, [1000 + 20 * c for c in range(40)], 20, 0),
    ("more sequences than warps", 70, 40, 1500, 16, 33, 17, [600 - 8 * c for c in range(70)], 25, 0),
]


def _script(run):
    """The calls of a run: ("reserve", counts), ("reassign", parents) or ("compact",)."""
    _, n_seqs, _, _, page, _, _, prompts, steps, seed = run
    rng = random.Random(seed)
    yield "reserve", list(prompts)
    yield "reassign", [max(c - 1, 0) for c in range(n_seqs)]     # pages shared before any is left behind
    yield "reserve", [1] * n_seqs
    for _ in range(steps):
        do = rng.choice(["step"] * 8 + ["jump", "fork", "star", "compact"])
        if do == "step":
            yield "reserve", [rng.choice([0, 1, 1, 2]) for _ in range(n_seqs)]
        elif do == "jump":
            yield "reserve", [rng.choice([0, 1, rng.randint(0, 3 * page)]) for _ in range(n_seqs)]
        elif do == "fork":
            yield "reassign", [rng.choice([c, c, c, c, rng.randrange(n_seqs), rng.choice([c, -1])])
                               for c in range(n_seqs)]
        elif do == "star":      # most become children of one
            one = rng.randrange(n_seqs)
            yield "reassign", [rng.choice([one, one, c]) for c in range(n_seqs)]
        else:
            yield "compact", None


def _apply(ref, do, arg, window, sinks):
    if do == "reserve":
        return ref.reserve(arg, window, sinks), []
    return ref.reassign(arg) if do == "reassign" else ref.compact()


def _model(run):
    _, n_seqs, max_pages, n_pages, page = run[:5]
    return kv8_ref.Pages(torch.full((n_seqs, max_pages), -1), torch.zeros(n_seqs, dtype=torch.int32),
                         torch.zeros(n_pages, dtype=torch.int32), page)


@pytest.mark.parametrize("run", RUNS, ids=lambda r: r[0])
def test_the_runs_reach_what_they_are_for(run):
    """On the lists alone: pages are given back, by more than a warp's 32 columns at once and
    from shared rows, and calls of both kinds find no room."""
    ref, window, sinks, page = _model(run), run[5], run[6], run[4]
    back = most = shared = 0
    refused = {"reserve": 0, "reassign": 0, "compact": 0}
    for do, arg in _script(run):
        held = [r[:] for r in ref.table]
        refs = ref.refs[:]
        info = _apply(ref, do, arg, window, sinks)[0]
        refused[do] += info[0] == 0
        if do == "reserve" and info[0]:
            back += info[2]
            for a, b in zip(held, ref.table):
                gone = [x for x, y in zip(a, b) if x >= 0 and y < 0]
                most, shared = max(most, len(gone)), shared + sum(refs[x] > 1 for x in gone)
    assert max(ref.lens) > 0
    if window:
        assert back > 0 and shared > 0, (back, shared)
    if run[0] in ("many columns at once", "no sinks", "plans that outgrow shared memory"):
        assert most > 32
    if "full" in run[0]:
        assert refused["reserve"] > 0 and refused["reassign"] > 0, refused


@pytest.mark.gpu
@pytest.mark.parametrize("run", RUNS, ids=lambda r: r[0])
def test_bookkeeping_matches_lists(cuda_lib, run):
    _, n_seqs, max_pages, n_pages, page, window, sinks = run[:7]
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.full((n_seqs, max_pages), -1, **i32), torch.zeros(n_seqs, **i32)
    refs, info, granted = torch.zeros(n_pages, **i32), torch.zeros(4, **i32), torch.ones(1, **i32)
    src, dst = (torch.zeros(max(n_seqs, n_pages // 2), **i32) for _ in range(2))
    ref = _model(run)
    for at, (do, arg) in enumerate(_script(run)):
        if do == "reserve":
            _lib.kvp_reserve(table, lens, refs, torch.tensor(arg, **i32), page, info, window=window, sinks=sinks,
                             granted=granted)
        elif do == "reassign":
            _lib.kvp_reassign(table, lens, refs, torch.tensor(arg, **i32), page, src, dst, info)
        else:
            _lib.kvp_compact(table, refs, src, dst, info)
        want, moves = _apply(ref, do, arg, window, sinks)
        assert info.tolist() == want, (at, do)
        if do == "reserve":
            assert granted.item() == want[0]
        assert list(zip(src.tolist(), dst.tolist()))[:len(moves)] == moves
        assert refs.tolist() == ref.refs and lens.tolist() == ref.lens and table.tolist() == ref.table, (at, do)
        assert _lib.sync_status() == (_lib.ATTN_OK if want[0] else _lib.ATTN_ERR_POOL)


@pytest.mark.gpu
@pytest.mark.parametrize("page,window,sinks,dtype", [(16, 40, 5, F16), (32, 33, 40, BF16)])
def test_a_windowed_run_with_forks(cuda_lib, page, window, sinks, dtype):
    """Two layers, decoding past the window while sequences fork, end and share pages that
    some of them give back: every few steps each row against the definition."""
    L, S, Hq, Hkv, D = 2, 4, 6, 2, 64
    cache = PagedKVCache(L, S, Hkv, D, n_pages=36, page_size=page, max_pages=16, window=window, sinks=sinks)
    g, rng = torch.Generator().manual_seed(21), random.Random(window)
    hist = [[[] for _ in range(S)] for _ in range(L)]
    back = 0

    def step(n_new, T, look):
        k, v, q = ([torch.randn(S, h, T, D, generator=g).to(dtype) for _ in range(L)] for h in (Hkv, Hkv, Hq))
        n = torch.tensor(n_new, dtype=torch.int32, device="cuda")
        cache.reserve(n)
        taken = cache.info.tolist()
        assert taken[0] == 1
        lens = cache.lens.tolist()
        for i in range(L):
            cache.append(i, k[i].cuda(), v[i].cuda(), n)
            out, lse = (t.double().cpu() for t in cache.attend(i, q[i].cuda(), n_new=n))
            for c in range(S):
                if not n_new[c]:
                    continue
                hist[i][c].append((k[i][c, :, :n_new[c]], v[i][c, :, :n_new[c]]))
                if not look:
                    continue
                pages = -(-lens[c] // page)
                kv = []
                for w in range(2):
                    pool, sc, at = torch.zeros(pages, Hkv, page, D).to(F8), torch.ones(pages, Hkv), 0
                    for call in hist[i][c]:
                        at += call[w].shape[1]
                        pool, sc = kv8_ref.append(call[w][None], pool, sc, torch.arange(pages)[None], [at],
                                                  [call[w].shape[1]])
                    kv += [pool, sc]
                ro, rl = kv8_ref.attention(q[i][c:c + 1, :, :n_new[c]], kv[0], kv[2], kv[1], kv[3],
                                           torch.arange(pages)[None], torch.tensor([lens[c]]), window, sinks)
                helpers.assert_fwd_close(out[c, :, :n_new[c]].numpy(), lse[c, :, :n_new[c]].numpy(), ro[0].numpy(),
                                         rl[0].numpy(), dtype, f"windowed run layer {i} sequence {c}")
        assert _lib.sync_status() == _lib.ATTN_OK
        return taken[2]

    def become(parents):
        cache.reassign(torch.tensor(parents, dtype=torch.int32, device="cuda"))
        assert _lib.sync_status() == _lib.ATTN_OK
        for i in range(L):
            old = [h[:] for h in hist[i]]
            hist[i] = [old[p][:] if p >= 0 else [] for p in parents]
    step([70, 20, 0, 33], 70, False)
    for at in range(100):
        back += step([rng.choice([0, 1, 1, 2]) for _ in range(S)], 2, at % 9 == 0)
        if at % 20 == 7:
            become([0, 0, 2, 3])
        if at % 20 == 13:
            become([1, 1, 1, 0])
        if at % 25 == 24:
            become([rng.randrange(S), 1, -1, 3])
            cache.compact()
    assert back > 1
    become([-1] * S)
    assert cache.refs.tolist() == [0] * 36 and bool((cache.table == -1).all())
