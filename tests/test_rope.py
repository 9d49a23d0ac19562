"""Rotary positions (rope.Rope, _lib.rope) against their definition in 64 bits.

Tolerances count the final rounding and the fp32 arithmetic (tests/rope_ref.py)."""
import math
from fractions import Fraction

import pytest
import torch

from tests import rope_ref
from tiled_memory_efficient_gb300 import _lib, sdpa
from tiled_memory_efficient_gb300.kvcache import PagedKVCache
from tiled_memory_efficient_gb300.rope import Rope, frequencies

F16, BF16 = torch.float16, torch.bfloat16
P = 256  # a fake, 16-byte-aligned "device" address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


# ------------------------------------------------------------------ on the CPU

def test_frequencies():
    f, a = frequencies(64)
    assert a == 1.0 and f[0] == 1.0 and math.isclose(f[31], 10000.0 ** (-62 / 64), rel_tol=1e-14)
    lin, _ = frequencies(64, scaling={"kind": "linear", "factor": 4.0})
    assert all(math.isclose(4 * x, y, rel_tol=1e-15) for x, y in zip(lin, f))
    ntk, _ = frequencies(64, scaling={"kind": "ntk", "factor": 8.0})
    assert ntk[0] == 1.0 and math.isclose(ntk[31] * 8, f[31], rel_tol=1e-12)
    assert frequencies(2, scaling={"kind": "ntk", "factor": 8.0})[0] == [1.0]
    s = {"kind": "yarn", "factor": 16.0, "original_len": 4096}
    y, a = frequencies(128, scaling=s)
    g, _ = frequencies(128)
    assert math.isclose(a, 0.1 * math.log(16.0) + 1.0)
    for i in range(64):
        turns = 4096 * g[i] / (2 * math.pi)
        if turns > 40:
            assert y[i] == g[i]
        if turns < 0.8:
            assert math.isclose(y[i], g[i] / 16, rel_tol=1e-14)
        assert g[i] / 16 * (1 - 1e-12) <= y[i] <= g[i]
    s = {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original_len": 8192}
    y, a = frequencies(128, 500000.0, s)
    g, _ = frequencies(128, 500000.0)
    assert a == 1.0
    for i in range(64):
        turns = 8192 * g[i] / (2 * math.pi)
        want = g[i] if turns >= 4 else g[i] / 8 if turns <= 1 else g[i] / 8 + (g[i] - g[i] / 8) * (turns - 1) / 3
        assert math.isclose(y[i], want, rel_tol=1e-12)


def test_turns_are_exact():
    """The 64-bit fractions of a turn give far positions' angles to 2^-32 of a turn."""
    rope = Rope(128, base=500000.0)
    words = rope.turns("cpu")
    assert words.dtype is torch.int64 and words.shape == (64,)
    per = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)
    for w, f in zip(words.tolist(), rope.inv_freq):
        for pos in (1, 4097, -3, 1 << 20, (1 << 31) - 1, -(1 << 31)):
            got = (pos * (w % 2 ** 64)) % 2 ** 64
            want = (Fraction(f) * per * pos) % 1
            d = abs(Fraction(got, 2 ** 64) - want)
            assert min(d, 1 - d) < Fraction(1, 2 ** 32)


@pytest.mark.parametrize("kw", [
    dict(head_dim=64, rotary_dim=63), dict(head_dim=64, rotary_dim=66), dict(head_dim=64, rotary_dim=0),
    dict(head_dim=64, base=0.5), dict(head_dim=64, base=float("inf")), dict(head_dim=64, amplitude=0.0),
    dict(head_dim=64, amplitude=float("nan")), dict(head_dim=64, inv_freq=[1.0]),
    dict(head_dim=64, rotary_dim=2, inv_freq=[float("nan")]),
    dict(head_dim=64, scaling={"kind": "cubic"}), dict(head_dim=64, scaling={"kind": "linear"}),
    dict(head_dim=64, scaling={"kind": "linear", "factor": -1.0}),
    dict(head_dim=64, scaling={"kind": "linear", "factor": 2.0, "low": 1.0}),
    dict(head_dim=64, scaling={"kind": "bands", "factor": 2.0, "low": 4.0, "high": 1.0, "original_len": 100}),
    dict(head_dim=64, scaling={"kind": "linear", "factor": 2.0}, inv_freq=[1.0] * 32),
])
def test_rope_refusals(kw):
    with pytest.raises(ValueError):
        Rope(**kw)


def test_other_head_dims_are_refused():
    with pytest.raises(NotImplementedError):
        Rope(96)


def _strides(*s):
    import ctypes
    return (ctypes.c_longlong * len(s))(*s)


ROWS = (512, 128, 64)
APPLY = dict(q=P, k=P, qo=2 * P, ko=2 * P, turns=P, pos=P, start=0, B=2, Hq=4, Hk=2, N=2, D=64, rot=64, inter=0, amp=1.0,
             back=0, st=_strides(*ROWS, *ROWS, *ROWS, *ROWS, 2, 1), dtype=0)


@pytest.mark.parametrize("change,code", [
    ({"q": 0}, 1), ({"qo": 0}, 1), ({"k": 0}, 1), ({"ko": 0}, 1), ({"Hk": 0}, 1), ({"turns": 0}, 1), ({"st": None}, 1),
    ({"B": 0}, 1), ({"N": -1}, 1), ({"Hq": 0}, 1), ({"rot": 66}, 1), ({"rot": 7}, 1), ({"rot": 0}, 1), ({"inter": 2}, 1),
    ({"amp": 0.0}, 1), ({"amp": float("inf")}, 1), ({"amp": float("nan")}, 1), ({"back": 2}, 1), ({"dtype": 2}, 1),
    ({"D": 96}, 2), ({"D": 256}, 2), ({"pos": 0, "start": (1 << 31) - 2}, 2), ({"B": 1 << 20, "N": 1 << 20}, 2),
    ({"q": P + 8}, 3), ({"ko": P + 2}, 3), ({"pos": P + 2}, 3), ({"turns": P + 4}, 3),
    ({"st": _strides(512, 128, 60, *ROWS, *ROWS, *ROWS, 2, 1)}, 3),
    ({"st": _strides(512, -128, 64, *ROWS, *ROWS, *ROWS, 2, 1)}, 1),
    ({"qo": P, "st": _strides(*ROWS, *ROWS, 1024, 128, 64, *ROWS, 2, 1)}, 1),   # in place with other strides
])
def test_c_refusals(lib, change, code):
    assert lib.rope_apply(*{**APPLY, **change}.values(), None) == code


# ------------------------------------------------------------------ on the GPU

def _rows(shape, dtype, seed, layout="bhnd"):
    x = torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    if layout == "bnhd":        # rows of a projection
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "fused":       # a slice of wider rows
        wide = torch.zeros(*shape[:3], shape[3] + 24, dtype=dtype, device="cuda")
        wide[..., 8:8 + shape[3]] = x
        return wide[..., 8:8 + shape[3]]
    if layout == "odd":         # rows that only a copy aligns
        flat = torch.zeros(x.numel() + 3, dtype=dtype, device="cuda")
        flat[3:] = x.flatten()
        return flat[3:].view(shape)
    return x


def _close(got, x, rope, positions, transposed=False, what=""):
    ref = rope_ref.rotate(x.cpu(), rope.inv_freq, positions.cpu(), rope.amplitude, rope.interleaved, transposed)
    tol = rope_ref.tolerance(x.cpu(), ref, x.dtype, rope.rotary_dim, rope.interleaved, rope.amplitude)
    over = (got.cpu().double() - ref).abs() / tol
    assert bool((over <= 1).all()), (what, float(over.max()))
    assert torch.equal(got[..., rope.rotary_dim:], x[..., rope.rotary_dim:])


CASES = [
    # D, rot, interleaved, scaling, B, Hq, Hk, N, far, layout, dtype
    (64, 64, False, None, 1, 1, 1, 1, 0, "bhnd", F16),
    (128, 128, False, None, 2, 4, 2, 33, 0, "bhnd", BF16),
    (128, 128, True, None, 2, 4, 4, 33, 1000000, "bnhd", BF16),
    (64, 64, True, {"kind": "linear", "factor": 3.0}, 3, 7, 1, 65, 5000, "fused", F16),
    (128, 32, False, {"kind": "yarn", "factor": 8.0, "original_len": 512}, 1, 9, 3, 100, 200000, "bnhd", BF16),
    (64, 16, True, {"kind": "ntk", "factor": 4.0}, 2, 2, 2, 17, 100, "bhnd", F16),
    (128, 48, False, {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original_len": 2048}, 1, 5, 1, 70,
     120000, "odd", F16),
    (64, 20, False, None, 2, 3, 1, 41, 999, "bhnd", F16),        # pairs that no 16-byte vector holds whole
    (128, 126, False, None, 1, 3, 2, 19, 70000, "fused", BF16),
    (128, 2, False, None, 1, 2, 1, 9, 30, "bhnd", BF16),
    (128, 2, True, None, 1, 2, 1, 9, 30, "bnhd", BF16),
    (64, 14, True, None, 2, 3, 2, 11, 500000, "bhnd", F16),
    (64, 62, True, None, 1, 1, 6, 5, 3, "odd", BF16),
    (128, 128, False, None, 1, 1, 1, 3000, 0, "bhnd", F16),      # one head: a thread takes one
    # long enough for four heads a thread, none of the sizes a multiple of what a CTA takes
    (128, 128, False, None, 2, 30, 11, 331, 50000, "bnhd", BF16),
    (64, 64, False, None, 1, 33, 5, 601, 50000, "bhnd", F16),
    (64, 20, False, None, 1, 33, 5, 601, 50000, "bnhd", BF16),
    (128, 30, True, None, 3, 13, 3, 251, 50000, "bhnd", F16),
    (64, 64, True, None, 1, 2, 1, 9001, 0, "bnhd", BF16),
    (128, 64, False, None, 1, 130, 7, 9, 100, "bhnd", F16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotations_match_the_definition(cuda_lib, case):
    D, rot, inter, scaling, B, Hq, Hk, N, far, layout, dtype = case
    rope = Rope(D, rot, interleaved=inter, scaling=scaling)
    q, k = _rows((B, Hq, N, D), dtype, 1, layout), _rows((B, Hk, N, D), dtype, 2, layout)
    g = torch.Generator().manual_seed(3)
    positions = torch.randint(-far, far + 1, (B, N), generator=g, dtype=torch.int32)
    keep = q.clone(), k.clone()
    yq, yk = rope(q, k, positions.cuda())
    assert yq.is_contiguous() and yk.is_contiguous() and yq.dtype is dtype
    _close(yq, q, rope, positions, what="q")
    _close(yk, k, rope, positions, what="k")
    # q alone, rows of positions that all sequences share, and turned back
    _close(rope(q, positions=positions[0].cuda()), q, rope, positions[:1].expand(B, N), what="q alone")
    tq, tk = _lib.rope(q, k, rope, positions.cuda(), transposed=True)
    _close(tq, q, rope, positions, transposed=True, what="back")
    _close(tk, k, rope, positions, transposed=True, what="back")
    # counted positions
    sq, sk = rope(q, k, start=far)
    ramp = far + torch.arange(N, dtype=torch.int32)
    _close(sq, q, rope, ramp[None].expand(B, N), what="start")
    _close(sk, k, rope, ramp[None].expand(B, N), what="start")
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1])
    # in place, where the rows allow it, and into other strides
    if layout != "odd":
        a, b = _rows((B, Hq, N, D), dtype, 1, layout), _rows((B, Hk, N, D), dtype, 2, layout)
        ra, rb = _lib.rope(a, b, rope, positions.cuda(), q_out=a, k_out=b)
        assert ra.data_ptr() == a.data_ptr() and torch.equal(a, yq) and torch.equal(b, yk)
    out = torch.empty(B, N, Hq, D, dtype=dtype, device="cuda").transpose(1, 2)
    _lib.rope(q, k, rope, positions.cuda(), q_out=out)
    assert torch.equal(out, yq)
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_in_place_leaves_neighbours_alone(cuda_lib):
    """Rows in the middle of wider ones: what stands beside them is not touched."""
    for rot, inter in ((64, False), (32, False), (20, False), (12, True)):
        wide = torch.randn(2, 3, 10, 64 + 24, device="cuda").to(F16)
        rope, keep = Rope(64, rot, interleaved=inter), wide.clone()
        x = wide[..., 8:72]
        want = rope(x.clone())
        _lib.rope(x, None, rope, q_out=x)
        assert torch.equal(x, want)
        assert torch.equal(wide[..., :8], keep[..., :8]) and torch.equal(wide[..., 72:], keep[..., 72:])


@pytest.mark.gpu
@pytest.mark.parametrize("rot,inter", [(64, False), (32, False), (20, False), (12, True), (64, True)])
def test_special_values(cuda_lib, rot, inter):
    """Infinities and NaN of dimensions that stay are kept; those of a pair stay within it."""
    rope = Rope(64, rot, interleaved=inter)
    x = torch.randn(1, 2, 4, 64, device="cuda").to(F16)
    x[0, 0, 1, 5], x[0, 1, 2, 0] = float("inf"), float("nan")
    if rot < 64:
        x[0, 0, 3, rot], x[0, 1, 3, 63] = float("-inf"), float("nan")
    y = rope(x, start=7)
    clean = rope(torch.where(torch.isfinite(x), x, torch.zeros_like(x)), start=7)
    touched = torch.zeros_like(x, dtype=torch.bool)
    for h, n, d in ((0, 1, 5), (1, 2, 0)):
        touched[0, h, n, d] = touched[0, h, n, (d ^ 1) if inter else (d + rot // 2) % rot] = True
    assert not bool(torch.isfinite(y[touched]).any())
    rest = ~touched & torch.isfinite(x)
    assert torch.equal(y[rest], clean[rest])
    if rot < 64:
        assert y[0, 0, 3, rot] == float("-inf") and bool(torch.isnan(y[0, 1, 3, 63]))


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot,inter,dtype", [(64, 64, False, F16), (128, 96, True, BF16), (64, 20, False, F16)])
def test_gradients(cuda_lib, D, rot, inter, dtype):
    """Against the formula, against differences, of expanded inputs, and a second time."""
    rope = Rope(D, rot, interleaved=inter, amplitude=1.25)
    positions = torch.tensor([[0, 5, 1000, 77777], [3, 4, 5, 6]], dtype=torch.int32, device="cuda")
    q, k = (_rows((2, h, 4, D), dtype, s).requires_grad_(True) for h, s in ((4, 1), (2, 2)))
    gq, gk = _rows((2, 4, 4, D), dtype, 3), _rows((2, 2, 4, D), dtype, 4, "bnhd")
    yq, yk = rope(q, k, positions)
    dq, dk = torch.autograd.grad((yq, yk), (q, k), (gq, gk))
    _close(dq, gq, rope, positions, transposed=True, what="dq")
    _close(dk, gk, rope, positions, transposed=True, what="dk")
    # one of the two alone
    for y, x, g, d in ((0, q, gq, dq), (1, k, gk, dk)):
        assert torch.equal(torch.autograd.grad(rope(q, k, positions)[y], x, g)[0], d)
    # differences: the rotation is linear, so y(q + h) - y(q - h) times g is 2 h times dq up to
    # the roundings of the four results (half a step each)
    h = _rows((2, 4, 4, D), dtype, 5)
    hi, lo = (q.detach() + h), (q.detach() - h)
    yhi, ylo = rope(hi, positions=positions), rope(lo, positions=positions)
    step = (hi.double() - lo.double())
    left = ((yhi.double() - ylo.double()) * gq.double()).sum()
    right = (step * dq.double()).sum()
    half = torch.finfo(dtype).eps / 2 * (1 + 2.0 ** -6)
    tol = half * (((yhi.double().abs() + ylo.double().abs()) * gq.double().abs()).sum()
                  + (step.abs() * dq.double().abs()).sum())
    assert abs(float(left - right)) <= float(tol)
    # keys that all query heads' groups share, through an expanded view
    one = _rows((2, 1, 4, D), dtype, 6).requires_grad_(True)
    y = rope(one.expand(2, 4, 4, D), positions=positions)
    (d1,) = torch.autograd.grad(y, one, gq)
    assert torch.equal(d1, dq.sum(1, keepdim=True))
    # a gradient of the gradient: of sum(dq * w) with respect to g it is the rotation of w
    g = gq.clone().requires_grad_(True)
    (d,) = torch.autograd.grad(rope(q, positions=positions), q, g, create_graph=True)
    (gg,) = torch.autograd.grad(d, g, h)
    assert torch.equal(gg, rope(h, positions=positions))


@pytest.mark.gpu
def test_positions_that_change_are_noticed(cuda_lib):
    rope, q = Rope(64), _rows((1, 2, 5, 64), F16, 1).requires_grad_(True)
    positions = torch.arange(5, dtype=torch.int32, device="cuda")
    y = rope(q, positions=positions)
    positions += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.gpu
def test_refusals(cuda_lib):
    rope, q = Rope(64), _rows((2, 4, 6, 64), F16, 1)
    k, pos = _rows((2, 2, 6, 64), F16, 2), torch.arange(6, dtype=torch.int32, device="cuda")
    for bad in (k[:, :, :5], k[:1], k.to(BF16), k.cpu(), k[0]):
        with pytest.raises((ValueError, TypeError)):
            rope(q, bad)
    for bad in (pos.long(), pos[:5], pos.cpu(), pos[None].expand(3, 6), pos.float()):
        with pytest.raises(ValueError, match="positions"):
            rope(q, k, bad)
    with pytest.raises(ValueError, match="rows"):
        Rope(128)(q, k)
    with pytest.raises(TypeError):
        rope(q.float())
    with pytest.raises(ValueError):
        rope(q, k, start=1 << 40)
    with pytest.raises(_lib.AttnError):
        rope(q, k, start=(1 << 31) - 3)
    with pytest.raises(ValueError, match="q_out"):
        _lib.rope(q, k, rope, q_out=k)
    with pytest.raises(ValueError, match="overlap"):
        _lib.rope(q, k, rope, q_out=q[:, :1].expand(2, 4, 6, 64))
    with pytest.raises(ValueError, match="k_out"):
        _lib.rope(q, None, rope, k_out=k)
    leaf = q.clone().requires_grad_(True)
    with pytest.raises(ValueError, match="autograd"):
        _lib.rope(leaf, k, rope, q_out=torch.empty_like(q))
    with torch.no_grad():
        assert torch.equal(_lib.rope(leaf, None, rope, q_out=torch.empty_like(q)), rope(q))
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_captured_and_on_other_streams(cuda_lib):
    """A training step captured with its backward, replayed on new inputs; and two streams at once."""
    rope = Rope(128, 64, interleaved=True)
    q, k = (_rows((2, h, 50, 128), BF16, h).requires_grad_(True) for h in (4, 2))
    g = [_rows((2, h, 50, 128), BF16, 9 + h) for h in (4, 2)]
    positions = torch.arange(50, dtype=torch.int32, device="cuda") + 11

    def both():
        y = rope(q, k, positions)
        return [t.detach() for t in y] + list(torch.autograd.grad(y, (q, k), g))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(both(), want))
    older = rope(q, k, positions)
    with pytest.raises(RuntimeError, match="recorded outside the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            both()
    del older
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    with torch.no_grad():
        q.mul_(2.0)
        positions.add_(1000)
    graph.replay()
    got = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(got, both()))
    assert not torch.equal(got[0], want[0])


@pytest.mark.gpu
def test_rotated_training_step(cuda_lib):
    """Rotation and attention together: the attention's scores depend on differences of positions
    alone, so shifting all positions changes nothing but rounding."""
    rope = Rope(64, base=500.0)
    q, k, v = (_rows((1, h, 130, 64), BF16, s).requires_grad_(True) for h, s in ((4, 1), (2, 2), (2, 3)))
    do = _rows((1, 4, 130, 64), BF16, 4)
    res = []
    for start in (0, 123456):
        rq, rk = rope(q, k, start=start)
        out = sdpa.window_attention(rq, rk, v, 60, 2)
        res.append([out.detach(), *torch.autograd.grad(out, (q, k, v), do)])
    # rotated rows are rounded to bf16 twice over: a relative 2^-8 of each score's factors
    for a, b in zip(*res):
        assert float((a.double() - b.double()).norm() / b.double().norm()) < 4 * 2.0 ** -8


@pytest.mark.gpu
def test_a_first_use_is_not_captured(cuda_lib):
    """The frequencies are copied to a device once: refused inside a capture, which goes on."""
    rope, q = Rope(64), _rows((1, 2, 5, 64), F16, 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="first use"):
            rope(q)
        twice = q * 2
    graph.replay()
    rope.turns("cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = rope(q)
    graph.replay()
    assert torch.equal(y, rope(q)) and torch.equal(twice, q * 2)


def test_frequencies_are_ordinary_tensors():
    """Whatever mode the first use runs in, the kept frequencies can be saved for a backward pass."""
    rope = Rope(64)
    with torch.inference_mode():
        words = rope.turns("cpu")
        assert torch.equal(Rope(64).turns("cpu"), words)
    assert not words.is_inference() and not rope.for_rows(torch.zeros(1, 1, 1, 64))[0].is_inference()


@pytest.mark.gpu
def test_a_first_use_under_inference_mode(cuda_lib):
    """Evaluation first, training afterwards: the rotation's gradient is what it is without the former."""
    q, k = _rows((1, 2, 5, 64), F16, 1), _rows((1, 2, 5, 64), F16, 2)
    g = _rows((1, 2, 5, 64), F16, 3)
    want = _lib.rope(g, None, Rope(64), transposed=True)
    cache = PagedKVCache(1, 1, 2, 64, n_pages=2, page_size=16)
    for first in ("rows", "append"):
        rope = Rope(64)
        with torch.inference_mode():
            if first == "rows":
                seen = rope(q, k)[0]
            else:
                cache.reserve(5)
                seen = cache.append(0, k, k, rope=rope, q=q)
        leaf = q.clone().requires_grad_(True)
        y = rope(leaf)
        assert torch.equal(y.detach(), rope(q)) and torch.equal(rope(q), Rope(64)(q)) and seen.is_inference()
        (d,) = torch.autograd.grad(y, leaf, g)
        assert torch.equal(d, want)
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_forward_mode_is_refused(cuda_lib):
    """A dual number's tangent does not vanish in silence: with or without gradients, of q or of k."""
    from torch.autograd import forward_ad
    rope, q, t = Rope(64), _rows((1, 2, 5, 64), F16, 1), _rows((1, 2, 5, 64), F16, 2)
    want = rope(q)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(q, t)
        for call in (lambda: rope(dual), lambda: rope(q, dual), lambda: _lib.rotary(dual, q, rope),
                     lambda: rope(dual, q.clone().requires_grad_(True))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
            with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        assert torch.equal(rope(q), want)
    with pytest.raises(RuntimeError):
        torch.func.jvp(rope, (q,), (t,))
    assert torch.equal(rope(q), want) and _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_one_row_of_positions_for_a_batch(cuda_lib):
    """[1, N], as models hold them: what [N] gives, forward, backward and of any strides."""
    rope, q, g = Rope(64), _rows((3, 2, 7, 64), BF16, 1).requires_grad_(True), _rows((3, 2, 7, 64), BF16, 2)
    pos = torch.randint(0, 9999, (7,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    want = rope(q, positions=pos)
    (dq,) = torch.autograd.grad(want, q, g)
    rows = torch.stack([pos, pos + 1], 1)   # every second element, and a batch stride that is nobody's
    for one in (pos[None], pos[None].expand(3, 7), rows[None, :, 0], rows.t()[:1]):
        got = rope(q, positions=one)
        assert torch.equal(got, want) and torch.equal(torch.autograd.grad(got, q, g)[0], dq)
        assert torch.equal(_lib.rope(q.detach(), None, rope, one), want)
    for bad in (pos[None, None], pos[None].expand(2, 7), pos[None, :6], pos[:1].expand(3, 1)):
        with pytest.raises(ValueError, match="positions"):
            rope(q, positions=bad)
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_results_that_overlap_are_refused(cuda_lib):
    """Results in each other's place, in another operand's, or with rows over rows: refused, and no version counted on;
    slices of one tensor that lie side by side are taken."""
    rope, q, k = Rope(64), _rows((2, 4, 6, 64), F16, 1), _rows((2, 4, 6, 64), F16, 2)
    spare, want = torch.empty_like(q), rope(q, k)
    flat = torch.zeros(2 * 4 * 6 * 64, dtype=F16, device="cuda")
    for bad, what in ((dict(q_out=k), "k does"), (dict(k_out=q), "q does"), (dict(q_out=spare, k_out=spare), "k_out does"),
                      (dict(q_out=spare, k_out=k[:, :2]), "k_out must"), (dict(q_out=k, k_out=q), "k does"),
                      (dict(q_out=flat.as_strided(q.shape, (1536, 384, 32, 1))), "overlap"),
                      (dict(k_out=flat.as_strided(q.shape, (384, 384, 64, 1))), "overlap")):
        keep = [(t, t.clone(), t._version) for t in (q, k, spare, flat)]
        with pytest.raises(ValueError, match=what):
            _lib.rope(q, k, rope, **bad)
        assert all(torch.equal(t.view(torch.uint8), c.view(torch.uint8)) and t._version == n for t, c, n in keep)
    with pytest.raises(ValueError, match="k does"):
        _lib.rope(q, q, rope, q_out=q, k_out=q)
    wide = torch.cat([q, k], 3)                        # [.., 128]: two slices, reaching over each other
    a, b = wide[..., :64], wide[..., 64:]
    n = wide._version
    got = _lib.rope(a, b, rope, q_out=a, k_out=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(wide, torch.cat(want, 3)) and wide._version > n
    cache = PagedKVCache(1, 2, 4, 64, n_pages=2, page_size=16)
    cache.reserve(6)
    pools = [t[0] for t in (cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale)]
    for out, what in ((k, "k does"), (flat.as_strided(q.shape, (1536, 384, 32, 1)), "overlap")):
        with pytest.raises(ValueError, match=what):
            _lib.kv8_append(k, k, *pools, cache.table, cache.lens, rope=rope, q=q, q_out=out)
    assert not cache.k_pages.view(torch.uint8).any()
    assert torch.equal(_lib.kv8_append(k, k, *pools, cache.table, cache.lens, rope=rope, q=q, q_out=spare), want[0])
    assert _lib.sync_status() == _lib.ATTN_OK


def test_a_first_use_inside_a_function_transform_is_refused():
    """What is made there ends with the transform: it is not kept, and the rotation goes on working."""
    from torch._subclasses import FakeTensorMode
    rope = Rope(64)

    def f(x):
        rope.turns("cpu")
        return x.sum()
    with pytest.raises(RuntimeError, match="function transform"):
        torch.func.grad(f)(torch.ones(3))
    with FakeTensorMode(), pytest.raises(RuntimeError, match="function transform"):
        rope.turns("cpu")
    words = rope.turns("cpu")
    assert type(words) is torch.Tensor and words.data_ptr() and torch.equal(words, Rope(64).turns("cpu"))
    assert torch.equal(torch.func.grad(f)(torch.ones(3)), torch.ones(3))


@pytest.mark.gpu
def test_function_transforms_are_refused(cuda_lib):
    """torch.func's transforms raise, whether they come first or not, and leave the rotation as it was."""
    q = _rows((1, 2, 5, 64), F16, 1)
    want = Rope(64)(q)
    for used in (False, True):
        rope = Rope(64)
        if used:
            rope(q)
        for transform in (lambda: torch.func.grad(lambda x: rope(x).float().sum())(q), lambda: torch.func.vjp(rope, q),
                          lambda: torch.func.jvp(rope, (q,), (q,)), lambda: torch.func.vmap(lambda x: rope(x[None])[0])(q)):
            with pytest.raises(RuntimeError):
                transform()
        leaf = q.clone().requires_grad_(True)
        y = rope(leaf)
        assert torch.equal(y.detach(), want) and torch.autograd.grad(y, leaf, q)[0].shape == q.shape
    assert _lib.sync_status() == _lib.ATTN_OK
