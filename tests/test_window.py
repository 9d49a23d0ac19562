"""Sliding-window attention with sinks (attn_fwd_window, attn_bwd_window and
sdpa.window_attention) against the fp64 definition, and its refusals.

Tolerances are those of the other forwards and backwards (tests/helpers.py):
the kernels are the same but for the key tiles they visit and the mask of the
edge tiles."""
import numpy as np
import pytest
import torch

from tests import helpers, window_ref
from tiled_memory_efficient_gb300 import _lib, inputs, sdpa

F16, BF16 = torch.float16, torch.bfloat16
P = 256  # a fake, 16-byte-aligned "device" address: validation fails before any use


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


# ------------------------------------------------------------------ CPU

def test_reference_gradients_agree_with_differences():
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(1, 1, n, 8, generator=g, dtype=torch.float64) for n in (5, 9, 9, 5))
    _, _, dq, dk, dv = window_ref.attention(q, k, v, 3, 2, dout=do)
    f = lambda: float((window_ref.attention(q, k, v, 3, 2)[0] * do).sum())
    eps = 1e-5
    for t, grad in ((q, dq), (k, dk), (v, dv)):
        for i in range(0, t.numel(), 7):
            old = t.view(-1)[i].item()
            t.view(-1)[i] = old + eps
            up = f()
            t.view(-1)[i] = old - eps
            down = f()
            t.view(-1)[i] = old
            # central difference: O(eps^2) truncation plus 1e-16 / eps cancellation
            assert abs((up - down) / (2 * eps) - float(grad.view(-1)[i])) < 1e-8


def test_reference_closed_forms():
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(1, 2, 12, 8, generator=g) for _ in range(3))
    out, lse = window_ref.attention(q, k, v, 1, 0)     # only itself
    assert torch.allclose(out, v.double()) and torch.allclose(
        lse, (q.double() * k.double()).sum(-1) * 8 ** -0.5)
    full = window_ref.attention(q, k, v, 12, 0)[0]     # a window as long as the sequence
    assert torch.equal(full, window_ref.attention(q, k, v, 3, 12)[0])   # every key a sink


@pytest.mark.parametrize("change,code", [
    ({"window": 0}, 1), ({"window": -1}, 1), ({"sinks": -1}, 1), ({"Nq": 129}, 1), ({"Hq": 3}, 1),
    ({"scale": 0.0}, 1), ({"dtype": 5}, 1), ({"D": 96}, 2), ({"q": 0}, 1), ({"q": P + 8}, 3),
    ({"out": P + 4}, 3), ({"lse": 0}, 1),
])
def test_forward_refusals(lib, change, code):
    a = dict(q=P, k=P, v=P, out=P, lse=P, ws=P, n=1 << 40, B=1, Hq=2, Hkv=2, Nq=128, Nk=128, D=64,
             scale=0.1, window=16, sinks=2, dtype=0)
    a.update(change)
    assert lib.attn_fwd_window(*a.values(), None) == code


def test_workspace_is_checked_first(lib):
    ws = lib.attn_fwd_window_workspace_size(64, 32, 2, 300, 300, 64, 16, 0, 1)
    assert ws >= 128 * 300 * 64 * 2 + 128 * 3   # bf16: the fp16 copy of v and its flags
    args = (64, 32, 2, 300, 300, 64, 0.1, 16, 0, 1, None)
    assert lib.attn_fwd_window(*[P] * 5, 0, ws, *args) == 1
    assert lib.attn_fwd_window(*[P] * 5, P + 8, ws, *args) == 3
    assert lib.attn_fwd_window(*[P] * 5, P, ws - 1, *args) == 6
    assert lib.attn_fwd_window_workspace_size(1, 2, 2, 300, 300, 64, 0, 0, 1) == 0
    assert lib.attn_fwd_window_workspace_size(1, 2, 2, 301, 300, 64, 4, 0, 1) == 0


@pytest.mark.parametrize("change,code", [
    ({"window": 0}, 1), ({"sinks": -1}, 1), ({"Nq": 129}, 1), ({"Hq": 3}, 1), ({"D": 32}, 2),
    ({"dout": 0}, 1), ({"dk": P + 8}, 3), ({"n": 16}, 6), ({"ws": 0}, 1),
])
def test_backward_refusals(lib, change, code):
    a = dict(q=P, k=P, v=P, out=P, dout=P, lse=P, dq=P, dk=P, dv=P, ws=P, n=1 << 40, B=1, Hq=2,
             Hkv=2, Nq=128, Nk=128, D=64, scale=0.1, window=16, sinks=2, dtype=0)
    a.update(change)
    assert lib.attn_bwd_window(*a.values(), None) == code
    # per head: 128 padded rows, two fp32 statistics
    assert lib.attn_bwd_window_workspace_size(1, 2, 2, 128, 128, 64, 16, 0, 0) >= 2 * 2 * 128 * 4
    assert lib.attn_bwd_window_workspace_size(1, 2, 2, 128, 128, 64, 0, 0, 0) == 0


def test_python_refusals():
    q = torch.zeros(1, 2, 8, 64, dtype=F16)
    with pytest.raises(NotImplementedError):     # no CPU fallback
        sdpa.window_attention(q, q, q, 4)
    with pytest.raises(ValueError):
        _lib.attn_fwd_window(q, q, q, 4)


# ------------------------------------------------------------------ GPU

CASES = [
    # B, Hq, Hkv, Nq, Nk, D, dtype, window, sinks
    (1, 2, 2, 256, 256, 64, F16, 64, 0),
    (1, 14, 2, 1000, 1000, 64, F16, 100, 4),        # one head per group, ragged
    (2, 4, 2, 300, 777, 128, BF16, 130, 17),        # a chunk against a longer cache
    (1, 14, 2, 1, 4133, 64, F16, 512, 4),           # decode: flattened heads, key ranges
    (1, 8, 1, 4, 3000, 128, BF16, 1000, 130),       # drafts, sinks over two tiles
    (1, 6, 2, 256, 1500, 128, F16, 300, 1),         # the longest flattened block
    (1, 7, 1, 257, 2000, 64, BF16, 256, 128),       # the shortest block of one head per group
    (1, 2, 1, 200, 200, 128, F16, 1, 0),            # a query sees itself alone
    (1, 2, 2, 513, 513, 64, BF16, 5000, 3),         # a window past the sequence
    (1, 3, 3, 640, 640, 128, F16, 128, 1000),       # every key a sink
    (1, 2, 2, 700, 700, 128, BF16, 333, 0),
    (2, 2, 1, 1, 1, 64, BF16, 1, 1),
    (1, 2, 2, 1100, 1100, 64, F16, 129, 129),
    (4, 8, 8, 1000, 1000, 64, F16, 130, 4),         # more key tiles than CTAs: each takes several
    (4, 8, 8, 300, 1500, 128, BF16, 200, 3),        # and most of them no query sees
    (5, 8, 8, 700, 700, 128, F16, 700, 0),
    (5, 8, 8, 1000, 1000, 128, BF16, 200, 130),     # D = 128 in more than a wave of Q tile pairs
    (6, 8, 4, 900, 2100, 128, F16, 300, 0),
    (8, 8, 8, 1100, 1100, 128, F16, 64, 1),         # pairs with one Q tile, several a CTA
    (3, 20, 4, 1025, 1025, 128, BF16, 129, 0),
]


def _inputs(B, Hq, Hkv, Nq, Nk, D, dtype, window, sinks):
    return inputs.make_custom(B, Hq, Hkv, Nq, Nk, D, dtype, seed=7 * Nq + window, with_grad=True)


def _assert_gradient(got, ref, dtype, what, name):
    """The gradient before its store lies within TOL_BWD of the definition, as the other
    backwards' do; the store rounds it by half a step more: |got - ref| <= |x - ref| +
    |round(x) - x| <= TOL_BWD + step / 2.  (At 4 to 8 half a bf16 step is 2^-6 = 0.0156 of
    the flat 0.02, which leaves 0.0044 for sums over a group of five heads.)"""
    assert np.all(np.isfinite(got)), f"{what}: non-finite {name}"
    err = np.abs(got - ref)
    # a step of the binade above ref's, where x may lie
    bound = helpers.TOL_BWD[dtype] + 0.5 * helpers.ulp(np.abs(ref) + helpers.TOL_BWD[dtype], dtype)
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert np.all(err <= bound), f"{what}: {name} off by {err[worst]:.3e} > {bound[worst]:.3e} at {ref[worst]:.3f}"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward_match_the_definition(cuda_lib, case):
    dtype, window, sinks = case[6:]
    x = _inputs(*case)
    q, k, v, do = (x[n].cuda() for n in ("q", "k", "v", "do"))
    out, lse = _lib.attn_fwd_window(q, k, v, window, sinks)
    grads = _lib.attn_bwd_window(q, k, v, out, do, lse, window, sinks)
    assert _lib.sync_status() == _lib.ATTN_OK
    ref = [t.numpy() for t in window_ref.attention(x["q"], x["k"], x["v"], window, sinks, dout=x["do"])]
    what = f"window {case[:6]} {window}+{sinks}"
    helpers.assert_fwd_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref[0], ref[1],
                             dtype, what)
    for name, g, r in zip(("dq", "dk", "dv"), grads, ref[2:]):
        _assert_gradient(g.double().cpu().numpy(), r, dtype, what, name)


@pytest.mark.gpu
def test_wide_bf16_values(cuda_lib):
    """Value tiles past fp16's range stay bf16, and P beside them; the other heads' do not."""
    B, H, N, D = 5, 8, 1000, 128
    x = inputs.make_custom(B, H, H, N, N, D, BF16, seed=50)
    v = x["v"].clone()
    v[1, 3, 400:410] *= 2.0 ** 20
    v[4, 7] *= 2.0 ** -12
    q, k = x["q"].cuda(), x["k"].cuda()
    out, lse = _lib.attn_fwd_window(q, k, v.cuda(), 150, 2)
    assert _lib.sync_status() == _lib.ATTN_OK
    plain, plain_lse = _lib.attn_fwd_window(q, k, x["v"].cuda(), 150, 2)
    ro, rl = window_ref.attention(x["q"], x["k"], v, 150, 2)
    assert torch.equal(lse, plain_lse)
    out = out.double().cpu()
    # bf16 P and output: 2^-9 of a term and of the result each (half a step of 8 bits), of
    # at most the largest value in sight
    for b, h in ((1, 3), (4, 7)):
        size = float(v[b, h].double().abs().max())
        assert float((out[b, h] - ro[b, h]).abs().max()) <= size * (2.0 ** -8 + 2.0 ** -8), (b, h)
    out[1, 3] = out[4, 7] = 0
    plain = plain.double().cpu()
    plain[1, 3] = plain[4, 7] = 0
    assert torch.equal(out, plain)


@pytest.mark.gpu
def test_a_window_over_everything_is_causal_attention(cuda_lib):
    x = inputs.make_custom(1, 4, 2, 512, 512, 128, F16, seed=11)
    q, k, v = (x[n].cuda() for n in "qkv")
    a, la = _lib.attn_fwd(q, k, v, causal=True)
    b, lb = _lib.attn_fwd_window(q, k, v, 1 << 40)
    torch.cuda.synchronize()
    # two roundings of one value and its sums: each within the forward's tolerance of the oracle
    assert (a.float() - b.float()).abs().max() <= 2 * helpers.TOL_O[F16]
    assert (la - lb).abs().max() <= 2 * helpers.TOL_LSE


@pytest.mark.gpu
def test_hidden_scores_do_not_matter(cuda_lib):
    """Keys no query of a row sees may score anything, an infinity or NaN too."""
    x = inputs.make_custom(1, 2, 2, 300, 900, 64, F16, seed=12)
    q, k, v = (x[n].cuda() for n in "qkv")
    a = _lib.attn_fwd_window(q, k, v, 128, 2)
    k2 = k.clone()
    k2[:, :, 2:400] = float("nan")        # the first query stands at 600 and sees 473 on
    k2[:, :, 400:470] = float("inf")
    b = _lib.attn_fwd_window(q, k2, v, 128, 2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_autograd_side_stream_and_strided_inputs(cuda_lib):
    """The differentiable function on a stream of its own, with inputs that are
    views of one projection, twice bit for bit and equal to the plain calls."""
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(2, 333, 8, 64, generator=g).to(BF16).cuda().requires_grad_(True)
    do = torch.randn(2, 4, 333, 64, generator=g).to(BF16).cuda()

    def once():
        q, k, v = (t.transpose(1, 2) for t in qkv.split((4, 2, 2), 2))
        out = sdpa.window_attention(q, k, v, 50, 3)
        return out.detach(), torch.autograd.grad(out, qkv, do)[0]
    a = once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = once()
    torch.cuda.current_stream().wait_stream(side)
    q, k, v = (t.transpose(1, 2).contiguous() for t in qkv.detach().split((4, 2, 2), 2))
    out, lse = _lib.attn_fwd_window(q, k, v, 50, 3)
    grads = _lib.attn_bwd_window(q, k, v, out, do, lse, 50, 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(a[0], out)
    assert torch.equal(a[1], torch.cat([t.transpose(1, 2) for t in grads], 2))
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_captured_and_replayed(cuda_lib):
    """Forward and backward captured into a graph and replayed on new inputs."""
    x = [inputs.make_custom(1, 4, 2, 400, 400, 64, F16, seed=s, with_grad=True) for s in (20, 21)]
    bufs = {n: x[0][n].cuda() for n in ("q", "k", "v", "do")}
    q, k, v, do = bufs.values()

    def both():
        out, lse = _lib.attn_fwd_window(q, k, v, 70, 5)
        return (out, lse) + _lib.attn_bwd_window(q, k, v, out, do, lse, 70, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for n, t in bufs.items():
        t.copy_(x[1][n])
    graph.replay()
    got = [t.clone() for t in held]
    for a, b in zip(got, both()):
        assert torch.equal(a, b)
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
@pytest.mark.parametrize("view", [False, True])
def test_captured_backward_beside_an_older_graph(cuda_lib, view):
    """Leaves that a graph outside the capture holds are refused, before anything of the
    backward is launched, and captured once that graph is gone."""
    x = inputs.make_custom(1, 2, 2, 200, 200, 64, F16, seed=30, with_grad=True)
    leaves = [x[n].cuda().requires_grad_(True) for n in "qkv"]
    do = x["do"].cuda()

    def both():
        q, k, v = (t[:, :] if view else t for t in leaves)
        out = sdpa.window_attention(q, k, v, 40, 2)
        return (out.detach(),) + torch.autograd.grad(out, leaves, do)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = both()
    torch.cuda.current_stream().wait_stream(side)
    older = sdpa.window_attention(*leaves, 40, 2)
    with pytest.raises(RuntimeError, match="recorded outside the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            both()
    del older
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    graph.replay()
    for a, b in zip(held, want):
        assert torch.equal(a, b)
    assert _lib.sync_status() == _lib.ATTN_OK


@pytest.mark.gpu
def test_two_streams_at_once(cuda_lib):
    """Forward and backward of two problems side by side give what each gives alone."""
    xs = [{n: t.cuda() for n, t in
           inputs.make_custom(2, 8, 2, 900, 900, 64, dt, seed=s, with_grad=True).items()}
          for s, dt in ((40, F16), (41, BF16))]

    def both(x):
        out, lse = _lib.attn_fwd_window(x["q"], x["k"], x["v"], 100, 3)
        return (out, lse) + _lib.attn_bwd_window(x["q"], x["k"], x["v"], out, x["do"], lse, 100, 3)
    want = [both(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = []
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(both(x))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(t, u) for t, u in zip(a, b))


@pytest.mark.gpu
def test_outputs_of_the_wrong_kind_are_refused(cuda_lib):
    q = torch.zeros(1, 2, 8, 64, dtype=F16, device="cuda")
    for bad in ({"out": q.bfloat16()}, {"lse": torch.zeros(1, 2, 8, device="cuda").half()},
                {"out": torch.zeros(1, 2, 9, 64, dtype=F16, device="cuda")}):
        with pytest.raises(ValueError):
            _lib.attn_fwd_window(q, q, q, 4, **bad)
    with pytest.raises(ValueError):
        sdpa.window_attention(q, q[:, :, :4], q[:, :, :4], 4)   # more queries than positions
    with pytest.raises(ValueError):
        sdpa.window_attention(q, q, q, 0)
    with pytest.raises(_lib.AttnError):
        _lib.attn_fwd_window(q, q, q, 0)
