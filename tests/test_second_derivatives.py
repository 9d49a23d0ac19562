"""Gradients taken with create_graph: the first derivatives are the same numbers, and a
second one through the attention raises instead of lacking its part."""
import pytest
import torch

from tests import helpers  # noqa: F401
from tiled_memory_efficient_gb300 import inputs, sdpa

F16, BF16 = torch.float16, torch.bfloat16


def _leaves(seed=60, dtype=F16):
    x = inputs.make_custom(1, 4, 2, 150, 150, 64, dtype, seed=seed, with_grad=True)
    return [x[n].cuda().requires_grad_(True) for n in "qkv"], x["do"].cuda()


def _check(call, dtype=F16):
    leaves, do = _leaves(dtype=dtype)
    want = torch.autograd.grad(call(*leaves), leaves, do)
    got = torch.autograd.grad(call(*leaves), leaves, do, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for g in got:       # alone, and beside a term that has a second derivative
        for loss in (g.float().square().sum(), g.float().square().sum() + leaves[0].float().pow(3).sum()):
            with pytest.raises(RuntimeError, match="second derivative"):
                torch.autograd.grad(loss, leaves[0], retain_graph=True)
    # what does not pass through the attention's gradients stays differentiable
    w = torch.tensor([2.0], device="cuda", requires_grad=True)
    loss = (call(*leaves).float() * do.float()).sum() + w.pow(3).sum()
    gw, gq = torch.autograd.grad(loss, (w, leaves[0]), create_graph=True)
    assert torch.autograd.grad(gw, w)[0].item() == 12.0
    # accumulated into .grad, and into it once more
    for _ in range(2):
        call(*leaves).backward(do, create_graph=True)
    for t, g in zip(leaves, want):
        assert torch.equal(t.grad.detach(), 2 * g)
        t.grad = None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_window_attention(cuda_lib, dtype):
    _check(lambda q, k, v: sdpa.window_attention(q, k, v, 40, 2), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_attention(cuda_lib, causal):
    _check(lambda q, k, v: sdpa.attention(q, k, v, is_causal=causal))


@pytest.mark.gpu
def test_masked_attention(cuda_lib):
    mask = torch.ones(1, 1, 150, 150, dtype=torch.bool, device="cuda").tril()
    _check(lambda q, k, v: sdpa.attention(q, k, v, attn_mask=mask))


@pytest.mark.gpu
def test_views_of_one_projection(cuda_lib):
    """Inputs that are not contiguous: the same gradients, and a second derivative raises."""
    g = torch.Generator().manual_seed(61)
    x = torch.randn(2, 100, 8, 64, generator=g).to(BF16).cuda().requires_grad_(True)
    do = torch.randn(2, 4, 100, 64, generator=g).to(BF16).cuda()
    for call in (lambda q, k, v: sdpa.attention(q, k, v, is_causal=True),
                 lambda q, k, v: sdpa.window_attention(q, k, v, 30, 1)):
        def once(x, **kw):
            return torch.autograd.grad(call(*(t.transpose(1, 2) for t in x.split((4, 2, 2), 2))), x, do, **kw)[0]
        parts = [t.transpose(1, 2).contiguous().detach().requires_grad_(True) for t in x.split((4, 2, 2), 2)]
        want = torch.cat([t.transpose(1, 2) for t in torch.autograd.grad(call(*parts), parts, do)], 2)
        assert torch.equal(once(x), want)
        first = once(x, create_graph=True)
        assert torch.equal(first, want)
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(first.float().square().sum() + x.float().pow(3).sum(), x)
