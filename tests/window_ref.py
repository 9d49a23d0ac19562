"""Sliding-window attention with sinks in fp64, one head at a time, from the
definition: every score, the visible set, softmax, weighted sum; gradients by
differentiating it."""
import torch


def visible(Nq, Nk, window, sinks):
    """[Nq, Nk] truth values: the queries are the last Nq positions; window 0: no window."""
    p = torch.arange(Nk - Nq, Nk).view(-1, 1)
    j = torch.arange(Nk).view(1, -1)
    ok = j <= p
    if window > 0:
        ok = ok & ((j > p - window) | (j < sinks))
    return ok


def head(q, k, v, window, sinks, scale, dout=None):
    q, k, v = (t.double().cpu().requires_grad_(dout is not None) for t in (q, k, v))
    s = (q @ k.t()) * scale
    s = s.masked_fill(~visible(q.shape[0], k.shape[0], window, sinks), float("-inf"))
    out = torch.softmax(s, 1) @ v
    lse = torch.logsumexp(s, 1)
    if dout is None:
        return out, lse
    grads = torch.autograd.grad(out, (q, k, v), dout.double().cpu())
    return out.detach(), lse.detach(), *grads


def attention(q, k, v, window, sinks, scale=None, dout=None):
    """out, lse and, with dout, dq, dk, dv of a [B, H, N, D] problem, as fp64."""
    B, Hq, Nq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = torch.empty(q.shape, dtype=torch.float64), torch.empty(q.shape[:3], dtype=torch.float64)
    dq = torch.empty(q.shape, dtype=torch.float64)
    dk, dv = (torch.zeros(k.shape, dtype=torch.float64) for _ in range(2))
    for b in range(B):
        for h in range(Hq):
            r = head(q[b, h], k[b, h // G], v[b, h // G], window, sinks, scale,
                     None if dout is None else dout[b, h])
            out[b, h], lse[b, h] = r[:2]
            if dout is not None:
                dq[b, h] = r[2]
                dk[b, h // G] += r[3]
                dv[b, h // G] += r[4]
    return (out, lse) if dout is None else (out, lse, dq, dk, dv)
