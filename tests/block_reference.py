"""Plain 64-bit forms of the block's operators (CPU), differentiable through torch autograd.

Written from the definitions, one time step at a time; nothing here is shared with the library.
"""
import torch

F64 = torch.float64


def wide(t, grad=False):
    return None if t is None else t.detach().cpu().to(F64).requires_grad_(grad)


def head_scan(x, delta, A_log, B, C, D, bias=None, softplus=True, h0=None):
    """y (b, L, H, P) and the last state (b, H, P, N), step by step."""
    b, L, H, P = x.shape
    G, N = B.shape[2:]
    raw = delta if bias is None else delta + bias
    step = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    A = -torch.exp(A_log)
    of = torch.arange(H) // (H // G)
    h = torch.zeros(b, H, P, N, dtype=x.dtype) if h0 is None else h0
    ys = []
    for t in range(L):
        h = torch.exp(step[:, t] * A)[..., None, None] * h \
            + (step[:, t, :, None] * x[:, t])[..., None] * B[:, t, of][:, :, None, :]
        ys.append((h * C[:, t, of][:, :, None, :]).sum(-1) + D[:, None] * x[:, t])
    y = torch.stack(ys, 1) if ys else x * D[:, None]
    return y, h


def residual_norm(x, w, residual=None, scale=None, eps=1e-5, stored=None):
    """(out, r); `stored`: the type r is kept in (its rounding passes gradients through)."""
    r = x if scale is None else x * scale
    r = r if residual is None else residual + r
    if stored is not None:
        r = r + (r.detach().float().to(stored).to(F64) - r.detach())
    return r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * w, r


def gated_norm(y, z, w, groups=1, eps=1e-5, before=False):
    gate = z / (1 + torch.exp(-z))
    v = (y if before else y * gate).unflatten(-1, (groups, -1))
    o = (v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)).flatten(-2) * w
    return o * gate if before else o


def rel(got, want):
    """2-norm of the difference over the 2-norm of what is wanted."""
    got, want = got.detach().cpu().to(F64), want.detach().to(F64)
    assert got.shape == want.shape, (got.shape, want.shape)
    if want.numel() == 0:
        return 0.0
    d, n = (got - want).norm().item(), want.norm().item()
    return d / n if n else (0.0 if d == 0 else float("inf"))
