"""The layers around the attention in 64 bits, from their formulas, with plain
torch operations (tests only).  Every function takes and returns float64
tensors on any device."""
import math

import torch


def act(z, name):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def act_slope(z, name):
    """The derivative, by autograd of act (so not the kernels' own formulas)."""
    if name == "none":
        return torch.ones_like(z)
    with torch.enable_grad():
        z = z.detach().clone().requires_grad_(True)
        act(z, name).sum().backward()
    return z.grad


def rotate(v, positions, inv_freq, rope, sign=1.0):
    """v [B, L, H, D], positions [B, L]; the first 2 len(inv_freq) elements turn."""
    if inv_freq is None:
        return v
    half = inv_freq.numel()
    a = (positions.double()[..., None] * inv_freq.double())[:, :, None, :]
    c, s = torch.cos(a), torch.sin(a) * sign
    if rope == "halves":
        i = torch.arange(half, device=v.device)
        j = i + half
    else:
        i = 2 * torch.arange(half, device=v.device)
        j = i + 1
    out = v.clone()
    out[..., i] = v[..., i] * c - v[..., j] * s
    out[..., j] = v[..., j] * c + v[..., i] * s
    return out


def norm(x, kind, eps):
    if kind == "none":
        return x
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)


def qk(x, weight, bias, kind, eps, inv_freq, rope, positions):
    """x [B, L, H, D] -> [B, H, L, D]."""
    v = norm(x, kind, eps)
    if weight is not None:
        v = v * weight
    if bias is not None:
        v = v + bias
    return rotate(v, positions, inv_freq, rope).transpose(1, 2)


def qk_grads(g, x, weight, bias, kind, eps, inv_freq, rope, positions):
    """Gradients of qk by the formulas: (dx, dweight, dbias)."""
    g = rotate(g.transpose(1, 2), positions, inv_freq, rope, -1.0)
    n = norm(x, kind, eps)
    dw, db = (g * n).sum((0, 1, 2)), g.sum((0, 1, 2))
    d = g if weight is None else g * weight
    if kind != "none":
        c = x - x.mean(-1, keepdim=True) if kind == "layer" else x
        r = 1 / torch.sqrt(c.square().mean(-1, keepdim=True) + eps)
        d = d - n * (d * n).mean(-1, keepdim=True)
        if kind == "layer":
            d = d - d.mean(-1, keepdim=True)  # n has mean zero: the same as g w's mean
        d = r * d
    return d, dw, db
