"""Definitions in 64 bits of the operators around the feed-forward block, for their tests."""
import math

import torch

TILE = 128


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def half_step(dtype):
    """How far a rounding to the type is off at most, relative to the value."""
    return torch.finfo(dtype).eps / 2


def strided(t, pad, at=0):
    """The same rows inside wider ones: row stride of `pad` more elements, `at` elements into the memory."""
    n, d = t.shape
    big = torch.full((n * (d + pad) + at,), float("nan"), dtype=torch.float32, device=t.device).to(t.dtype)
    view = big[at:].as_strided((n, d), (d + pad, 1))
    view.copy_(t)
    return view


def norm(x, weight, eps, residual=None, dy=None, d_total=None):
    """total, y, and with dy dx and d_weight."""
    if residual is not None:
        x = (x.double() + residual.double()).to(x.dtype)
    out = {"total": x}
    s, w = x.double(), weight.double()
    rstd = 1 / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    out["y"] = s * rstd * w
    if dy is not None:
        d = dy.double()
        g, h = d * w, s * rstd
        out["dx"] = rstd * (g - h * (g * h).mean(-1, keepdim=True))
        # what the two terms' roundings are relative to
        out["dx_mag"] = rstd * (g.abs() + h.abs() * (g * h).abs().mean(-1, keepdim=True))
        if d_total is not None:
            out["dx"] = out["dx"] + d_total.double()
        out["d_weight"] = (d * h).sum(0)
        out["d_weight_mag"] = (d * h).abs().sum(0)
    return out


def route(ids, experts):
    """offsets and place, choice by choice."""
    lists = [[] for _ in range(experts)]
    flat = ids.cpu().reshape(-1).tolist()
    for c, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(c)
    offsets, place = [0], [-1] * len(flat)
    for some in lists:
        for i, c in enumerate(some):
            place[c] = offsets[-1] + i
        offsets.append(offsets[-1] + len(some))
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(place, dtype=torch.int32).view(ids.shape[0], -1)


def gate(z, act):
    """(activation, its derivative), float64."""
    if act is None:
        return z, torch.ones_like(z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    a = math.sqrt(2 / math.pi)
    u = torch.tanh(a * (z + 0.044715 * z**3))
    return 0.5 * z * (1 + u), 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * a * (1 + 3 * 0.044715 * z * z)
