"""The model operators' definitions in 64 bits, for their tests."""
import torch

TILE = 128


def blocks(n):
    return -(-n // TILE)


def fp8_weight(g, *shape, sigma=0.02):
    """Codes of normal weights and uneven block scales, on the generator's device."""
    dev = g.device
    w = (torch.randn(shape, generator=g, device=dev) * 107).clamp(-448, 448)
    codes = w.to(torch.float8_e4m3fn).view(torch.uint8)
    scale = (torch.rand(shape[:-2] + (blocks(shape[-2]), blocks(shape[-1])), generator=g, device=dev) + 0.2) * (sigma / 107)
    return codes, scale


def decode(codes, scale):
    """[E, R, C] values in float64, from the format: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    def value(c):
        e, m = (c >> 3) & 15, c & 7
        v = float("nan") if c & 127 == 127 else m / 8 * 2.0**-6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        return -v if c & 128 else v

    v = torch.tensor([value(c) for c in range(256)], dtype=torch.float64, device=codes.device)[codes.int()]
    r, k = codes.shape[-2:]
    s = scale.double().repeat_interleave(TILE, -2)[..., :r, :].repeat_interleave(TILE, -1)[..., :k]
    return v * s


def runs(offsets, experts, tokens):
    if offsets is None:
        return [(0, tokens)]
    o = offsets.tolist()
    return [(o[e], o[e + 1]) for e in range(experts)]


def ffn(x, wgu, wd, spans, dy=None):
    """y, and with dy also dx, d_gate_up, d_down; and the sums of magnitudes that bound y's and dx's roundings."""
    x = x.double()
    f = wd.shape[1]
    out = {k: torch.zeros_like(x) for k in ("y", "y_mag", "dx", "dx_mag")}
    out["d_gate_up"], out["d_down"] = torch.zeros_like(wgu), torch.zeros_like(wd)
    for e, (lo, hi) in enumerate(spans):
        xe = x[lo:hi]
        g, u = xe @ wgu[e][:, :f], xe @ wgu[e][:, f:]
        s = 1 / (1 + torch.exp(-g))
        a = g * s
        h = a * u
        out["y"][lo:hi] = h @ wd[e]
        out["y_mag"][lo:hi] = h.abs() @ wd[e].abs()
        if dy is None:
            continue
        d = dy[lo:hi].double()
        dh = d @ wd[e].T
        dgu = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * a], 1)
        out["d_down"][e] = h.T @ d
        out["d_gate_up"][e] = xe.T @ dgu
        out["dx"][lo:hi] = dgu @ wgu[e].T
        out["dx_mag"][lo:hi] = dgu.abs() @ wgu[e].abs().T
    return out


def distill(z, ids, teacher, tau, weight):
    """(loss, gradient) row by row, float64."""
    rows, vocab = z.shape
    z = z.double()
    loss, grad = torch.zeros(rows, dtype=torch.float64), torch.zeros(rows, vocab, dtype=torch.float64)
    for r in range(rows):
        w = 1.0 if weight is None else float(weight[r])
        listed = [(int(j), float(t)) for j, t in zip(ids[r], teacher[r])
                  if 0 <= int(j) < vocab and float(t) != -float("inf")]
        if w == 0 or not listed:
            continue
        j = torch.tensor([a for a, _ in listed])
        lp = torch.log_softmax(torch.tensor([b for _, b in listed], dtype=torch.float64) / tau, 0)
        lq = torch.log_softmax(z[r].cpu() / tau, 0)
        p = lp.exp()
        loss[r] = tau * tau * (p * (lp - lq[j])).sum()
        full = torch.zeros(vocab, dtype=torch.float64).index_add_(0, j, p)
        grad[r] = w * tau * (lq.exp() - full)
    return loss, grad
