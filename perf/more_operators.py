"""What is timed of the operators around the gated feed-forward block, and their plain forms.

Three operators of a pre-norm block whose weights live as the optimizer writes them:

* ``norm``: root-mean-square norm of rows, the residual added first; its result in the rows' type or in 8 bits
  with a scale for every 128 columns; with ``train`` the backward pass too.
* ``route``: tokens sorted by expert (``offsets`` as the feed-forward block takes them), their rows gathered and the
  experts' rows joined again with weights; with ``train`` the gradients of both.
* ``linear``: a matrix product with an FP8 weight, or its transpose, of BF16 rows or of the norm's 8-bit rows, with
  bias, activation and residual; with ``train`` the gradients of rows, weight and bias.

``run`` computes them in elementary torch operations in 32 bits, or with ``own`` through the package's entry
points.  ``exact`` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False

TILE = 128  # a scale covers 128 x 128 codes of a weight, 128 neighbours of a row
EPS = 1e-6
GELU = math.sqrt(8.0 / math.pi)  # gelu_tanh(z) = z sigmoid(GELU (z + 0.044715 z^3))


def _blocks(n):
    return -(-n // TILE)


# ---------------------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # a decode step's rows before a projection: latency
        {"name": "norm decode fp8", "op": "norm", "train": False, "fp8": True, "rows": 32, "dim": 7168, "residual": True, "type": "bf16"},
        # a prefill batch before a projection, the residual stream updated
        {"name": "norm prefill fp8", "op": "norm", "train": False, "fp8": True, "rows": 16384, "dim": 7168, "residual": True, "type": "bf16"},
        # a training micro-batch, forward and backward
        {"name": "norm train", "op": "norm", "train": True, "fp8": False, "rows": 8192, "dim": 7168, "residual": True, "type": "bf16"},
        # FP32 rows of an odd width that no vector load fits
        {"name": "norm train ragged", "op": "norm", "train": True, "fp8": False, "rows": 2003, "dim": 4097, "residual": False, "type": "f32"},
        # one decode step of a batch over the repository's 32 experts: latency
        {"name": "route decode", "op": "route", "train": False, "tokens": 61, "top": 8, "experts": 32, "dim": 7168, "dropped": 0.0, "type": "bf16"},
        # a training micro-batch over them
        {"name": "route train", "op": "route", "train": True, "tokens": 8192, "top": 8, "experts": 32, "dim": 7168, "dropped": 0.0, "type": "bf16"},
        # FP32 rows of an odd width; a tenth of the choices dropped
        {"name": "route train ragged", "op": "route", "train": True, "tokens": 3001, "top": 3, "experts": 17, "dim": 1001, "dropped": 0.1, "type": "f32"},
        # one token's 8-bit row through the dense configuration's wider projection: bound by the codes it reads
        {"name": "linear decode fp8", "op": "linear", "train": False, "x": "fp8", "tokens": 1, "rows": 4096, "cols": 14336, "transposed": False, "act": "silu", "bias": False, "residual": False, "out": "bf16"},
        # a decode batch added to the residual stream
        {"name": "linear decode batch", "op": "linear", "train": False, "x": "bf16", "tokens": 61, "rows": 7168, "cols": 4096, "transposed": False, "act": "none", "bias": False, "residual": True, "out": "bf16"},
        # a prefill chunk of 8-bit rows
        {"name": "linear prefill fp8", "op": "linear", "train": False, "x": "fp8", "tokens": 4096, "rows": 7168, "cols": 4096, "transposed": False, "act": "none", "bias": True, "residual": False, "out": "bf16"},
        # a training micro-batch of the dense configuration's widening product
        {"name": "linear train", "op": "linear", "train": True, "x": "bf16", "tokens": 2051, "rows": 4096, "cols": 14336, "transposed": False, "act": "gelu_tanh", "bias": True, "residual": False, "out": "bf16"},
        # the logits of a tied embedding table with an odd vocabulary, and their gradients
        {"name": "linear train head", "op": "linear", "train": True, "x": "bf16", "tokens": 1001, "rows": 50001, "cols": 4096, "transposed": True, "act": "none", "bias": False, "residual": False, "out": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "linear", "linear"])
    if op == "norm":
        rows, dim = _log(rng, 1, 16384), _log(rng, 64, 8192)
        rows = max(1, min(rows, (8192 * 7168) // dim))
        train = rng.random() < 0.5
        return {"op": op, "train": train, "fp8": not train and rng.random() < 0.7, "rows": rows, "dim": dim, "residual": rng.random() < 0.6, "type": rng.choice(["bf16", "bf16", "f32"])}
    if op == "route":
        top, dim = rng.randint(1, 8), _log(rng, 64, 7168)
        kind = rng.choice(["bf16", "bf16", "f32"])
        tokens = max(1, min(_log(rng, 1, 16384), (32768 * 7168) // (top * dim)))
        return {"op": op, "train": rng.random() < 0.5, "tokens": tokens, "top": top, "experts": rng.randint(2, 256), "dim": dim, "dropped": rng.choice([0.0, 0.0, 0.1, 0.5]), "type": kind}
    transposed = rng.random() < 0.4
    cols = 16 * _log(rng, 2, 900)
    rows = _log(rng, 32, 50001) if transposed else 16 * _log(rng, 2, 448) + rng.choice([0, 0, 1, 8])
    tokens = _log(rng, 1, 8192)
    train = rng.random() < 0.5
    x = "bf16" if train or (not transposed and rows % 16) else rng.choice(["bf16", "fp8"])
    tokens = max(1, min(tokens, (2051 * 4096 * 14336) // (2 * rows * cols)))
    return {"op": op, "train": train, "x": x, "tokens": tokens, "rows": rows, "cols": cols, "transposed": transposed, "act": rng.choice(["none", "none", "silu", "gelu_tanh"]), "bias": rng.random() < 0.5, "residual": rng.random() < 0.4, "out": rng.choice(["bf16", "bf16", "f32"])}


def _type(case, key="type"):
    return torch.bfloat16 if case[key] == "bf16" else torch.float32


def _inner_outer(case):
    """The widths of the product's rows and of its result."""
    return (case["cols"], case["rows"]) if case["transposed"] else (case["rows"], case["cols"])


def work(case):
    op = case["op"]
    if op == "norm":
        n, d = case["rows"] * case["dim"], case["dim"]
        size = 2 if case["type"] == "bf16" else 4
        b = n * size * (3 if case["residual"] else 1) + 4 * d
        b += n + 4 * case["rows"] * _blocks(d) if case["fp8"] else n * size
        if case["train"]:
            b += 3 * n * size + 8 * d  # dy and the summed rows again, dx; the weight and its gradient
        return {"bytes": b, "flops": (14 if case["train"] else 5) * n}
    if op == "route":
        t, k, d = case["tokens"], case["top"], case["dim"]
        size = 2 if case["type"] == "bf16" else 4
        kept = int(t * k * (1.0 - case["dropped"]))
        # ids, order and places; the tokens' rows once and the experts' rows written; those read with weights, the result
        b = t * k * (8 + 4 + 4) + size * d * (t + t * k) + size * d * (kept + t) + 4 * t * k
        if case["train"]:
            # dy and the experts' rows read, their gradients written, with the weights'; the rows' gradients read, the tokens' written
            b += size * d * (t + kept + t * k) + 8 * t * k + size * d * (kept + t)
        return {"bytes": b, "flops": (6 if case["train"] else 2) * kept * d}
    t, r, c = case["tokens"], case["rows"], case["cols"]
    inner, outer = _inner_outer(case)
    y = t * outer * (2 if case["out"] == "bf16" else 4)
    b = r * c + 4 * _blocks(r) * _blocks(c) + t * inner * (2 if case["x"] == "bf16" else 1) + y
    b += (4 * outer if case["bias"] else 0) + (2 * t * outer if case["residual"] else 0)
    if case["train"]:
        b += y + r * c + 4 * _blocks(r) * _blocks(c) + 2 * 2 * t * inner + 4 * r * c + (4 * outer if case["bias"] else 0)
    return {"bytes": b, "flops": (6 if case["train"] else 2) * t * r * c}


# ---------------------------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _weight(g, rows, cols):
    """E4M3 codes of normal weights whose block scales put about 4.2 sigma at 448, and those scales."""
    w = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.bfloat16).mul_(107.0).clamp_(-448.0, 448.0)
    codes = w.to(torch.float8_e4m3fn).view(torch.uint8)
    scale = (torch.rand((_blocks(rows), _blocks(cols)), generator=g, device="cuda") + 0.5) * 1.9e-4
    return codes, scale


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)

    def normal(*shape, dtype=torch.bfloat16, by=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(by)

    if op == "norm":
        shape, dtype = (case["rows"], case["dim"]), _type(case)
        s["x"] = normal(*shape, dtype=dtype)
        s["residual"] = normal(*shape, dtype=dtype, by=3.0) if case["residual"] else None
        s["weight"] = normal(case["dim"], dtype=torch.float32, by=0.2) + 1.0
        if case["train"]:
            s["dy"] = normal(*shape, dtype=dtype, by=0.1)
            # what reaches the summed rows past the norm
            s["d_total"] = normal(*shape, dtype=dtype, by=0.1) if case["residual"] else None
    elif op == "route":
        t, k, e, d, dtype = case["tokens"], case["top"], case["experts"], case["dim"], _type(case)
        # each token's own experts, some liked better; a dropped choice is -1
        liked = torch.rand(e, generator=g, device="cuda") * 2.0
        pick = torch.rand(t, max(e, k), generator=g, device="cuda")
        pick[:, :e] += liked
        ids = pick.argsort(1, descending=True)[:, :k].int() % e
        s["ids"] = torch.where(torch.rand(t, k, generator=g, device="cuda") < case["dropped"], torch.full_like(ids, -1), ids)
        w = torch.rand(t, k, generator=g, device="cuda") + 0.05
        s["weight"] = w / w.sum(1, keepdim=True)
        s["x"] = normal(t, d, dtype=dtype)
        s["rows"] = normal(t * k, d, dtype=dtype)  # what the experts made of their rows
        s["residual"] = normal(t, d, dtype=dtype)
        if case["train"]:
            s["dy"] = normal(t, d, dtype=dtype, by=0.1)
            s["d_rows"] = normal(t * k, d, dtype=dtype, by=0.1)  # and what came back through them
    else:
        t = case["tokens"]
        inner, outer = _inner_outer(case)
        s["codes"], s["scale"] = _weight(g, case["rows"], case["cols"])
        s["x"] = normal(t, inner)
        s["x_scale"] = None
        if case["x"] == "fp8":
            x = s["x"].float().mul_(107.0).clamp_(-448.0, 448.0)
            s["x"] = x.to(torch.float8_e4m3fn)
            s["x_scale"] = (torch.rand(t, _blocks(inner), generator=g, device="cuda") + 0.5) / 107.0
        s["bias"] = normal(outer, dtype=torch.float32, by=0.5) if case["bias"] else None
        s["residual"] = normal(t, outer) if case["residual"] else None
        if case["train"]:
            s["dy"] = normal(t, outer, dtype=_type(case, "out"), by=0.1)
    return s


# ---------------------------------------------------------------------------------------------------------
# plain forms


def _norm(s):
    x, w, dim = s["x"], s["weight"], s["dim"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
    f = x.float()
    rstd = 1.0 / torch.sqrt((f * f).sum(1, keepdim=True) / dim + EPS)
    y = f * rstd * w
    out = {"total": x} if s["residual"] is not None else {}
    if s["fp8"]:
        n = _blocks(dim)
        groups = torch.zeros(y.shape[0], n * TILE, device="cuda")
        groups[:, :dim] = y
        groups = groups.view(-1, n, TILE)
        top = groups.abs().amax(2)
        scale = torch.where(top == 0.0, torch.ones_like(top), top / 448.0)
        codes = (groups / scale[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        return {**out, "codes": codes.view(-1, n * TILE)[:, :dim].contiguous(), "scale": scale}
    out["y"] = y.to(x.dtype)
    if s["train"]:
        dy, hat = s["dy"].float(), f * rstd
        g = dy * w
        dx = rstd * (g - hat * ((g * hat).sum(1, keepdim=True) / dim))
        if s["d_total"] is not None:
            dx = dx + s["d_total"].float()
        out["dx"] = dx.to(x.dtype)
        out["d_weight"] = (dy * hat).sum(0)
    return out


def _route(s):
    t, k, e, dtype = s["tokens"], s["top"], s["experts"], s["x"].dtype
    ids = s["ids"].reshape(-1).long()
    there = (ids >= 0) & (ids < e)
    key = torch.where(there, ids, torch.full_like(ids, e))
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(t * k, device="cuda")
    n = (key[:, None] < torch.arange(1, e + 1, device="cuda")).sum(0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), n])
    place = torch.where(there, place, torch.full_like(place, -1)).view(t, k)
    took = torch.arange(t * k, device="cuda")[:, None] < offsets[e]
    rows = torch.where(took, s["x"][order // k], torch.zeros((), dtype=dtype, device="cuda"))
    mine, w = place.clamp(min=0), torch.where(place >= 0, s["weight"], torch.zeros_like(s["weight"]))

    def joined(v, w, more=None):
        got = torch.where((place >= 0)[:, :, None], v[mine].float(), torch.zeros((), device="cuda"))
        got = (got * w[:, :, None]).sum(1) if w is not None else got.sum(1)
        return (got if more is None else got + more.float()).to(dtype)

    out = {"offsets": offsets.int(), "place": place.int(), "rows": rows, "y": joined(s["rows"], w, s["residual"])}
    if s["train"]:
        dy = s["dy"].float()
        token = order // k
        at = w.reshape(-1)[order]
        out["d_rows"] = torch.where(took, dy[token] * at[:, None], torch.zeros((), device="cuda")).to(dtype)
        dot = (dy[token] * s["rows"].float()).sum(1)
        d_weight = torch.zeros(t * k, device="cuda")
        d_weight[order] = torch.where(took[:, 0], dot, torch.zeros_like(dot))
        out["d_weight"] = d_weight.view(t, k)
        out["dx"] = joined(s["d_rows"], None)
    return out


def _spread(scale, rows, cols):
    return scale.repeat_interleave(TILE, 0)[:rows].repeat_interleave(TILE, 1)[:, :cols]


def _gate(z, act):
    """The factor of z in its activation, and the derivative of their product."""
    c = z if act == "silu" else GELU * (z + 0.044715 * z * z * z)
    dc = torch.ones_like(z) if act == "silu" else GELU * (1.0 + 3.0 * 0.044715 * z * z)
    sig = 1.0 / (1.0 + torch.exp(-c))
    return sig, sig + z * sig * (1.0 - sig) * dc


def _linear(s):
    t, (inner, outer) = s["tokens"], _inner_outer(s)
    w = s["codes"].view(torch.float8_e4m3fn).float() * _spread(s["scale"], s["rows"], s["cols"])
    w = w.t() if s["transposed"] else w
    x = s["x"].float()
    if s["x_scale"] is not None:
        x = x * s["x_scale"].repeat_interleave(TILE, 1)[:, :inner]
    z = x @ w
    if s["bias"] is not None:
        z = z + s["bias"]
    sig, slope = _gate(z, s["act"]) if s["act"] != "none" else (None, None)
    y = z if sig is None else z * sig
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(_type(s, "out"))}
    if s["train"]:
        dz = s["dy"].float() if slope is None else s["dy"].float() * slope
        out["dx"] = (dz @ w.t()).bfloat16()
        out["d_weight"] = dz.t() @ x if s["transposed"] else x.t() @ dz
        if s["bias"] is not None:
            out["d_bias"] = dz.sum(0)
    return out


def _run_own(s):
    from blockwise_fp8_zero_fold_gb300 import ops

    if s["op"] == "norm":
        if s["fp8"]:
            got = ops.rms_norm_fp8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
            return {"codes": got[0], "scale": got[1], **({"total": got[2]} if len(got) > 2 else {})}
        y = ops.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        y, total = y if s["residual"] is not None else (y, s["x"])
        out = {"y": y} if s["residual"] is None else {"y": y, "total": total}
        if s["train"]:
            out["dx"], out["d_weight"] = ops.rms_norm_grad(s["dy"], total, s["weight"], eps=EPS, d_total=s["d_total"])
        return out
    if s["op"] == "route":
        r = ops.route(s["ids"], s["experts"])
        out = {"offsets": r.offsets, "place": r.place, "rows": ops.dispatch(s["x"], r)}
        out["y"] = ops.combine(s["rows"], r, s["weight"], residual=s["residual"])
        if s["train"]:
            out["d_rows"], out["d_weight"] = ops.combine_grad(s["dy"], s["rows"], r, s["weight"])
            out["dx"] = ops.dispatch_grad(s["d_rows"], r)
        return out
    act = None if s["act"] == "none" else s["act"]
    keep = s["train"] and act is not None
    y = ops.linear(s["x"], s["codes"], s["scale"], x_scale=s["x_scale"], bias=s["bias"], activation=act, residual=s["residual"], transposed=s["transposed"], dtype=_type(s, "out"), save=keep)
    y, pre = y if keep else (y, None)
    if not s["train"]:
        return {"y": y}
    dx, d_weight, d_bias = ops.linear_grad(s["dy"], s["x"], s["codes"], s["scale"], activation=act, pre=pre, transposed=s["transposed"], bias=s["bias"] is not None)
    return {"y": y, "dx": dx, "d_weight": d_weight, **({"d_bias": d_bias} if s["bias"] is not None else {})}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "route": _route, "linear": _linear}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _values():
    """What each of the 256 E4M3 codes stands for: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    got = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if c & 127 == 127 else (m / 8 * 2.0**-6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        got.append(-v if c & 128 else v)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _exact_norm(s):
    x, w, d = s["x"].double(), s["weight"].double(), s["dim"]
    out = {}
    if s["residual"] is not None:
        # the norm is that of the summed rows as they are kept, in the rows' type
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
        out["total"] = x
    norm = torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x / norm * w
    if s["fp8"]:
        top = torch.stack([y[:, i : i + TILE].abs().amax(1) for i in range(0, d, TILE)], 1)
        scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
        column = torch.arange(d, device="cuda") // TILE
        return {**out, "codes": y / scale[:, column], "scale": scale}
    out["y"] = y
    if s["train"]:
        # y_j = x_j w_j / norm, and d norm / d x_i = x_i / (d norm)
        dy = s["dy"].double()
        inner = (dy * w * x).sum(1, keepdim=True)
        out["dx"] = dy * w / norm - x * inner / (d * norm**3)
        if s["d_total"] is not None:
            out["dx"] += s["d_total"].double()
        out["d_weight"] = (dy * x / norm).sum(0)
    return out


def _exact_route(s):
    t, k, e = s["tokens"], s["top"], s["experts"]
    ids = s["ids"].cpu().tolist()
    lists = [[] for _ in range(e)]
    for token, mine in enumerate(ids):
        for j, expert in enumerate(mine):
            if 0 <= expert < e:
                lists[expert].append((token, j))
    ends, order = [0], []
    for some in lists:
        order += some
        ends.append(len(order))
    place = torch.full((t, k), -1, dtype=torch.int32)
    n = len(order)
    tokens = torch.tensor([a for a, _ in order], dtype=torch.int64, device="cuda")
    slots = torch.tensor([b for _, b in order], dtype=torch.int64, device="cuda")
    place[tokens.cpu(), slots.cpu()] = torch.arange(n, dtype=torch.int32)
    w = s["weight"].double()
    rows = torch.zeros(t * k, s["dim"], dtype=torch.float64, device="cuda")
    rows[:n] = s["x"].double()[tokens]
    y = s["residual"].double()
    y.index_put_((tokens,), s["rows"][:n].double() * w[tokens, slots][:, None], accumulate=True)
    out = {"offsets": torch.tensor(ends, dtype=torch.int32), "place": place, "rows": rows, "y": y}
    if s["train"]:
        dy = s["dy"].double()
        out["d_rows"] = torch.zeros_like(rows)
        out["d_rows"][:n] = dy[tokens] * w[tokens, slots][:, None]
        out["d_weight"] = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        out["d_weight"][tokens, slots] = torch.einsum("nd,nd->n", dy[tokens], s["rows"][:n].double())
        out["dx"] = torch.zeros(t, s["dim"], dtype=torch.float64, device="cuda")
        out["dx"].index_put_((tokens,), s["d_rows"][:n].double(), accumulate=True)
    return out


def _exact_linear(s):
    r, c = s["rows"], s["cols"]
    at_r, at_c = torch.arange(r, device="cuda") // TILE, torch.arange(c, device="cuda") // TILE
    w = _values()[s["codes"].int()].mul_(s["scale"].double()[at_r][:, at_c])
    w = w.T if s["transposed"] else w
    x = s["x"].double()
    if s["x_scale"] is not None:
        x *= s["x_scale"].double()[:, torch.arange(x.shape[1], device="cuda") // TILE]
    z = x @ w
    if s["bias"] is not None:
        z += s["bias"].double()
    slope = None
    if s["act"] == "silu":
        y = z * torch.sigmoid(z)
        slope = torch.sigmoid(z) * (1 + z * torch.sigmoid(-z))
    elif s["act"] == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        u = torch.tanh(a * (z + 0.044715 * z**3))
        y = 0.5 * z * (1 + u)
        slope = 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * a * (1 + 3 * 0.044715 * z * z)
    else:
        y = z.clone()
    if s["residual"] is not None:
        y += s["residual"].double()
    out = {"y": y}
    if s["train"]:
        dz = s["dy"].double() if slope is None else s["dy"].double() * slope
        out["dx"] = dz @ w.T
        out["d_weight"] = dz.T @ x if s["transposed"] else x.T @ dz
        if s["bias"] is not None:
            out["d_bias"] = dz.sum(0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "linear": _exact_linear}[case["op"]](s)
