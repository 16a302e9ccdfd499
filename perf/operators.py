"""What is timed of the model operators that run next to the optimizer step, and their plain forms.

Three operators, which take the FP8 weights and the 128x128 block scales as the optimizer writes them and hand
back the FP32 weight gradients that its next step reads:

* ``embed`` / ``embed_grad``: rows of an FP8 embedding table, scaled; and the table's gradient.
* ``ffn``: the gated feed-forward block of each expert on its own tokens, ``(silu(x Wg) * (x Wu)) Wd``, and with
  ``train`` its backward pass too (dx and both weight gradients).
* ``distill``: the distillation loss against a teacher's top logits, and with ``train`` the logits' gradient.

``run`` computes them in elementary torch operations in 32 bits, or with ``own`` through the package's entry
points.  ``exact`` is the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TILE = 128  # a scale covers 128 x 128 codes


def _blocks(n):
    return -(-n // TILE)


# ---------------------------------------------------------------------------------------------------------
# cases


def listed():
    return [
        # one token of a dense block of the repository's dense configuration: serving, bound by the codes it reads
        {"name": "ffn decode dense", "op": "ffn", "train": False, "experts": 1, "active": 1, "hidden": 4096, "inner": 14336, "tokens": 1},
        # one decode step of a batch over the repository's 32 experts: about two tokens on each of 27 of them
        {"name": "ffn decode experts", "op": "ffn", "train": False, "experts": 32, "active": 27, "hidden": 7168, "inner": 2048, "tokens": 61},
        # a prefill chunk over the experts, forward only, one expert without a token
        {"name": "ffn prefill experts", "op": "ffn", "train": False, "experts": 32, "active": 31, "hidden": 7168, "inner": 2048, "tokens": 5003},
        # a training micro-batch over the experts, forward and backward
        {"name": "ffn train experts", "op": "ffn", "train": True, "experts": 32, "active": 31, "hidden": 7168, "inner": 2048, "tokens": 8192},
        # a training micro-batch of the dense block
        {"name": "ffn train dense", "op": "ffn", "train": True, "experts": 1, "active": 1, "hidden": 4096, "inner": 14336, "tokens": 2051},
        # a small model's training step: a width that ends inside a 128-block, few tokens
        {"name": "ffn train small", "op": "ffn", "train": True, "experts": 4, "active": 3, "hidden": 304, "inner": 256, "tokens": 333},
        # the tokens of one decode step of a batch: latency
        {"name": "embed decode", "op": "embed", "vocab": 131072, "dim": 7168, "tokens": 32, "alpha": 1.0, "out": "bf16"},
        # the tokens of a prefill or training batch, scaled by sqrt(dim)
        {"name": "embed batch", "op": "embed", "vocab": 131072, "dim": 7168, "tokens": 16384, "alpha": 84.664, "out": "bf16"},
        # the table's gradient for a training batch: few rows have tokens, the commonest have hundreds
        {"name": "embed grad", "op": "embed_grad", "vocab": 131072, "dim": 4096, "tokens": 16384, "alpha": 64.0, "grad": "bf16"},
        # evaluation of a few rows: the loss alone
        {"name": "distill eval", "op": "distill", "train": False, "rows": 16, "vocab": 32000, "top": 16, "temperature": 1.0, "logits": "f32"},
        # a training micro-batch with a large vocabulary
        {"name": "distill train", "op": "distill", "train": True, "rows": 4096, "vocab": 131072, "top": 64, "temperature": 1.0, "logits": "bf16"},
        # FP32 logits of a vocabulary whose rows are not aligned, softened
        {"name": "distill train ragged", "op": "distill", "train": True, "rows": 1001, "vocab": 50001, "top": 32, "temperature": 2.0, "logits": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn", "embed", "embed_grad", "distill", "distill"])
    if op == "ffn":
        experts = rng.choice([1, 1, rng.randint(2, 32), rng.randint(2, 32)])
        hidden = 16 * _log(rng, 8, 448)
        inner = min(TILE * _log(rng, 1, 112), TILE * max(1, (32 * 7168 * 2048) // (experts * hidden * TILE)))
        train = rng.random() < 0.5
        tokens = _log(rng, 1, 8192)
        tokens = max(1, min(tokens, int(8192 * 7168 * 2048 / (hidden * inner))))
        return {"op": op, "train": train, "experts": experts, "active": rng.randint((experts + 1) // 2, experts), "hidden": hidden, "inner": inner, "tokens": tokens}
    if op == "embed":
        return {"op": op, "vocab": _log(rng, 1000, 131072), "dim": _log(rng, 64, 7168), "tokens": _log(rng, 1, 16384), "alpha": round(rng.uniform(0.5, 90.0), 3), "out": rng.choice(["bf16", "bf16", "f32"])}
    if op == "embed_grad":
        vocab = _log(rng, 1000, 131072)
        dim = min(_log(rng, 64, 7168), (131072 * 4096) // vocab)
        return {"op": op, "vocab": vocab, "dim": dim, "tokens": _log(rng, 1, 16384), "alpha": round(rng.uniform(0.5, 90.0), 3), "grad": rng.choice(["bf16", "bf16", "f32"])}
    vocab = _log(rng, 1000, 131072)
    rows = max(1, min(_log(rng, 1, 8192), (4096 * 131072) // (2 * vocab)))
    return {"op": op, "train": rng.random() < 0.7, "rows": rows, "vocab": vocab, "top": _log(rng, 1, 128), "temperature": rng.choice([1.0, 1.0, 2.0, 4.0]), "logits": rng.choice(["bf16", "f32"])}


def _loads(case):
    """Tokens of each expert that has some, largest first: between once and four times the smallest share."""
    n = min(case["active"], case["tokens"])
    share = [1.0 + 3.0 * i / n for i in range(n, 0, -1)]
    got = [max(1, int(case["tokens"] * s / sum(share))) for s in share]
    i = 0
    while sum(got) != case["tokens"]:
        step = 1 if sum(got) < case["tokens"] else -1
        if got[i % n] + step >= 1:
            got[i % n] += step
        i += 1
    return got


def work(case):
    op = case["op"]
    if op == "ffn":
        t, h, f = case["tokens"], case["hidden"], case["inner"]
        n = len(_loads(case))
        codes = n * 3 * h * f
        scales = 4 * n * (_blocks(h) * _blocks(2 * f) + _blocks(f) * _blocks(h))
        b = codes + scales + 2 * t * h * 2
        if case["train"]:
            # read x and dy again with the codes, write dx and every expert's two weight gradients
            b += codes + scales + 3 * t * h * 2 + 4 * case["experts"] * 3 * h * f
        return {"bytes": b, "flops": (18 if case["train"] else 6) * t * h * f}
    if op == "embed":
        t, d = case["tokens"], case["dim"]
        return {"bytes": t * (8 + d + 4 * _blocks(d) + d * (2 if case["out"] == "bf16" else 4)), "flops": 2 * t * d}
    if op == "embed_grad":
        t, d = case["tokens"], case["dim"]
        return {"bytes": t * (8 + d * (2 if case["grad"] == "bf16" else 4)) + 4 * case["vocab"] * d, "flops": 2 * t * d}
    n = case["rows"] * case["vocab"] * (2 if case["logits"] == "bf16" else 4)
    return {"bytes": n * (2 if case["train"] else 1) + case["rows"] * (8 * case["top"] + 8), "flops": (6 if case["train"] else 4) * case["rows"] * case["vocab"]}


# ---------------------------------------------------------------------------------------------------------
# inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _weight(g, *shape):
    """E4M3 codes of normal weights whose block scales put about 4.2 sigma at 448, and those scales."""
    w = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16).mul_(107.0).clamp_(-448.0, 448.0)
    codes = w.to(torch.float8_e4m3fn).view(torch.uint8)
    grid = shape[:-2] + (_blocks(shape[-2]), _blocks(shape[-1]))
    scale = (torch.rand(grid, generator=g, device="cuda") + 0.5) * 1.9e-4
    return codes, scale


def _zipf(g, n, vocab):
    """Token ids with frequency about 1 / rank; a few -1 (no token)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab + 1.0)).long().clamp_(1, vocab) - 1
    ids = (rank * 7919 + 13) % vocab
    none = torch.rand(n, generator=g, device="cuda") < 0.01
    return torch.where(none, torch.full_like(ids, -1), ids)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "ffn":
        e, h, f, t = case["experts"], case["hidden"], case["inner"], case["tokens"]
        order = torch.randperm(e, generator=torch.Generator().manual_seed(seed)).tolist()
        counts = [0] * e
        for i, n in enumerate(_loads(case)):
            counts[order[i]] = n
        ends = np.concatenate([[0], np.cumsum(counts)])
        s["counts"] = counts
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["gate_up"], s["gate_up_scale"] = _weight(g, e, h, 2 * f)
        s["down"], s["down_scale"] = _weight(g, e, f, h)
        s["x"] = torch.randn(t, h, generator=g, device="cuda", dtype=torch.bfloat16)
        if case["train"]:
            # loss-scaled gradients of the block's output
            s["dy"] = torch.randn(t, h, generator=g, device="cuda").mul_(1024 * 1e-4).bfloat16()
    elif op == "embed":
        s["table"], s["scale"] = _weight(g, case["vocab"], case["dim"])
        s["ids"] = _zipf(g, case["tokens"], case["vocab"])
    elif op == "embed_grad":
        s["ids"] = _zipf(g, case["tokens"], case["vocab"])
        s["dy"] = torch.randn(case["tokens"], case["dim"], generator=g, device="cuda").mul_(1024 * 1e-4)
        s["dy"] = s["dy"].bfloat16() if case["grad"] == "bf16" else s["dy"]
    else:
        r, v, k = case["rows"], case["vocab"], case["top"]
        dtype = torch.bfloat16 if case["logits"] == "bf16" else torch.float32
        s["z"] = torch.randn(r, v, generator=g, device="cuda", dtype=dtype).mul_(2.5)
        # distinct ids in no order; logits from the highest down; some rows give fewer than k (-1 and -inf)
        ids = torch.randint(1, v // k + 1, (r, k), generator=g, device="cuda").cumsum(1) - 1
        ids = ids.gather(1, torch.rand(r, k, generator=g, device="cuda").argsort(1))
        logits = (torch.randn(r, k, generator=g, device="cuda") * 3 + 8).sort(1, descending=True).values
        fewer = torch.randint(1, 2 * k + 1, (r, 1), generator=g, device="cuda")
        gone = torch.arange(k, device="cuda") >= fewer
        s["ids"] = torch.where(gone, torch.full_like(ids, -1), ids).int()
        s["teacher"] = torch.where(gone, torch.full_like(logits, -math.inf), logits)
        s["weight"] = (torch.rand(r, generator=g, device="cuda") > 0.1).float() * (1024.0 / r)
    return s


# ---------------------------------------------------------------------------------------------------------
# plain forms


def _decode(codes, scale):
    w = codes.view(torch.float8_e4m3fn).float()
    r, c = codes.shape[-2:]
    return w * scale.repeat_interleave(TILE, -2)[..., :r, :].repeat_interleave(TILE, -1)[..., :c]


def _ffn(s):
    x, f = s["x"].float(), s["inner"]
    gate_up, down = _decode(s["gate_up"], s["gate_up_scale"]), _decode(s["down"], s["down_scale"])
    # token t is row `at` of expert `of`: every expert's tokens padded to the longest list
    many = max(s["counts"])
    t = torch.arange(x.shape[0], device="cuda")
    of = torch.searchsorted(s["offsets"][1:].contiguous(), t.int(), right=True)
    at = t - s["offsets"][of]

    def spread(v):
        out = torch.zeros(s["experts"], many, v.shape[1], device="cuda")
        out[of, at] = v
        return out

    xs = spread(x)
    gu = torch.bmm(xs, gate_up)
    gate, up = gu[..., :f], gu[..., f:]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sig
    hid = act * up
    y = torch.bmm(hid, down)[of, at].bfloat16()
    if not s["train"]:
        return {"y": y}
    dys = spread(s["dy"].float())
    dhid = torch.bmm(dys, down.transpose(1, 2))
    d_down = torch.bmm(hid.transpose(1, 2), dys)
    dgu = torch.cat([dhid * up * sig * (1.0 + gate * (1.0 - sig)), dhid * act], 2)
    d_gate_up = torch.bmm(xs.transpose(1, 2), dgu)
    dx = torch.bmm(dgu, gate_up.transpose(1, 2))[of, at].bfloat16()
    return {"y": y, "dx": dx, "d_gate_up": d_gate_up, "d_down": d_down}


def _embed(s):
    ids = s["ids"]
    there = (ids >= 0)[:, None]
    row = ids.clamp(min=0)
    scale = s["scale"][row // TILE].repeat_interleave(TILE, 1)[:, : s["dim"]]
    out = s["table"][row].view(torch.float8_e4m3fn).float() * scale * s["alpha"]
    return torch.where(there, out, torch.zeros_like(out)).to(torch.bfloat16 if s["out"] == "bf16" else torch.float32)


def _embed_grad(s):
    there = s["ids"] >= 0
    d = torch.zeros(s["vocab"] + 1, s["dim"], device="cuda")
    d.index_add_(0, torch.where(there, s["ids"], torch.full_like(s["ids"], s["vocab"])), s["dy"].float() * s["alpha"])
    return d[: s["vocab"]]


def _distill(s):
    tau = s["temperature"]
    z = s["z"].float() / tau
    top = z.amax(1, keepdim=True)
    ex = torch.exp(z - top)
    total = ex.sum(1, keepdim=True)
    there = (s["ids"] >= 0) & (s["teacher"] > -math.inf)
    ids = s["ids"].clamp(min=0).long()
    t = torch.where(there, s["teacher"] / tau, torch.full_like(s["teacher"], -math.inf))
    t = t - t.amax(1, keepdim=True)
    p = torch.exp(t)
    mass = p.sum(1, keepdim=True)
    p = p / mass
    log_q = z.gather(1, ids) - top - torch.log(total)
    each = torch.where(there, p * (t - torch.log(mass) - log_q), torch.zeros_like(p))
    used = s["weight"] != 0
    loss = torch.where(used, tau * tau * each.sum(1), torch.zeros_like(s["weight"]))
    if not s["train"]:
        return {"loss": loss}
    d = ex / total
    d.scatter_add_(1, ids, -p)
    d = d * (tau * s["weight"])[:, None]
    return {"loss": loss, "dlogits": d.to(s["z"].dtype)}


def _run_own(s):
    from blockwise_fp8_zero_fold_gb300 import ops

    op = s["op"]
    if op == "ffn":
        w = (s["gate_up"], s["gate_up_scale"], s["down"], s["down_scale"])
        if not s["train"]:
            return {"y": ops.ffn_forward(s["x"], *w, offsets=s["offsets"])}
        y, saved = ops.ffn_forward(s["x"], *w, offsets=s["offsets"], save=True)
        dx, d_gate_up, d_down = ops.ffn_backward(s["dy"], s["x"], saved, *w, offsets=s["offsets"])
        return {"y": y, "dx": dx, "d_gate_up": d_gate_up, "d_down": d_down}
    if op == "embed":
        return ops.embed(s["ids"], s["table"], s["scale"], alpha=s["alpha"], dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)
    if op == "embed_grad":
        return ops.embed_grad(s["ids"], s["dy"], s["vocab"], alpha=s["alpha"])
    if not s["train"]:
        return {"loss": ops.distill_loss(s["z"], s["ids"], s["teacher"], temperature=s["temperature"], row_weight=s["weight"])}
    loss, d = ops.distill_loss_grad(s["z"], s["ids"], s["teacher"], temperature=s["temperature"], row_weight=s["weight"])
    return {"loss": loss, "dlogits": d}


def run(state):
    if own:
        return _run_own(state)
    return {"ffn": _ffn, "embed": _embed, "embed_grad": _embed_grad, "distill": _distill}[state["op"]](state)


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


def _matrix(codes, scale, values):
    r, c = codes.shape
    at_r, at_c = torch.arange(r, device="cuda") // TILE, torch.arange(c, device="cuda") // TILE
    return values[codes.int()].mul_(scale.double()[at_r][:, at_c])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ffn":
        f, values = case["inner"], _values()
        x = s["x"].double()
        out = {"y": torch.zeros_like(x)}
        if case["train"]:
            out["dx"] = torch.zeros_like(x)
            out["d_gate_up"] = torch.zeros(s["gate_up"].shape, dtype=torch.float64, device="cuda")
            out["d_down"] = torch.zeros(s["down"].shape, dtype=torch.float64, device="cuda")
        lo = 0
        for e, n in enumerate(s["counts"]):
            mine, lo = slice(lo, lo + n), lo + n
            if not n:
                continue
            wgu = _matrix(s["gate_up"][e], s["gate_up_scale"][e], values)
            wd = _matrix(s["down"][e], s["down_scale"][e], values)
            g, u = x[mine] @ wgu[:, :f], x[mine] @ wgu[:, f:]
            a = g * torch.sigmoid(g)
            out["y"][mine] = (a * u) @ wd
            if not case["train"]:
                continue
            dy = s["dy"][mine].double()
            dh = dy @ wd.T
            out["d_down"][e] = (a * u).T @ dy
            # silu' = silu + sigmoid (1 - silu)
            dg, du = dh * u * (a + torch.sigmoid(g) * (1 - a)), dh * a
            out["d_gate_up"][e, :, :f], out["d_gate_up"][e, :, f:] = x[mine].T @ dg, x[mine].T @ du
            out["dx"][mine] = dg @ wgu[:, :f].T + du @ wgu[:, f:].T
        return out
    if op == "embed":
        values, ids = _values(), s["ids"].tolist()
        where = torch.tensor([i for i, t in enumerate(ids) if t >= 0], device="cuda")
        rows = torch.tensor([t for t in ids if t >= 0], device="cuda")
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        col = torch.arange(case["dim"], device="cuda") // TILE
        if len(rows):
            out[where] = values[s["table"][rows].int()] * s["scale"].double()[rows // TILE][:, col] * case["alpha"]
        return out
    if op == "embed_grad":
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        real = (s["ids"] >= 0).nonzero()[:, 0]
        out.index_put_((s["ids"][real],), s["dy"][real].double() * case["alpha"], accumulate=True)
        return out
    tau, v = case["temperature"], case["vocab"]
    losses, grads = [], []
    for lo in range(0, case["rows"], 512):
        some = slice(lo, lo + 512)
        log_q = torch.log_softmax(s["z"][some].double() / tau, 1)
        ids = s["ids"][some].long()
        there = ids >= 0
        log_p = torch.log_softmax(s["teacher"][some].double() / tau, 1)
        p = log_p.exp()
        # the teacher's distribution over the whole vocabulary, and a column beyond it for absent entries
        full = torch.zeros(len(ids), v + 1, dtype=torch.float64, device="cuda")
        full.scatter_(1, torch.where(there, ids, torch.full_like(ids, v)), p)
        full = full[:, :v]
        w = s["weight"][some].double()
        entropy = torch.where(there, p * log_p, torch.zeros_like(p)).sum(1)
        losses.append(torch.where(w != 0, tau * tau * (entropy - (full * log_q).sum(1)), torch.zeros_like(w)))
        if case["train"]:
            grads.append((log_q.exp() - full) * (tau * w)[:, None])
    out = {"loss": torch.cat(losses)}
    if case["train"]:
        out["dlogits"] = torch.cat(grads)
    return out
