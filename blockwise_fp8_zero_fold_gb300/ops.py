"""Model operators next to the optimizer step, on torch tensors.

They take the FP8 weights as the optimizer writes them -- row-major E4M3 codes
[E, R, C] (uint8) and FP32 block scales [E, ceil(R/128), ceil(C/128)]
(``ShardOptimizer.step``'s FP8 params and ``scale_views()``) -- and give back
FP32 [E, R, C] weight gradients, which ``ShardOptimizer.step`` reads:

  embed, embed_grad          rows of an FP8 table, and the table's gradient;
  ffn_forward, ffn_backward  the gated feed-forward block of each expert;
  distill_loss, distill_loss_grad
                             distillation from a teacher's top logits;
  rms_norm, rms_norm_fp8, rms_norm_grad
                             root-mean-square norm, the residual added first;
  route, dispatch, combine, dispatch_grad, combine_grad
                             tokens sorted by expert for ``ffn_forward``, and back;
  linear, linear_grad        a matrix product with bias, activation and residual.

Each is one call of libfp8z1.so's entry point of the same name (include/
fp8z1_ops.h has the formulas); this module checks the tensors, allocates
outputs and workspaces through torch and enqueues on ``stream`` (a
``torch.cuda.Stream``; None is torch's current stream).  With a ``stream``
that is not current, the outputs and workspaces are allocated as that stream's
and the outputs marked as used on the current one too; the order of the two
streams, and the inputs' memory until the work is done, are the caller's to
see to.  Tensors that do not fit raise ValueError, what the library refuses
raises Fp8z1Error.  Should a wait between the warps of a matrix product's or
the norm's gradient's kernel ever run out, what it belongs to is NaN
(``fp8z1.fp8z1_ffn_timeouts``, ``fp8z1_linear_timeouts`` and
``fp8z1_rms_norm_timeouts`` count them); the optimizer skips a step with such
gradients.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import fp8z1 as F

# The calls are small next to a few microseconds of kernel, so the checks here
# build no message, wrapper or list before something is wrong.

_TYPES = {torch.float32: F.F32, torch.bfloat16: F.BF16}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
_raw_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice


def _bad(what: str):
    raise ValueError(what)


def _begin(dev: int, stream):
    """(raw stream to enqueue on, the torch stream when it is not the current one)"""
    if dev < 0:
        _bad("the operators need CUDA tensors")
    if dev != _device():
        _bad("the tensors are not on the current device")
    now = _raw_stream(dev)
    if stream is None:
        return now, None
    if not isinstance(stream, torch.cuda.Stream) or stream.device.index != dev:
        _bad("stream must be a torch.cuda.Stream of the tensors' device")
    return stream.cuda_stream, stream if stream.cuda_stream != now else None


def _scratch(shape, dtype, dev: int, other):
    """Memory of one call, from the pool of the stream that the call is enqueued on.  (The current stream's
    pool may give out a block that the current stream's kernels still use: in order there, not on ``other``.)"""
    if other is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(other):
        return torch.empty(shape, dtype=dtype, device=dev)


def _new(shape, dtype, dev: int, other):
    """An output: the same, and kept until what the caller's stream does with it is done."""
    t = _scratch(shape, dtype, dev, other)
    if other is not None:
        t.record_stream(torch.cuda.current_stream(dev))
    return t


def _given(t: torch.Tensor, shape, dtype, dev: int, what: str):
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _bad(f"{what} must be {dtype} of shape {tuple(shape)} on the inputs' device")
    return t


def _same_device(dev: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            _bad("the tensors are on several devices")


def _rows(t: torch.Tensor, what: str) -> int:
    """The row stride of a 2-D tensor whose rows are dense and apart."""
    n, cols = t.shape
    ld, one = t.stride()
    if cols > 1 and one != 1:
        _bad(f"{what}'s rows must be dense")
    if n <= 1:  # a single row's stride is whatever it was cut from, and no alignment is asked of it
        return cols
    if ld < cols:
        _bad(f"{what}'s rows must not overlap")
    return ld


def _stride_of(t: torch.Tensor, dim: int, what: str) -> int:
    """The row stride of [*, dim]: contiguous, or 2-D of any row stride."""
    if t.is_contiguous():
        return dim
    if t.dim() != 2:
        _bad(f"{what} must be contiguous, or 2-D")
    return _rows(t, what)


def _fits(t: torch.Tensor, shape, dtype, dev: int, dim: int, what: str) -> int:
    """The row stride of a tensor that has to be of this shape, type and device."""
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _bad(f"{what} must be {dtype} of shape {tuple(shape)} on the inputs' device")
    return dim if t.is_contiguous() else _stride_of(t, dim, what)


def _fp8_weight(codes: torch.Tensor, scale: torch.Tensor, what: str):
    """(E, R, C) of an FP8 weight after checking its codes and block scales."""
    shape = codes.shape
    if len(shape) == 2:
        e, (r, c) = 1, shape
    elif len(shape) == 3:
        e, r, c = shape
    else:
        _bad(f"{what} must be [E, R, C] or [R, C] codes")
    if codes.dtype not in (torch.uint8, torch.float8_e4m3fn) or not codes.is_contiguous():
        _bad(f"{what} must be contiguous E4M3 codes (uint8)")
    if (scale.dtype != torch.float32 or scale.shape[-2:] != ((r + 127) // 128, (c + 127) // 128)
            or scale.numel() != e * ((r + 127) // 128) * ((c + 127) // 128) or not scale.is_contiguous()):
        _bad(f"{what}'s scales must be contiguous float32 [E, ceil(R/128), ceil(C/128)]")
    return e, r, c


# ---- embedding -----------------------------------------------------------------


def embed(ids: torch.Tensor, table: torch.Tensor, scale: torch.Tensor, *, alpha: float = 1.0,
          dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``alpha * table[ids]``, [*ids.shape, dim]; rows of ids outside the table are zero."""
    e, vocab, dim = _fp8_weight(table, scale, "the table")
    nbytes, kind = _ID_BYTES.get(ids.dtype), _TYPES.get(dtype)
    if e != 1:
        _bad("an embedding table is [vocab, dim]")
    if nbytes is None or not ids.is_contiguous():
        _bad("ids must be contiguous int32 or int64")
    if kind is None:
        _bad(f"no embedding output of {dtype}")
    dev = ids.get_device()
    raw, other = _begin(dev, stream)
    _same_device(dev, table, scale)
    shape = ids.shape + (dim,)
    ld = dim
    if out is None:
        out = _new(shape, dtype, dev, other)
    else:
        _given(out, shape, dtype, dev, "out")
        if out.dim() == 2:
            ld = _rows(out, "out")
        elif not out.is_contiguous():
            _bad("out must be contiguous")
    F.fp8z1_embed(vocab, dim, table, scale, ids, nbytes, ids.numel(), alpha, out, kind, ld, raw)
    return out


def embed_grad(ids: torch.Tensor, dy: torch.Tensor, vocab: int, *, alpha: float = 1.0,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The FP32 [vocab, dim] gradient of ``embed``'s table from ``dy``
    [*ids.shape, dim] (every row written; repeatable bit for bit)."""
    nbytes, kind = _ID_BYTES.get(ids.dtype), _TYPES.get(dy.dtype)
    if nbytes is None or not ids.is_contiguous():
        _bad("ids must be contiguous int32 or int64")
    if kind is None:
        _bad(f"no gradient of {dy.dtype}")
    if dy.dim() < 1 or dy.shape[:-1] != ids.shape:
        _bad("dy must be [*ids.shape, dim]")
    dim, n = dy.shape[-1], ids.numel()
    dev = ids.get_device()
    raw, other = _begin(dev, stream)
    _same_device(dev, dy)
    ld = dim
    if dy.dim() == 2:
        ld = _rows(dy, "dy")
    elif not dy.is_contiguous():
        _bad("dy must be contiguous")
    if out is None:
        out = _new((vocab, dim), torch.float32, dev, other)
    elif not _given(out, (vocab, dim), torch.float32, dev, "out").is_contiguous():
        _bad("out must be contiguous")
    ws = _scratch(F.fp8z1_embed_grad_workspace(vocab, dim, n), torch.uint8, dev, other)
    F.fp8z1_embed_grad(vocab, dim, ids, nbytes, n, alpha, dy, kind, ld, out, ws, raw)
    return out


# ---- gated feed-forward block -----------------------------------------------------


def _ffn_dims(x, gate_up, gate_up_scale, down, down_scale, offsets):
    e, h, f2 = _fp8_weight(gate_up, gate_up_scale, "gate_up")
    e2, f, h2 = _fp8_weight(down, down_scale, "down")
    if e != e2 or h != h2 or f2 != 2 * f:
        _bad(f"gate_up [{e}, {h}, {f2}] and down [{e2}, {f}, {h2}] do not match: [E, hidden, 2 inner] and "
             "[E, inner, hidden]")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != h:
        _bad(f"x must be bfloat16 [tokens, {h}]")
    if offsets is None:
        if e != 1:
            _bad("several experts need offsets")
    elif offsets.dtype != torch.int32 or offsets.shape != (e + 1,) or not offsets.is_contiguous():
        _bad(f"offsets must be contiguous int32 [{e + 1}]")
    return F.fp8z1_ffn_dims(x.shape[0], h, f, e)


def ffn_forward(x: torch.Tensor, gate_up: torch.Tensor, gate_up_scale: torch.Tensor, down: torch.Tensor,
                down_scale: torch.Tensor, *, offsets: Optional[torch.Tensor] = None, save: bool = False,
                out: Optional[torch.Tensor] = None, stream=None):
    """``(silu(x Wg) * (x Wu)) Wd`` of each expert on its rows of ``x``
    (bfloat16 [tokens, hidden], grouped by expert: expert e has rows
    [offsets[e], offsets[e + 1])).  With ``save`` also the buffer that
    ``ffn_backward`` reads: (y, saved)."""
    dims = _ffn_dims(x, gate_up, gate_up_scale, down, down_scale, offsets)
    dev = x.get_device()
    raw, other = _begin(dev, stream)
    _same_device(dev, gate_up, gate_up_scale, down, down_scale, offsets)
    if out is None:
        out = _new(x.shape, torch.bfloat16, dev, other)
    else:
        _given(out, x.shape, torch.bfloat16, dev, "out")
    saved_bytes, forward_bytes, _ = F.fp8z1_ffn_sizes(dims)
    saved = _new(saved_bytes, torch.uint8, dev, other) if save else None
    ws = _scratch(forward_bytes, torch.uint8, dev, other)
    F.fp8z1_ffn_forward(dims, x, _rows(x, "x"), offsets, gate_up, gate_up_scale, down, down_scale, out,
                        _rows(out, "out"), saved, ws, raw)
    return (out, saved) if save else out


def ffn_backward(dy: torch.Tensor, x: torch.Tensor, saved: torch.Tensor, gate_up: torch.Tensor,
                 gate_up_scale: torch.Tensor, down: torch.Tensor, down_scale: torch.Tensor, *,
                 offsets: Optional[torch.Tensor] = None, need_dx: bool = True,
                 d_gate_up: Optional[torch.Tensor] = None, d_down: Optional[torch.Tensor] = None, stream=None):
    """(dx, d_gate_up, d_down) of ``ffn_forward(..., save=True)`` with the same
    arguments: dx bfloat16 (None without ``need_dx``), the weight gradients
    FP32 in the weights' shapes."""
    dims = _ffn_dims(x, gate_up, gate_up_scale, down, down_scale, offsets)
    if dy.dtype != torch.bfloat16 or dy.shape != x.shape:
        _bad("dy must be bfloat16 of x's shape")
    dev = x.get_device()
    raw, other = _begin(dev, stream)
    _same_device(dev, dy, saved, gate_up, gate_up_scale, down, down_scale, offsets)
    saved_bytes, _, backward_bytes = F.fp8z1_ffn_sizes(dims)
    if saved.dtype != torch.uint8 or saved.numel() < saved_bytes:
        _bad("saved is not from ffn_forward of these sizes")
    dx = _new(x.shape, torch.bfloat16, dev, other) if need_dx else None
    grads = []
    for given, w, what in ((d_gate_up, gate_up, "d_gate_up"), (d_down, down, "d_down")):
        if given is None:
            given = _new(w.shape, torch.float32, dev, other)
        elif not _given(given, w.shape, torch.float32, dev, what).is_contiguous():
            _bad(f"{what} must be contiguous")
        grads.append(given)
    ws = _scratch(backward_bytes, torch.uint8, dev, other)
    F.fp8z1_ffn_backward(dims, dy, _rows(dy, "dy"), x, _rows(x, "x"), offsets, gate_up, gate_up_scale, down,
                         down_scale, saved, dx, _rows(dx, "dx") if need_dx else 0, grads[0], grads[1], ws, raw)
    return dx, grads[0], grads[1]


# ---- distillation --------------------------------------------------------------------


def _distill(logits, teacher_ids, teacher_logits, temperature, row_weight, grad, out, stream):
    kind = _TYPES.get(logits.dtype)
    if kind is None or logits.dim() != 2:
        _bad("logits must be float32 or bfloat16 [rows, vocab]")
    rows, vocab = logits.shape
    shape = teacher_ids.shape
    if teacher_ids.dtype != torch.int32 or len(shape) != 2 or shape[0] != rows or not teacher_ids.is_contiguous():
        _bad("teacher_ids must be contiguous int32 [rows, top]")
    if teacher_logits.dtype != torch.float32 or teacher_logits.shape != shape or not teacher_logits.is_contiguous():
        _bad("teacher_logits must be contiguous float32 of teacher_ids' shape")
    if row_weight is not None and (row_weight.dtype != torch.float32 or row_weight.shape != (rows,)
                                   or not row_weight.is_contiguous()):
        _bad("row_weight must be contiguous float32 [rows]")
    dev = logits.get_device()
    raw, other = _begin(dev, stream)
    _same_device(dev, teacher_ids, teacher_logits, row_weight)
    ld, ld_d = _rows(logits, "logits"), 0
    if grad:
        if out is None:
            out = _new(logits.shape, logits.dtype, dev, other)
            ld_d = vocab
        else:
            ld_d = _rows(_given(out, logits.shape, logits.dtype, dev, "out"), "out")
    loss = _new(rows, torch.float32, dev, other)
    F.fp8z1_distill(logits, kind, ld, rows, vocab, teacher_ids, teacher_logits, shape[1], temperature, row_weight,
                    loss, out, ld_d, raw)
    return loss, out


def distill_loss(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                 temperature: float = 1.0, row_weight: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Each row's ``temperature^2 * KL(p || q)`` against the teacher's listed
    logits, float32 [rows] (0 in rows of weight 0 or without a teacher entry)."""
    return _distill(logits, teacher_ids, teacher_logits, temperature, row_weight, False, None, stream)[0]


def distill_loss_grad(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                      temperature: float = 1.0, row_weight: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, stream=None):
    """(loss, dlogits): ``distill_loss`` and the gradient of
    ``(row_weight * loss).sum()`` in the logits' type.  ``out`` may be
    ``logits`` itself."""
    return _distill(logits, teacher_ids, teacher_logits, temperature, row_weight, True, out, stream)


# ---- root-mean-square norm -------------------------------------------------------------


def _norm(x, weight, residual, eps, fp8, out, total, stream):
    shape, dtype = x.shape, x.dtype
    kind = _TYPES.get(dtype)
    if kind is None or not shape:
        _bad("x must be float32 or bfloat16 [*, dim]")
    dim = shape[-1]
    if weight.dtype != torch.float32 or weight.shape != (dim,) or not weight.is_contiguous():
        _bad(f"weight must be contiguous float32 [{dim}]")
    ld_x = _stride_of(x, dim, "x")
    dev = x.get_device()
    raw, other = _begin(dev, stream)
    if weight.get_device() != dev:
        _bad("the tensors are on several devices")
    ld_r, ld_t, ld_y, scale = 0, dim, dim, None
    if residual is not None:
        ld_r = _fits(residual, shape, dtype, dev, dim, "residual")
        if total is None:
            total = _new(shape, dtype, dev, other)
        else:
            ld_t = _fits(total, shape, dtype, dev, dim, "total")
    elif total is not None:
        _bad("total is the sum with a residual")
    y, codes = out, None
    if out is not None:
        ld_y = _fits(out, shape, dtype, dev, dim, "out")
    if fp8:
        codes = out = _new(shape, torch.float8_e4m3fn, dev, other)
        scale = _new((*shape[:-1], (dim + 127) // 128), torch.float32, dev, other)
    elif out is None:
        y = out = _new(shape, dtype, dev, other)
    F.fp8z1_rms_norm(x.numel() // dim if dim else 0, dim, x, kind, ld_x, residual, ld_r, weight, eps, total, ld_t, y, ld_y,
                     codes, scale, raw)
    return out, scale, total


def rms_norm(x: torch.Tensor, weight: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             out: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None, stream=None):
    """``s * (mean(s^2) + eps)^-1/2 * weight`` of each row s of ``x`` (float32 or
    bfloat16 [*, dim]; weight float32 [dim]), in x's type.  With ``residual``
    s = x + residual, and the result is (y, s); ``total`` takes s (it may be
    ``x`` or ``residual`` itself, as ``out`` may)."""
    y, _, total = _norm(x, weight, residual, eps, False, out, total, stream)
    return y if residual is None else (y, total)


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 out: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None, stream=None):
    """``rms_norm`` in 8 bits: (codes, scale), E4M3 codes (float8_e4m3fn) and a float32
    scale for every 128 columns, [*, ceil(dim / 128)]; with ``residual`` (codes,
    scale, s).  ``out`` takes the result in x's type as well, which ``linear_grad`` needs
    where the product before it took the codes."""
    codes, scale, total = _norm(x, weight, residual, eps, True, out, total, stream)
    return (codes, scale) if residual is None else (codes, scale, total)


def rms_norm_grad(dy: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, *, eps: float = 1e-6,
                  d_total: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                  d_weight: Optional[torch.Tensor] = None, stream=None):
    """(dx, d_weight) of ``rms_norm`` from the rows that it normed (its ``total``, or x):
    dx in their type, which is the residual's gradient too, with ``d_total`` (what
    reaches the sum past the norm) added; d_weight float32 [dim]."""
    shape, dtype = total.shape, total.dtype
    kind = _TYPES.get(dtype)
    if kind is None or not shape:
        _bad("total must be float32 or bfloat16 [*, dim]")
    dim = shape[-1]
    if weight.dtype != torch.float32 or weight.shape != (dim,) or not weight.is_contiguous():
        _bad(f"weight must be contiguous float32 [{dim}]")
    ld_s = _stride_of(total, dim, "total")
    dev = total.get_device()
    raw, other = _begin(dev, stream)
    if weight.get_device() != dev:
        _bad("the tensors are on several devices")
    ld_dy = _fits(dy, shape, dtype, dev, dim, "dy")
    ld_t, ld_dx = 0, dim
    if d_total is not None:
        ld_t = _fits(d_total, shape, dtype, dev, dim, "d_total")
    if dx is None:
        dx = _new(shape, dtype, dev, other)
    else:
        ld_dx = _fits(dx, shape, dtype, dev, dim, "dx")
    if d_weight is None:
        d_weight = _new((dim,), torch.float32, dev, other)
    elif not _given(d_weight, (dim,), torch.float32, dev, "d_weight").is_contiguous():
        _bad("d_weight must be contiguous")
    rows = total.numel() // dim if dim else 0
    ws = _scratch(F.fp8z1_rms_norm_grad_workspace(rows, dim), torch.uint8, dev, other)
    F.fp8z1_rms_norm_grad(rows, dim, dy, kind, ld_dy, total, ld_s, weight, eps, d_total, ld_t, dx, ld_dx, d_weight, ws,
                          raw)
    return dx, d_weight


# ---- routing --------------------------------------------------------------------------


class Route(NamedTuple):
    """Where tokens' rows go: expert e has rows [offsets[e], offsets[e + 1]) of
    tokens * top (int32 [experts + 1], as ``ffn_forward`` takes them), and choice j of
    token t row place[t, j] (int32 [tokens, top], -1: none)."""
    offsets: torch.Tensor
    place: torch.Tensor


def route(ids: torch.Tensor, experts: int, *, stream=None) -> Route:
    """Sorts the choices ids[t, j] (int32 or int64 [tokens, top], or [tokens]) by
    expert, each expert's in the order of the choices; an id outside [0, experts)
    is no choice."""
    nbytes, shape = _ID_BYTES.get(ids.dtype), ids.shape
    if nbytes is None or len(shape) not in (1, 2) or not ids.is_contiguous():
        _bad("ids must be contiguous int32 or int64 [tokens, top]")
    tokens, top = shape if len(shape) == 2 else (shape[0], 1)
    raw, other = _begin(dev := ids.get_device(), stream)
    if not 1 <= experts <= 1024:
        _bad("experts must be 1 to 1024")
    offsets = _new(experts + 1, torch.int32, dev, other)
    place = _new((tokens, top), torch.int32, dev, other)
    F.fp8z1_route(ids, nbytes, tokens, top, experts, offsets, place, raw)
    return Route(offsets, place)


def _route_dims(r: Route, dev: int):
    offsets, place = r
    shape, ends = place.shape, offsets.shape
    if place.dtype != torch.int32 or len(shape) != 2 or not place.is_contiguous():
        _bad("place must be contiguous int32 [tokens, top]")
    if offsets.dtype != torch.int32 or len(ends) != 1 or ends[0] < 2 or not offsets.is_contiguous():
        _bad("offsets must be contiguous int32 [experts + 1]")
    if offsets.get_device() != dev or place.get_device() != dev:
        _bad("the tensors are on several devices")
    return shape[0], shape[1], ends[0] - 1


def _plain_rows(t: torch.Tensor, rows: int, what: str):
    """(type, dim, row stride) of float32 or bfloat16 [rows, dim]."""
    kind, shape = _TYPES.get(t.dtype), t.shape
    if kind is None or len(shape) != 2 or shape[0] != rows:
        _bad(f"{what} must be float32 or bfloat16 [{rows}, dim]")
    dim = shape[1]
    return kind, dim, dim if t.is_contiguous() else _rows(t, what)


def _choice_weight(weight, shape, dev: int):
    if weight.dtype != torch.float32 or weight.shape != shape or not weight.is_contiguous() or weight.get_device() != dev:
        _bad(f"weight must be contiguous float32 {tuple(shape)} on the rows' device")


def dispatch(x: torch.Tensor, r: Route, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The experts' rows, [tokens * top, dim]: row place[t, j] is x[t] (float32 or
    bfloat16 [tokens, dim]); rows of no choice, behind the last expert's, are zero."""
    dev = x.get_device()
    tokens, top, experts = _route_dims(r, dev)
    kind, dim, ld = _plain_rows(x, tokens, "x")
    raw, other = _begin(dev, stream)
    ld_o, shape = dim, (tokens * top, dim)
    if out is None:
        out = _new(shape, x.dtype, dev, other)
    else:
        ld_o = _fits(out, shape, x.dtype, dev, dim, "out")
    F.fp8z1_dispatch(tokens, top, experts, dim, x, kind, ld, r[0], r[1], out, ld_o, raw)
    return out


def combine(rows: torch.Tensor, r: Route, weight: Optional[torch.Tensor] = None, *,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Each token's ``residual + sum_j weight[t, j] * rows[place[t, j]]``, [tokens, dim] in
    the rows' type (rounded once; weight float32 [tokens, top], None for 1).  ``out``
    may be ``residual`` itself."""
    dev = rows.get_device()
    tokens, top, _ = _route_dims(r, dev)
    kind, dim, ld = _plain_rows(rows, tokens * top, "rows")
    if weight is not None:
        _choice_weight(weight, (tokens, top), dev)
    raw, other = _begin(dev, stream)
    shape, ld_r, ld_y = (tokens, dim), 0, dim
    if residual is not None:
        ld_r = _fits(residual, shape, rows.dtype, dev, dim, "residual")
    if out is None:
        out = _new(shape, rows.dtype, dev, other)
    else:
        ld_y = _fits(out, shape, rows.dtype, dev, dim, "out")
    F.fp8z1_combine(tokens, top, dim, rows, kind, ld, r[1], weight, residual, ld_r, out, ld_y, raw)
    return out


def dispatch_grad(d_rows: torch.Tensor, r: Route, *, add: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``dispatch``'s gradient, the sum of each token's rows of ``d_rows``; ``add``
    (what reaches x otherwise) joins it."""
    return combine(d_rows, r, residual=add, out=out, stream=stream)


def combine_grad(dy: torch.Tensor, rows: torch.Tensor, r: Route, weight: torch.Tensor, *,
                 out: Optional[torch.Tensor] = None, stream=None):
    """(d_rows, d_weight) of ``combine``: d_rows in the rows' type (zero in rows of no
    choice), d_weight float32 [tokens, top] (0 where there is no row)."""
    dev = rows.get_device()
    tokens, top, experts = _route_dims(r, dev)
    kind, dim, ld = _plain_rows(rows, tokens * top, "rows")
    _choice_weight(weight, (tokens, top), dev)
    raw, other = _begin(dev, stream)
    ld_dy, ld_d = _fits(dy, (tokens, dim), rows.dtype, dev, dim, "dy"), dim
    if out is None:
        out = _new(rows.shape, rows.dtype, dev, other)
    else:
        ld_d = _fits(out, rows.shape, rows.dtype, dev, dim, "out")
    d_weight = _new((tokens, top), torch.float32, dev, other)
    F.fp8z1_combine_grad(tokens, top, experts, dim, dy, kind, ld_dy, rows, ld, r[0], r[1], weight, out, ld_d, d_weight,
                         raw)
    return out, d_weight


# ---- matrix product ---------------------------------------------------------------------

_ACTS = {None: F.ACT_NONE, "silu": F.ACT_SILU, "gelu_tanh": F.ACT_GELU_TANH}
_CODES = (torch.uint8, torch.float8_e4m3fn)


def _linear_dims(x, weight, scale, transposed, activation, y_type):
    """(dims, width of x, width of y, row stride of x)"""
    e, r, c = _fp8_weight(weight, scale, "the weight")
    act, kind, shape = _ACTS.get(activation, -1), _TYPES.get(y_type), x.shape
    if e != 1:
        _bad("a product's weight is [rows, cols]")
    if act < 0:
        _bad(f"no activation {activation!r}: None, 'silu' or 'gelu_tanh'")
    if kind is None:
        _bad(f"no product of {y_type}")
    inner, outer = (c, r) if transposed else (r, c)
    if len(shape) != 2 or shape[1] != inner:
        _bad(f"x must be [tokens, {inner}]")
    x_type = F.BF16 if x.dtype == torch.bfloat16 else F.E4M3 if x.dtype in _CODES else _bad("x must be bfloat16 or E4M3 codes")
    dims = F.fp8z1_linear_dims(shape[0], r, c, 1 if transposed else 0, act, x_type, kind)
    return dims, inner, outer, inner if x.is_contiguous() else _rows(x, "x")


def linear(x: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor, *, x_scale: Optional[torch.Tensor] = None,
           bias: Optional[torch.Tensor] = None, activation: Optional[str] = None, residual: Optional[torch.Tensor] = None,
           transposed: bool = False, dtype: torch.dtype = torch.bfloat16, save: bool = False,
           out: Optional[torch.Tensor] = None, stream=None):
    """``act(x w + bias) + residual`` with an FP8 weight [rows, cols] (cols a multiple of
    16), or ``x w^T`` with ``transposed``, in float32 or bfloat16.  ``x``: bfloat16
    [tokens, width], or E4M3 codes with ``x_scale`` as ``rms_norm_fp8`` gives them
    (width a multiple of 16 then).  ``bias`` float32, ``residual`` bfloat16;
    ``activation`` None, "silu" or "gelu_tanh".  With ``save`` also z = x w + bias,
    float32, which ``linear_grad`` reads where there is an activation: (y, z)."""
    dims, inner, outer, ld_x = _linear_dims(x, weight, weight_scale, transposed, activation, dtype)
    tokens = x.shape[0]
    dev = x.get_device()
    raw, other = _begin(dev, stream)
    if dims.x_type == F.E4M3:
        if (x_scale is None or x_scale.dtype != torch.float32 or x_scale.shape != (tokens, (inner + 127) // 128)
                or not x_scale.is_contiguous()):
            _bad("E4M3 codes need x_scale, contiguous float32 [tokens, ceil(width / 128)]")
        if tokens == 1:
            ld_x = (inner + 15) // 16 * 16  # a single row's stride is whatever it was cut from
    elif x_scale is not None:
        _bad("bfloat16 rows have no x_scale")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (outer,) or not bias.is_contiguous()):
        _bad(f"bias must be contiguous float32 [{outer}]")
    _same_device(dev, weight, weight_scale, x_scale, bias)
    shape, ld_r, ld_y = (tokens, outer), 0, outer
    if residual is not None:
        ld_r = _fits(residual, shape, torch.bfloat16, dev, outer, "residual")
    if out is None:
        out = _new(shape, dtype, dev, other)
    else:
        ld_y = _fits(out, shape, dtype, dev, outer, "out")
    pre = _new(shape, torch.float32, dev, other) if save else None
    size = F.fp8z1_linear_sizes(dims)[0]
    ws = _scratch(size, torch.uint8, dev, other) if size else None
    F.fp8z1_linear(dims, x, ld_x, x_scale, weight, weight_scale, bias, residual, ld_r, out, ld_y, pre, ws, raw)
    return (out, pre) if save else out


def linear_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor, *,
                activation: Optional[str] = None, pre: Optional[torch.Tensor] = None, transposed: bool = False,
                bias: bool = False, need_dx: bool = True, need_weight: bool = True,
                d_weight: Optional[torch.Tensor] = None, d_bias: Optional[torch.Tensor] = None, stream=None):
    """(dx, d_weight, d_bias) of ``linear`` for bfloat16 ``x`` and dy in its result's type: dx
    bfloat16 (None without ``need_dx``), d_weight float32 in the weight's shape (None
    without ``need_weight``), d_bias float32 (None without ``bias``).  ``pre``: z of
    ``linear(..., save=True)``, with an activation.  The residual's gradient is dy."""
    dims, inner, outer, ld_x = _linear_dims(x, weight, weight_scale, transposed, activation, dy.dtype)
    tokens = x.shape[0]
    if dims.x_type != F.BF16:
        _bad("the gradients need bfloat16 x")
    if dy.shape != (tokens, outer):
        _bad(f"dy must be [{tokens}, {outer}]")
    if activation is None:
        pre = None
    elif pre is None or pre.dtype != torch.float32 or pre.shape != dy.shape or not pre.is_contiguous():
        _bad("pre must be contiguous float32 of dy's shape, from linear(..., save=True)")
    dev = x.get_device()
    raw, other = _begin(dev, stream)
    _same_device(dev, dy, weight, weight_scale, pre)
    if not (need_dx or need_weight or bias):
        _bad("no gradient is wanted")
    dx = _new(x.shape, torch.bfloat16, dev, other) if need_dx else None
    if not need_weight:
        d_weight = None
    elif d_weight is None:
        d_weight = _new(weight.shape, torch.float32, dev, other)
    elif not _given(d_weight, weight.shape, torch.float32, dev, "d_weight").is_contiguous():
        _bad("d_weight must be contiguous")
    if not bias:
        d_bias = None
    elif d_bias is None:
        d_bias = _new((outer,), torch.float32, dev, other)
    elif not _given(d_bias, (outer,), torch.float32, dev, "d_bias").is_contiguous():
        _bad("d_bias must be contiguous")
    ws = _scratch(F.fp8z1_linear_sizes(dims)[1], torch.uint8, dev, other)
    F.fp8z1_linear_grad(dims, dy, outer if dy.is_contiguous() else _rows(dy, "dy"), x, ld_x, weight, weight_scale, pre, dx,
                        inner, d_weight, d_bias, ws, raw)
    return dx, d_weight, d_bias
