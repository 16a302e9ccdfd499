"""Model operators next to the optimizer step, on torch tensors.

They take the FP8 weights as the optimizer writes them -- row-major E4M3 codes
[E, R, C] (uint8) and FP32 block scales [E, ceil(R/128), ceil(C/128)]
(``ShardOptimizer.step``'s FP8 params and ``scale_views()``) -- and give back
FP32 [E, R, C] weight gradients, which ``ShardOptimizer.step`` reads:

  embed, embed_grad          rows of an FP8 table, and the table's gradient;
  ffn_forward, ffn_backward  the gated feed-forward block of each expert;
  distill_loss, distill_loss_grad
                             distillation from a teacher's top logits.

Each is one call of libfp8z1.so's entry point of the same name (include/
fp8z1_ops.h has the formulas); this module checks the tensors, allocates
outputs and workspaces through torch and enqueues on ``stream`` (a
``torch.cuda.Stream``; None is torch's current stream).  With a ``stream``
that is not current, the outputs and workspaces are allocated as that stream's
and the outputs marked as used on the current one too; the order of the two
streams, and the inputs' memory until the work is done, are the caller's to
see to.  Tensors that do not fit raise ValueError, what the library refuses
raises Fp8z1Error.  Should a wait between the feed-forward kernels' warps ever
run out, what it belongs to is NaN (``fp8z1.fp8z1_ffn_timeouts`` counts them);
the optimizer skips a step with such gradients.
"""
from __future__ import annotations

from typing import Optional

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
