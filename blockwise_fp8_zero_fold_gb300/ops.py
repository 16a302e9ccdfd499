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
that is not current, the outputs and workspaces are marked as used there; the
inputs' memory is the caller's to keep until the work is done.  Tensors that
do not fit raise ValueError, what the library refuses raises Fp8z1Error.
"""
from __future__ import annotations

import ctypes as C
from typing import Optional, Tuple

import torch

from . import fp8z1 as F

_TYPES = {torch.float32: F.F32, torch.bfloat16: F.BF16}


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _stream_of(device, stream):
    """(torch stream to enqueue on, whether it is not the current one)"""
    if stream is None:
        return torch.cuda.current_stream(device), False
    _need(isinstance(stream, torch.cuda.Stream), "stream must be a torch.cuda.Stream or None")
    return stream, stream != torch.cuda.current_stream(device)


class _Call:
    """Allocations of one call: on its stream, so that their reuse is ordered."""

    def __init__(self, device, stream):
        _need(device.type == "cuda", "the operators need CUDA tensors")
        self.device = device
        self.stream, self.other = _stream_of(device, stream)
        _need(self.stream.device == device, f"a stream of {self.stream.device} for tensors on {device}")

    def empty(self, shape, dtype):
        if not self.other:
            return torch.empty(shape, dtype=dtype, device=self.device)
        t = torch.empty(shape, dtype=dtype, device=self.device)
        t.record_stream(self.stream)
        return t

    def bytes(self, n):
        return self.empty((max(1, int(n)),), torch.uint8)

    def out(self, given, shape, dtype, what):
        if given is None:
            return self.empty(shape, dtype)
        _need(tuple(given.shape) == tuple(shape) and given.dtype == dtype and given.device == self.device,
              f"{what} must be {dtype} of shape {tuple(shape)} on {self.device}")
        return given


def _on(device, *tensors):
    for t in tensors:
        _need(t is None or t.device == device, f"a tensor on {t.device if t is not None else None}, others on {device}")


def _rows(t: torch.Tensor, what: str):
    """The row stride of a 2-D tensor whose rows are dense."""
    _need(t.dim() == 2 and (t.shape[1] <= 1 or t.stride(1) == 1), f"{what} must be 2-D with dense rows")
    ld = t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0))
    _need(ld >= t.shape[1], f"{what}'s rows must not overlap")
    return ld


def _fp8_weight(codes: torch.Tensor, scale: torch.Tensor, what: str) -> Tuple[int, int, int]:
    """(E, R, C) of an FP8 weight after checking its codes and block scales."""
    _need(codes.dim() in (2, 3) and codes.is_contiguous(), f"{what} must be contiguous [E, R, C] or [R, C] codes")
    _need(codes.dtype == torch.uint8 or codes.dtype == torch.float8_e4m3fn, f"{what} must hold E4M3 codes (uint8)")
    e, r, c = ((1,) + tuple(codes.shape))[-3:]
    grid = (e, -(-r // F.TILE), -(-c // F.TILE))
    _need(scale.dtype == torch.float32 and scale.is_contiguous() and scale.numel() == grid[0] * grid[1] * grid[2]
          and tuple(scale.shape[-2:]) == grid[1:], f"{what}'s scales must be contiguous float32 {grid}")
    return e, r, c


def _ids(ids: torch.Tensor) -> int:
    _need(ids.dtype in (torch.int32, torch.int64) and ids.is_contiguous(), "ids must be contiguous int32 or int64")
    return ids.element_size()


# ---- embedding -----------------------------------------------------------------


def embed(ids: torch.Tensor, table: torch.Tensor, scale: torch.Tensor, *, alpha: float = 1.0,
          dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``alpha * table[ids]``, [*ids.shape, dim]; rows of ids outside the table are zero."""
    e, vocab, dim = _fp8_weight(table, scale, "the table")
    _need(e == 1, "an embedding table is [vocab, dim]")
    _need(dtype in _TYPES, f"no embedding output of {dtype}")
    nbytes = _ids(ids)
    call = _Call(ids.device, stream)
    _on(ids.device, table, scale)
    n = ids.numel()
    out = call.out(out, tuple(ids.shape) + (dim,), dtype, "out")
    _need(out.dim() == 2 or out.is_contiguous(), "out must be contiguous")
    ld = _rows(out, "out") if out.dim() == 2 else dim
    F.fp8z1_embed(vocab, dim, table, scale, ids, nbytes, n, alpha, out, _TYPES[dtype], ld, call.stream)
    return out


def embed_grad(ids: torch.Tensor, dy: torch.Tensor, vocab: int, *, alpha: float = 1.0,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The FP32 [vocab, dim] gradient of ``embed``'s table from ``dy``
    [*ids.shape, dim] (every row written; repeatable bit for bit)."""
    nbytes = _ids(ids)
    _need(dy.dtype in _TYPES, f"no gradient of {dy.dtype}")
    _need(dy.dim() >= 1 and tuple(dy.shape[:-1]) == tuple(ids.shape), "dy must be [*ids.shape, dim]")
    dim, n = dy.shape[-1], ids.numel()
    call = _Call(ids.device, stream)
    _on(ids.device, dy)
    _need(dy.dim() == 2 or dy.is_contiguous(), "dy must be contiguous")
    ld = _rows(dy, "dy") if dy.dim() == 2 else dim
    out = call.out(out, (vocab, dim), torch.float32, "out")
    _need(out.is_contiguous(), "out must be contiguous")
    ws = call.bytes(F.fp8z1_embed_grad_workspace(vocab, dim, n))
    F.fp8z1_embed_grad(vocab, dim, ids, nbytes, n, alpha, dy, _TYPES[dy.dtype], ld, out, ws, call.stream)
    return out


# ---- gated feed-forward block -----------------------------------------------------


def _ffn_dims(x, gate_up, gate_up_scale, down, down_scale, offsets):
    e, h, f2 = _fp8_weight(gate_up, gate_up_scale, "gate_up")
    e2, f, h2 = _fp8_weight(down, down_scale, "down")
    _need(e == e2 and h == h2 and f2 == 2 * f, f"gate_up [{e}, {h}, {f2}] and down [{e2}, {f}, {h2}] do not match: "
          "[E, hidden, 2 inner] and [E, inner, hidden]")
    _need(x.dim() == 2 and x.shape[1] == h and x.dtype == torch.bfloat16, f"x must be bfloat16 [tokens, {h}]")
    if offsets is not None:
        _need(offsets.dtype == torch.int32 and offsets.is_contiguous() and tuple(offsets.shape) == (e + 1,),
              f"offsets must be contiguous int32 [{e + 1}]")
    else:
        _need(e == 1, "several experts need offsets")
    _on(x.device, gate_up, gate_up_scale, down, down_scale, offsets)
    return F.fp8z1_ffn_dims(x.shape[0], h, f, e)


def ffn_forward(x: torch.Tensor, gate_up: torch.Tensor, gate_up_scale: torch.Tensor, down: torch.Tensor,
                down_scale: torch.Tensor, *, offsets: Optional[torch.Tensor] = None, save: bool = False,
                out: Optional[torch.Tensor] = None, stream=None):
    """``(silu(x Wg) * (x Wu)) Wd`` of each expert on its rows of ``x``
    (bfloat16 [tokens, hidden], grouped by expert: expert e has rows
    [offsets[e], offsets[e + 1])).  With ``save`` also the buffer that
    ``ffn_backward`` reads: (y, saved)."""
    dims = _ffn_dims(x, gate_up, gate_up_scale, down, down_scale, offsets)
    call = _Call(x.device, stream)
    y = call.out(out, tuple(x.shape), torch.bfloat16, "out")
    saved_bytes, forward_bytes, _ = F.fp8z1_ffn_sizes(dims)
    saved = call.bytes(saved_bytes) if save else None
    ws = call.bytes(forward_bytes)
    F.fp8z1_ffn_forward(dims, x, _rows(x, "x"), offsets, gate_up, gate_up_scale, down, down_scale, y, _rows(y, "out"),
                        saved, ws, call.stream)
    return (y, saved) if save else y


def ffn_backward(dy: torch.Tensor, x: torch.Tensor, saved: torch.Tensor, gate_up: torch.Tensor,
                 gate_up_scale: torch.Tensor, down: torch.Tensor, down_scale: torch.Tensor, *,
                 offsets: Optional[torch.Tensor] = None, need_dx: bool = True,
                 d_gate_up: Optional[torch.Tensor] = None, d_down: Optional[torch.Tensor] = None, stream=None):
    """(dx, d_gate_up, d_down) of ``ffn_forward(..., save=True)`` with the same
    arguments: dx bfloat16 (None without ``need_dx``), the weight gradients
    FP32 in the weights' shapes."""
    dims = _ffn_dims(x, gate_up, gate_up_scale, down, down_scale, offsets)
    _need(dy.dtype == torch.bfloat16 and tuple(dy.shape) == tuple(x.shape), "dy must be bfloat16 of x's shape")
    call = _Call(x.device, stream)
    _on(x.device, dy, saved)
    saved_bytes, _, backward_bytes = F.fp8z1_ffn_sizes(dims)
    _need(saved.dtype == torch.uint8 and saved.numel() >= saved_bytes, "saved is not from ffn_forward of these sizes")
    dx = call.empty(tuple(x.shape), torch.bfloat16) if need_dx else None
    d_gate_up = call.out(d_gate_up, tuple(gate_up.shape), torch.float32, "d_gate_up")
    d_down = call.out(d_down, tuple(down.shape), torch.float32, "d_down")
    _need(d_gate_up.is_contiguous() and d_down.is_contiguous(), "the weight gradients must be contiguous")
    ws = call.bytes(backward_bytes)
    F.fp8z1_ffn_backward(dims, dy, _rows(dy, "dy"), x, _rows(x, "x"), offsets, gate_up, gate_up_scale, down,
                         down_scale, saved, dx, _rows(dx, "dx") if need_dx else 0, d_gate_up, d_down, ws, call.stream)
    return dx, d_gate_up, d_down


# ---- distillation --------------------------------------------------------------------


def _distill(logits, teacher_ids, teacher_logits, temperature, row_weight, dlogits, call):
    _need(logits.dtype in _TYPES, f"no logits of {logits.dtype}")
    ld = _rows(logits, "logits")
    rows, vocab = logits.shape
    _need(teacher_ids.dtype == torch.int32 and teacher_ids.dim() == 2 and teacher_ids.shape[0] == rows
          and teacher_ids.is_contiguous(), "teacher_ids must be contiguous int32 [rows, top]")
    _need(teacher_logits.dtype == torch.float32 and teacher_logits.shape == teacher_ids.shape
          and teacher_logits.is_contiguous(), "teacher_logits must be contiguous float32 of teacher_ids' shape")
    if row_weight is not None:
        _need(row_weight.dtype == torch.float32 and row_weight.is_contiguous() and tuple(row_weight.shape) == (rows,),
              "row_weight must be contiguous float32 [rows]")
    _on(logits.device, teacher_ids, teacher_logits, row_weight)
    loss = call.empty((rows,), torch.float32)
    F.fp8z1_distill(logits, _TYPES[logits.dtype], ld, rows, vocab, teacher_ids, teacher_logits, teacher_ids.shape[1],
                    temperature, row_weight, loss, dlogits, 0 if dlogits is None else _rows(dlogits, "dlogits"),
                    call.stream)
    return loss


def distill_loss(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                 temperature: float = 1.0, row_weight: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Each row's ``temperature^2 * KL(p || q)`` against the teacher's listed
    logits, float32 [rows] (0 in rows of weight 0 or without a teacher entry)."""
    call = _Call(logits.device, stream)
    return _distill(logits, teacher_ids, teacher_logits, temperature, row_weight, None, call)


def distill_loss_grad(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logits: torch.Tensor, *,
                      temperature: float = 1.0, row_weight: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, stream=None):
    """(loss, dlogits): ``distill_loss`` and the gradient of
    ``(row_weight * loss).sum()`` in the logits' type.  ``out`` may be
    ``logits`` itself."""
    call = _Call(logits.device, stream)
    d = call.out(out, tuple(logits.shape), logits.dtype, "out")
    return _distill(logits, teacher_ids, teacher_logits, temperature, row_weight, d, call), d
