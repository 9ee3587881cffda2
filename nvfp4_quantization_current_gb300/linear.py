"""A linear layer on the blockwise FP8 copies, with dropout and the residual sum behind it:

    y = residual + dropout(x W^T)

Forward: the activations in 1x128 tiles and the weights in 128x128 tiles
(:func:`q_blockwise`), their product (:func:`mm_blockwise`), then
:func:`drop_add`.  Backward: :func:`drop_q_blockwise` draws the dropout's
decisions again and casts the gradient behind it in one read; the input
gradient is the product of its rowwise copy with the weights' transposed copy
and the weight gradient the product of the two transposed copies.  The layer
keeps FP8 copies for the backward pass, no mask and no BF16 activation.

The recipe is the DeepSeek-V3-like one of "Mixed-precision training: fp16 to
fp8", "Blockwise scaling".
"""
from __future__ import annotations

from typing import Optional

import torch

from . import BlockwiseTensor, _ready, drop_add, drop_q_blockwise, mm_blockwise, q_blockwise


def _cast_rows(x, rowwise, colwise, status):
    """1x128 copies of x [M, K].  The transposed copy needs M % 128 == 0: a
    ragged x is cast with zero rows below it, which add nothing to the weight
    gradient; the rowwise copy is cut back to M rows."""
    M = x.shape[0]
    if not colwise or M % 128 == 0:
        return q_blockwise(x, "1x128", rowwise, colwise, status=status)
    t = q_blockwise(torch.nn.functional.pad(x, (0, 0, 0, -M % 128)), "1x128", rowwise, True, status=status)
    if rowwise:
        t.q_row, t.s_row = t.q_row[:M], t.s_row[:M]
    return t


class _Once(torch.autograd.Function):
    """A gradient as it is.  Its own derivative, which the FP8 casts do not have, raises: a graph of the
    backward pass that ended here would lose that part without a word (`start` begins one where dy has none)."""
    @staticmethod
    def forward(ctx, g, dy, start):
        return g.view_as(g)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("BlockwiseLinear has no second derivative")


class _BlockwiseLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, w, p, seed, offset, main_grad, train, status):
        need_x, need_w = (train and n for n in ctx.needs_input_grad[:2])
        if need_x and w.q_colT is None:
            raise ValueError("copies lacks the transposed copy, which the input gradient reads")
        out_shape = (*x.shape[:-1], weight.shape[0])
        x2 = _ready(x.reshape(-1, x.shape[-1]))
        if residual is not None and residual.shape not in (out_shape, (x2.shape[0], weight.shape[0])):
            raise ValueError(f"residual must have the result's shape {out_shape}, not {tuple(residual.shape)}")
        xq = _cast_rows(x2, True, need_w, status)
        y = mm_blockwise(xq.q_row, xq.s_row, w.q_row, w.s_row, dtype=x.dtype, status=status)
        if p > 0 or residual is not None:
            drop_add(y, p, seed, offset, None if residual is None else _ready(residual.reshape(y.shape)), out=y)
        ctx.save_for_backward(*((w.q_colT, w.s_colT) if need_x else (None, None)),
                              *((xq.q_colT, xq.s_colT) if need_w else (None, None)))
        ctx.args = (p, seed, offset, main_grad, weight.dtype, x.shape, None if residual is None else residual.shape, status)
        return y.view(out_shape)

    @staticmethod
    def backward(ctx, dy):
        with torch.no_grad():
            dx, dw = _BlockwiseLinear.gradients(ctx, dy)
        if torch.is_grad_enabled():   # create_graph
            dx, dw = (None if g is None else _Once.apply(g, dy, torch.zeros((), requires_grad=True)) for g in (dx, dw))
        return (dx, dw, None if ctx.args[6] is None else dy.reshape(ctx.args[6])) + (None,) * 7

    @staticmethod
    def gradients(ctx, dy):
        w_q, w_s, x_q, x_s = ctx.saved_tensors
        p, seed, offset, main_grad, w_dtype, x_shape, _, status = ctx.args
        need_x, need_w = ctx.needs_input_grad[:2]
        if not (need_x or need_w):
            return None, None
        dx = dw = None
        d = _ready(dy.reshape(-1, dy.shape[-1]))
        M = d.shape[0]
        if need_w and M % 128 != 0:   # zero rows below, as in the forward pass; the draws are by flat index
            d = torch.nn.functional.pad(d, (0, 0, 0, -M % 128))
        g = drop_q_blockwise(d, p, seed, offset, need_x, need_w, status=status)
        if need_x:
            dx = mm_blockwise(g.q_row[:M], g.s_row[:M], w_q, w_s, dtype=dy.dtype, status=status).view(x_shape)
        if need_w:
            dw = mm_blockwise(g.q_colT, g.s_colT, x_q, x_s, tile_b="1x128", dtype=w_dtype, out=main_grad,
                              accumulate=main_grad is not None, status=status)
        return dx, None if main_grad is not None else dw


def _drawn() -> int:
    """A number below 2^62 from torch's CPU generator: far from any other one, in counters."""
    return int(torch.empty((), dtype=torch.int64, device="cpu").random_(0, 1 << 62))


class BlockwiseLinear(torch.nn.Module):
    """``y = residual + dropout(x W^T)`` on blockwise FP8 copies.

    ``in_features`` and ``out_features`` are multiples of 128; x is bfloat16 or
    float32 with any number of rows and any strides, the residual alike and of
    x's type.  With ``main_grad`` set (FP32, the weight's shape) the weight
    gradient is added to it and ``weight.grad`` stays unset.  ``copies`` takes the
    result of :meth:`quantize_weight`, made once for the micro-batches of a step,
    or once for serving.  There is no second derivative: one that is asked for
    raises.

    Dropout runs in training mode; its decisions follow from the layer's ``seed``
    and the ``offset`` of the call (in counters of 8 elements).  Neither has to be
    given: a seed is drawn when a layer with dropout is made, an offset at every
    call, both from torch's CPU generator, so that masks differ from call to call
    and layer to layer, repeat under ``torch.manual_seed``, and a checkpointed
    forward pass draws its own again.  Who gives offsets gives each step its own,
    e.g. ``step * rows * out_features // 8``.  A call that is captured into a CUDA
    graph has to be given one (every replay draws what it was captured with).

    ``status`` (a one-element int32 tensor on the layer's device) collects what
    the layer's casts and products report: ``Q_ST_NONFINITE`` where x, the
    weight or a gradient was not finite, ``Q_ST_TIMEOUT`` where a kernel gave up
    waiting and a result is not whole.  Look at it where the host waits anyway
    (before the optimizer's step, say) and zero it."""

    def __init__(self, in_features: int, out_features: int, p: float = 0.0, seed: Optional[int] = None, device="cuda",
                 dtype=torch.bfloat16):
        super().__init__()
        if in_features % 128 or out_features % 128:
            raise ValueError("in_features and out_features must be multiples of 128")
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)
        self.p = float(p)
        self.seed = int(seed) if seed is not None else _drawn() if p > 0 else 0
        self.main_grad: Optional[torch.Tensor] = None
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def _status_on(self, device):
        if self.status.device != device:   # the layer was moved
            self.status = torch.zeros_like(self.status, device=device) if self.status.is_meta else self.status.to(device)
        return self.status

    def quantize_weight(self, colwise=True) -> BlockwiseTensor:
        """The weight's 128x128 copies (``colwise``: also the transposed one, for the input gradient)."""
        return q_blockwise(self.weight.detach(), "128x128", rowwise=True, colwise=colwise,
                           status=self._status_on(self.weight.device))

    def forward(self, x, residual=None, offset: Optional[int] = None, copies: Optional[BlockwiseTensor] = None):
        train = torch.is_grad_enabled()
        p = self.p if self.training else 0.0
        if offset is None:
            if p > 0 and x.is_cuda and torch.cuda.is_current_stream_capturing():
                raise ValueError("a captured call with dropout needs its offset: a drawn one would be every replay's")
            offset = _drawn() if p > 0 else 0
        if copies is None:
            copies = self.quantize_weight(colwise=train and x.requires_grad)
        return _BlockwiseLinear.apply(x, self.weight, residual, copies, p, self.seed,
                                      int(offset), self.main_grad, train, self._status_on(x.device))
