"""Linear layers on the library's copies, and the norm ahead of them.

:class:`BlockwiseLinear` works on the blockwise FP8 copies, with dropout and the residual sum behind it:

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

:class:`NormBlockwiseLinear` has the root-mean-square norm and the residual's
addition ahead of it, y = norm(x + residual) W^T: :func:`norm_q_blockwise` makes
the copies while it norms, and :func:`norm_grad` takes the input gradient's
product back through the norm.  :class:`RMSNorm` is the norm by itself.

:class:`NVFP4Linear` works on NVFP4 copies as the recipe of "From BF16 to
FP8/FP4: low-precision and mixed-precision LLM pretraining", 2.4, has it: 1x16
blocks for activations and gradients, 16x16 blocks for weights, stochastic
rounding on gradients, the random Hadamard transform on both inputs of the
weight gradient, and :func:`matmul_nvfp4` for the three products.

A backward pass may be captured into a CUDA graph if no eager graph of the same
parameters or inputs is alive then: let go of earlier results and losses first.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (BlockwiseTensor, NVFP4Tensor, _once, _ready, _word, drop_add, drop_q_blockwise, matmul_nvfp4, mm_blockwise, norm_add,
               norm_grad, norm_q_blockwise, q_blockwise, q_nvfp4, q_nvfp4_recipe, q_nvfp4_rht_colT)


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


def _link(wanted):
    """An output of a layer's function without elements, kept for its backward pass (None where there is none): it leads to
    all of the function's inputs, which themselves are not kept, for :func:`_once` to stand on the way to them."""
    return torch.empty(0) if wanted else None


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
        link = _link(need_x or need_w)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(*((w.q_colT, w.s_colT) if need_x else (None, None)),
                              *((xq.q_colT, xq.s_colT) if need_w else (None, None)), link)
        ctx.args = (p, seed, offset, main_grad, weight.dtype, x.shape, None if residual is None else residual.shape, status)
        return y.view(out_shape), link

    @staticmethod
    def backward(ctx, dy, _):
        *saved, link = ctx.saved_tensors   # once: a checkpoint unpacks each a single time
        with torch.no_grad():
            grads = _BlockwiseLinear.gradients(ctx, dy, saved)
        dx, dw = _once("BlockwiseLinear", grads, dy, link)
        return (dx, dw, None if ctx.args[6] is None else dy.reshape(ctx.args[6])) + (None,) * 7

    @staticmethod
    def gradients(ctx, dy, saved):
        w_q, w_s, x_q, x_s = saved
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
    x's type; the weight may lie on any address.  With ``main_grad`` set (FP32, the
    weight's shape, on a 16-byte boundary) the weight gradient is added to it and ``weight.grad`` stays unset.  ``copies`` takes the
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
        return q_blockwise(_ready(self.weight.detach()), "128x128", rowwise=True, colwise=colwise,
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
                                      int(offset), self.main_grad, train, self._status_on(x.device))[0]


class RMSNorm(torch.nn.Module):
    """``y = h rsqrt(mean(h^2) + eps) weight`` over the last dimension, h = x or
    x + residual; with a residual the result is ``(y, h)``, h being the new
    residual.  x is bfloat16 or float32 with any strides, the residual of its shape
    and type.  ``amax`` (a one-element float32 tensor) receives max|y|, for
    :class:`NVFP4Linear` to be given.  ``status`` is as in :class:`BlockwiseLinear`:
    ``Q_ST_TIMEOUT`` where a kernel of either pass gave up waiting, and with ``amax``
    ``Q_ST_NONFINITE`` where that maximum is not finite."""

    def __init__(self, features: int, eps: float = 1e-6, device="cuda", dtype=torch.bfloat16):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(features, device=device, dtype=dtype))
        self.eps = float(eps)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    _status_on = BlockwiseLinear._status_on

    def forward(self, x, residual=None, amax: Optional[torch.Tensor] = None):
        y, h, _ = norm_add(_ready(x), _ready(self.weight), self.eps, None if residual is None else _ready(residual), amax=amax,
                           status=self._status_on(x.device))
        return y if residual is None else (y, h)


def _rows_to(x, step):
    """x [M, K] with zero rows below it up to a multiple of `step`."""
    return x if x.shape[0] % step == 0 else torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % step))


class _NormBlockwiseLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, norm_weight, weight, residual, w, eps, main_grad, train, status):
        need = [train and n for n in ctx.needs_input_grad[:4]]
        through, need_w = need[0] or need[1] or need[3], need[2]
        if through and w.q_colT is None:
            raise ValueError("copies lacks the transposed copy, which the input gradient reads")
        if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
            raise ValueError(f"residual must have x's shape {tuple(x.shape)} and type, not {tuple(residual.shape)}, {residual.dtype}")
        x2, r2 = (None if t is None else _ready(t.reshape(-1, t.shape[-1])) for t in (x, residual))
        M = x2.shape[0]
        if need_w and M % 128 != 0:   # zero rows below: their norm is zero and adds nothing to the weight gradient
            x2, r2 = _rows_to(x2, 128), None if r2 is None else _rows_to(r2, 128)
        xq, h, rstd = norm_q_blockwise(x2, _ready(norm_weight.detach()), eps, r2, rowwise=True, colwise=need_w, status=status)
        y = mm_blockwise(xq.q_row[:M], xq.s_row[:M], w.q_row, w.s_row, dtype=x.dtype, status=status)
        ctx.set_materialize_grads(False)
        link = _link(through or need_w)
        ctx.save_for_backward(*((h[:M], rstd[:M], norm_weight, w.q_colT, w.s_colT) if through else (None,) * 5),
                              *((xq.q_colT, xq.s_colT) if need_w else (None, None)), link)
        ctx.args = (main_grad, weight.dtype, x.shape, residual is not None, status)
        y = y.view(*x.shape[:-1], weight.shape[0])
        return (y, link, h[:M].reshape(x.shape)) if residual is not None else (y, link)

    @staticmethod
    def backward(ctx, dy, _, dh=None):
        if dy is None:   # the sum alone was used
            return (dh, None, None, dh) + (None,) * 5
        *saved, link = ctx.saved_tensors   # once: a checkpoint unpacks each a single time
        with torch.no_grad():
            grads = _NormBlockwiseLinear.gradients(ctx, dy, dh, saved)
        dx, dn, dw = _once("NormBlockwiseLinear", grads, dy, dh, link)
        return (dx, dn, dw, dx if ctx.args[3] else None) + (None,) * 5

    @staticmethod
    def gradients(ctx, dy, dh, saved):
        h, rstd, norm_weight, w_q, w_s, x_q, x_s = saved
        main_grad, w_dtype, x_shape, _, status = ctx.args
        need = ctx.needs_input_grad
        through, need_w = need[0] or need[1] or need[3], need[2]
        d = _ready(dy.reshape(-1, dy.shape[-1]))
        M = d.shape[0]
        g = _cast_rows(d, through, need_w, status)
        dx = dn = dw = None
        if through:
            dn_in = mm_blockwise(g.q_row, g.s_row, w_q, w_s, dtype=dy.dtype, status=status)
            dx, dn = norm_grad(dn_in, h, rstd, _ready(norm_weight), None if dh is None else _ready(dh.reshape(-1, dh.shape[-1])), need_dw=need[1],
                               out=dn_in, status=status)
            dx = dx.view(x_shape)
        if need_w:
            dw = mm_blockwise(g.q_colT, g.s_colT, x_q, x_s, tile_b="1x128", dtype=w_dtype, out=main_grad,
                              accumulate=main_grad is not None, status=status)
        return dx, dn, None if main_grad is not None else dw


class NormBlockwiseLinear(BlockwiseLinear):
    """``y = norm(x + residual) W^T`` on blockwise FP8 copies, the norm that of
    :class:`RMSNorm` with the parameter ``norm_weight``; with a residual the result is
    ``(y, h)``, h = x + residual being the new residual.  x and the residual are
    bfloat16 or float32, of one type and shape, with any strides.  ``main_grad``,
    ``copies`` and ``status`` are those of :class:`BlockwiseLinear`; there is no second
    derivative: one that is asked for raises."""

    def __init__(self, in_features: int, out_features: int, eps: float = 1e-6, device="cuda", dtype=torch.bfloat16):
        super().__init__(in_features, out_features, device=device, dtype=dtype)
        if not eps > 0:   # rows of zeros, padding among them, have no norm without it
            raise ValueError("eps must be positive")
        self.norm_weight = torch.nn.Parameter(torch.ones(in_features, device=device, dtype=dtype))
        self.eps = float(eps)

    def forward(self, x, residual=None, copies: Optional[BlockwiseTensor] = None):
        train = torch.is_grad_enabled()
        if copies is None:
            through = x.requires_grad or self.norm_weight.requires_grad or residual is not None and residual.requires_grad
            copies = self.quantize_weight(colwise=train and through)
        y, _, *h = _NormBlockwiseLinear.apply(x, self.norm_weight, self.weight, residual, copies, self.eps, self.main_grad, train,
                                              self._status_on(x.device))
        return (y, *h) if h else y


class _NVFP4Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, w, sign_mask, seed, offset, main_grad, train, status, amax):
        need_x, need_w = (train and n for n in ctx.needs_input_grad[:2])
        if need_x and w.q_colT is None:
            raise ValueError("copies lacks the transposed copy, which the input gradient reads")
        x2 = _ready(x.reshape(-1, x.shape[-1]))
        M = x2.shape[0]
        col = None
        if need_w:   # the product over tokens takes 32 of them at a time: zero rows below add nothing
            row, col = q_nvfp4_recipe(_rows_to(x2, 32), sign_mask, status=status)
        else:
            if amax is not None:
                _word("amax", amax, x.device)
            row = q_nvfp4(_rows_to(x2, 16), amax=amax, status=status)
        y = matmul_nvfp4(row.q_row[:M], row.sb_row[:M], row.s_global, w.q_row, w.sb_row, w.s_global, dtype=x.dtype, status=status)
        link = _link(need_x or need_w)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(*((w.q_colT, w.sb_colT, w.s_global) if need_x else (None,) * 3),
                              *((col.q_colT, col.sb_colT, col.s_global) if need_w else (None,) * 3), link)
        ctx.args = (sign_mask, seed, offset, main_grad, weight.dtype, x.shape, status)
        return y.view(*x.shape[:-1], weight.shape[0]), link

    @staticmethod
    def backward(ctx, dy, _):
        *saved, link = ctx.saved_tensors   # once: a checkpoint unpacks each a single time
        with torch.no_grad():
            grads = _NVFP4Linear.gradients(ctx, dy, saved)
        return _once("NVFP4Linear", grads, dy, link) + (None,) * 8

    @staticmethod
    def gradients(ctx, dy, saved):
        w, x = saved[:3], saved[3:]
        sign_mask, seed, offset, main_grad, w_dtype, x_shape, status = ctx.args
        need_x, need_w = ctx.needs_input_grad[:2]
        d = _ready(dy.reshape(-1, dy.shape[-1]))
        M = d.shape[0]
        dx = dw = row = col = None
        if need_x and need_w:
            row, col = q_nvfp4_recipe(_rows_to(d, 32), sign_mask, "sr", seed, offset, status=status)
        elif need_x:
            row = q_nvfp4(_rows_to(d, 16), "1x16", "sr", seed, offset, status=status)
        elif need_w:
            col = q_nvfp4_rht_colT(_rows_to(d, 32), sign_mask, "sr", seed, offset, status=status)
        if need_x:
            dx = matmul_nvfp4(row.q_row[:M], row.sb_row[:M], row.s_global, *w, dtype=dy.dtype, status=status).view(x_shape)
        if need_w:
            dw = matmul_nvfp4(col.q_colT, col.sb_colT, col.s_global, *x, blk_b="1x16", dtype=w_dtype, out=main_grad,
                              accumulate=main_grad is not None, status=status)
        return dx, None if main_grad is not None else dw


class NVFP4Linear(torch.nn.Module):
    """``y = x W^T`` on NVFP4 copies.

    ``in_features`` and ``out_features`` are multiples of 32; x is bfloat16 or float32
    with any number of rows and any strides.  ``main_grad`` (FP32, the weight's shape),
    ``copies`` (of :meth:`quantize_weight`) and ``status`` are as in
    :class:`BlockwiseLinear`.  ``amax`` (a one-element float32 tensor holding max|x|, as
    :class:`RMSNorm` gives it) saves a read of x where no weight gradient is wanted;
    with one, both of the recipe's maxima take a single read in any case.

    Gradients are rounded stochastically.  The numbers follow from the layer's ``seed``
    and the call's ``offset`` (in counters of 16 elements), which are drawn from
    torch's CPU generator where they are not given; a call with gradients that is
    captured into a CUDA graph has to be given its offset (every replay draws what it
    was captured with).  ``sign_mask`` is that of the Hadamard transform of both inputs
    of the weight gradient.  There is no second derivative: one that is asked for
    raises."""

    def __init__(self, in_features: int, out_features: int, seed: Optional[int] = None, sign_mask: int = 0xB4E1, device="cuda",
                 dtype=torch.bfloat16):
        super().__init__()
        if in_features % 32 or out_features % 32:
            raise ValueError("in_features and out_features must be multiples of 32")
        if not 0 <= sign_mask <= 0xFFFF:
            raise ValueError("sign_mask must have 16 bits")
        self.weight = torch.nn.Parameter(torch.empty(out_features, in_features, device=device, dtype=dtype))
        torch.nn.init.normal_(self.weight, std=0.02)
        self.seed = int(seed) if seed is not None else _drawn()
        self.sign_mask = int(sign_mask)
        self.main_grad: Optional[torch.Tensor] = None
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    _status_on = BlockwiseLinear._status_on

    def quantize_weight(self, colwise=True) -> NVFP4Tensor:
        """The weight's 16x16 copies (``colwise``: also the transposed one, for the input gradient)."""
        return q_nvfp4(_ready(self.weight.detach()), "16x16", rowwise=True, colwise=colwise, status=self._status_on(self.weight.device))

    def forward(self, x, offset: Optional[int] = None, copies: Optional[NVFP4Tensor] = None, amax: Optional[torch.Tensor] = None):
        train = torch.is_grad_enabled()
        if offset is None:
            draws = train and (x.requires_grad or self.weight.requires_grad)
            if draws and x.is_cuda and torch.cuda.is_current_stream_capturing():
                raise ValueError("a captured call with gradients needs its offset: a drawn one would be every replay's")
            offset = _drawn() if draws else 0
        if copies is None:
            copies = self.quantize_weight(colwise=train and x.requires_grad)
        return _NVFP4Linear.apply(x, self.weight, copies, self.sign_mask, self.seed, int(offset), self.main_grad, train,
                                  self._status_on(x.device), amax)[0]
