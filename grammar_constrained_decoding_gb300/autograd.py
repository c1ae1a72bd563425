"""Autograd form of the distillation loss: cg_distill_loss forward,
cg_distill_grad backward, nothing kept but the inputs and the normaliser, two
values a row (one would lose it in rows far from zero)."""

from __future__ import annotations

import contextlib

import torch


@contextlib.contextmanager
def on_ctx_stream(ctx, *tensors):
    """Runs the body's library calls, which go to the context's stream, after what
    torch's current stream holds so far, and makes that stream wait for them.
    The tensors' memory is kept from reuse until the context's stream has passed."""
    cur = torch.cuda.current_stream(ctx.stream.device)
    if cur == ctx.stream:
        yield
        return
    ctx.stream.wait_stream(cur)
    yield  # a refused tensor raises here
    for t in tensors:
        if t is not None:
            t.record_stream(ctx.stream)
    cur.wait_stream(ctx.stream)


class DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(fn, logits, ctx, ids, teacher, temp, bitmask):
        B = logits.shape[0]
        loss = torch.empty(B, dtype=torch.float32, device=logits.device)
        norm = torch.empty((B, 2), dtype=torch.float32, device=logits.device)
        with on_ctx_stream(ctx, logits, ids, teacher, bitmask, loss, norm):
            ctx.distill_loss(logits, ids, teacher, loss, temp=temp, bitmask=bitmask, out_norm=norm)
        fn.save_for_backward(logits, ids, teacher, bitmask, norm)
        fn.ctx, fn.temp = ctx, temp
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fn, grad_loss):
        logits, ids, teacher, bitmask, norm = fn.saved_tensors
        grad_loss = grad_loss.contiguous()  # an expanded scalar (loss.sum()) is one value with stride 0
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        with on_ctx_stream(fn.ctx, logits, ids, teacher, bitmask, norm, grad_loss, grad):
            fn.ctx.distill_grad(logits, ids, teacher, None, grad, temp=fn.temp, bitmask=bitmask,
                                grad_loss=grad_loss, norm=norm)
        return grad, None, None, None, None, None
