"""Autograd forms of the losses and the embedding.  The distillation loss:
cg_distill_loss forward, cg_distill_grad backward, nothing kept but the inputs
and the normaliser, two values a row (one would lose it in rows far from zero).
The output layer's cross entropy: cg_head_loss and cg_head_grad, which keep the
losses besides, no logits.  The embedding: cg_embed and cg_embed_grad."""

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


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(fn, table, ctx, tokens, scale):
        out = torch.empty((tokens.shape[0], table.shape[1]), dtype=table.dtype, device=table.device)
        with on_ctx_stream(ctx, table, tokens, out):
            ctx.embed(table, tokens, out, scale=scale)
        fn.save_for_backward(tokens)
        fn.ctx, fn.scale = ctx, scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fn, grad):
        (tokens,) = fn.saved_tensors
        grad = grad.contiguous()
        out = torch.empty((fn.ctx.V, grad.shape[1]), dtype=grad.dtype, device=grad.device)
        with on_ctx_stream(fn.ctx, grad, tokens, out):
            fn.ctx.embed_grad(grad, tokens, out, scale=fn.scale)
        return out, None, None, None


class HeadLoss(torch.autograd.Function):
    @staticmethod
    def forward(fn, hidden, weight, ctx, target, temp, bitmask):
        B = hidden.shape[0]
        loss = torch.empty(B, dtype=torch.float32, device=hidden.device)
        norm = torch.empty((B, 2), dtype=torch.float32, device=hidden.device)
        with on_ctx_stream(ctx, hidden, weight, target, bitmask, loss, norm):
            ctx.head_loss(hidden, weight, target, loss, temp=temp, bitmask=bitmask, out_norm=norm)
        fn.save_for_backward(hidden, weight, target, bitmask, loss, norm)
        fn.ctx, fn.temp = ctx, temp
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(fn, grad_loss):
        hidden, weight, target, bitmask, loss, norm = fn.saved_tensors
        grad_loss = grad_loss.contiguous()  # an expanded scalar (loss.sum()) is one value with stride 0
        new = lambda t, wanted: torch.empty(t.shape, dtype=t.dtype, device=t.device) if wanted else None  # noqa: E731
        dh, dw = new(hidden, fn.needs_input_grad[0]), new(weight, fn.needs_input_grad[1])
        if dh is None and dw is None:
            return (None,) * 6
        with on_ctx_stream(fn.ctx, hidden, weight, target, bitmask, loss, norm, grad_loss, dh, dw):
            fn.ctx.head_grad(hidden, weight, target, loss, norm, dh, dw, temp=fn.temp, bitmask=bitmask,
                             grad_loss=grad_loss)
        return dh, dw, None, None, None, None
