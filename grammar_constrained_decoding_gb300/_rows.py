"""Argument checks of the vocabulary operators' Python entry points.  A tensor of
another shape, type, device (the context's is wanted) or layout raises CgError
with CG_E_ARG before the library sees its pointer."""

from __future__ import annotations

import torch

from . import _lib as L

DTYPE = {torch.float32: L.CG_F32, torch.bfloat16: L.CG_BF16}
LOGITS, F32, U32 = (torch.bfloat16, torch.float32), (torch.float32,), (torch.int32, torch.uint32)


def _refuse(call: str, what: str, dtypes: tuple, shape: tuple, dev: int, layout: str):
    kinds = " or ".join(str(d).removeprefix("torch.") for d in dtypes)
    raise L.CgError(call, L.CG_E_ARG, f"{what}: a {layout} tensor {kinds} {list(shape)} on cuda:{dev} is wanted")


def want(call: str, t, what: str, dtypes: tuple, shape: tuple, dev: int = 0) -> int:
    """Pointer of a contiguous tensor of one of the dtypes and the shape on CUDA device dev."""
    if t.get_device() != dev or t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        _refuse(call, what, dtypes, shape, dev, "contiguous")
    return t.data_ptr()


def opt(call: str, t, what: str, dtypes: tuple, shape: tuple, dev: int = 0) -> int | None:
    return None if t is None else want(call, t, what, dtypes, shape, dev)


def rows_of(call: str, t, what: str, dtypes: tuple, shape: tuple, dev: int = 0) -> tuple[int, int]:
    """(pointer, row stride in elements) of a matrix on CUDA device dev whose rows are contiguous."""
    if t.get_device() != dev or t.dtype not in dtypes or t.shape != shape or (t.stride(1) != 1 and shape[1] != 1):
        _refuse(call, what, dtypes, shape, dev, "row-contiguous")
    return t.data_ptr(), (t.stride(0) if shape[0] > 1 else shape[1])


def matrix_of(call: str, t, what: str, dtype, rows: int, dev: int = 0) -> tuple[int, int, int]:
    """(pointer, row stride in elements, columns) of a matrix of `rows` rows and any width (dtype None: of
    either float type)."""
    if t.dim() != 2:
        raise L.CgError(call, L.CG_E_ARG, f"{what}: a matrix is wanted")
    shape = (rows, t.shape[1])
    return *rows_of(call, t, what, LOGITS if dtype is None else (dtype,), shape, dev), t.shape[1]


try:  # the handle alone: a microsecond less than the stream object
    from torch._C import _cuda_getCurrentRawStream as raw_stream
except ImportError:  # a build of torch without CUDA, or one that names it otherwise
    def raw_stream(dev: int) -> int:
        return torch.cuda.current_stream(dev).cuda_stream

KEPT_WORKSPACE = 64 << 20   # bytes: what a thread keeps between its calls; larger ones are allocated for each


def with_workspace(ctx, call: str, given, need, entry, args) -> None:
    """entry(*args, workspace, its bytes) in the caller's workspace (a u8 tensor), or in one that the library's own
    need() says the size of:
      - the one that this thread's calls on the context's stream have kept (allocating in every call costs as
        much host time as a small call itself), tried before need() is asked;
      - a new one, which belongs to the context's stream: in a graph capture, which has to own what its replays
        use, for a stream that is not torch's current one, and for large calls."""
    if given is not None:
        want(call, given, "workspace", (torch.uint8,), given.shape, ctx._dev)
        L.check(call, entry(*args, given.data_ptr(), given.numel()))
        return
    here = raw_stream(ctx._dev) == ctx._stream
    may_keep = here and not torch.cuda.is_current_stream_capturing()
    kept = getattr(ctx._kept, "workspace", None) if may_keep else None
    if kept is not None:
        rc = entry(*args, kept.data_ptr(), kept.numel())
        if rc != L.CG_E_NOMEM:
            L.check(call, rc)
            return
    nbytes = max(need(), 256)
    if here:
        new = torch.empty(max(nbytes, 1 << 20) if may_keep else nbytes, dtype=torch.uint8, device=ctx._dev)
        if may_keep and nbytes <= KEPT_WORKSPACE:
            ctx._kept.workspace = new
    else:
        with torch.cuda.stream(ctx.stream):
            new = torch.empty(nbytes, dtype=torch.uint8, device=ctx._dev)
    L.check(call, entry(*args, new.data_ptr(), new.numel()))
