"""Argument checks of the per-row operators' Python entry points.  A tensor of
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
