"""GB300-native grammar-constrained decoding: Python binding of libcg.so.

Every operation runs in the C/CUDA library (include/cg.h); this module only
marshals arguments: numpy arrays for host data, torch CUDA tensors (pointers
and the current stream) for device data.

    g = Grammar.compile(source, kind="json", bounds=Bounds())
    v = Vocab(list_of_token_bytes)
    ctx = Ctx([g], v)                        # binds torch's current CUDA stream
    ctx.fill_bitmask(states, bitmask, gid=None, forced=None)
    ctx.mask_and_sample(logits, bitmask, temp, top_p, seed, step, out_tok)
    ctx.accept(states, toks, out_states, out_flags)

On the same masked rows, with settings and random numbers per row, the best
tokens, and a student's distillation loss (see distill() for autograd):

    ctx.sample_rows(logits, uniform, out_tok, bitmask, temp, top_k, top_p, min_p)
    ctx.top_logprobs(logits, out_ids, out_logprobs, bitmask)
    ctx.distill_loss(logits, ids, teacher, out_loss, temp, bitmask)

And the model's two ends, where tokens become rows and rows become logits (see
embed() and head_loss() for autograd):

    ctx.embed(table, tokens, out, scale)
    ctx.head_loss(hidden, weight, target, out_loss, temp, bitmask)
"""

from __future__ import annotations

import ctypes as C
import threading
from dataclasses import dataclass

import numpy as np

from . import _lib as L
from ._lib import (CG_DEAD, CG_FLAG_CAPPED, CG_FLAG_DONE, CG_FLAG_FORCED_NEXT,  # noqa: F401
                   CG_FLAG_NO_TOKEN, CG_FLAG_REJECTED, CG_NO_TOKEN, CG_STATE_ACCEPT,
                   CG_STATE_FORCED_ONLY, CG_STATE_SINK, CgError)


@dataclass(frozen=True)
class Bounds:
    ws_max: int = 4
    max_len_default: int = 256
    depth_max: int = 5
    max_items_default: int = 16
    max_tokens: int = 2048

    def c(self) -> L.cg_bounds:
        return L.cg_bounds(self.ws_max, self.max_len_default, self.depth_max, self.max_items_default,
                           self.max_tokens)


def _u32p(x):
    return C.byref(x)


class Grammar:
    def __init__(self, handle):
        self._h = C.c_void_p(handle)

    @classmethod
    def compile(cls, source: str | bytes, kind: str = "gbnf", bounds: Bounds = Bounds()) -> "Grammar":
        data = source.encode("utf-8") if isinstance(source, str) else bytes(source)
        out = C.c_void_p()
        err = C.create_string_buffer(512)
        k = {"gbnf": L.CG_GBNF, "json": L.CG_JSON_SCHEMA, "structtag": L.CG_STRUCTURAL_TAG}[kind]
        b = bounds.c()
        rc = L.lib().cg_compile(data, len(data), k, C.byref(b), C.byref(out), err, len(err))
        L.check("cg_compile", rc, err.value.decode("utf-8", "replace"))
        return cls(out.value)

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value:
            L.lib().cg_grammar_destroy(self._h)
            self._h = C.c_void_p()

    def info(self) -> dict:
        n, cols, start = C.c_uint32(), C.c_uint32(), C.c_uint32()
        L.check("cg_grammar_info", L.lib().cg_grammar_info(self._h, C.byref(n), C.byref(cols), C.byref(start)))
        return {"n_states": n.value, "n_cols": cols.value, "start": start.value}

    def export(self) -> tuple[np.ndarray, np.ndarray]:
        S = self.info()["n_states"]
        nxt = np.empty((S, 512), dtype=np.int32)
        flags = np.empty(S, dtype=np.uint8)
        L.check("cg_grammar_export", L.lib().cg_grammar_export(self._h, nxt.ctypes.data, flags.ctypes.data))
        return nxt, flags

    def try_input(self, data: bytes, injected: np.ndarray | None = None) -> tuple[int, int, bool]:
        ref, end, acc = C.c_size_t(), C.c_uint32(), C.c_int()
        inj = None
        if injected is not None:
            injected = np.ascontiguousarray(injected, dtype=np.uint8)
            inj = injected.ctypes.data
        L.check("cg_try_input", L.lib().cg_try_input(self._h, data, len(data), inj, C.byref(ref), C.byref(end),
                                                      C.byref(acc)))
        return ref.value, end.value, bool(acc.value)

    def live_states(self) -> np.ndarray:
        n = C.c_uint32()
        L.check("cg_live_states", L.lib().cg_live_states(self._h, None, 0, C.byref(n)))
        out = np.empty(n.value, dtype=np.uint32)
        L.check("cg_live_states", L.lib().cg_live_states(self._h, out.ctypes.data, n.value, C.byref(n)))
        return out


class Vocab:
    def __init__(self, tokens: list[bytes]):
        off = np.zeros(len(tokens) + 1, dtype=np.uint32)
        off[1:] = np.cumsum([len(t) for t in tokens])
        data = np.frombuffer(b"".join(tokens), dtype=np.uint8).copy()
        h = C.c_void_p()
        L.check("cg_vocab_create", L.lib().cg_vocab_create(data.ctypes.data, off.ctypes.data, len(tokens), C.byref(h)))
        self._h = h
        self.V = len(tokens)

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value:
            L.lib().cg_vocab_destroy(self._h)
            self._h = C.c_void_p()

    def tokenize_greedy(self, text: bytes) -> list[int]:
        out = np.empty(len(text) + 1, dtype=np.uint32)
        n = C.c_size_t()
        L.check("cg_tokenize_greedy", L.lib().cg_tokenize_greedy(self._h, text, len(text), out.ctypes.data,
                                                                  len(out), C.byref(n)))
        return out[:n.value].tolist()


def eval_arith(span: bytes, fmt: str) -> tuple[bytes, bool]:
    f = {"calc_tag": L.CG_RESULT_CALC_TAG, "json_answer": L.CG_RESULT_JSON_ANSWER}[fmt]
    buf = C.create_string_buffer(256)
    n, ok = C.c_size_t(), C.c_int()
    L.check("cg_eval_arith", L.lib().cg_eval_arith(span, len(span), f, buf, len(buf), C.byref(n), C.byref(ok)))
    return buf.raw[:n.value], bool(ok.value)


def mask_classes(grammars: list["Grammar"], max_len: int) -> tuple[np.ndarray, int]:
    """Joint mask classes of grammars used in one context: (class of every
    state, grammar after grammar; number of classes)."""
    arr = (C.c_void_p * len(grammars))(*[g._h.value for g in grammars])
    S, n = C.c_uint32(), C.c_uint32()
    L.check("cg_mask_classes", L.lib().cg_mask_classes(arr, len(grammars), max_len, None, 0, C.byref(S), C.byref(n)))
    out = np.zeros(S.value, dtype=np.uint32)
    L.check("cg_mask_classes", L.lib().cg_mask_classes(arr, len(grammars), max_len, out.ctypes.data, S.value,
                                                        C.byref(S), C.byref(n)))
    return out, n.value


def eval_strop(span: bytes) -> tuple[bytes, bool]:
    """A string operation's forced bytes (<result>V</result> or <result_error>code</result_error>)."""
    buf = C.create_string_buffer(256)
    n, ok = C.c_size_t(), C.c_int()
    L.check("cg_eval_strop", L.lib().cg_eval_strop(span, len(span), buf, len(buf), C.byref(n), C.byref(ok)))
    return buf.raw[:n.value], bool(ok.value)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


class Ctx:
    """Device context bound to one CUDA stream (torch's current stream by default)."""

    def __init__(self, grammars: list[Grammar], vocab: Vocab, stream=None):
        import torch
        from . import _rows
        if stream is None:
            stream = torch.cuda.current_stream()
        self.stream = stream
        self._stream = stream.cuda_stream
        self._kept = threading.local()  # a workspace for each thread's calls
        self._dev = torch.cuda.current_device()  # where the library creates the context
        self._rows = _rows  # an import in every call would be a twentieth of the smallest
        arr = (C.c_void_p * len(grammars))(*[g._h.value for g in grammars])
        h = C.c_void_p()
        L.check("cg_ctx_create", L.lib().cg_ctx_create(arr, len(grammars), vocab._h, C.c_void_p(stream.cuda_stream),
                                                       C.byref(h)))
        self._h = h
        self.V = vocab.V
        self.W = (vocab.V + 31) // 32

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value:
            L.lib().cg_ctx_destroy(self._h)
            self._h = C.c_void_p()

    def info(self) -> dict:
        nc, cb, V, W = C.c_uint32(), C.c_uint64(), C.c_uint32(), C.c_uint32()
        L.check("cg_ctx_info", L.lib().cg_ctx_info(self._h, C.byref(nc), C.byref(cb), C.byref(V), C.byref(W)))
        return {"n_classes": nc.value, "cache_bytes": cb.value, "V": V.value, "W": W.value}

    def status(self) -> int:
        code = C.c_uint32()
        rc = L.lib().cg_ctx_status(self._h, C.byref(code))
        if rc not in (L.CG_OK, L.CG_E_DEVICE):
            L.check("cg_ctx_status", rc)
        return code.value

    def prefill(self) -> None:
        L.check("cg_ctx_prefill", L.lib().cg_ctx_prefill(self._h))

    def cache_stats(self) -> dict:
        """Mask-cache counters (synchronises the stream): lookups and class masks
        computed by the segmented fused step's pre-pass, and the class masks in
        the cache now by any path ("ready", of info()["n_classes"])."""
        lk, cm, rd = C.c_uint64(), C.c_uint64(), C.c_uint32()
        L.check("cg_ctx_cache_stats", L.lib().cg_ctx_cache_stats(self._h, C.byref(lk), C.byref(cm), C.byref(rd)))
        return {"lookups": lk.value, "computed": cm.value, "ready": rd.value}

    def fill_bitmask(self, states, bitmask, gid=None, forced=None) -> None:
        B = states.shape[0]
        L.check("cg_fill_bitmask", L.lib().cg_fill_bitmask(self._h, _ptr(states), _ptr(gid), _ptr(forced), B,
                                                            _ptr(bitmask)))

    def mask_and_sample(self, logits, bitmask, temp: float, top_p: float, seed: int, step: int, out_tok,
                        probs=None, inplace: bool = False) -> None:
        import torch
        dtype = {torch.float32: L.CG_F32, torch.bfloat16: L.CG_BF16}[logits.dtype]
        B, V = logits.shape
        L.check("cg_mask_and_sample", L.lib().cg_mask_and_sample(
            self._h, _ptr(logits), dtype, B, V, _ptr(bitmask), float(temp), float(top_p), int(seed), int(step),
            _ptr(out_tok), _ptr(probs), L.CG_SAMPLE_INPLACE if inplace else 0))

    def mask_and_sample_noalloc(self, logits, bitmask, temp: float, top_p: float, seed: int, step: int, out_tok,
                                probs=None, inplace: bool = False) -> None:
        """mask_and_sample on the library's fixed scratch (no device allocation;
        B <= CG_NOALLOC_MAX_ROWS; overlapping calls on one device race)."""
        import torch
        dtype = {torch.float32: L.CG_F32, torch.bfloat16: L.CG_BF16}[logits.dtype]
        B, V = logits.shape
        L.check("cg_mask_and_sample_noalloc", L.lib().cg_mask_and_sample_noalloc(
            self._h, _ptr(logits), dtype, B, V, _ptr(bitmask), float(temp), float(top_p), int(seed), int(step),
            _ptr(out_tok), _ptr(probs), L.CG_SAMPLE_INPLACE if inplace else 0))

    def accept(self, states, toks, out_states, out_flags, gid=None, forced=None, counts=None,
               max_tokens: int = 2048) -> None:
        B = states.shape[0]
        L.check("cg_accept", L.lib().cg_accept(self._h, _ptr(states), _ptr(gid), _ptr(toks), _ptr(forced), B,
                                                _ptr(counts), max_tokens, _ptr(out_states), _ptr(out_flags)))


    def step(self, states, logits, temp: float, top_p: float, seed: int, step: int, out_tok, out_states, out_flags,
             gid=None, forced=None, counts=None, max_tokens: int = 2048, bitmask=None) -> None:
        """fill_bitmask + mask_and_sample + accept in one call (one segmented
        kernel for bf16 logits); bitmask, when given, receives the row masks."""
        import torch
        dtype = {torch.float32: L.CG_F32, torch.bfloat16: L.CG_BF16}[logits.dtype]
        B, V = logits.shape
        L.check("cg_step", L.lib().cg_step(
            self._h, _ptr(states), _ptr(gid), _ptr(forced), B, _ptr(logits), dtype, V, float(temp), float(top_p),
            int(seed), int(step), _ptr(counts), max_tokens, _ptr(bitmask), _ptr(out_tok), _ptr(out_states),
            _ptr(out_flags)))


    def accept_many(self, states, draft, draft_len, out_states, out_n, out_flags, gid=None, forced=None,
                    counts=None, max_tokens: int = 2048, path=None) -> None:
        """Speculative verification: the longest grammatical prefix of each row's
        draft ([B, K] ids, draft_len per row); forced [B, K] pins positions."""
        B, K = draft.shape
        L.check("cg_accept_many", L.lib().cg_accept_many(
            self._h, _ptr(states), _ptr(gid), _ptr(draft), _ptr(draft_len), _ptr(forced), B, K, _ptr(counts),
            max_tokens, _ptr(out_states), _ptr(out_n), _ptr(out_flags), _ptr(path)))

    def step_host(self, states, h_logits, temp: float, top_p: float, seed: int, step: int, h_out_tok, out_states,
                  out_flags, gid=None, forced=None, counts=None, max_tokens: int = 2048, out_tok=None) -> None:
        """cg_step with the logits in (page-locked) host memory and the ids
        copied back to host memory; asynchronous until sync()."""
        import torch
        dtype = {torch.float32: L.CG_F32, torch.bfloat16: L.CG_BF16}[h_logits.dtype]
        B, V = h_logits.shape
        L.check("cg_step_host", L.lib().cg_step_host(
            self._h, _ptr(states), _ptr(gid), _ptr(forced), B, _ptr(h_logits), dtype, V, float(temp), float(top_p),
            int(seed), int(step), _ptr(counts), max_tokens, _ptr(h_out_tok), _ptr(out_tok), _ptr(out_states),
            _ptr(out_flags)))

    def sample_rows(self, logits, uniform, out_tok, bitmask=None, temp=None, top_k=None, top_p=None, min_p=None,
                    out_logprob=None) -> None:
        """One token per row: temperature, top-k, top-p and min-p of each row's
        own ([B] tensors or None), drawn with the given random numbers uniform
        [B, V] (a [1, V] or expanded tensor shares one row; None for an all-greedy
        batch); out_logprob receives log p of the token before any cut."""
        R, call, dev, B, W = self._rows, "cg_sample_rows", self._dev, logits.shape[0], self.W
        x, ld = R.rows_of(call, logits, "logits", R.LOGITS, (B, self.V), dev)
        u, ldu = None, 0
        if uniform is not None:
            shared = uniform.shape[0] == 1
            u, ldu = R.rows_of(call, uniform, "uniform", R.F32, (1 if shared else B, self.V), dev)
            ldu = 0 if shared else ldu
        each = (B,)
        rc = L.lib().cg_sample_rows(
            self._h, x, R.DTYPE[logits.dtype], B, self.V, ld, R.opt(call, bitmask, "bitmask", R.U32, (B, W), dev),
            R.opt(call, temp, "temp", R.F32, each, dev), R.opt(call, top_k, "top_k", R.U32, each, dev),
            R.opt(call, top_p, "top_p", R.F32, each, dev), R.opt(call, min_p, "min_p", R.F32, each, dev), u, ldu,
            R.want(call, out_tok, "out_tok", R.U32, each, dev),
            R.opt(call, out_logprob, "out_logprob", R.F32, each, dev))
        L.check(call, rc)

    def top_logprobs(self, logits, out_ids, out_logprobs, bitmask=None, out_lse=None) -> None:
        """The n best allowed tokens of each row (n = out_ids.shape[1]), best
        first, with their log-probabilities."""
        R, call, dev, B, n = self._rows, "cg_top_logprobs", self._dev, logits.shape[0], out_ids.shape[1]
        x, ld = R.rows_of(call, logits, "logits", R.LOGITS, (B, self.V), dev)
        rc = L.lib().cg_top_logprobs(
            self._h, x, R.DTYPE[logits.dtype], B, self.V, ld,
            R.opt(call, bitmask, "bitmask", R.U32, (B, self.W), dev), n,
            R.want(call, out_ids, "out_ids", R.U32, (B, n), dev),
            R.want(call, out_logprobs, "out_logprobs", R.F32, (B, n), dev),
            R.opt(call, out_lse, "out_lse", R.F32, (B,), dev))
        L.check(call, rc)

    def distill_loss(self, logits, ids, teacher, out_loss, temp: float = 1.0, bitmask=None, out_lse=None,
                     out_grad=None, grad_loss=None, out_norm=None) -> None:
        """Loss of each row against the teacher's listed tokens (ids, teacher
        [B, K]); with out_grad also the gradient by the logits, times grad_loss [B].
        out_norm [B, 2] receives the normaliser as distill_grad takes it."""
        R, call, dev, B, K = self._rows, "cg_distill_loss", self._dev, logits.shape[0], ids.shape[1]
        x, ld = R.rows_of(call, logits, "logits", R.LOGITS, (B, self.V), dev)
        g, ldg = None, 0
        if out_grad is not None:
            g, ldg = R.rows_of(call, out_grad, "out_grad", (logits.dtype,), (B, self.V), dev)
        rc = L.lib().cg_distill_loss_norm(
            self._h, x, R.DTYPE[logits.dtype], B, self.V, ld, R.opt(call, bitmask, "bitmask", R.U32, (B, self.W), dev),
            R.want(call, ids, "ids", R.U32, (B, K), dev), R.want(call, teacher, "teacher", R.F32, (B, K), dev), K, temp,
            R.want(call, out_loss, "out_loss", R.F32, (B,), dev), R.opt(call, out_lse, "out_lse", R.F32, (B,), dev),
            R.opt(call, out_norm, "out_norm", R.F32, (B, 2), dev),
            R.opt(call, grad_loss, "grad_loss", R.F32, (B,), dev), g, ldg)
        L.check(call, rc)

    def distill_grad(self, logits, ids, teacher, lse, out_grad, temp: float = 1.0, bitmask=None,
                     grad_loss=None, norm=None) -> None:
        """The gradient alone, from the normaliser that distill_loss left in out_norm
        (norm, with lse None) or, to the rounding of one value a row, in out_lse."""
        R, call, dev, B, K = self._rows, "cg_distill_grad", self._dev, logits.shape[0], ids.shape[1]
        x, ld = R.rows_of(call, logits, "logits", R.LOGITS, (B, self.V), dev)
        g, ldg = R.rows_of(call, out_grad, "out_grad", (logits.dtype,), (B, self.V), dev)
        if (lse is None) == (norm is None):
            raise L.CgError(call, L.CG_E_ARG, "lse or norm: one of the two is wanted")
        if norm is None:
            entry, kept = L.lib().cg_distill_grad, R.want(call, lse, "lse", R.F32, (B,), dev)
        else:
            entry, kept = L.lib().cg_distill_grad_norm, R.want(call, norm, "norm", R.F32, (B, 2), dev)
        rc = entry(
            self._h, x, R.DTYPE[logits.dtype], B, self.V, ld, R.opt(call, bitmask, "bitmask", R.U32, (B, self.W), dev),
            R.want(call, ids, "ids", R.U32, (B, K), dev), R.want(call, teacher, "teacher", R.F32, (B, K), dev), K, temp,
            kept, R.opt(call, grad_loss, "grad_loss", R.F32, (B,), dev), g, ldg)
        L.check(call, rc)

    def embed(self, table, tokens, out, scale: float = 1.0) -> None:
        """out[i] = scale * table[tokens[i]] (zeros where tokens[i] is CG_NO_TOKEN): table [V, D], tokens [N], out [N, D]."""
        R, call, dev, N = self._rows, "cg_embed", self._dev, tokens.shape[0]
        t, ld, D = R.matrix_of(call, table, "table", None, self.V, dev)
        o, ldo = R.rows_of(call, out, "out", (table.dtype,), (N, D), dev)
        L.check(call, L.lib().cg_embed(self._h, t, R.DTYPE[table.dtype], self.V, D, ld,
                                       R.want(call, tokens, "tokens", R.U32, (N,), dev), N, scale, o, ldo))

    def embed_workspace(self, grad, tokens) -> int:
        """Bytes that embed_grad works in."""
        n, call, N = C.c_size_t(), "cg_embed_workspace", tokens.shape[0]
        D = self._rows.matrix_of(call, grad, "grad", None, N, self._dev)[2]
        L.check(call, L.lib().cg_embed_workspace(self._h, self._rows.DTYPE[grad.dtype], N, D, C.byref(n)))
        return n.value

    def embed_grad(self, grad, tokens, out_grad, scale: float = 1.0, accumulate: bool = False, workspace=None) -> None:
        """out_grad[v] = scale * sum of grad[i] over the i with tokens[i] == v, or added to it: grad [N, D],
        tokens [N], out_grad [V, D].  workspace: u8 tensor of embed_workspace() bytes, else one is allocated."""
        R, call, dev, N = self._rows, "cg_embed_grad", self._dev, tokens.shape[0]
        g, ld, D = R.matrix_of(call, grad, "grad", None, N, dev)
        o, ldo = R.rows_of(call, out_grad, "out_grad", (grad.dtype,), (self.V, D), dev)
        tok = R.want(call, tokens, "tokens", R.U32, (N,), dev)
        R.with_workspace(self, call, workspace, lambda: self.embed_workspace(grad, tokens), L.lib().cg_embed_grad,
                         (self._h, g, R.DTYPE[grad.dtype], N, self.V, D, ld, tok, scale, int(accumulate), o, ldo))

    def _head_operands(self, call, hidden, weight):
        """(what the calls take of the two matrices, B, D)."""
        R, dev, B = self._rows, self._dev, hidden.shape[0]
        h, ldh, D = R.matrix_of(call, hidden, "hidden", None, B, dev)
        w, ldw = R.rows_of(call, weight, "weight", (hidden.dtype,), (self.V, D), dev)
        return (self._h, h, w, R.DTYPE[hidden.dtype], B, self.V, D, ldh, ldw), B, D

    def _head_bytes(self, operands, grad) -> int:
        n = C.c_size_t()
        L.check("cg_head_workspace", L.lib().cg_head_workspace(*operands, grad, C.byref(n)))
        return n.value

    def head_workspace(self, hidden, weight, grad: bool = False) -> int:
        """Bytes that head_loss (or head_grad) works in."""
        return self._head_bytes(self._head_operands("cg_head_workspace", hidden, weight)[0], int(grad))

    def head_loss(self, hidden, weight, target, out_loss, temp: float = 1.0, bitmask=None, out_lse=None,
                  out_norm=None, workspace=None) -> None:
        """Cross entropy of each row of hidden [B, D] against its target token [B] over the allowed tokens, the
        logits hidden @ weight.T (weight [V, D]) never stored; out_norm [B, 2] receives the normaliser as
        head_grad takes it.  workspace: u8 tensor of head_workspace() bytes, else one is allocated."""
        R, call, dev = self._rows, "cg_head_loss", self._dev
        operands, B, _ = self._head_operands(call, hidden, weight)
        mask = R.opt(call, bitmask, "bitmask", R.U32, (B, self.W), dev)
        t, loss = R.want(call, target, "target", R.U32, (B,), dev), R.want(call, out_loss, "out_loss", R.F32, (B,), dev)
        lse, norm = R.opt(call, out_lse, "out_lse", R.F32, (B,), dev), R.opt(call, out_norm, "out_norm", R.F32, (B, 2), dev)
        R.with_workspace(self, call, workspace, lambda: self._head_bytes(operands, 0), L.lib().cg_head_loss,
                         (*operands, mask, t, temp, loss, lse, norm))

    def head_grad(self, hidden, weight, target, loss, norm, out_grad_hidden=None, out_grad_weight=None,
                  temp: float = 1.0, bitmask=None, grad_loss=None, workspace=None) -> None:
        """The gradients of the sum of grad_loss [B] * loss by hidden and by weight (one of them may be None), from
        the loss and the normaliser that head_loss left.  workspace: of head_workspace(..., grad=True) bytes."""
        R, call, dev = self._rows, "cg_head_grad", self._dev
        operands, B, D = self._head_operands(call, hidden, weight)
        dh, lddh, dw, lddw = None, 0, None, 0
        if out_grad_hidden is not None:
            dh, lddh = R.rows_of(call, out_grad_hidden, "out_grad_hidden", (hidden.dtype,), (B, D), dev)
        if out_grad_weight is not None:
            dw, lddw = R.rows_of(call, out_grad_weight, "out_grad_weight", (hidden.dtype,), (self.V, D), dev)
        mask = R.opt(call, bitmask, "bitmask", R.U32, (B, self.W), dev)
        t, kept = R.want(call, target, "target", R.U32, (B,), dev), R.want(call, loss, "loss", R.F32, (B,), dev)
        norm = R.want(call, norm, "norm", R.F32, (B, 2), dev)
        up = R.opt(call, grad_loss, "grad_loss", R.F32, (B,), dev)
        R.with_workspace(self, call, workspace, lambda: self._head_bytes(operands, 1), L.lib().cg_head_grad,
                         (*operands, mask, t, temp, kept, norm, up, dh, lddh, dw, lddw))

    def self_test_cluster_timeout(self, out) -> None:
        """Make a block of a cluster give up while others still send to it (the status then
        reads CG_DEV_TIMEOUT); out [1] receives the number of messages it stayed for (6)."""
        call = "cg_self_test_cluster_timeout"
        L.check(call, L.lib().cg_self_test_cluster_timeout(
            self._h, self._rows.want(call, out, "out", self._rows.U32, (1,), self._dev)))

    def self_test_wait_timeout(self) -> None:
        """Make one bounded device wait run out (the status then reads CG_DEV_TIMEOUT)."""
        L.check("cg_self_test_wait_timeout", L.lib().cg_self_test_wait_timeout(self._h))

    def sync(self) -> None:
        L.check("cg_ctx_sync", L.lib().cg_ctx_sync(self._h))


class PdaGrammar:
    """A recursive GBNF grammar compiled to a pushdown automaton with a stack
    bound of ``depth`` frames (cg_pda_compile)."""

    def __init__(self, source: str | bytes, depth: int):
        data = source.encode("utf-8") if isinstance(source, str) else bytes(source)
        out = C.c_void_p()
        L.check("cg_pda_compile", L.lib().cg_pda_compile(data, len(data), int(depth), C.byref(out)))
        self._h = out

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value:
            L.lib().cg_pda_grammar_destroy(self._h)
            self._h = C.c_void_p()

    def info(self) -> dict:
        n, r, cols, d = C.c_uint32(), C.c_uint32(), C.c_uint32(), C.c_uint32()
        L.check("cg_pda_grammar_info", L.lib().cg_pda_grammar_info(self._h, C.byref(n), C.byref(r), C.byref(cols),
                                                                    C.byref(d)))
        return {"n_states": n.value, "n_rules": r.value, "n_cols": cols.value, "depth": d.value}

    def try_input(self, data: bytes, injected: np.ndarray | None = None) -> tuple[int, bool, int]:
        """(bytes walked before the first refused one, complete, stack level)."""
        n, acc, lvl = C.c_size_t(), C.c_int(), C.c_uint32()
        inj = None
        if injected is not None:
            injected = np.ascontiguousarray(injected, dtype=np.uint8)
            inj = injected.ctypes.data
        L.check("cg_pda_try_input", L.lib().cg_pda_try_input(self._h, data, len(data), inj, C.byref(n),
                                                              C.byref(acc), C.byref(lvl)))
        return n.value, bool(acc.value), lvl.value


class Pda:
    """Pushdown rows on a context (cg_pda_create).  Row configurations are a
    u32 tensor [B, depth + 2]: state, stack level, return states."""

    def __init__(self, ctx: Ctx, vocab: Vocab, grammar: PdaGrammar):
        h = C.c_void_p()
        L.check("cg_pda_create", L.lib().cg_pda_create(ctx._h, vocab._h, grammar._h, C.byref(h)))
        self._h = h
        self._ctx = ctx  # destroyed before its context
        self.depth = grammar.info()["depth"]
        self.row_words = self.depth + 2

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value:
            L.lib().cg_pda_destroy(self._h)
            self._h = C.c_void_p()

    def info(self) -> dict:
        k, m, cb, nc = C.c_uint32(), C.c_uint32(), C.c_uint64(), C.c_uint32()
        L.check("cg_pda_info", L.lib().cg_pda_info(self._h, C.byref(k), C.byref(m), C.byref(cb), C.byref(nc)))
        return {"n_keys": k.value, "n_masks": m.value, "cache_bytes": cb.value, "n_candidates": nc.value}

    def fill_bitmask(self, cfg, bitmask, forced=None) -> None:
        L.check("cg_pda_fill_bitmask", L.lib().cg_pda_fill_bitmask(self._h, _ptr(cfg), cfg.shape[0], _ptr(forced),
                                                                    _ptr(bitmask)))

    def accept(self, cfg, toks, out_flags, forced=None, counts=None, max_tokens: int = 0) -> None:
        L.check("cg_pda_accept", L.lib().cg_pda_accept(self._h, _ptr(cfg), cfg.shape[0], _ptr(toks), _ptr(forced),
                                                        _ptr(counts), int(max_tokens), _ptr(out_flags)))

    def step(self, cfg, logits, temp: float, top_p: float, seed: int, step: int, out_tok, out_flags, forced=None,
             counts=None, max_tokens: int = 0, bitmask=None) -> None:
        """mask, sample and accept in one call (one kernel on the bf16 top-p path)."""
        import torch
        dtype = {torch.float32: L.CG_F32, torch.bfloat16: L.CG_BF16}[logits.dtype]
        B, V = logits.shape
        L.check("cg_pda_step", L.lib().cg_pda_step(
            self._h, _ptr(cfg), B, _ptr(logits), dtype, V, float(temp), float(top_p), int(seed), int(step),
            _ptr(forced), _ptr(counts), int(max_tokens), _ptr(bitmask), _ptr(out_tok), _ptr(out_flags)))

    def accept_many(self, cfg, draft, draft_len, out_n, out_flags, forced=None, counts=None,
                    max_tokens: int = 0) -> None:
        """Speculative verification of drafts [B, K] against the rows' configurations."""
        B, K = draft.shape
        L.check("cg_pda_accept_many", L.lib().cg_pda_accept_many(
            self._h, _ptr(cfg), B, _ptr(draft), _ptr(draft_len), _ptr(forced), K, _ptr(counts), int(max_tokens),
            _ptr(out_n), _ptr(out_flags)))

    def accept_fill(self, cfg, toks, out_flags, bitmask, forced=None, counts=None, max_tokens: int = 0,
                    forced_next=None) -> None:
        """accept, then fill_bitmask of the next step, in one launch."""
        L.check("cg_pda_accept_fill", L.lib().cg_pda_accept_fill(
            self._h, _ptr(cfg), cfg.shape[0], _ptr(toks), _ptr(forced), _ptr(counts), int(max_tokens),
            _ptr(out_flags), _ptr(forced_next), _ptr(bitmask)))


class Driver:
    """Host driver of forced tokens (evaluator-aware grammars)."""

    def __init__(self, vocab: Vocab, B: int, gid: np.ndarray | None, rules: list[tuple[bytes, bytes, int]]):
        self._keep = []
        arr = (L.cg_span_rule * len(rules))()
        for i, (op, cl, fmt) in enumerate(rules):
            bo = C.create_string_buffer(op, len(op) or 1)
            bc = C.create_string_buffer(cl, len(cl) or 1)
            self._keep += [bo, bc]
            arr[i] = L.cg_span_rule(C.cast(bo, C.c_void_p), len(op), C.cast(bc, C.c_void_p), len(cl), fmt)
        g = None
        if gid is not None:
            self._gid = np.ascontiguousarray(gid, dtype=np.uint16)
            g = self._gid.ctypes.data
        h = C.c_void_p()
        L.check("cg_driver_create", L.lib().cg_driver_create(vocab._h, B, g, arr, len(rules), C.byref(h)))
        self._h = h
        self.B = B

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value:
            L.lib().cg_driver_destroy(self._h)
            self._h = C.c_void_p()

    def update(self, toks: np.ndarray, flags: np.ndarray, forced_used: np.ndarray, forced_next: np.ndarray) -> int:
        n = C.c_uint32()
        L.check("cg_driver_update", L.lib().cg_driver_update(self._h, toks.ctypes.data, flags.ctypes.data,
                                                              forced_used.ctypes.data, forced_next.ctypes.data,
                                                              C.byref(n)))
        return n.value


def distill(ctx: Ctx, logits, ids, teacher, temp: float = 1.0, bitmask=None):
    """Distillation loss of each row, f32 [B], differentiable by logits (and by
    nothing else): Ctx.distill_loss forward, Ctx.distill_grad backward.  Runs on
    the context's stream, ordered after and before torch's current one."""
    from .autograd import DistillLoss
    return DistillLoss.apply(logits, ctx, ids, teacher, float(temp), bitmask)


def embed(ctx: Ctx, table, tokens, scale: float = 1.0):
    """scale * table[tokens], [N, D] of the table's dtype (zeros where a token is CG_NO_TOKEN), differentiable by
    table [V, D]: Ctx.embed forward, Ctx.embed_grad backward.  Ordered with torch's current stream as distill()."""
    from .autograd import Embed
    return Embed.apply(table, ctx, tokens, float(scale))


def head_loss(ctx: Ctx, hidden, weight, target, temp: float = 1.0, bitmask=None):
    """Cross entropy of each row, f32 [B], of the output layer hidden [B, D] @ weight [V, D].T over the allowed
    tokens, differentiable by hidden and weight, no logits kept: Ctx.head_loss forward, Ctx.head_grad backward.
    Rows whose target is CG_NO_TOKEN or forbidden have loss 0.  Ordered with torch's current stream as distill()."""
    from .autograd import HeadLoss
    return HeadLoss.apply(hidden, weight, ctx, target, float(temp), bitmask)
