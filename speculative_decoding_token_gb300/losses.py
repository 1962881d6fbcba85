"""Log-probabilities of given tokens and distillation of a draft: the binding of the ``specverify_token_logprobs*`` and
``specverify_distill_*`` calls of ``include/specverify.h``, as methods of :class:`SpecVerify`.

A training step of a draft on text that its target has scored::

    sv = SpecVerify(1, 1, V)
    top = sv.token_logprobs(target_logits, tokens, T, k=64)                 # tokens [rows]; kept with the text
    grad, loss = sv.distill_grad(draft_logits, top.topk_idx, top.topk_logprob, weight, T, "fkl")
    draft_logits.backward(grad)                                             # on into the draft

and what a server returns of the tokens that a step emitted::

    n, tokens = sv.verify(target, draft, p_off, q_off, drafts, gamma, T, seed)
    r = sv.token_logprobs(target, tokens, T, k=5, row_off=p_off)            # r.logprob [B, gamma_max + 1]
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

torch = None  # imported by bind(), when the library is loaded: this module, like its package, does without until then

FP32, BF16 = 0, 1
MAX_ALTERNATIVES, MAX_LIST = 128, 256
MAX_INT32 = 2 ** 31 - 1
DIVERGENCES = {"fkl": 0, "rkl": 1, "jsd": 2, "tvd": 3}
FORMS = {"logprobs": 0, "logits": 1}

_DTYPES, _lib, _check = {}, None, None  # filled by bind()


class SpecverifyLists(ctypes.Structure):
    """Mirror of ``specverify_lists`` (include/specverify.h)."""
    _fields_ = [("K", ctypes.c_int32), ("target_dtype", ctypes.c_int32), ("form", ctypes.c_int32),
                ("divergence", ctypes.c_int32), ("beta", ctypes.c_float), ("ids", ctypes.c_void_p),
                ("target", ctypes.c_void_p)]


class TokenLogprobs(NamedTuple):
    """What :meth:`RowLosses.token_logprobs` returns, each of the tokens' shape (the top tokens with k more); None where
    it was not asked for."""
    logprob: torch.Tensor
    entropy: torch.Tensor | None
    lse: torch.Tensor | None
    rank: torch.Tensor | None
    topk_logprob: torch.Tensor | None
    topk_idx: torch.Tensor | None


def bind(lib):
    global torch, _lib, _check
    import torch
    from . import _check
    _lib = lib
    _DTYPES.update({torch.float32: FP32, torch.bfloat16: BF16})
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    rows = [vp, vp, i32, i64, i64, i64, f32]
    lib.specverify_token_logprobs.argtypes = rows + [i32, i32, vp, vp, vp, i32] + [vp] * 7
    lib.specverify_token_logprobs_grad.argtypes = rows + [vp, vp, vp, vp, i64, vp, vp, vp]
    lib.specverify_distill_loss.argtypes = rows + [vp, vp, vp]
    lib.specverify_distill_grad.argtypes = rows + [vp, vp, vp, i64, vp, vp]
    for name in ("token_logprobs", "token_logprobs_grad", "distill_loss", "distill_grad"):
        getattr(lib, "specverify_" + name).restype = ctypes.c_int


def _array(name, t, index, shape, dtype):
    """The address of a contiguous tensor of that shape and type on CUDA device `index`; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, not "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _one_of(name, x, among):
    if x not in among:
        raise ValueError(f"{name} must be one of {', '.join(among)}, not {x!r}")
    return among[x]


class RowLosses:
    """The methods; the class that takes them has a handle ``h`` on CUDA device ``device``."""

    def _rows(self, name, x):
        """Address, dtype, rows, V and row stride of logits or of their gradient."""
        dt = _DTYPES.get(x.dtype)
        if dt is None or x.dim() != 2 or x.get_device() != self.device:
            raise ValueError(f"{name} must be a 2-D float32 or bfloat16 tensor on cuda:{self.device}, not {x.dtype} "
                             f"{tuple(x.shape)} on {x.device}")
        rows, V = x.shape
        stride, one = x.stride()
        if one != 1 and V != 1:
            raise ValueError(f"{name} must have unit column stride")
        # a single row's stride says nothing; the library wants whole 16-byte pieces
        return x.data_ptr(), dt, rows, V, stride if rows > 1 else -(-V // 8) * 8

    def _raw(self, stream):
        return torch._C._cuda_getCurrentRawStream(self.device) if stream is None else stream.cuda_stream

    def _new(self, stream, shape, dtype=None):
        device, dtype = f"cuda:{self.device}", dtype or torch.float32
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)

    def _grad_rows(self, logits, grad, stream):
        if grad is None:
            rows, V = logits.shape
            grad = self._new(stream, (rows, -(-V // 8) * 8), logits.dtype)[:, :V]
        elif grad.shape != logits.shape or grad.dtype is not logits.dtype:
            raise ValueError("grad must have the logits' shape and dtype")
        at, _, _, _, stride = self._rows("grad", grad)
        return grad, at, stride

    def token_logprobs_buffers(self, *shape, k=0, entropy=True, lse=True, rank=False, stream=None) -> TokenLogprobs:
        """Buffers for :meth:`token_logprobs` of tokens of that shape, to pass as ``out``."""
        one = lambda want, dtype=None, more=(): self._new(stream, (*shape, *more), dtype) if want else None  # noqa: E731
        return TokenLogprobs(one(True), one(entropy), one(lse), one(rank, torch.int32), one(k > 0, more=(k,)),
                             one(k > 0, torch.int32, (k,)))

    def token_logprobs(self, logits, tokens, temperature=1.0, *, k=0, row_off=None, path=None, entropy=True, lse=True,
                       rank=False, out=None, stream=None) -> TokenLogprobs:
        """Log-probabilities of ``tokens`` (int32; -1: not asked for) under softmax(logits / temperature), with the rows'
        entropy, logsumexp, the tokens' rank and the ``k`` most likely tokens.

        ``tokens`` [rows], a token a row; or [B, M] with ``row_off`` int64 [B], token (b, m) under row row_off[b] + m, or
        row_off[b] + path[b, m] with ``path`` int32 [B, M]: the outputs of a verify call with its row offsets, or those of
        a tree verify with its path. ``out``: buffers to use, which then say what is computed."""
        at, dt, rows, V, stride = self._rows("logits", logits)
        shape = tokens.shape
        if row_off is None:
            if tokens.numel() != rows or path is not None:
                raise ValueError("tokens without row_off must be one for each row, and have no path")
            B, M = rows, 1
        elif tokens.dim() != 2:
            raise ValueError("tokens with row_off must be [B, M]")
        else:
            B, M = shape
        if max(B, M) > MAX_INT32:
            raise ValueError(f"no more than {MAX_INT32} rows a call, or sequences, or tokens of one")
        if not 0 <= k <= MAX_ALTERNATIVES:
            raise ValueError(f"k must be 0 to {MAX_ALTERNATIVES}, not {k}")
        if out is None:
            out = self.token_logprobs_buffers(*shape, k=k, entropy=entropy, lse=lse, rank=rank, stream=stream)
        if (k > 0) != (out.topk_idx is not None) or (k > 0) != (out.topk_logprob is not None):
            raise ValueError("out must have buffers for the top tokens where k > 0, and only there")
        d, f32, i32 = self.device, torch.float32, torch.int32
        top = (*shape, k)
        rc = _lib.specverify_token_logprobs(
            self.h, at, dt, rows, V, stride, temperature, B, M, _array("tokens", tokens, d, shape, i32),
            _array("row_off", row_off, d, (B,), torch.int64), _array("path", path, d, shape, i32), k,
            _array("logprob", out.logprob, d, shape, f32), _array("entropy", out.entropy, d, shape, f32),
            _array("lse", out.lse, d, shape, f32), _array("rank", out.rank, d, shape, i32),
            _array("topk_logprob", out.topk_logprob, d, top, f32), _array("topk_idx", out.topk_idx, d, top, i32),
            self._raw(stream))
        if rc:
            _check(rc, "specverify_token_logprobs")
        return out

    def token_logprobs_grad(self, logits, tokens, grad_logprob, grad_entropy=None, temperature=1.0, *, grad=None,
                            logprob=None, entropy=None, stream=None):
        """Gradient of sum(grad_logprob * logprob + grad_entropy * entropy) with respect to the logits, for one token a row
        (int32 [rows]; -1: a row that counts for nothing); returns (grad, logprob, entropy). ``grad`` may be the logits
        themselves, which it then replaces."""
        at, dt, rows, V, stride = self._rows("logits", logits)
        grad, gat, gstride = self._grad_rows(logits, grad, stream)
        logprob = self._new(stream, (rows,)) if logprob is None else logprob
        entropy = self._new(stream, (rows,)) if entropy is None else entropy
        d, f32, one = self.device, torch.float32, (rows,)
        rc = _lib.specverify_token_logprobs_grad(
            self.h, at, dt, rows, V, stride, temperature,
            _array("tokens", tokens, d, one, torch.int32), _array("grad_logprob", grad_logprob, d, one, f32),
            _array("grad_entropy", grad_entropy, d, one, f32), gat, gstride, _array("logprob", logprob, d, one, f32),
            _array("entropy", entropy, d, one, f32), self._raw(stream))
        if rc:
            _check(rc, "specverify_token_logprobs_grad")
        return grad, logprob, entropy

    def _lists(self, rows, ids, target, divergence, form, beta):
        shape, dt = ids.shape, _DTYPES.get(target.dtype)
        if len(shape) != 2 or shape[0] != rows or not 1 <= shape[1] <= MAX_LIST or dt is None:
            raise ValueError(f"ids must be [rows, 1 to {MAX_LIST}], and target of its shape, float32 or bfloat16")
        return ctypes.byref(SpecverifyLists(
            shape[1], dt, _one_of("form", form, FORMS), _one_of("divergence", divergence, DIVERGENCES), beta,
            _array("ids", ids, self.device, shape, torch.int32),
            _array("target", target, self.device, shape, target.dtype)))

    def distill_loss(self, draft, ids, target, temperature=1.0, divergence="fkl", *, form="logprobs", beta=0.5, loss=None,
                     stream=None):
        """Divergence (``fkl``, ``rkl``, ``jsd`` with ``beta``, ``tvd``) of each row of draft logits from the target's listed
        tokens; returns loss [rows].

        ``ids`` int32 [rows, K]: the listed tokens, -1 where a list is shorter. ``target`` [rows, K]: their
        log-probabilities at this temperature (``form="logprobs"``: what they leave of one is the rest of the
        vocabulary's), or their logits (``form="logits"``: softmax over the list)."""
        at, dt, rows, V, stride = self._rows("draft", draft)
        loss = self._new(stream, (rows,)) if loss is None else loss
        rc = _lib.specverify_distill_loss(
            self.h, at, dt, rows, V, stride, temperature, self._lists(rows, ids, target, divergence, form, beta),
            _array("loss", loss, self.device, (rows,), torch.float32), self._raw(stream))
        if rc:
            _check(rc, "specverify_distill_loss")
        return loss

    def distill_grad(self, draft, ids, target, weight=None, temperature=1.0, divergence="fkl", *, form="logprobs", beta=0.5,
                     grad=None, loss=None, stream=None):
        """:meth:`distill_loss` and the gradient of sum(weight * loss) with respect to the draft's logits, in one pass over
        them; returns (grad, loss). ``weight`` float32 [rows], or None for ones. ``grad`` may be the logits themselves."""
        at, dt, rows, V, stride = self._rows("draft", draft)
        grad, gat, gstride = self._grad_rows(draft, grad, stream)
        loss = self._new(stream, (rows,)) if loss is None else loss
        d, one = self.device, (rows,)
        rc = _lib.specverify_distill_grad(
            self.h, at, dt, rows, V, stride, temperature, self._lists(rows, ids, target, divergence, form, beta),
            _array("weight", weight, d, one, torch.float32), gat, gstride, _array("loss", loss, d, one, torch.float32),
            self._raw(stream))
        if rc:
            _check(rc, "specverify_distill_grad")
        return grad, loss
