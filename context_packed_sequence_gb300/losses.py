"""Losses of a packed batch on its logits: the torch-facing binding.

The batch is what ``pack_docs`` and ``roll_labels`` (or, in the zigzag layout,
``roll_labels_zigzag``) leave: T rows, int32 labels, a uint8 loss mask and the
padded document boundaries.  As in ``api``, functions here only check shapes,
allocate outputs and pass pointers through the C ABI; the formulas are in
include/thd.h.  Nothing is differentiated by autograd: every loss returns its
gradient (``dlogits``, or ``dlogprobs`` for ``token_logprobs_backward``), which
the caller hands to its model's backward pass.

    w, docs = thd.loss_weights(loss_mask, cu_seqlens_padded, cp, thd.DOC_MEAN)
    out = thd.policy_loss(logits, labels, w, old_logprobs, advantages, doc_ids=docs)
    logits_of_the_model.backward(out.dlogits)
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib as L
from .api import ThdError, _need_cuda, _ptr, _raise_host, _range, _stream

TOKEN_MEAN = L.TOKEN_MEAN
DOC_MEAN = L.DOC_MEAN
TOKEN_SUM = L.TOKEN_SUM

_DTYPES = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16, torch.float16: L.DTYPE_F16}


class PolicyLoss(NamedTuple):
    loss: torch.Tensor            # float32, 0-d
    kl: torch.Tensor              # float32, 0-d
    clip_fraction: torch.Tensor   # float32, 0-d
    logprobs: torch.Tensor        # float32 [T]
    dlogits: Optional[torch.Tensor]


class PreferenceLoss(NamedTuple):
    loss: torch.Tensor            # float32, 0-d
    margins: torch.Tensor         # float32 [pairs]
    doc_logprobs: torch.Tensor    # float32 [documents]
    dlogprobs: torch.Tensor       # float32 [T]


class DistillLoss(NamedTuple):
    loss: torch.Tensor            # float32, 0-d
    token_losses: torch.Tensor    # float32 [T]
    dlogits: Optional[torch.Tensor]


def _rows(t, name):
    """A [T, V] CUDA matrix whose rows are dense; returns (T, V, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] < 1:
        raise ValueError(f"{name} must be [T, V] with V >= 1, got shape {tuple(t.shape)}")
    T, V = t.shape
    stride = t.stride(0) if T > 1 else max(t.stride(0), V)
    if (V > 1 and t.stride(1) != 1) or stride < V:
        raise ValueError(f"{name} must have dense rows that do not overlap, got strides {t.stride()}")
    return T, V, stride


def _vector(t, name, n, dtype, device):
    _need_cuda(t, name, dtype)
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} values, got shape {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    return t.data_ptr()


def _optional(t, name, n, dtype, device):
    return None if t is None else _vector(t, name, n, dtype, device)


def _logits(logits, temperature):
    T, V, stride = _rows(logits, "logits")
    return T, V, L.ThdLogits(logits.data_ptr(), T, stride, V, _DTYPES[logits.dtype], float(temperature), 0)


def _empty(shape, dtype, device, stream):
    """An output on the stream its kernel runs on: memory that another stream
    still uses is not handed out."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _gradient(logits, out, grad_scale, stream):
    """(gradient tensor, its struct); out None: a new contiguous one."""
    if out is None:
        out = _empty(logits.shape, logits.dtype, logits.device, stream)
    _, _, stride = _rows(out, "out")
    if out.shape != logits.shape or out.dtype != logits.dtype or out.device != logits.device:
        raise ValueError("out must match logits in shape, dtype and device")
    return out, L.ThdGradient(out.data_ptr(), stride, float(grad_scale), 0)


def loss_weights(loss_mask, cu_seqlens_padded, cp: int = 1, reduction: int = TOKEN_MEAN, status=None, stream=None):
    """(weights float32 [T], doc_ids int32 [T]) of the rows of a packed batch.

    TOKEN_MEAN: every row with loss counts the same; DOC_MEAN: every document
    with such a row does; TOKEN_SUM: 1 per row.  Rows are in the zigzag layout
    of ``cp`` ranks, or in the contiguous layout (cp = 1).  A row's weight may
    be changed before it is handed to a loss (a normaliser over several
    microbatches, say); a weight of 0 leaves the row out."""
    _need_cuda(cu_seqlens_padded, "cu_seqlens_padded", torch.int32)
    _need_cuda(loss_mask, "loss_mask", torch.uint8)
    dev, T, n = loss_mask.device, loss_mask.numel(), cu_seqlens_padded.numel() - 1
    buf = _empty(2 * T + max(n, 0), torch.int32, dev, stream)
    weights, doc_ids, ws = buf[:T].view(torch.float32), buf[T:2 * T], buf[2 * T:]
    with _range("thd_loss_weights"):
        code = L.load().thd_loss_weights(loss_mask.data_ptr(), cu_seqlens_padded.data_ptr(), n, T, int(cp),
                                         int(reduction), weights.data_ptr(), doc_ids.data_ptr(), ws.data_ptr(),
                                         4 * max(n, 0), _ptr(status), _stream(stream))
    _raise_host(code, "thd_loss_weights")
    return weights, doc_ids


def token_logprobs(logits, labels, loss_mask=None, temperature: float = 1.0, status=None, stream=None):
    """(logprobs, lse), float32 [T]: the labels' log-probabilities under
    softmax(logits / temperature) and the rows' log-sum-exp.  Rows whose
    loss_mask is 0 are not read and give 0."""
    T, V, z = _logits(logits, temperature)
    dev = logits.device
    labels_p = _vector(labels, "labels", T, torch.int32, dev)
    mask_p = _optional(loss_mask, "loss_mask", T, torch.uint8, dev)
    out = _empty((2, T), torch.float32, dev, stream)
    p = out.data_ptr()
    with _range("thd_token_logprobs"):
        code = L.load().thd_token_logprobs(ctypes.byref(z), labels_p, mask_p, p, p + 4 * T, _ptr(status),
                                           _stream(stream))
    _raise_host(code, "thd_token_logprobs")
    return out[0], out[1]


def token_logprobs_backward(logits, labels, lse, dlogprobs, temperature: float = 1.0, grad_scale: float = 1.0,
                            out=None, status=None, stream=None):
    """dlogits [T, V] of ``token_logprobs`` for the incoming gradient dlogprobs
    [T], rounded once to the logits' type.  ``out`` may be the logits."""
    T, V, z = _logits(logits, temperature)
    dev = logits.device
    labels_p = _vector(labels, "labels", T, torch.int32, dev)
    lse_p = _vector(lse, "lse", T, torch.float32, dev)
    g_p = _vector(dlogprobs, "dlogprobs", T, torch.float32, dev)
    out, g = _gradient(logits, out, grad_scale, stream)
    with _range("thd_token_logprobs_backward"):
        code = L.load().thd_token_logprobs_backward(ctypes.byref(z), labels_p, lse_p, g_p, ctypes.byref(g),
                                                    _ptr(status), _stream(stream))
    _raise_host(code, "thd_token_logprobs_backward")
    return out


def policy_loss(logits, labels, weights, old_logprobs, advantages, ref_logprobs=None, doc_ids=None,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0,
                grad_scale: float = 1.0, need_dlogits: bool = True, out=None, status=None, stream=None) -> PolicyLoss:
    """Clipped policy loss with a KL term against the reference, and its
    gradient, in one pass over the logits.

    advantages: one per row, or with ``doc_ids`` (from loss_weights) one per
    document.  The loss is the weighted sum of the rows' losses."""
    T, V, z = _logits(logits, temperature)
    dev = logits.device
    labels_p = _vector(labels, "labels", T, torch.int32, dev)
    weights_p = _vector(weights, "weights", T, torch.float32, dev)
    old_p = _vector(old_logprobs, "old_logprobs", T, torch.float32, dev)
    ref_p = _optional(ref_logprobs, "ref_logprobs", T, torch.float32, dev)
    docs_p = _optional(doc_ids, "doc_ids", T, torch.int32, dev)
    n_adv = advantages.numel() if docs_p is not None and isinstance(advantages, torch.Tensor) else T
    adv_p = _vector(advantages, "advantages", n_adv, torch.float32, dev)
    if need_dlogits:
        out, g = _gradient(logits, out, grad_scale, stream)
    buf = _empty(3 + 4 * T, torch.float32, dev, stream)
    base = buf.data_ptr()
    params = L.ThdPolicy(old_p, ref_p, adv_p, docs_p, n_adv if docs_p is not None else 0, float(clip_low),
                         float(clip_high), float(kl_coef))
    with _range("thd_policy_loss"):
        code = L.load().thd_policy_loss(ctypes.byref(z), labels_p, weights_p, ctypes.byref(params),
                                        ctypes.byref(g) if need_dlogits else None, base + 12, base, base + 12 + 4 * T,
                                        12 * T, _ptr(status), _stream(stream))
    _raise_host(code, "thd_policy_loss")
    return PolicyLoss(buf[0], buf[1], buf[2], buf[3:3 + T], out if need_dlogits else None)


def preference_loss(logprobs, loss_mask, cu_seqlens_padded, chosen, rejected, ref_logprobs=None, cp: int = 1,
                    beta: float = 0.1, label_smoothing: float = 0.0, margin: float = 0.0,
                    length_normalized: bool = False, status=None, stream=None) -> PreferenceLoss:
    """Preference loss over pairs of the batch's documents and its gradient
    with respect to the label log-probabilities (token_logprobs_backward
    carries it on to the logits).

    chosen, rejected: int32 document indices, one pair per entry.  Rows are in
    the zigzag layout of ``cp`` ranks, or contiguous (cp = 1)."""
    _need_cuda(logprobs, "logprobs", torch.float32)
    _need_cuda(cu_seqlens_padded, "cu_seqlens_padded", torch.int32)
    dev, T, n = logprobs.device, logprobs.numel(), cu_seqlens_padded.numel() - 1
    mask_p = _vector(loss_mask, "loss_mask", T, torch.uint8, dev)
    ref_p = _optional(ref_logprobs, "ref_logprobs", T, torch.float32, dev)
    _need_cuda(chosen, "chosen", torch.int32)
    P = chosen.numel()
    rejected_p = _vector(rejected, "rejected", P, torch.int32, dev)
    if n < 0:
        raise ThdError(L.ERR_INVALID_ARG, "preference_loss: cu_seqlens_padded is empty")
    buf = _empty(1 + P + 3 * n + T, torch.float32, dev, stream)
    base = buf.data_ptr()
    params = L.ThdPreference(ref_p, float(beta), float(label_smoothing), float(margin), int(bool(length_normalized)))
    with _range("thd_preference_loss"):
        code = L.load().thd_preference_loss(logprobs.data_ptr(), mask_p, cu_seqlens_padded.data_ptr(), n, T, int(cp),
                                            chosen.data_ptr(), rejected_p, P, ctypes.byref(params), base, base + 4,
                                            base + 4 * (1 + P), base + 4 * (1 + P + n), base + 4 * (1 + P + n + T),
                                            8 * n, _ptr(status), _stream(stream))
    _raise_host(code, "thd_preference_loss")
    return PreferenceLoss(buf[0], buf[1:1 + P], buf[1 + P:1 + P + n], buf[1 + P + n:1 + P + n + T])


def distill_topk_loss(logits, teacher_ids, teacher_scores, weights, temperature: float = 1.0, normalize: bool = True,
                      grad_scale: float = 1.0, need_dlogits: bool = True, out=None, status=None,
                      stream=None) -> DistillLoss:
    """Distillation from the entries a teacher kept of each row, and its
    gradient, in one pass over the logits.

    teacher_ids int32 [T, K] (negative: absent), teacher_scores [T, K]: the
    teacher's logits, over which q = softmax(scores / temperature), or with
    normalize=False its log-probabilities.  The loss is the weighted sum of the
    rows' tau^2 sum_k q_k (ln q_k - lp(id_k))."""
    T, V, z = _logits(logits, temperature)
    dev = logits.device
    _need_cuda(teacher_ids, "teacher_ids", torch.int32)
    _need_cuda(teacher_scores, "teacher_scores")
    if teacher_ids.dim() != 2 or teacher_ids.shape[0] != T or teacher_scores.shape != teacher_ids.shape:
        raise ValueError(f"teacher_ids and teacher_scores must both be [{T}, K], got shapes "
                         f"{tuple(teacher_ids.shape)} and {tuple(teacher_scores.shape)}")
    if teacher_scores.dtype not in _DTYPES:
        raise TypeError(f"teacher_scores must be float32, bfloat16 or float16, got {teacher_scores.dtype}")
    if teacher_ids.device != dev or teacher_scores.device != dev:
        raise ValueError(f"the teacher's entries must be on {dev}")
    weights_p = _vector(weights, "weights", T, torch.float32, dev)
    if need_dlogits:
        out, g = _gradient(logits, out, grad_scale, stream)
    buf = _empty(1 + T, torch.float32, dev, stream)
    base = buf.data_ptr()
    teacher = L.ThdTeacher(teacher_ids.data_ptr(), teacher_scores.data_ptr(), teacher_ids.shape[1],
                           _DTYPES[teacher_scores.dtype], int(bool(normalize)), 0)
    with _range("thd_distill_topk_loss"):
        code = L.load().thd_distill_topk_loss(ctypes.byref(z), ctypes.byref(teacher), weights_p,
                                              ctypes.byref(g) if need_dlogits else None, base + 4, base,
                                              _ptr(status), _stream(stream))
    _raise_host(code, "thd_distill_topk_loss")
    return DistillLoss(buf[0], buf[1:], out if need_dlogits else None)
