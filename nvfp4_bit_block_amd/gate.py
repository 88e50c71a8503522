"""The expert gate (``include/nvfp4_gate.h``): routing ids and weights for the
routed-expert layers from router logits, and the gradient of those weights.
Argument marshalling only, as in the package's ``__init__``."""
from __future__ import annotations

import functools
import math

import torch

import nvfp4_bit_block_amd as nv

SCORE_SOFTMAX = "softmax"
SCORE_SIGMOID = "sigmoid"
_SCORES = {SCORE_SOFTMAX: 0, SCORE_SIGMOID: 1}
_LOGITS = (torch.float32, torch.bfloat16)


@functools.lru_cache(maxsize=256)
def _config(T, E, top_k, n_group, topk_group, group_top, score, renormalize, bf16, scale):
    """The C struct of one problem (a pure function of its numbers)."""
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    if top_k < 1:
        raise ValueError(f"top_k must be at least 1, got {top_k}")
    if not (math.isfinite(scale) and scale > 0.0):
        raise ValueError(f"scale must be finite and > 0, got {scale}")
    return nv.GateConfig(T, E, top_k, n_group, topk_group, group_top, _SCORES[score], 1 if renormalize else 0,
                         1 if bf16 else 0, scale)


def moe_gate(logits, top_k, score=SCORE_SOFTMAX, bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True,
             scale=1.0, ids=None, weights=None, stream=None):
    """nvfp4_moe_gate: returns (ids int32 [T, top_k], weights fp32 [T, top_k]).

    ``logits`` fp32 or bf16 [T, E]; -inf or NaN takes an expert out of a row.
    ``bias`` fp32 [E] is added to the scores for the choice only (there is no
    gradient to it).  ``n_group`` runs of experts, of which the ``topk_group``
    with the largest sum of their ``group_top`` best choice values stay.  A
    row with fewer candidates than ``top_k`` ends in ids -1 of weight 0."""
    T, E, dev = nv._matrix(logits, "logits", _LOGITS)
    if bias is not None:
        nv._arg(bias, "bias", nv._F32, (E,), dev)
    c = _config(T, E, top_k, n_group, topk_group, group_top, score, bool(renormalize),
                logits.dtype is torch.bfloat16, float(scale))

    def body(s):
        i = nv._out(ids, "ids", torch.int32, (T, top_k), dev)
        w = nv._out(weights, "weights", torch.float32, (T, top_k), dev)
        nv._check(nv.lib().nvfp4_moe_gate(c, logits.data_ptr(), None if bias is None else bias.data_ptr(),
                                          i.data_ptr(), w.data_ptr(), s), "nvfp4_moe_gate")
        return i, w
    return nv._launch(dev, stream, body)


def moe_gate_backward(logits, ids, dweights, score=SCORE_SOFTMAX, renormalize=True, scale=1.0, dlogits=None,
                      stream=None):
    """nvfp4_moe_gate_backward: the gradient of the forward call's weights with
    respect to its logits, [T, E] in their type, at the ids that it chose."""
    T, E, dev = nv._matrix(logits, "logits", _LOGITS)
    rows, top_k, _ = nv._matrix(ids, "ids", nv._I32)
    if rows != T:
        raise ValueError(f"ids: {rows} rows, logits has {T}")
    nv._cuda(ids, "ids", dev)
    nv._arg(dweights, "dweights", nv._F32, (T, top_k), dev)
    c = _config(T, E, top_k, 1, 1, 1, score, bool(renormalize), logits.dtype is torch.bfloat16, float(scale))

    def body(s):
        d = nv._out(dlogits, "dlogits", logits.dtype, (T, E), dev)
        nv._check(nv.lib().nvfp4_moe_gate_backward(c, logits.data_ptr(), ids.data_ptr(), dweights.data_ptr(),
                                                   d.data_ptr(), s), "nvfp4_moe_gate_backward")
        return d
    return nv._launch(dev, stream, body)
