"""The expert gate (``include/nvfp4_gate.h``): routing ids and weights for the
routed-expert layers from router logits, and the gradient of those weights.
Argument marshalling only, as in the package's ``__init__``."""
from __future__ import annotations

import ctypes
import math

import torch

import nvfp4_bit_block_amd as nv

SCORE_SOFTMAX = "softmax"
SCORE_SIGMOID = "sigmoid"
_SCORES = {SCORE_SOFTMAX: 0, SCORE_SIGMOID: 1}
_LOGITS = (torch.float32, torch.bfloat16)


def _config(logits, top_k, n_group, topk_group, group_top, score, renormalize, scale):
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    scale = float(scale)
    if not (math.isfinite(scale) and scale > 0.0):
        raise ValueError(f"scale must be finite and > 0, got {scale}")
    T, E = logits.shape
    return nv.GateConfig(T, E, top_k, n_group, topk_group, group_top, _SCORES[score], 1 if renormalize else 0,
                         0 if logits.dtype == torch.float32 else 1, scale)


def moe_gate(logits, top_k, score=SCORE_SOFTMAX, bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True,
             scale=1.0, ids=None, weights=None, stream=None):
    """nvfp4_moe_gate: returns (ids int32 [T, top_k], weights fp32 [T, top_k]).

    ``logits`` fp32 or bf16 [T, E]; -inf or NaN takes an expert out of a row.
    ``bias`` fp32 [E] is added to the scores for the choice only (there is no
    gradient to it).  ``n_group`` runs of experts, of which the ``topk_group``
    with the largest sum of their ``group_top`` best choice values stay.  A
    row with fewer candidates than ``top_k`` ends in ids -1 of weight 0."""
    nv._req(logits, "logits", _LOGITS, (None, None))
    T, E = logits.shape
    dev = nv._cuda(logits, "logits").device
    if bias is not None:
        nv._req(bias, "bias", nv._F32, (E,), dev)
    c = _config(logits, top_k, n_group, topk_group, group_top, score, renormalize, scale)
    with nv._launch(dev, stream) as s:
        ids = nv._empty((T, top_k), torch.int32, dev) if ids is None else nv._req(ids, "ids", nv._I32, (T, top_k), dev)
        weights = (nv._empty((T, top_k), torch.float32, dev) if weights is None else
                   nv._req(weights, "weights", nv._F32, (T, top_k), dev))
        nv._check(nv.lib().nvfp4_moe_gate(ctypes.byref(c), logits.data_ptr(),
                                          None if bias is None else bias.data_ptr(), ids.data_ptr(),
                                          weights.data_ptr(), s), "nvfp4_moe_gate")
    return ids, weights


def moe_gate_backward(logits, ids, dweights, score=SCORE_SOFTMAX, renormalize=True, scale=1.0, dlogits=None,
                      stream=None):
    """nvfp4_moe_gate_backward: the gradient of the forward call's weights with
    respect to its logits, [T, E] in their type, at the ids that it chose."""
    nv._req(logits, "logits", _LOGITS, (None, None))
    T, E = logits.shape
    dev = nv._cuda(logits, "logits").device
    nv._req(ids, "ids", nv._I32, (T, None), dev)
    top_k = ids.shape[1]
    nv._req(dweights, "dweights", nv._F32, (T, top_k), dev)
    c = _config(logits, top_k, 1, 1, 1, score, renormalize, scale)
    with nv._launch(dev, stream) as s:
        dlogits = (nv._empty((T, E), logits.dtype, dev) if dlogits is None else
                   nv._req(dlogits, "dlogits", (logits.dtype,), (T, E), dev))
        nv._check(nv.lib().nvfp4_moe_gate_backward(ctypes.byref(c), logits.data_ptr(), ids.data_ptr(),
                                                   dweights.data_ptr(), dlogits.data_ptr(), s),
                  "nvfp4_moe_gate_backward")
    return dlogits
