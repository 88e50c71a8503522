"""What an element of the gate's gradient may differ by from its 64-bit
definition (tests/mx_reference.py): its own terms' magnitudes times the
roundings they take.

A term is a weight (64 + 4 |l| roundings of 2^-24, as in tests/test_gpu_gate.py,
|l| the row's largest logit) times dw, or times the row's sum of top_k such
products, once more times a weight or a probability p_e (an exponential of
l_e - max, whose argument is off by 2^-24 of itself, and a sum over the row:
no more than a weight's) and 1 - s_e (a dozen).  So at most
3 (64 + 4 |l|) + 2 top_k + 32 roundings; bf16 outputs add half a step, 2^-8
relative.  Values below fp32's (bf16's) range may flush to 0."""
from __future__ import annotations

import numpy as np

from tests import mx_reference as ref

EPS = 2.0 ** -24


def gradient_bound(l, ids, dw, score, renorm, scale, want, bf16):
    T, E = l.shape
    size = np.zeros((T, E))
    w = ref.gate_weights(l, ids, score, renorm, scale)
    for t in range(T):
        live = l[t] > -np.inf
        slots = [(i, e) for i, e in enumerate(ids[t]) if 0 <= e < E and live[e]]
        dot = sum(abs(w[t, i] * dw[t, i]) for i, _ in slots)
        if score == "softmax" and not renorm and live.any():
            p = np.where(live, np.exp(l[t] - l[t][live].max()), 0.0)
            size[t] += dot * p / p.sum()
        for i, e in slots:
            g = w[t, i] * (abs(dw[t, i]) + (dot / scale if renorm else 0.0))
            size[t, e] += g / (1.0 + np.exp(l[t, e])) if score == "sigmoid" else g
    big = np.where(np.isfinite(l), np.abs(l), 0.0).max(axis=1, initial=1.0)[:, None]
    bound = (3 * (64 + 4 * big) + 2 * ids.shape[1] + 32) * EPS * size + 1e-37
    return bound + (2.0 ** -8 * (np.abs(want) + bound) if bf16 else 0.0)


# T, E, top_k: every form of the kernel, four tokens a wave and one
CASES = [(1, 256, 8), (37, 60, 6), (5, 1, 1), (130, 7, 7), (19, 129, 16), (3, 384, 8), (9, 130, 17), (3, 700, 33),
         (2, 1024, 64), (2, 1500, 8), (2, 4096, 8), (3, 4095, 64)]


def case(T, E, k, score, dtype_round, masked):
    """logits (fp32), ids, dw: few large logits, so that their experts have most
    of the probability, and others of a hundredth of it."""
    rng = np.random.default_rng(T + E + k)
    x = rng.standard_normal((T, E)).astype(np.float32) * np.float32(1.5)
    x[rng.random((T, E)) < 0.02] += np.float32(4.0)
    if masked:
        x[rng.random((T, E)) < 0.1] = -np.inf
        x[rng.random(T) < 0.1] = -np.inf
    x = dtype_round(x)
    l64 = x.astype(np.float64)
    ids, _ = ref.gate(l64, k, score=score)
    return x, l64, ids, rng.standard_normal((T, k)).astype(np.float32)
