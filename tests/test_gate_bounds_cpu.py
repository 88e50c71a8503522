"""The gradient's bound (tests/gate_bounds.py) on the host: it rejects
gradients that lack a part of a term."""
import numpy as np
import pytest

from tests import gate_bounds as gb
from tests import mx_reference as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", gb.CASES)
@pytest.mark.parametrize("bf16", [False, True])
def test_bound_rejects_wrong_gradients(bf16, score, renorm, T, E, k):
    for masked in (False, True):
        _, l, ids, dw = gb.case(T, E, k, score, lambda v: v, masked)
        dw = dw.astype(np.float64)
        want = ref.gate_gradient(l, ids, dw, score, renorm, 2.5)
        bound = gb.gradient_bound(l, ids, dw, score, renorm, 2.5, want, bf16)
        if not want.any():                                        # one expert: its weight does not move
            continue
        taken = np.zeros(want.shape, bool)
        for t, row in enumerate(ids):
            taken[t, row[row >= 0]] = True
        wrong = {"nothing": np.zeros_like(want), "a fifth": 0.2 * want}
        if score == "softmax" and not renorm and E > 2 * k:
            wrong["no dense term"] = np.where(taken, want, 0.0)
            wrong["a fifth of the dense term"] = np.where(taken, want, 0.2 * want)
            wrong["dense term 2 % off"] = np.where(taken, want, 1.02 * want)
            last = want.copy()
            last[:, E - 1 - (~taken[:, ::-1] & (l[:, ::-1] > -np.inf)).argmax(axis=1)] = 0.0
            wrong["last expert"] = last
        if renorm or score == "softmax":                          # the share of the row's sum left out
            w = ref.gate_weights(l, ids, score, renorm, 2.5)
            part = np.zeros_like(want)
            for t, row in enumerate(ids):
                for i, e in enumerate(row):
                    if e >= 0:
                        part[t, e] = w[t, i] * dw[t, i] / (1.0 + np.exp(l[t, e]) if score == "sigmoid" else 1.0)
            wrong["no shared term"] = part
        for name, v in wrong.items():
            assert (np.abs(v - want) > bound).any(), name
