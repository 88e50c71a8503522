"""The layer's error bound (tests/mx_bounds.py) on the host: it lets a layer
through that rounds where the definition does, and nothing else."""
import numpy as np
import pytest

from tests import mx_bounds
from tests import mx_reference as ref
from tests.test_gpu_mx_experts import CASES


def _round(v):
    return ref.bf16_values(ref.bf16_round(v))


def _slots(x, ids, tw, w13, w2):
    """Each slot's weighted down product [T, top_k, H]."""
    T, H = x.shape
    I = w2[0].shape[-1] * 2
    xh = ref.mx_decode(*ref.mx_encode(x))
    y = np.zeros((T, ids.shape[1], H))
    for e in range(w13[0].shape[0]):
        t, j = np.nonzero(ids == e)
        if t.size:
            gu = xh[t] @ ref.mx_decode(w13[0][e], w13[1][e]).T
            g = gu[:, :I]
            h = ref.mx_decode(*ref.mx_encode(ref.bf16_round(g / (1.0 + np.exp(-g)) * gu[:, I:])))
            y[t, j] = h @ ref.mx_decode(w2[0][e], w2[1][e]).T
    return y


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]))
def test_bound_rejects_wrong_layers(case):
    args = mx_bounds.experts_case(*case[:-1])
    want, bound = mx_bounds.experts(*args)
    slots, w = _slots(*args), args[2].astype(np.float64)[:, :, None]
    good = _round((slots * w).sum(axis=1))
    mx_bounds.check(good, want, bound)
    live = np.nonzero((args[1] >= 0).any(axis=1))[0]
    wrong = {"zeros": np.zeros_like(good), "half": 0.5 * good}
    for name, row in (("first", live[0]), ("last", live[-1])):
        for part, f in (("zeroed", 0.0), ("halved", 0.5)):
            wrong[f"{name} row {part}"] = good.copy()
            wrong[f"{name} row {part}"][row] *= f
    wrong["last 16 columns of a row halved"] = good.copy()
    wrong["last 16 columns of a row halved"][live[-1], -16:] *= 0.5
    if (args[1] >= 0).sum(axis=1).max() > 1 and good.size >= 4096:
        wrong["slots rounded to bf16"] = _round((_round(slots) * w).sum(axis=1))
    for name, y in wrong.items():
        with pytest.raises(AssertionError, match="outside the bound"):
            mx_bounds.check(y, want, bound)
            pytest.fail(f"{name}: let through")
