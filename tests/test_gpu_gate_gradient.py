"""The gate's gradient against the 64-bit definition, each element within the
roundings of its own terms (tests/gate_bounds.py)."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_amd as nv
from tests import gate_bounds as gb
from tests import mx_reference as ref
from tests.gpu_common import device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", gb.CASES)
def test_every_element(dtype, score, renorm, T, E, k):
    for masked in (False, True):
        x, l64, ids, dw = gb.case(T, E, k, score, lambda v: torch.from_numpy(v).to(dtype).float().numpy(), masked)
        scale = 2.5 if masked else 1.0
        got = nv.moe_gate_backward(torch.from_numpy(x).to(dtype).to(device()), torch.from_numpy(ids).to(device()),
                                   torch.from_numpy(dw).to(device()), score=score, renormalize=renorm, scale=scale)
        got = got.cpu().double().numpy()
        want = ref.gate_gradient(l64, ids, dw.astype(np.float64), score, renorm, scale)
        bound = gb.gradient_bound(l64, ids, dw.astype(np.float64), score, renorm, scale, want, dtype == torch.bfloat16)
        err = np.abs(got - want)
        assert (err <= bound).all(), (np.argwhere(err > bound)[:4], np.max(err / bound))
        assert (got[~np.isfinite(l64)] == 0).all()
