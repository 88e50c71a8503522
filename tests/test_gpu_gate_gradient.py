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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [12, 21, 300])                      # rows of whole fours, of none, a wave per token
@pytest.mark.parametrize("bits", [0x7FC00000, 0x7FFFFFFF, -1, 0x7F800000])
def test_weight_gradients_that_are_not_finite(dtype, score, renorm, E, bits):
    """A NaN of any pattern (memory filled with ones is one) or an infinity in
    dw reaches the logits' gradient and no other row."""
    x = torch.randn((5, E), generator=torch.Generator().manual_seed(E)).to(dtype)
    ids = torch.from_numpy(ref.gate(x.double().numpy(), 3, score=score)[0])
    dw = torch.ones((5, 3))
    clean = nv.moe_gate_backward(x.to(device()), ids.to(device()), dw.to(device()), score=score, renormalize=renorm).cpu()
    dw.view(torch.int32)[2, 1] = bits
    got = nv.moe_gate_backward(x.to(device()), ids.to(device()), dw.to(device()), score=score, renormalize=renorm).cpu()
    assert not torch.isfinite(got[2, ids[2, 1]]).item()
    if bits != 0x7F800000:
        assert torch.isnan(got[2, ids[2, 1]]).item()
    if score == "softmax" and not renorm:
        assert not torch.isfinite(got[2]).any()
    rest = [0, 1, 3, 4]
    assert torch.equal(got[rest], clean[rest]) and torch.isfinite(clean).all()
