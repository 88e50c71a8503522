"""The gate's choice value where two scores are one number in 64 bits although
their logits differ: with a rank of two values (group_top = 2) or a bias the
score decides, equal scores go to the lower index, and that also where every
group is kept; otherwise the logit decides."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_amd as nv
from tests import mx_reference as ref
from tests.gpu_common import device

pytestmark = pytest.mark.gpu

# sigmoid: 1.0 above a logit of about 37; softmax: 0.0 below about -745 of the largest
ROWS = {"sigmoid": [[40.0, 50.0, 45.0, 1.0, 39.0, 90.0, 2.0, 41.0], [-3.0, 60.0, -2.0, 70.0, 38.0, -1.0, 99.0, 64.0]],
        "softmax": [[-900.0, 0.0, -800.0, -850.0, -790.0, -799.0, -1e4, -900.5],
                    [-2000.0, -1900.0, 5.0, -1800.0, 4.0, -1700.0, -1600.0, -1500.0]]}


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("T", [2, 2050])                          # a wave, a quarter wave per token
@pytest.mark.parametrize("with_bias", [False, True])
def test_equal_scores_go_by_index(score, G, T, with_bias):
    x = torch.tensor(ROWS[score], dtype=torch.float32).repeat(T // 2, 1)
    bias = torch.zeros(8) if with_bias else None
    for group_top in (1, 2):
        ids, w = nv.moe_gate(x.to(device()), 6, score=score, n_group=G, topk_group=G, group_top=group_top,
                             bias=None if bias is None else bias.to(device()))
        rid, rw = ref.gate(x[:2].double().numpy(), 6, score=score, n_group=G, topk_group=G, group_top=group_top,
                           bias=None if bias is None else bias.double().numpy())
        # the definition orders by the score in the one case and by the logit in the other
        by_logit = np.argsort(-np.array(ROWS[score]), axis=1, kind="stable")[:, :6]
        assert np.array_equal(rid, by_logit) == (group_top == 1 and not with_bias)
        assert np.array_equal(ids.cpu().numpy(), np.tile(rid, (T // 2, 1)))
        # weights: as in tests/test_gpu_gate.py; below fp32's range they may flush to 0
        big = np.abs(np.array(ROWS[score])).max()
        assert np.allclose(w.cpu().numpy(), np.tile(rw, (T // 2, 1)), rtol=(64 + 4 * big) * 2.0 ** -24, atol=1e-37)
