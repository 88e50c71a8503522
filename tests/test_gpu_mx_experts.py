"""The MXFP4 routed-expert layer against its 64-bit definition, every element
of every row within the error that its own roundings allow (derived in
tests/mx_bounds.py), in each of the layer's plans: slot by slot, sorted in row
tiles of 16, sorted in row tiles of 192."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_amd as nv
from tests import mx_bounds
from tests.gpu_common import dev, dev_bf16, device, host_bf16_f32

pytestmark = pytest.mark.gpu

SLOTS, ROWS16, ROWS192 = "slots", "row tiles of 16", "row tiles of 192"

# seed, T, E, top_k, H, I, part of the slots without an expert, tokens that all
# take expert 0, plan
CASES = [
    (1, 200, 8, 2, 256, 256, 0.0, 0, ROWS192),
    (2, 60, 8, 4, 544, 352, 0.1, 0, ROWS192),
    (3, 40, 32, 4, 256, 96, 0.0, 40, ROWS16),
    (4, 3, 16, 4, 512, 96, 0.0, 0, SLOTS),
]


def _align(v):
    return (v + 255) // 256 * 256


def run_and_plan(x, ids, tw, w13, w2):
    """The layer's output and the plan that it took, as its workspace shows:
    the sorted plans need more of it, and leave the first row tile of each
    expert behind the first row of each."""
    T, H = x.shape
    E, I, k = w13[0].shape[0], w2[0].shape[-1] * 2, ids.shape[1]
    need = nv.mx_moe_workspace_size(T, E, k, H, I)
    ws = torch.zeros(need, dtype=torch.uint8, device=device())
    y = nv.mx_moe(dev_bf16(x), dev(ids), dev(tw), dev(w13[0]), dev(w13[1]), dev(w2[0]), dev(w2[1]), ws=ws)
    y = host_bf16_f32(y).astype(np.float64)
    S = T * k
    if need == _align(S * I // 2) + _align(S * I // 32):
        return y, SLOTS
    tiles = ws[_align(4 * (E + 1)):][:4 * (E + 1)].cpu().numpy().view(np.int32)
    rows = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    assert rows.max() > 16, "both sorted plans have one tile an expert"
    for bm, plan in ((16, ROWS16), (192, ROWS192)):
        if np.array_equal(np.diff(tiles), (rows + bm - 1) // bm):
            return y, plan
    raise AssertionError("unknown plan")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c[:6]))
def test_every_row(case):
    args = mx_bounds.experts_case(*case[:-1])
    y, plan = run_and_plan(*args)
    assert plan == case[-1]
    mx_bounds.check(y, *mx_bounds.experts(*args))
