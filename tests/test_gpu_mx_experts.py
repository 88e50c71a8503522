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
    # slots: K units of two steps and of one in either product, one token and
    # several, the most slots
    (5, 1, 8, 2, 256, 256, 0.0, 0, SLOTS),
    (6, 1, 8, 8, 512, 512, 0.0, 0, SLOTS),
    (7, 2, 16, 3, 96, 768, 0.2, 0, SLOTS),
    (8, 7, 40, 9, 96, 64, 0.0, 0, SLOTS),
    (9, 1, 200, 128, 64, 32, 0.1, 0, SLOTS),
    (10, 16, 256, 8, 64, 32, 0.0, 0, SLOTS),
    # rows of h too long for the waves' LDS
    (11, 1, 4, 2, 64, 11520, 0.0, 0, SLOTS),
    (12, 2, 4, 2, 64, 11552, 0.0, 0, SLOTS),
    # one slot more than the slot form takes; several row tiles of an expert,
    # whole and with one row
    (13, 43, 200, 3, 64, 32, 0.0, 43, ROWS16),
    (14, 40, 32, 4, 256, 256, 0.1, 33, ROWS16),
    (15, 64, 32, 5, 512, 512, 0.0, 48, ROWS16),
    (16, 48, 40, 4, 96, 544, 0.0, 17, ROWS16),
    (17, 33, 24, 5, 1024, 128, 0.2, 20, ROWS16),
    # tiles of whole and odd blocks, one expert, a row past a tile
    (18, 61, 4, 3, 544, 352, 0.0, 0, ROWS192),
    (19, 400, 2, 2, 256, 512, 0.0, 0, ROWS192),
    (20, 193, 1, 1, 128, 128, 0.0, 0, ROWS192),
    (21, 300, 5, 3, 160, 96, 0.1, 100, ROWS192),
    # many experts, and many slots (sorted by several launches)
    (22, 40, 4096, 8, 64, 32, 0.0, 40, ROWS16),
    (23, 1100, 600, 8, 64, 32, 0.1, 0, ROWS16),
    (24, 2100, 20, 4, 160, 96, 0.1, 0, ROWS192),
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


@pytest.mark.parametrize("T,plan", [(1, SLOTS), (200, ROWS16), (2500, ROWS192)])
def test_last_expert_past_32_bits(T, plan):
    """600 experts, the last one's weights past 2 GiB, in each plan; the other
    experts' weights decode as NaN."""
    E, H, I = 600, 2048, 2048
    x, _, tw, w13, w2 = mx_bounds.experts_case(T, T, 1, 1, H, I)
    d = device()
    assert (E - 1) * w13[0].size > 2 ** 31
    full = []
    for t in (*w13, *w2):
        big = torch.full((E, *t.shape[1:]), 255, dtype=torch.uint8, device=d)
        big[-1] = torch.from_numpy(t[0])
        full.append(big)
    ids = torch.full((T, 1), E - 1, dtype=torch.int32, device=d)
    ws = torch.zeros(nv.mx_moe_workspace_size(T, E, 1, H, I), dtype=torch.uint8, device=d)
    y = nv.mx_moe(dev_bf16(x), ids, dev(tw), *full, ws=ws)
    if plan != SLOTS:
        tiles = ws[_align(4 * (E + 1)):][:4 * (E + 1)].cpu().numpy().view(np.int32)
        assert tiles[-1] == -(-T // (16 if plan == ROWS16 else 192))
    else:
        assert ws.numel() == _align(T * I // 2) + _align(T * I // 32)
    some = np.linspace(0, T - 1, min(T, 200)).astype(int)           # of the rows, the first and the last
    args = (x[some], np.zeros((some.size, 1), np.int32), tw[some], w13, w2)
    mx_bounds.check(host_bf16_f32(y).astype(np.float64)[some], *mx_bounds.experts(*args))
