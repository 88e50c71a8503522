"""The expert gate and its gradient against the 64-bit definition
(tests/mx_reference.py).

ids are compared for equality.  Weights: fp32 arithmetic of a dozen roundings
(each at most 2^-24 relative) and functions of a few ulps on terms that are
all positive, so 64 * 2^-24 relative, plus the logits' own size where the
logarithm of the sigmoid, itself rounded to 2^-24 |l|, is exponentiated.
Gradients are sums of products of such weights with both signs: the same
bound relative to the terms' magnitudes."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_amd as nv
from tests import mx_reference as ref
from tests.gpu_common import device

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _logits(rng, T, E, dtype, masked=False, spread=1.0):
    x = rng.standard_normal((T, E)).astype(np.float32) * np.float32(spread)
    if masked:
        x[rng.random((T, E)) < 0.1] = -np.inf
        x[rng.random(T) < 0.1] = -np.inf
    t = torch.from_numpy(x).to(dtype)
    return t, t.double().numpy()


def _weight_bound(l64, w):
    big = np.where(np.isfinite(l64), np.abs(l64), 0.0).max(axis=1, initial=1.0)[:, None]
    return (64 + 4 * big) * EPS * np.abs(w) + 1e-37


def _check(l, l64, k, **kw):
    bias = kw.pop("bias", None)
    ids, w = nv.moe_gate(l.to(device()), k, bias=None if bias is None else bias.to(device()), **kw)
    rid, rw = ref.gate(l64, k, bias=None if bias is None else bias.double().numpy(), **kw)
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:4]
    assert (np.abs(w - rw) <= _weight_bound(l64, rw)).all(), np.abs(w - rw).max()
    return ids


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (37, 60, 6), (5, 1, 1), (130, 7, 7), (19, 129, 16), (3, 384, 8),
                                   (9, 130, 17), (2, 1024, 64), (2, 4096, 8), (17, 16, 1)])
def test_gate_plain(dtype, score, renorm, T, E, k):
    rng = np.random.default_rng(T * 1000 + E + k)
    for masked in (False, True):
        l, l64 = _logits(rng, T, E, dtype, masked)
        _check(l, l64, k, score=score, renormalize=renorm, scale=2.5 if masked else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("T,E,k,G,kg", [(1, 256, 8, 8, 4), (33, 60, 6, 5, 2), (6, 256, 4, 256, 9), (7, 24, 3, 8, 1),
                                        (3, 1024, 8, 16, 3), (2, 4096, 8, 4096, 40), (4, 30, 10, 3, 1)])
def test_gate_groups_and_bias(score, group_top, with_bias, T, E, k, G, kg):
    rng = np.random.default_rng(E + G + k)
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * np.float32(0.2)) if with_bias else None
    for masked in (False, True):
        l, l64 = _logits(rng, T, E, torch.float32, masked)
        _check(l, l64, k, score=score, bias=bias, n_group=G, topk_group=kg, group_top=group_top, scale=1.5)


def test_gate_ties_and_order():
    # few distinct logits, both zeros: equal experts go by index
    rng = np.random.default_rng(0)
    x = rng.integers(-2, 3, (64, 48)).astype(np.float32) * np.float32(0.5)
    x[x == 0] = np.where(rng.random((x == 0).sum()) < 0.5, np.float32(0.0), np.float32(-0.0))
    l = torch.from_numpy(x)
    for kw in (dict(), dict(score="sigmoid"), dict(n_group=6, topk_group=2), dict(n_group=6, topk_group=3, group_top=2),
               dict(score="sigmoid", bias=torch.zeros(48)), dict(bias=torch.full((48,), 0.25))):
        _check(l, l.double().numpy(), 7, **kw)
    ids, w = nv.moe_gate(torch.zeros((2, 300), device=device()), 5)
    assert ids.cpu().tolist() == [[0, 1, 2, 3, 4]] * 2 and torch.equal(w.cpu(), torch.full((2, 5), 0.2))


def test_gate_close_scores_order_in_64_bits():
    # scores that fp32 cannot tell apart: a bias of 1 swallows differences below 2^-24
    l = torch.tensor([[-18.0, -17.5, -17.0, -16.5, -19.0, -16.75, -30.0, -29.0]])
    bias = torch.ones(8)
    ids = _check(l, l.double().numpy(), 8, score="sigmoid", bias=bias)
    assert ids[0].tolist() == [3, 5, 2, 1, 0, 4, 7, 6]


def test_gate_extreme_logits():
    big = float(torch.finfo(torch.float32).max)
    l = torch.tensor([
        [np.inf, 1.0, np.nan, -np.inf, 2.0, big, -big, 0.0],
        [-big] * 8,                                        # a mask of the type's lowest value on every expert
        [-big, -big, 3.0, -big, 1.0, -big, -big, -big],
        [np.nan] * 8,
        [-np.inf] * 7 + [5.0],
        [-200.0, -300.0, -1e30, -250.0, -np.inf, np.nan, -220.0, -1e4],
        [88.0, 90.0, 200.0, -90.0, -104.0, 1e30, 3.0, 0.0],
    ], dtype=torch.float32)
    l64 = l.double().numpy()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for kw in (dict(), dict(n_group=4, topk_group=3, group_top=2)):
                ids, w = nv.moe_gate(l.to(device()), 3, score=score, renormalize=renorm, **kw)
                rid, rw = ref.gate(l64, 3, score=score, renormalize=renorm, **kw)
                assert np.array_equal(ids.cpu().numpy(), rid)
                w = w.cpu().numpy()
                assert np.isfinite(w).all()
                # the logits' own rounding is exact here; sigmoids below fp32's range may flush to 0
                assert np.allclose(w, rw, rtol=2e-5, atol=1e-37)
    # a bias takes experts out (-inf, NaN) or puts one first (+inf)
    bias = torch.tensor([-np.inf, 0.0, 0.0, 0.0, np.nan, 0.0, np.inf, 0.0])
    x = torch.arange(8, dtype=torch.float32).repeat(3, 1)
    ids, w = nv.moe_gate(x.to(device()), 7, bias=bias.to(device()))
    assert ids[0].tolist() == [6, 7, 5, 3, 2, 1, -1] and w[0, 6].item() == 0.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (37, 60, 6), (5, 1, 1), (130, 7, 7), (19, 129, 16), (3, 384, 8),
                                   (9, 130, 17), (2, 1024, 64), (2, 4096, 8)])
def test_gate_gradient(dtype, score, renorm, T, E, k):
    rng = np.random.default_rng(T + E + k)
    for masked in (False, True):
        l, l64 = _logits(rng, T, E, dtype, masked)
        ids, _ = ref.gate(l64, k, score=score)
        dw = rng.standard_normal((T, k)).astype(np.float32)
        scale = 2.5 if masked else 1.0
        got = nv.moe_gate_backward(l.to(device()), torch.from_numpy(ids).to(device()), torch.from_numpy(dw).to(device()),
                                   score=score, renormalize=renorm, scale=scale)
        assert got.dtype == dtype and got.shape == (T, E)
        got = got.cpu().double().numpy()
        want = ref.gate_gradient(l64, ids, dw.astype(np.float64), score, renorm, scale)
        # each value is w dw less a share of D, |D| <= sum |w dw| <= scale max |dw|
        size = 2 * scale * np.abs(dw).max()
        bound = 256 * EPS * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0.0)
        assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max()
        assert (got[~np.isfinite(l64)] == 0).all()


def test_gate_gradient_against_differences():
    rng = np.random.default_rng(3)
    l, l64 = _logits(rng, 6, 20, torch.float32, masked=True)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            ids, _ = ref.gate(l64, 4, score=score)
            dw = rng.standard_normal((6, 4))
            got = nv.moe_gate_backward(l.to(device()), torch.from_numpy(ids).to(device()),
                                       torch.from_numpy(dw.astype(np.float32)).to(device()), score=score,
                                       renormalize=renorm, scale=2.0).cpu().double().numpy()
            step = 1e-5
            for t in range(6):
                for e in range(20):
                    if not np.isfinite(l64[t, e]):
                        continue
                    up, dn = l64.copy(), l64.copy()
                    up[t, e] += step
                    dn[t, e] -= step
                    d = ((ref.gate_weights(up, ids, score, renorm, 2.0) - ref.gate_weights(dn, ids, score, renorm, 2.0))
                         * dw).sum() / (2 * step)
                    # central differences: step^2 / 6 of a third derivative below 2 * 2 * |dw|, and fp32
                    assert abs(got[t, e] - d) <= 1e-5, (score, renorm, t, e)


def test_gate_gradient_repeated_and_foreign_ids():
    l = torch.randn((3, 12), generator=torch.Generator().manual_seed(1))
    ids = torch.tensor([[4, 4, 4, 7], [-1, 12, 3, 2 ** 31 - 1], [-1, -1, -1, -1]], dtype=torch.int32)
    dw = torch.tensor([[1.0, 2.0, -0.5, 0.25]] * 3)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            got = nv.moe_gate_backward(l.to(device()), ids.to(device()), dw.to(device()), score=score,
                                       renormalize=renorm).cpu().double().numpy()
            want = ref.gate_gradient(l.double().numpy(), ids.numpy(), dw.double().numpy(), score, renorm, 1.0)
            assert np.abs(got - want).max() <= 256 * EPS * 4


def test_gate_on_a_stream_and_in_a_graph():
    dev = device()
    g = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn((300, 256), generator=g, device=dev)
    bias = torch.randn(256, generator=g, device=dev) * 0.1
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)
    want = nv.moe_gate(x, 8, bias=bias, **kw)
    dw = torch.randn((300, 8), generator=g, device=dev)
    wantd = nv.moe_gate_backward(x, want[0], dw, score="sigmoid", scale=2.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.moe_gate(x, 8, bias=bias, stream=side, **kw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ids, w = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    dl = torch.zeros_like(x)
    src = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.moe_gate(src, 8, bias=bias, ids=ids, weights=w, **kw)
        nv.moe_gate_backward(src, ids, dw, score="sigmoid", scale=2.5, dlogits=dl)
    for i in range(3):
        src.copy_(x if i % 2 == 0 else x.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        order = slice(None) if i % 2 == 0 else slice(None, None, -1)
        assert np.array_equal(ids.cpu().numpy(), want[0].cpu().numpy()[order])
        assert np.array_equal(w.cpu().numpy(), want[1].cpu().numpy()[order])
        if i % 2 == 0:
            assert torch.equal(dl, wantd)


def test_gate_leaves_other_memory_alone():
    dev = device()
    x = torch.randn((5, 60), device=dev)
    ids = torch.full((9, 6), 77, dtype=torch.int32, device=dev)
    w = torch.full((9, 6), 7.0, device=dev)
    nv.moe_gate(x, 6, ids=ids[:5], weights=w[:5])
    assert (ids[5:] == 77).all() and (w[5:] == 7.0).all()
    d = torch.full((9, 60), 7.0, device=dev)
    nv.moe_gate_backward(x, ids[:5].contiguous(), w[:5].contiguous(), dlogits=d[:5])
    assert (d[5:] == 7.0).all()
    empty = nv.moe_gate(x[:0], 6)
    assert empty[0].shape == (0, 6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,G,kg,group_top,score,renorm", [
    (2049, 7, 3, 1, 1, 1, "softmax", False), (2051, 60, 6, 5, 2, 2, "sigmoid", True),
    (2050, 128, 16, 128, 20, 1, "softmax", True), (3001, 256, 8, 8, 4, 2, "sigmoid", True),
    (2049, 256, 8, 1, 1, 1, "softmax", False), (2049, 250, 16, 2, 1, 1, "sigmoid", False)])
@pytest.mark.parametrize("with_bias", [True, False])
def test_gate_many_tokens(dtype, T, E, k, G, kg, group_top, score, renorm, with_bias):
    """Four tokens to a wave."""
    rng = np.random.default_rng(T + E + k + G)
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * np.float32(0.2)) if with_bias else None
    l, l64 = _logits(rng, T, E, dtype, masked=True)
    _check(l, l64, k, score=score, renormalize=renorm, bias=bias, n_group=G, topk_group=kg, group_top=group_top)
