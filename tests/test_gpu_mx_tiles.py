"""MXFP4 products bit for bit: on the large tiles (256 x 192 and 256 x 256,
which take about a tile for every CU), and in every smaller form.

The scale bytes lie so close together that every sum is a whole number of
quanta below 2^20 of them, in any order: fp32 holds them all, and the one
rounding to bf16 is the definition's."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_amd as nv
import workloads as wl
from tests import mx_bounds
from tests import mx_reference as ref
from tests.gpu_common import dev, dev_bf16, device, host_bf16_f32

pytestmark = pytest.mark.gpu

# 2048 x 6144: 256 tiles of 256 x 192, against 192 of 256 x 256 and one and a
# half rounds of 128 x 128; K from less than one step of 256 to many, whole and
# odd numbers of 128 and (through the unaligned form) of 32
TILES_192 = [(2048, 6144, 128), (2048, 6144, 384), (2000, 6141, 256), (1793, 6139, 640), (2048, 6144, 2048), (2037, 6100, 8320),
             (2048, 6144, 32), (2000, 6141, 96), (2048, 6144, 160), (1800, 6139, 544), (2048, 6144, 1056), (2037, 6100, 8224)]
# 4096 x 4096: 256 tiles of 256 x 256
TILES_256 = [(4096, 4096, 128), (4096, 4096, 256), (4001, 4093, 384), (3841, 4089, 512), (4096, 4096, 896), (4090, 4095, 2176)]


def _exact(a, w):
    off = mx_bounds.sum_error(ref.mx_decode(*a), mx_bounds.quantum(*a), ref.mx_decode(*w), mx_bounds.quantum(*w))[1]
    assert (off == 0).all(), "sums are not exact"
    return ref.bf16_values(ref.bf16_round(ref.product(a, w)))


@pytest.mark.parametrize("M,N,K", TILES_192 + TILES_256)
def test_large_tiles(M, N, K):
    rng = np.random.default_rng(M + N + K)
    a, w = ref.random_mx(rng, M, K, lo=126, hi=128), ref.random_mx(rng, N, K, lo=121, hi=123)
    ws = torch.full((max(16, nv.mx_gemm_packed_workspace_size(M, N, K)),), 255, dtype=torch.uint8, device=device())
    out = torch.full((M + 1, N), 3.0, dtype=torch.bfloat16, device=device())
    ad, wd = (dev(a[0]), dev(a[1])), (dev(w[0]), dev(w[1]))
    nv.mx_gemm_packed(*ad, *wd, out=out[:M], ws=ws)
    assert np.array_equal(host_bf16_f32(out[:M]).astype(np.float64), _exact(a, w))
    assert (out[M] == 3.0).all()
    assert torch.equal(nv.mx_gemm_packed(*ad, *wd), out[:M])       # and again


def test_weight_gradient_of_a_training_batch():
    """dW = dY^T X of 544 tokens from columnwise copies, on the unaligned 256 x
    192 tiles."""
    rng = np.random.default_rng(7)
    T, N, K = 544, 2048, 6144
    dy, x = wl.normal_bf16(rng, (T, N), 1.0), wl.normal_bf16(rng, (T, K), 1.0)
    got = nv.mx_gemm_packed(*nv.mx_quantize_columnwise(dev_bf16(dy)), *nv.mx_quantize_columnwise(dev_bf16(x)))
    a, w = (ref.mx_encode(np.ascontiguousarray(v.T)) for v in (dy, x))
    want = ref.product(a, w)
    off = mx_bounds.sum_error(ref.mx_decode(*a), mx_bounds.quantum(*a), ref.mx_decode(*w), mx_bounds.quantum(*w))[1]
    assert (off == 0).mean() > 0.99                                 # (where a row holds a small block: 2^-23 K)
    err = np.abs(host_bf16_f32(got).astype(np.float64) - want)
    assert (err <= off + 2.0 ** -8 * (np.abs(want) + off)).all()


# the streaming kernel's forms, the 128 x 128 tiles and their K splits, as in
# tests/test_gpu_mx.py
SMALL = [(1, 16, 32), (1, 1, 64), (1, 257, 4096), (2, 40, 96), (5, 4099, 512), (8, 100, 2080), (16, 64, 1024), (17, 33, 544),
         (33, 130, 256), (64, 256, 768), (100, 70, 1312), (128, 128, 512), (129, 257, 288), (300, 515, 2048),
         (257, 256, 8192), (65, 129, 4096), (70, 33, 4128), (200, 255, 8224), (128, 6, 16384), (520, 700, 2304),
         (2, 6144, 4096), (1, 70, 16384), (1, 70, 8448), (1, 70, 8480), (3, 70, 8448), (4, 33, 8224), (1, 8200, 4352),
         (2, 8209, 160), (1, 16500, 544), (20, 100, 2304), (20, 8200, 256), (40, 130, 1280), (64, 65, 2080),
         (12, 70, 8192), (12, 70, 8448), (16, 8200, 4352), (16, 33, 8224)]


@pytest.mark.parametrize("M,N,K", SMALL)
def test_smaller_forms(M, N, K):
    rng = np.random.default_rng(M + N + K)
    a, w = ref.random_mx(rng, M, K, lo=126, hi=128), ref.random_mx(rng, N, K, lo=121, hi=123)
    wd = (dev(w[0]), dev(w[1]))
    want = _exact(a, w)
    got = nv.mx_gemm_packed(dev(a[0]), dev(a[1]), *wd)
    assert np.array_equal(host_bf16_f32(got).astype(np.float64), want)
    # a bf16 activation whose MXFP4 is `a`: a block's scale stays where it is if
    # its largest code is 4 or 6
    v = ref.mx_decode(*a).reshape(M, K // 32, 32)
    v[..., 0] = 6 * np.exp2(a[1] - 127.0)
    v = v.reshape(M, K)
    x = ref.bf16_round(v)
    got = nv.mx_gemm(dev_bf16(x), *wd)
    assert np.array_equal(host_bf16_f32(got).astype(np.float64), _exact(ref.mx_encode(x), w))


@pytest.mark.parametrize("M,K", [(8, 32), (8, 256), (80, 32), (80, 128), (80, 2080), (300, 8192)])
def test_scale_bytes_at_their_ends(M, K):
    """Scales of 2^-127 and 2^127 that meet in one product, sums below fp32's
    normal numbers, and NaN scales: every row and column has one scale."""
    rng = np.random.default_rng(M + K)
    N = 72
    sa = rng.choice([0, 1, 2, 60, 127, 128, 190, 250, 253, 255], M).astype(np.uint8)
    sw = rng.choice([0, 1, 2, 60, 127, 128, 190, 253, 255], N).astype(np.uint8)
    a = rng.integers(0, 256, (M, K // 2), dtype=np.uint8), np.repeat(sa[:, None], K // 32, axis=1)
    w = rng.integers(0, 256, (N, K // 2), dtype=np.uint8), np.repeat(sw[:, None], K // 32, axis=1)
    got = host_bf16_f32(nv.mx_gemm_packed(dev(a[0]), dev(a[1]), dev(w[0]), dev(w[1]))).astype(np.float64)
    nan = (sa == 255)[:, None] | (sw == 255)[None, :]
    assert np.isnan(got[nan]).all() and nan.any()
    A, W = (ref.mx_decode(c, np.full_like(s, 127)) for c, s in (a, w))
    scale = np.exp2(sa.astype(np.float64)[:, None] + sw.astype(np.float64)[None, :] - 254.0)
    want, mag = A @ W.T * scale, np.abs(A) @ np.abs(W).T * scale
    # (sums of whole quarters below 36 K: exact)
    normal = ~nan & (mag < 2.0 ** 127) & (np.abs(want) >= 2.0 ** -126)
    assert normal.sum() > 50
    rounded = ref.bf16_values(ref.bf16_round(np.where(normal, want, 0.0)))
    assert np.array_equal(got[normal], rounded[normal])
    # below the normal numbers a sum may flush to 0.  (Where the magnitudes add up
    # past fp32's range nothing is required: of 2^127 + .. - 2^127 - .. = 0 the
    # partial sums can be infinite in fp32.)
    tiny = ~nan & (mag < 2.0 ** 127) & (np.abs(want) < 2.0 ** -126)
    assert tiny.sum() > 50
    assert (np.abs(got[tiny]) <= 2.0 ** -126).all()
