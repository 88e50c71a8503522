"""MXFP4 quantize, dequantize, products and the routed-expert layer against
the 64-bit definition (tests/mx_reference.py).

Quantize and dequantize: bit for bit.  Products: the codes' products are exact
and are summed in fp32 in some order, so the sum is off by at most
K * 2^-23 of the sum of magnitudes (2^-23 rather than a half step: the matrix
units may truncate), then one rounding to bf16, 2^-8 relative.  The layer's
bound here leaves room for a rounding of each slot's result to bf16 (2^-8 of
the sum of their magnitudes), which the layer does not make
(tests/test_gpu_mx_experts.py bounds it without), and
adds the rounding of h to bf16 and to MXFP4, which the definition has too: an
h that lies closer to a border than the error of its sum may take the
neighbouring code, so the layer's inputs here give sums that fp32 holds
exactly up to silu, and the bound counts one such code (an eighth of the
slot's magnitude at most, since the block's largest element has a step of a
third) in a hundredth of the rows."""
import numpy as np
import pytest
import torch

import nvfp4_bit_block_amd as nv
import workloads as wl
from tests import mx_reference as ref
from tests.gpu_common import dev, dev_bf16, device, host_bf16_f32, host_u8

pytestmark = pytest.mark.gpu


def _blocks(rng, rows, cols):
    """bf16 patterns over the whole range: normals, ties, zeros, subnormals, the largest."""
    x = rng.integers(0, 1 << 16, (rows, cols), dtype=np.uint16)
    x[(x & 0x7F80) == 0x7F80] &= 0x7F7F                       # finite
    near = rng.random((rows, cols // 32)) < 0.6               # blocks of one magnitude range
    e = np.repeat(rng.integers(1, 254, (rows, cols // 32)), 32, axis=1)
    d = rng.integers(0, 5, (rows, cols))
    y = ((x & 0x8000) | (np.maximum(e - d, 0) << 7) | (x & 0x60)).astype(np.uint16)  # few mantissa bits: ties
    x = np.where(np.repeat(near, 32, axis=1), y, x)
    x[rng.random((rows, cols)) < 0.05] = 0x8000
    x[0, :32] = 0
    return x


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (128, 2048), (33, 6144), (257, 64)])
def test_quantize_and_dequantize_bit_exact(rows, cols):
    x = _blocks(np.random.default_rng(rows + cols), rows, cols)
    c, s = nv.mx_quantize(dev_bf16(x))
    rc, rs = ref.mx_encode(x)
    assert np.array_equal(host_u8(s), rs)
    assert np.array_equal(host_u8(c), rc)
    y = host_bf16_f32(nv.mx_dequantize(c, s))
    assert np.array_equal(y.astype(np.float64), ref.mx_decode(rc, rs))


@pytest.mark.parametrize("rows,cols", [(32, 1), (32, 65), (96, 130), (512, 1021), (256, 64), (544, 72), (64, 3)])
def test_quantize_columnwise_bit_exact(rows, cols):
    x = _blocks(np.random.default_rng(rows + cols), rows, max(32, (cols + 31) // 32 * 32))[:, :cols].copy()
    c, s = nv.mx_quantize_columnwise(dev_bf16(x))
    rc, rs = ref.mx_encode(np.ascontiguousarray(x.T))
    assert np.array_equal(host_u8(s), rs)
    assert np.array_equal(host_u8(c), rc)


def test_infinities_and_nan_mark_their_block():
    x = wl.to_bf16_bits(np.random.default_rng(0).standard_normal((4, 128)).astype(np.float32))
    x[0, 5], x[1, 40], x[2, 127] = 0x7F80, 0xFFC0, 0xFF80
    c, s = nv.mx_quantize(dev_bf16(x))
    rc, rs = ref.mx_encode(x)
    assert np.array_equal(host_u8(s), rs) and (rs == 255).sum() == 3
    y = host_bf16_f32(nv.mx_dequantize(c, s))
    assert np.isnan(y).reshape(4, 4, 32).all(axis=2).sum() == 3 and np.isnan(y).sum() == 96
    # the product carries them to the outputs that use the block, and to no other
    wc, ws = ref.random_mx(np.random.default_rng(1), 40, 128)
    y = host_bf16_f32(nv.mx_gemm(dev_bf16(x), dev(wc), dev(ws)))
    assert np.isnan(y[:3]).all() and np.isfinite(y[3]).all()


def test_every_scale_byte_decodes():
    s = np.arange(256, dtype=np.uint8)[:, None]
    c = np.tile(np.arange(16, dtype=np.uint8) * 17, (256, 1))
    y = host_bf16_f32(nv.mx_dequantize(dev(c), dev(s)))
    want = ref.mx_decode(c, s)
    with np.errstate(over="ignore"):
        assert np.array_equal(y, want.astype(np.float32), equal_nan=True)


def _check_product(y, a, w):
    A, W = ref.mx_decode(*a), ref.mx_decode(*w)
    want, mag = A @ W.T, np.abs(A) @ np.abs(W).T
    bound = A.shape[1] * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(want)
    y = y.astype(np.float64)
    assert np.isfinite(y).all()
    err = np.abs(y - want)
    assert (err <= bound).all(), (err / bound).max()


SHAPES = [(1, 16, 32), (1, 1, 64), (1, 257, 4096), (2, 40, 96), (5, 4099, 512), (8, 100, 2080), (16, 64, 1024),
          (17, 33, 544), (33, 130, 256), (64, 256, 768), (100, 70, 1312), (128, 128, 512), (129, 257, 288),
          (300, 515, 2048), (257, 256, 8192), (31, 1, 32),
          (65, 129, 4096), (70, 33, 4128), (200, 255, 8224), (128, 6, 16384), (520, 700, 2304), (2, 6144, 4096)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, w = ref.random_mx(rng, M, K, lo=120, hi=130), ref.random_mx(rng, N, K)
    wd = (dev(w[0]), dev(w[1]))
    _check_product(host_bf16_f32(nv.mx_gemm_packed(dev(a[0]), dev(a[1]), *wd)), a, w)
    x = wl.normal_bf16(rng, (M, K), 1.0)
    y = nv.mx_gemm(dev_bf16(x), *wd)
    _check_product(host_bf16_f32(y), ref.mx_encode(x), w)
    # the two forms are one product
    assert torch.equal(y, nv.mx_gemm_packed(*nv.mx_quantize(dev_bf16(x)), *wd))


def test_product_leaves_other_rows_alone_and_repeats():
    rng = np.random.default_rng(4)
    a, w = ref.random_mx(rng, 37, 544), ref.random_mx(rng, 67, 544)
    A, W = (dev(a[0]), dev(a[1])), (dev(w[0]), dev(w[1]))
    out = torch.full((40, 67), 3.0, dtype=torch.bfloat16, device=device())
    nv.mx_gemm_packed(*A, *W, out=out[:37])
    first = out.clone()
    assert (out[37:] == 3.0).all()
    for _ in range(3):
        nv.mx_gemm_packed(*A, *W, out=out[:37])
        assert torch.equal(out, first)


def test_gradients_of_a_linear_layer():
    # y = x W^T: dX = dY W and dW = dY^T X from columnwise copies
    rng = np.random.default_rng(6)
    M, N, K = 96, 160, 224
    x, w, dy = (wl.normal_bf16(rng, s, 1.0) for s in ((M, K), (N, K), (M, N)))
    wt = nv.mx_quantize_columnwise(dev_bf16(w))                     # [K, N]
    dx = nv.mx_gemm(dev_bf16(dy), *wt)
    tr = lambda b: ref.mx_encode(np.ascontiguousarray(b.T))         # noqa: E731
    _check_product(host_bf16_f32(dx), ref.mx_encode(dy), tr(w))
    dw = nv.mx_gemm_packed(*nv.mx_quantize_columnwise(dev_bf16(dy)), *nv.mx_quantize_columnwise(dev_bf16(x)))
    _check_product(host_bf16_f32(dw), tr(dy), tr(x))


def _experts_case(rng, T, E, k, H, I, skip=0.0):
    x = wl.normal_bf16(rng, (T, H), 1.0)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    if skip:
        ids[rng.random((T, k)) < skip] = -1
    tw = rng.random((T, k)).astype(np.float32)
    w13, w2 = ref.random_mx(rng, E, 2 * I, H), ref.random_mx(rng, E, H, I)
    return x, ids, tw, w13, w2


def _run_experts(x, ids, tw, w13, w2, **kw):
    return nv.mx_moe(dev_bf16(x), dev(ids), dev(tw), dev(w13[0]), dev(w13[1]), dev(w2[0]), dev(w2[1]), **kw)


def _check_experts(y, x, ids, tw, w13, w2):
    want, mag, slots = ref.experts(x, ids, tw, w13, w2)
    I = w2[0].shape[-1] * 2
    y = host_bf16_f32(y).astype(np.float64)
    assert np.isfinite(y).all()
    err = np.abs(y - want)
    tight = I * 2.0 ** -23 * mag + 2.0 ** -8 * (1 + 2.0 ** -8) * (np.abs(want) + slots) + ids.shape[1] * 2.0 ** -8 * mag / np.sqrt(I)
    rows = (err > tight).any(axis=1)
    assert rows.mean() <= 0.01 or rows.sum() <= 1, (rows.sum(), (err / tight).max())
    assert (err <= tight + mag / 8).all()


@pytest.mark.parametrize("T,E,k,H,I", [(1, 8, 2, 64, 32), (1, 4, 4, 512, 96), (3, 16, 4, 96, 64), (7, 3, 1, 288, 160),
                                       (16, 8, 2, 256, 128), (61, 4, 3, 544, 352), (40, 64, 8, 128, 64),
                                       (200, 2, 2, 256, 64), (300, 5, 3, 160, 96), (33, 1, 1, 64, 32)])
def test_experts(T, E, k, H, I):
    rng = np.random.default_rng(T + 10 * E + 100 * k + H + I)
    case = _experts_case(rng, T, E, k, H, I)
    _check_experts(_run_experts(*case), *case)


@pytest.mark.parametrize("T", [1, 4, 50])
def test_experts_skipped_slots_and_repeated_experts(T):
    rng = np.random.default_rng(T)
    x, ids, tw, w13, w2 = _experts_case(rng, T, 6, 4, 128, 96, skip=0.4)
    ids[0] = -1                                                  # a token without an expert
    if T > 1:
        ids[1] = [2, 2, 2, 5]                                    # the same expert three times
        ids[2] = [6, 2 ** 31 - 1, -7, 0]                         # outside the experts
    y = _run_experts(x, ids, tw, w13, w2)
    assert (y[0] == 0).all()
    _check_experts(y, x, ids, tw, w13, w2)
    all_out = _run_experts(x, np.full_like(ids, -1), tw, w13, w2)
    assert (all_out == 0).all()


def test_experts_one_expert_takes_all_and_repeats():
    rng = np.random.default_rng(9)
    x, ids, tw, w13, w2 = _experts_case(rng, 150, 8, 2, 256, 64)
    ids[:, 0], ids[:, 1] = 3, np.where(np.arange(150) < 3, 5, -1)
    y = _run_experts(x, ids, tw, w13, w2)
    _check_experts(y, x, ids, tw, w13, w2)
    ws = nv.workspace(nv.mx_moe_workspace_size(150, 8, 2, 256, 64), device())
    for fill in (0, 255):                                        # nothing is read from an earlier call
        ws.fill_(fill)
        out = torch.full((152, 256), 9.0, dtype=torch.bfloat16, device=device())
        _run_experts(x, ids, tw, w13, w2, ws=ws, out=out[:150])
        assert torch.equal(out[:150], y) and (out[150:] == 9.0).all()


@pytest.mark.parametrize("T", [1, 48])
def test_gate_feeds_the_experts(T):
    """Router logits -> gate -> routed experts, eager, on a side stream, and
    captured; the MXFP4 and the NVFP4 layer take the gate's output alike."""
    rng = np.random.default_rng(T)
    E, k, H, I = 16, 4, 256, 64
    x, _, _, w13, w2 = _experts_case(rng, T, E, k, H, I)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[-1, 2:] = -np.inf                                     # two candidates: slots 2 and 3 are skipped
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)
    xd, ld, bd = dev_bf16(x), dev(logits), dev(bias)
    W = (dev(w13[0]), dev(w13[1]), dev(w2[0]), dev(w2[1]))

    def layer(**s):
        ids, w = nv.moe_gate(ld, k, bias=bd, **kw, **s)
        return nv.mx_moe(xd, ids, w, *W, **s)

    rid, rw = ref.gate(logits.astype(np.float64), k, bias=bias, **kw)
    y = layer()
    _check_experts(y, x, rid, rw.astype(np.float32), w13, w2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = layer(stream=side)
    side.synchronize()
    assert torch.equal(y, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = layer()
    keep = xd.clone()
    for i in range(3):
        xd.copy_(keep if i != 1 else torch.zeros_like(keep))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, y) if i != 1 else bool((z == 0).all())
    # the NVFP4 layer on the same routing
    c13, s13, g13 = wl.random_nvfp4((E,), 2 * I, H, 1, device())
    c2, s2, g2 = wl.random_nvfp4((E,), H, I, 2, device())
    ids, w = nv.moe_gate(ld, k, bias=bd, **kw)
    y4 = nv.moe_grouped_gemm(xd, ids, w, c13, s13, g13, c2, s2, g2)
    assert torch.isfinite(y4.float()).all()


def test_product_in_a_graph():
    rng = np.random.default_rng(2)
    for M in (1, 20, 150):
        w = ref.random_mx(rng, 200, 544)
        W = (dev(w[0]), dev(w[1]))
        x = dev_bf16(wl.normal_bf16(rng, (M, 544), 1.0)).view(torch.bfloat16)
        x2 = dev_bf16(wl.normal_bf16(rng, (M, 544), 1.0)).view(torch.bfloat16)
        want = [nv.mx_gemm(v, *W) for v in (x, x2)]
        src = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = nv.mx_gemm(src, *W)
        for i in range(4):
            src.copy_((x, x2)[i % 2])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want[i % 2])


def test_offsets_past_32_bits():
    """Operands of more than 2^31 code bytes and 2^32 elements: the last rows
    equal those of a small call on copies of them."""
    d = device()
    g = torch.Generator(device=d).manual_seed(0)
    rows, cols = (1 << 32) // 4096 + 65, 4096
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=d)
    x[:1000].normal_(generator=g)
    x[-1000:].normal_(generator=g)
    c, s = nv.mx_quantize(x)
    tc, ts = nv.mx_quantize(x[-1000:].clone())
    assert torch.equal(c[-1000:], tc) and torch.equal(s[-1000:], ts)
    assert torch.equal(nv.mx_dequantize(c, s)[-1000:], nv.mx_dequantize(tc, ts))
    del x
    w = (torch.randint(0, 256, (40, cols // 2), generator=g, device=d, dtype=torch.uint8),
         torch.randint(118, 122, (40, cols // 32), generator=g, device=d, dtype=torch.uint8))
    y = nv.mx_gemm_packed(c, s, *w)                                    # large activation
    z = nv.mx_gemm_packed(tc, ts, *w)
    assert (y[-1000:].float() - z.float()).abs().max() <= 2.0 ** -7 * z.float().abs().max()
    y = nv.mx_gemm_packed(*w, c, s)                                    # large weight
    z = nv.mx_gemm_packed(*w, tc, ts)
    assert (y[:, -1000:].float() - z.float()).abs().max() <= 2.0 ** -7 * z.float().abs().max()
    y = nv.mx_gemm_packed(w[0][:3], w[1][:3], c, s)                    # and through the streaming kernel
    assert (y[:, -1000:].float() - z[:3].float()).abs().max() <= 2.0 ** -7 * z.float().abs().max()


def test_experts_past_32_bits():
    """A last expert whose weights start past 2 GiB."""
    d = device()
    g = torch.Generator(device=d).manual_seed(1)
    E, H, I = 600, 2048, 2048
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=d, dtype=torch.uint8)  # noqa: E731
    w13 = (torch.empty((E, 2 * I, H // 2), dtype=torch.uint8, device=d), r(118, 122, E, 2 * I, H // 32))
    w2 = (torch.empty((E, H, I // 2), dtype=torch.uint8, device=d), r(118, 122, E, H, I // 32))
    assert (E - 1) * w13[0][0].numel() > 2 ** 31
    w13[0][-1], w2[0][-1] = r(0, 256, 2 * I, H // 2), r(0, 256, H, I // 2)
    for T in (2, 40, 4000):                                            # slots, slots, tiles
        x = torch.randn((T, H), generator=g, device=d).to(torch.bfloat16)
        ids = torch.full((T, 1), E - 1, dtype=torch.int32, device=d)
        tw = torch.ones((T, 1), device=d)
        y = nv.mx_moe(x, ids, tw, *w13, *w2)
        z = nv.mx_moe(x, torch.zeros_like(ids), tw, *[t[-1:].clone() for t in (*w13, *w2)])
        assert (y.float() - z.float()).norm() <= 0.01 * z.float().norm()


def test_misaligned_views_are_refused():
    d = device()
    c = torch.zeros(4 * 64 + 8, dtype=torch.uint8, device=d)[8:].view(4, 64)
    s = torch.zeros((4, 4), dtype=torch.uint8, device=d)
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device=d)
    for call in (lambda: nv.mx_dequantize(c, s), lambda: nv.mx_gemm(x, c, s)):
        with pytest.raises(nv.Nvfp4Error, match="aligned"):
            call()
    with pytest.raises(ValueError, match="shape"):
        nv.mx_gemm(x, c.clone(), s, out=torch.empty((2, 5), dtype=torch.bfloat16, device=d))
    with pytest.raises(nv.Nvfp4Error, match="workspace"):
        nv.mx_gemm(torch.zeros((70, 128), dtype=torch.bfloat16, device=d), c.clone(), s,
                   ws=torch.empty(16, dtype=torch.uint8, device=d))


def test_two_streams_at_once():
    """Calls that run together on two streams, each with its own temporaries."""
    rng = np.random.default_rng(8)
    case = _experts_case(rng, 90, 8, 3, 256, 128)
    w = ref.random_mx(rng, 300, 1024)
    xb = dev_bf16(wl.normal_bf16(rng, (80, 1024), 1.0))
    W = (dev(w[0]), dev(w[1]))
    args = [dev_bf16(case[0]), dev(case[1]), dev(case[2]), *map(dev, case[3]), *map(dev, case[4])]
    want = (nv.mx_moe(*args), nv.mx_gemm(xb, *W))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(8):
        got.append((nv.mx_moe(*args, stream=s1), nv.mx_gemm(xb, *W, stream=s2)))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


# many experts (bounds searched in two steps), many slots (sorted by several
# launches), in row tiles of 16 and on the large ones
MANY = [(40, 4096, 8, 64, 32), (300, 130, 8, 96, 64), (1100, 600, 8, 64, 32), (2100, 20, 4, 160, 96)]


@pytest.mark.parametrize("T,E,k,H,I", MANY)
def test_experts_many(T, E, k, H, I):
    rng = np.random.default_rng(T + E)
    case = _experts_case(rng, T, E, k, H, I, skip=0.1)
    _check_experts(_run_experts(*case), *case)


@pytest.mark.parametrize("T,E,k,H,I", [MANY[1], MANY[3]])
def test_experts_in_a_graph(T, E, k, H, I):
    """Replays with other tokens and other routing, eager work between them."""
    rng = np.random.default_rng(T)
    x, ids, tw, w13, w2 = _experts_case(rng, T, E, k, H, I)
    x2, ids2 = wl.normal_bf16(rng, (T, H), 1.0), np.full_like(ids, 1)
    W = (dev(w13[0]), dev(w13[1]), dev(w2[0]), dev(w2[1]))
    xs, idss, twd = [dev_bf16(x), dev_bf16(x2)], [dev(ids), dev(ids2)], dev(tw)
    want = [nv.mx_moe(xs[i], idss[i], twd, *W) for i in range(2)]
    xd, idd = xs[0].clone(), idss[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv.mx_moe(xd, idd, twd, *W)
    for i in range(4):
        xd.copy_(xs[i % 2])
        idd.copy_(idss[i % 2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i % 2])
        assert torch.equal(nv.mx_moe(xs[1], idss[1], twd, *W), want[1])


@pytest.mark.parametrize("T", [2, 40, 200])
@pytest.mark.parametrize("bad", [0x7FC0, 0x7F80, 0xFF80])
def test_a_token_that_is_not_finite_stays_by_itself(T, bad):
    rng = np.random.default_rng(T)
    x, ids, tw, w13, w2 = _experts_case(rng, T, 4, 2, 128, 64)
    clean = host_bf16_f32(_run_experts(x, ids, tw, w13, w2))
    p = dev_bf16(x)
    W = (dev(w2[0][0]), dev(w2[1][0]))                            # [128, 64]: takes 64 columns
    product = host_bf16_f32(nv.mx_gemm(p[:, :64].contiguous(), *W))
    xb = x.copy()
    xb[1, 5] = bad
    y = host_bf16_f32(_run_experts(xb, ids, tw, w13, w2))
    z = host_bf16_f32(nv.mx_gemm(dev_bf16(xb)[:, :64].contiguous(), *W))
    rest = np.arange(T) != 1
    assert np.array_equal(y[rest], clean[rest]) and np.isnan(y[1]).all()
    assert np.array_equal(z[rest], product[rest]) and np.isnan(z[1]).all()


# the streaming kernel's forms: one, two and four weight tiles a wave, one, two
# and four activation tiles, short and long rows, whole and odd blocks
@pytest.mark.parametrize("M,N,K", [(1, 70, 16384), (2, 70, 12288), (1, 70, 8448), (1, 70, 8480), (3, 70, 8448), (4, 33, 8224),
                                   (1, 8200, 4352), (2, 8209, 160), (3, 8200, 4352), (1, 16500, 544), (1, 16400, 512),
                                   (20, 100, 2304), (20, 8200, 256), (20, 8200, 96), (40, 130, 1280), (64, 65, 2080)])
def test_product_streaming(M, N, K):
    test_product(M, N, K)


@pytest.mark.parametrize("T,E,k,H,I", [(16, 256, 8, 64, 32), (7, 40, 9, 96, 64), (10, 300, 10, 256, 160), (2, 8, 2, 544, 352),
                                       (1, 200, 128, 64, 32), (1, 200, 129, 64, 32)])
def test_experts_slot_by_slot(T, E, k, H, I):
    rng = np.random.default_rng(T * E + k)
    case = _experts_case(rng, T, E, k, H, I, skip=0.1)
    _check_experts(_run_experts(*case), *case)


# activations too large for the waves' LDS
@pytest.mark.parametrize("M,N,K", [(12, 70, 8192), (12, 70, 8448), (16, 8200, 4352), (16, 33, 8224)])
def test_product_streaming_from_memory(M, N, K):
    test_product(M, N, K)


@pytest.mark.parametrize("T,I", [(1, 11520), (2, 11552)])
def test_experts_wide_slots(T, I):
    rng = np.random.default_rng(I)
    case = _experts_case(rng, T, 4, 2, 64, I)
    _check_experts(_run_experts(*case), *case)
