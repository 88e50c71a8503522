"""Host-side checks of the gate and MXFP4 entry points: every call below fails
a check or is a zero-size no-op, so nothing reaches a GPU."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import nvfp4_bit_block_amd as nv
from tests import mx_reference as ref

pytestmark = pytest.mark.skipif(not os.path.exists(nv.LIB_PATH), reason="libnvfp4.so not built")

OK, NULL, SHAPE, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4, 5
A, MIS = 4096, 4097
INCLUDE = os.path.dirname(nv.HEADER)


def test_every_declared_function_is_exported_and_bound():
    L = nv.lib()
    for header in ("nvfp4_gate.h", "nvfp4_mx.h"):
        text = open(os.path.join(INCLUDE, header)).read()
        names = re.findall(r"^(?:size_t|int32_t)\s+(nvfp4_\w+)\s*\(", text, re.M)
        assert names
        for n in names:
            assert getattr(L, n).argtypes is not None, n
        assert f'#include "{header}"' in open(nv.HEADER).read()


def _gate(**over):
    c = dict(T=4, E=16, top_k=2, n_group=1, topk_group=1, group_top=1, score=0, renormalize=1, logits_dtype=0, scale=1.0)
    c.update(over)
    return nv.GateConfig(**c)


@pytest.mark.parametrize("over", [
    dict(T=-1), dict(E=0), dict(top_k=0), dict(top_k=17), dict(score=2), dict(score=-1), dict(logits_dtype=2),
    dict(renormalize=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_gate_shape_checks(over):
    L = nv.lib()
    c = ctypes.byref(_gate(**over))
    assert L.nvfp4_moe_gate(c, A, None, A, A, None) == SHAPE
    assert L.nvfp4_moe_gate_backward(c, A, A, A, A, None) == SHAPE


@pytest.mark.parametrize("over", [dict(n_group=3), dict(n_group=0), dict(n_group=32), dict(topk_group=2), dict(topk_group=0),
                                  dict(group_top=0), dict(group_top=3), dict(n_group=16, topk_group=1)])
def test_gate_group_checks(over):
    assert nv.lib().nvfp4_moe_gate(ctypes.byref(_gate(**over)), A, None, A, A, None) == SHAPE


def test_gate_other_checks():
    L = nv.lib()
    g, b = L.nvfp4_moe_gate, L.nvfp4_moe_gate_backward
    ok = ctypes.byref(_gate())
    assert g(None, A, None, A, A, None) == NULL
    for bad in (dict(E=4097), dict(E=128, top_k=65), dict(T=1 << 26)):
        assert g(ctypes.byref(_gate(**bad)), A, None, A, A, None) == UNSUP
        assert b(ctypes.byref(_gate(**bad)), A, A, A, A, None) == UNSUP
    for args in ((None, None, A, A), (A, None, None, A), (A, None, A, None)):
        assert g(ok, *args, None) == NULL
    for args in ((MIS, None, A, A), (A, A + 2, A, A), (A, None, A + 2, A), (A, None, A, A + 1)):
        assert g(ok, *args, None) == ALIGN
    for i in range(4):
        assert b(ok, *[None if j == i else A for j in range(4)], None) == NULL
        assert b(ok, *[A + 2 if j == i else A for j in range(4)], None) == ALIGN
    assert g(ctypes.byref(_gate(T=0)), None, None, None, None, None) == OK
    assert b(ctypes.byref(_gate(T=0)), None, None, None, None, None) == OK
    assert g(ok, A + 8, None, A, A, None) == ALIGN and b"16-byte" in L.nvfp4_last_error()


def test_quantize_checks():
    L = nv.lib()
    q, c, d = L.nvfp4_mx_quantize, L.nvfp4_mx_quantize_columnwise, L.nvfp4_mx_dequantize
    assert q(A, 4, 48, A, A, None) == SHAPE and q(A, -1, 32, A, A, None) == SHAPE and q(A, 4, 0, A, A, None) == SHAPE
    assert q(A, 1 << 40, 1 << 20, A, A, None) == UNSUP
    assert q(None, 4, 32, A, A, None) == NULL and q(A, 4, 32, A, None, None) == NULL
    assert q(MIS, 4, 32, A, A, None) == ALIGN and q(A, 4, 32, A + 8, A, None) == ALIGN
    assert q(None, 0, 32, None, None, None) == OK
    assert c(A, 48, 4, A, A, None) == SHAPE and c(A, 32, -1, A, A, None) == SHAPE
    assert c(A, 1 << 40, 1 << 20, A, A, None) == UNSUP
    assert c(A, 32, 4, None, A, None) == NULL and c(A, 32, 4, A, MIS, None) == ALIGN
    assert c(None, 0, 4, None, None, None) == OK and c(None, 32, 0, None, None, None) == OK
    assert d(A, A, 4, 33, A, None) == SHAPE and d(A, A, 1 << 62, 32, A, None) == UNSUP
    assert d(A, None, 4, 32, A, None) == NULL and d(A, A, 4, 32, A + 2, None) == ALIGN
    assert d(None, None, 0, 32, None, None) == OK


def test_product_checks():
    L = nv.lib()
    g, p = L.nvfp4_mx_gemm, L.nvfp4_mx_gemm_packed
    big = 1 << 40
    for M, N, K, want in ((-1, 4, 64, SHAPE), (4, -1, 64, SHAPE), (4, 4, 0, SHAPE), (4, 4, 48, SHAPE),
                          (4, 4, 1 << 24, UNSUP), (1 << 30, 1, 32, UNSUP), (1, 1 << 30, 32, UNSUP),
                          (1 << 20, 1 << 20, 32, UNSUP)):
        assert g(A, M, N, K, A, A, A, A, big, None) == want
        assert p(A, A, M, N, K, A, A, A, A, big, None) == want
        assert L.nvfp4_mx_gemm_workspace_size(M, N, K) == 0
    ws = L.nvfp4_mx_gemm_workspace_size(100, 300, 544)
    assert g(A, 100, 300, 544, A, A, A, None, 0, None) == (WS if ws else OK)
    assert ws == 0 or g(A, 100, 300, 544, A, A, A, A, ws - 1, None) == WS
    for i in range(4):
        bad = [A] * 4
        bad[i] = None
        assert g(bad[0], 4, 4, 64, bad[1], bad[2], bad[3], A, big, None) == NULL
        bad[i] = A + 8
        assert g(bad[0], 4, 4, 64, bad[1], bad[2], bad[3], A, big, None) == ALIGN
    for i in range(5):
        bad = [A] * 5
        bad[i] = None
        assert p(bad[0], bad[1], 4, 4, 64, *bad[2:], A, big, None) == NULL
        bad[i] = A + 8
        assert p(bad[0], bad[1], 4, 4, 64, *bad[2:], A, big, None) == ALIGN
    assert g(A, 4, 4, 64, A, A, A, A + 8, big, None) == ALIGN
    assert g(None, 0, 4, 64, None, None, None, None, 0, None) == OK
    assert p(None, None, 4, 0, 64, None, None, None, None, 0, None) == OK


def test_experts_checks():
    L = nv.lib()

    def call(ws=1 << 50, null=None, shift=None, tensors=True, wsp=A, **over):
        p = dict(T=4, E=8, top_k=2, H=64, I=32)
        p.update(over)
        t = {n: A for n, _ in nv.MxMoeTensors._fields_}
        if null:
            t[null] = None
        if shift:
            t[shift] = A + 2
        return L.nvfp4_mx_moe(ctypes.byref(nv.MxMoeProblem(**p)),
                              ctypes.byref(nv.MxMoeTensors(**t)) if tensors else None, wsp, ws, None)

    for over in (dict(T=-1), dict(E=0), dict(top_k=0), dict(H=0), dict(H=48), dict(I=0), dict(I=80)):
        assert call(**over) == SHAPE
    for over in (dict(E=4097), dict(T=1 << 30), dict(T=1 << 62, top_k=4), dict(T=1 << 20, H=4096), dict(H=1 << 16, I=1 << 15),
                 dict(T=1 << 20, top_k=8, I=1024), dict(H=1 << 40)):
        assert call(**over) == UNSUP
    assert call(tensors=False) == NULL
    for n, _ in nv.MxMoeTensors._fields_:
        assert call(null=n) == NULL and call(shift=n) == ALIGN
    assert call(wsp=None) == WS and call(ws=100) == WS and call(wsp=A + 8) == ALIGN
    assert L.nvfp4_mx_moe(None, None, None, 0, None) == NULL
    assert call(T=0, null="x", wsp=None, ws=0) == OK
    p = nv.MxMoeProblem(T=4, E=8, top_k=2, H=64, I=32)
    assert L.nvfp4_mx_moe_workspace_size(ctypes.byref(p)) > 0
    assert nv.mx_moe_workspace_size(0, 8, 2, 64, 32) == 0 and nv.mx_moe_workspace_size(4, 8, 2, 48, 32) == 0


def test_binding_rejects_bad_tensors():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    wc, ws = torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((8, 2), dtype=torch.uint8)
    with pytest.raises(TypeError, match="x"):
        nv.mx_gemm(x.float(), wc, ws)
    with pytest.raises(ValueError, match="CUDA"):
        nv.mx_gemm(x, wc, ws)
    with pytest.raises(ValueError, match="contiguous"):
        nv.mx_quantize(torch.zeros((64, 4), dtype=torch.bfloat16).t())
    with pytest.raises(ValueError, match="scales"):
        nv.mx_dequantize(wc, torch.zeros((8, 4), dtype=torch.uint8))
    with pytest.raises(ValueError, match="blocks"):
        nv.mx_dequantize(torch.zeros((8, 24), dtype=torch.uint8), torch.zeros((8, 1), dtype=torch.uint8))
    with pytest.raises(TypeError, match="logits"):
        nv.moe_gate(torch.zeros((4, 8), dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="CUDA"):
        nv.moe_gate(torch.zeros((4, 8)), 2)
    with pytest.raises(TypeError, match="topk_ids"):
        nv.mx_moe(x, torch.zeros((4, 2), dtype=torch.int64), torch.zeros((4, 2)), wc[None], ws[None], wc[None], ws[None])


def test_reference_against_worked_values():
    """The definition itself, on values worked by hand."""
    # 6, 3.1 and ties under scale 1 (amax 6: floor(log2 6) - 2 = 0)
    x = np.zeros((1, 32), np.float32)
    x[0, :9] = [6.0, 2.5, 3.5, 5.0, -0.25, 0.75, -7.0, 1.25, 3.125]
    x[0, 6] = -5.5
    bits = (torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy()).view(np.uint16)
    c, s = ref.mx_encode(bits)
    assert s[0, 0] == 127
    assert ref.mx_decode(c, s)[0, :9].tolist() == [6.0, 2.0, 4.0, 4.0, -0.0, 1.0, -6.0, 1.0, 3.0]
    assert ref.mx_encode(np.zeros((1, 32), np.uint16))[1][0, 0] == 0
    one = np.full((1, 32), 0x3F80, np.uint16)                  # 1.0: scale 2^-2, code of 4
    c, s = ref.mx_encode(one)
    assert s[0, 0] == 125 and (c == 0x66).all()
    assert np.array_equal(ref.bf16_round(np.array([1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, -0.0])),
                          np.array([0x3F80, 0x3F82, 0x8000], np.uint16))
    ids, w = ref.gate(np.array([[0.0, 1.0, 1.0, -np.inf]]), 3)
    e = np.exp(-1.0)
    assert ids.tolist() == [[1, 2, 0]] and np.allclose(w[0], np.array([1, 1, e]) / (2 + e))


def test_lds_loads_of_the_mx_kernels_have_their_wait_states(tmp_path):
    """As tests/test_dma_hazards.py, for the MXFP4 kernels' global-to-LDS loads."""
    import subprocess
    from nvfp4_bit_block_amd import build
    from tests.test_dma_hazards import hazards
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not found")
    out = str(tmp_path / "mx_gemm.s")
    r = subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-S", "-x", "hip",
                        os.path.join(build.CSRC, "mx_gemm.hip"), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    asm = open(out).read()
    assert re.search(r"buffer_load_\w+\s.*\blds$", asm, re.M)
    bad = hazards(asm)
    assert not bad, bad[:3]


def test_a_stream_of_another_device_is_refused():
    class Stream:
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        nv._launch(torch.device("cuda", 0), Stream(), lambda s: s)


def test_binding_refuses_an_odd_number_of_gate_up_rows():
    x, ids, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8)
    with pytest.raises(ValueError, match="gate and up"):
        nv.mx_moe(x, ids, w, u8(3, 65, 32), u8(3, 64, 2), u8(3, 64, 16), u8(3, 64, 1))


def test_binding_refuses_a_top_k_below_one():
    from nvfp4_bit_block_amd import gate
    for top_k in (0, -1):
        with pytest.raises(ValueError, match="top_k"):
            gate._config(4, 16, top_k, 1, 1, 1, "softmax", True, False, 1.0)


def test_product_limits():
    """One launch holds fewer than 2^32 threads: N of 2^28 and more is refused."""
    L = nv.lib()
    for N in (1 << 28, (1 << 30) - 1):
        assert L.nvfp4_mx_gemm(A, 1, N, 32, A, A, A, A, 1 << 40, None) == UNSUP
        assert L.nvfp4_mx_gemm_packed(A, A, 1, N, 32, A, A, A, A, 1 << 40, None) == UNSUP
