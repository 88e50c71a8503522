"""MXFP4 (``include/nvfp4_mx.h``): quantize, dequantize, products and the
routed-expert layer.  Argument marshalling only, as in the package's
``__init__``; an MXFP4 tensor [R, C] is a pair of uint8 tensors, codes
[R, C/2] and E8M0 scale bytes [R, C/32]."""
from __future__ import annotations

import torch

import nvfp4_bit_block_amd as nv


def _mx_tensor(codes, scales, name, device=None):
    """codes uint8 [R, C/2], scales uint8 [R, C/32], C a multiple of 32, on
    one device (`device` if given); returns (R, C, device)."""
    # dtypes and shapes first, then the devices
    nv._req(codes, name + "codes", nv._U8, (None, None))
    rows, half = codes.shape
    if half % 16:
        raise ValueError(f"{name}codes: rows of {half} bytes are not whole blocks of 32 elements")
    dev = codes.device
    nv._arg(scales, name + "scales", nv._U8, (rows, half // 16), None if dev.type != "cuda" else dev)
    nv._cuda(codes, name + "codes", device)
    return rows, 2 * half, dev


def _activation(x):
    return nv._matrix(x, "x", nv._BF16)


def _mx_weights(w_codes, w_scales, K, dev):
    N, Kw, _ = _mx_tensor(w_codes, w_scales, "w_", dev)
    if Kw != K:
        raise ValueError(f"w_codes: rows of {Kw} elements, the activation has {K}")
    return N


def _workspace(ws, need, dev):
    """(tensor to hold on to, address, bytes) of the caller's workspace, or of
    a new one of `need` bytes (none for 0)."""
    if ws is not None:
        nv._req(ws, "ws", nv._U8, device=dev)
    elif need:
        ws = nv.workspace(need, dev)
    return (None, None, 0) if ws is None else (ws, ws.data_ptr(), ws.numel())


def mx_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(nv.lib().nvfp4_mx_gemm_workspace_size(M, N, K))


def mx_gemm_packed_workspace_size(M: int, N: int, K: int) -> int:
    return int(nv.lib().nvfp4_mx_gemm_packed_workspace_size(M, N, K))


def mx_moe_workspace_size(T, E, top_k, H, I) -> int:
    return int(nv.lib().nvfp4_mx_moe_workspace_size(nv.MxMoeProblem(T, E, top_k, H, I)))


def mx_quantize(x, codes=None, scales=None, stream=None):
    """nvfp4_mx_quantize: bf16 [R, C] -> (codes [R, C/2], scales [R, C/32])."""
    rows, cols, dev = _activation(x)

    def body(s):
        c = nv._out(codes, "codes", torch.uint8, (rows, cols // 2), dev)
        e = nv._out(scales, "scales", torch.uint8, (rows, cols // 32), dev)
        nv._check(nv.lib().nvfp4_mx_quantize(x.data_ptr(), rows, cols, c.data_ptr(), e.data_ptr(), s),
                  "nvfp4_mx_quantize")
        return c, e
    return nv._launch(dev, stream, body)


def mx_quantize_columnwise(x, codes=None, scales=None, stream=None):
    """nvfp4_mx_quantize_columnwise: the MXFP4 of x^T, bf16 [R, C] -> (codes
    [C, R/2], scales [C, R/32])."""
    rows, cols, dev = _activation(x)

    def body(s):
        c = nv._out(codes, "codes", torch.uint8, (cols, rows // 2), dev)
        e = nv._out(scales, "scales", torch.uint8, (cols, rows // 32), dev)
        nv._check(nv.lib().nvfp4_mx_quantize_columnwise(x.data_ptr(), rows, cols, c.data_ptr(), e.data_ptr(), s),
                  "nvfp4_mx_quantize_columnwise")
        return c, e
    return nv._launch(dev, stream, body)


def mx_dequantize(codes, scales, out=None, stream=None):
    """nvfp4_mx_dequantize: the exact bf16 values [R, C]."""
    rows, cols, dev = _mx_tensor(codes, scales, "")

    def body(s):
        y = nv._out(out, "out", torch.bfloat16, (rows, cols), dev)
        nv._check(nv.lib().nvfp4_mx_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, y.data_ptr(), s),
                  "nvfp4_mx_dequantize")
        return y
    return nv._launch(dev, stream, body)


def mx_gemm(x, w_codes, w_scales, out=None, ws=None, stream=None):
    """nvfp4_mx_gemm: bf16 [M, K] x MXFP4 [N, K] -> bf16 [M, N], the activation
    quantized within the call."""
    M, K, dev = _activation(x)
    N = _mx_weights(w_codes, w_scales, K, dev)

    def body(s):
        y = nv._out(out, "out", torch.bfloat16, (M, N), dev)
        L = nv.lib()
        hold, wp, wn = _workspace(ws, 0 if ws is not None else L.nvfp4_mx_gemm_workspace_size(M, N, K), dev)
        nv._check(L.nvfp4_mx_gemm(x.data_ptr(), M, N, K, w_codes.data_ptr(), w_scales.data_ptr(), y.data_ptr(),
                                  wp, wn, s), "nvfp4_mx_gemm")
        return y
    return nv._launch(dev, stream, body)


def mx_gemm_packed(a_codes, a_scales, w_codes, w_scales, out=None, ws=None, stream=None):
    """nvfp4_mx_gemm_packed: MXFP4 [M, K] x MXFP4 [N, K] -> bf16 [M, N]."""
    M, K, dev = _mx_tensor(a_codes, a_scales, "a_")
    N = _mx_weights(w_codes, w_scales, K, dev)

    def body(s):
        y = nv._out(out, "out", torch.bfloat16, (M, N), dev)
        L = nv.lib()
        hold, wp, wn = _workspace(ws, 0 if ws is not None else L.nvfp4_mx_gemm_packed_workspace_size(M, N, K), dev)
        nv._check(L.nvfp4_mx_gemm_packed(a_codes.data_ptr(), a_scales.data_ptr(), M, N, K, w_codes.data_ptr(),
                                         w_scales.data_ptr(), y.data_ptr(), wp, wn, s), "nvfp4_mx_gemm_packed")
        return y
    return nv._launch(dev, stream, body)


def mx_moe(x, topk_ids, topk_weights, w13_codes, w13_scales, w2_codes, w2_scales, out=None, ws=None, stream=None):
    """nvfp4_mx_moe: the routed-expert layer on MXFP4 experts.  topk_ids int32
    and topk_weights fp32 [T, k], as ``moe_gate`` gives them (ids outside
    [0, E) are skipped)."""
    # every dtype and shape first, then the devices
    nv._bf16(x, "x", (None, None))
    T, H = x.shape
    nv._req(topk_ids, "topk_ids", nv._I32, (T, None))
    k = topk_ids.shape[1]
    nv._req(topk_weights, "topk_weights", nv._F32, (T, k))
    nv._req(w13_codes, "w13_codes", nv._U8, (None, None, H // 2))
    E, twoI, _ = w13_codes.shape
    if twoI % 2:
        raise ValueError(f"w13_codes: {twoI} rows per expert, need gate and up rows, the same number of each")
    I = twoI // 2
    nv._req(w13_scales, "w13_scales", nv._U8, (E, 2 * I, H // 32))
    nv._req(w2_codes, "w2_codes", nv._U8, (E, H, I // 2))
    nv._req(w2_scales, "w2_scales", nv._U8, (E, H, I // 32))
    dev = nv._cuda(x, "x").device
    for t, n in ((topk_ids, "topk_ids"), (topk_weights, "topk_weights"), (w13_codes, "w13_codes"),
                 (w13_scales, "w13_scales"), (w2_codes, "w2_codes"), (w2_scales, "w2_scales")):
        nv._cuda(t, n, dev)

    def body(s):
        y = nv._out(out, "out", torch.bfloat16, (T, H), dev)
        L = nv.lib()
        p = nv.MxMoeProblem(T, E, k, H, I)
        hold, wp, wn = _workspace(ws, 0 if ws is not None else L.nvfp4_mx_moe_workspace_size(p), dev)
        t = nv.MxMoeTensors(x.data_ptr(), topk_ids.data_ptr(), topk_weights.data_ptr(), w13_codes.data_ptr(),
                            w13_scales.data_ptr(), w2_codes.data_ptr(), w2_scales.data_ptr(), y.data_ptr())
        nv._check(L.nvfp4_mx_moe(p, t, wp, wn, s), "nvfp4_mx_moe")
        return y
    return nv._launch(dev, stream, body)
