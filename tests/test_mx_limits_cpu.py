"""Sizes at the ends of the documented ranges, on a machine without a GPU:
what is out of range is refused by the host's own checks, and what is in range
passes them and the launchers' and ends at the missing device."""
import pytest
import torch

import nvfp4_bit_block_amd as nv

UNSUP, HIP = 4, 6
A = 4096


def test_columnwise_quantize_refuses_sizes_near_2_63():
    L = nv.lib()
    for rows, cols in ((2 ** 63 - 32, 1), (2 ** 63 - 224, 64), (32, 2 ** 63 - 1), (32, 2 ** 63 - 63),
                       (2 ** 63 - 32, 2 ** 63 - 1)):
        assert L.nvfp4_mx_quantize_columnwise(None, rows, cols, None, None, None) == UNSUP, (rows, cols)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls below may not reach a device")
@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 64, 65])
def test_products_at_the_largest_sizes_have_a_launch(M):
    """Every size inside the documented limits gets past the launchers' own
    checks (fewer than 2^32 threads in a launch)."""
    L = nv.lib()
    sizes = [((1 << 28) - 1, 32), ((1 << 28) - 1, 8192), ((1 << 26) + 16, 8192), ((1 << 26) - 16, 8192), (1 << 24, 16384)]
    for N, K in sizes:
        for call in (lambda: L.nvfp4_mx_gemm(A, M, N, K, A, A, A, A, 1 << 60, None),
                     lambda: L.nvfp4_mx_gemm_packed(A, A, M, N, K, A, A, A, A, 1 << 60, None)):
            assert call() == HIP and b"no ROCm-capable device" in L.nvfp4_last_error(), (N, K, L.nvfp4_last_error())
