"""Sizes at the ends of the documented ranges, on a machine without a GPU:
what is out of range is refused by the host's own checks, and what is in range
passes them and the launchers' and ends at the missing device."""
import nvfp4_bit_block_amd as nv

UNSUP = 4


def test_columnwise_quantize_refuses_sizes_near_2_63():
    L = nv.lib()
    for rows, cols in ((2 ** 63 - 32, 1), (2 ** 63 - 224, 64), (32, 2 ** 63 - 1), (32, 2 ** 63 - 63),
                       (2 ** 63 - 32, 2 ** 63 - 1)):
        assert L.nvfp4_mx_quantize_columnwise(None, rows, cols, None, None, None) == UNSUP, (rows, cols)
