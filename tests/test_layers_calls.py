"""Calls of the layers around the mixer whose sizes pass the integers that carry them (no GPU needed)."""
import ctypes

import pytest

import gated_delta_rule_wy_b200 as g
from gated_delta_rule_wy_b200 import binding as b

P, Q, S = (ctypes.c_void_p(v) for v in (0x10000, 0x20000, 0x30000))
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_wy_b200 import build

    build.build()
    return g.load_library()


@pytest.mark.parametrize("N,T,H", [(1 << 21, 1 << 21, 1 << 21), (MOST, MOST, MOST), (MOST, 0, MOST), (1 << 20, 0, 1 << 20),
                                   (1, 1, MOST), (1 << 24, 1 << 10, 1 << 10)])
def test_convolution_gradients_refuse_sizes_whose_products_wrap(lib, N, T, H):
    """Elements, scratch bytes or blocks past their integers, also where a product of them is a small number again."""
    st = lib.gdr2_short_conv_silu_backward(N, T, H, 64, b.GDR2_BF16, 4, 0, ctypes.c_float(1e-6), P, P, None, Q, None, S, S,
                                           None, P, ctypes.c_size_t((1 << 64) - 1), None)
    assert st == b.GDR2_ERR_INVALID_ARG and b"too large" in lib.gdr2_last_error()


def test_a_first_position_past_32_bits_is_not_taken_for_its_low_half():
    import torch

    q = torch.zeros(1, 4, 2, 64)
    for first in (2 ** 31, 2 ** 32 + 3, -2 ** 31 - 1, -2 ** 32 + 3):
        with pytest.raises(ValueError, match="first_position"):
            g.gdr2_head_norm_rope(q, first_position=first)
        with pytest.raises(ValueError, match="first_position"):
            g.gdr2_head_norm_rope_backward(q, None, q, first_position=first)


def test_norm_and_rotation_refuse_one_buffer_for_both_outputs(lib):
    common = (1, 4, 2, 2, 64, b.GDR2_BF16, 1, ctypes.c_float(1e-6), P, 128, P, 128, None, None, 64, 0, P, 16, None, 0)
    assert lib.gdr2_head_norm_rope(*common, Q, Q, None) == b.GDR2_ERR_INVALID_ARG and b"same" in lib.gdr2_last_error()
    for dq, dk, dqw, dkw in ((Q, Q, None, None), (Q, S, ctypes.c_void_p(0x50000), ctypes.c_void_p(0x50000))):
        st = lib.gdr2_head_norm_rope_backward(*common, P, P, dq, dk, dqw, dkw, P, ctypes.c_size_t(1 << 40), None)
        assert st == b.GDR2_ERR_INVALID_ARG and b"same" in lib.gdr2_last_error()
