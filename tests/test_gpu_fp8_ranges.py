"""The FP8 block-scaled operators at the ends of their ranges, against 64-bit plain forms."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
import microscaling_quantized_linear_b200 as nvq
from test_gpu_fp8_block import check, operand, product_bounds

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ scales

@pytest.mark.parametrize("big", [105, -109])
@pytest.mark.parametrize("M,N,K", [(40, 136, 272), (300, 400, 528)])
def test_products_of_opposing_scales(M, N, K, big):
    """One operand's scales near the end of FP32, the other's bringing their product back, and codes of 256 to
    448 of one sign, whose blocks sum to 2^24: exact, in steps of 2^12."""
    small = -60 if big > 0 else 64
    for op, kinds, shapes in ((nvq.fp8_block_linear, ("rows", "tiles"), ((M, K), (N, K))),
                              (nvq.fp8_block_linear_dgrad, ("rows", "tiles"), ((M, N), (N, K))),
                              (nvq.fp8_block_linear_wgrad, ("columns", "columns"), ((M, N), (M, K)))):
        for ea, eb in ((big, small), (small, big)):
            a, b = (operand(*s, k, i, True) for i, (s, k) in enumerate(zip(shapes, kinds)))
            for codes, _ in (a, b):
                codes.bitwise_and_(7).bitwise_or_(0x78).clamp_(max=0x7E)
            a[1].mul_(2.0 ** ea)
            b[1].mul_(2.0 ** eb)
            A, B = ref.value(*a, kinds[0]), ref.value(*b, kinds[1])
            if op is nvq.fp8_block_linear_dgrad:
                B, T = B.T, N
            elif op is nvq.fp8_block_linear_wgrad:
                A, B, T = A.T, B.T, M
            else:
                T = K
            want, _ = product_bounds(A, B, T, True)
            check(op(*a, *b), want, 0.0, unit=2.0 ** -24 if op is nvq.fp8_block_linear_wgrad else 2.0 ** -8)
    assert nvq.device_status() == 0
