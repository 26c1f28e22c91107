"""ans_gated_grad beside row scales that a trained layer's are not: large ones, and gradients near fp32's end."""
import pytest
import torch

from rans_decode_gemm_b200 import ans

from test_gpu_gated import ACTS, Block, check_grad, inputs, run_grad

pytestmark = pytest.mark.gpu


def scaled(dtype, by, seed=3):
    """A block whose row scales are times `by` (a number, or one for each row)."""
    B = Block(dtype, 512, 128, seed=seed)
    for L in (B.gate, B.up):
        f = torch.as_tensor(by, dtype=torch.float64).expand(512)
        L.scales = (L.scales.double() * f.to(L.scales.device)).float()
        L.w = L.w * f[:, None]
    return B


@pytest.mark.parametrize("dtype", [ans.INT8, ans.FP8_E4M3, ans.FP4_PAIRS])
@pytest.mark.parametrize("M", [7, 150])
def test_gradients_near_the_end_of_fp32(cuda, dtype, M):
    """Row scales of 2 to 8 (2^11 of the usual 1e-3 to 4e-3) beside products of dH and x of 1e-38 to 1e-40: dX of 1e-33."""
    B = scaled(dtype, 2048.0)
    for size_x, size_h in ((1e-22, 1e-16), (1e-21, 1e-16), (1e-16, 1e-22), (1e-10, 1e-10)):
        x, dh = inputs(B, M, 9, size_x)
        dh = (dh.float() * size_h).bfloat16()
        for act in ACTS:
            check_grad(B, x, dh, act)
    # a token without a gradient, and one of zeros, beside them
    x, dh = inputs(B, M, 9, 1e-22)
    dh = (dh.float() * 1e-16).bfloat16()
    x[1], dh[2] = 0, 0
    dx, dg, du = run_grad(B, x, dh, ans.ACT_SILU)
    assert not dx[1:3].any() and not dg[1:3].any() and not du[1:3].any()
