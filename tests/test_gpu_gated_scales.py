"""ans_gated_grad beside row scales that a trained layer's are not: large ones, and gradients near fp32's end."""
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import BF16
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


@pytest.mark.parametrize("dtype", [ans.INT8, ans.FP8_E4M3])
@pytest.mark.parametrize("M", [5, 150, 700])
@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 12, 2.0 ** 14, 2.0 ** 17])
def test_one_row_of_far_larger_scales(cuda, dtype, M, ratio):
    """A row of far larger scales in both layers, with no part in the gradients of half the tokens: the others'
    keep theirs.  dX is off by two roundings to bf16 at most (dG and dU, and dX), each of some 0.43 BF16 of its
    norm: 0.6 BF16 together."""
    by = torch.ones(512, dtype=torch.float64)
    by[77] = ratio
    B = scaled(dtype, by)
    x, dh = inputs(B, M, 13)
    dx, dg, du = run_grad(B, x, dh, ans.ACT_RELU)
    g, u, d = x.double() @ B.gate.w.T, x.double() @ B.up.w.T, dh.double()
    want_g, want_u = torch.where(g > 0, d * u, 0.0), torch.where(g > 0, d * g, 0.0)
    want = want_g @ B.gate.w + want_u @ B.up.w
    assert (want_g[:, 77] == 0).any() and (want_g[:, 77] != 0).any()
    off = (dx.cpu().double() - want).norm(dim=1) / want.norm(dim=1)
    assert (off <= BF16).all(), f"{off.max().item():.3g}"
    again = run_grad(B, x, dh, ans.ACT_RELU)
    assert all(torch.equal(a, b) for a, b in zip((dx, dg, du), again))
    # and, whatever comes with it, a token's row is the same
    few = run_grad(B, x[:3], dh[:3], ans.ACT_RELU)
    assert torch.equal(few[1], dg[:3]) and torch.equal(few[2], du[:3])
