"""ans_gated over batches of changing size, as a program that decodes and takes prompts in turn calls it."""
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import status, within, workspace
from test_gpu_gated import Block, forward_reference, inputs, run_forward, run_grad

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,N,K", [(ans.BF16_SPLIT, 512, 512), (ans.INT8, 640, 1024), (ans.INT4_PAIRS, 512, 1024)])
def test_one_workspace_serves_every_batch(cuda, dtype, N, K):
    """Prompts, single tokens and gradients in turn, in one workspace: the bits of a fresh one each time."""
    B = Block(dtype, N, K, seed=4)
    order = (300, 1, 40, 32, 300, 5, 16, 2, 129, 32)
    size = max(max(ans.ans_gated_workspace(B.layout, M, B.kind), ans.ans_gated_grad_workspace(B.layout, M, B.kind))
               for M in order)
    ws, st = workspace(size), status()
    for turn, M in enumerate(order):
        x, dh = inputs(B, M, turn)
        h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        ans.ans_gated(x.cuda(), M, *B.args(ans.ACT_SILU), h, ws, size, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert torch.equal(h, run_forward(B, x, ans.ACT_SILU)), f"M {M}, turn {turn}"
        if turn % 3 == 2:
            dx, dg, du = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty_like(h), torch.empty_like(h)
            ans.ans_gated_grad(x.cuda(), dh.cuda(), M, *B.args(ans.ACT_SILU), dx, dg, du, ws, size, st)
            torch.cuda.synchronize()
            assert int(st.item()) == 0
            assert all(torch.equal(a, b) for a, b in zip((dx, dg, du), run_grad(B, x, dh, ans.ACT_SILU)))


@pytest.mark.parametrize("dtype", [ans.INT8, ans.FP8_E4M3, ans.INT4_PAIRS, ans.INT4, ans.FP4_E2M1, ans.BF16_SPLIT])
@pytest.mark.parametrize("M", [1, 16, 32, 33])
def test_rows_of_any_size_in_batches_of_any_size(cuda, dtype, M):
    """Rows far outside f16's range, below and above: a token's result does not depend on how many come with it."""
    B = Block(dtype, 512, 256, seed=7)
    x, _ = inputs(B, M, 11)
    sizes = torch.tensor([1e-7, 1e6, 1e-15, 1e12, 1.0, 7e4])
    for first in range(6 if M == 1 else 1):
        y = (x.float() * sizes[(torch.arange(M) + first) % 6][:, None]).bfloat16()
        for act in (ans.ACT_SILU, ans.ACT_RELU):
            h = run_forward(B, y, act)
            within(h, *forward_reference(B, y, act), f"h {act} {first}")
            # and within two roundings of those of a batch that is large enough to be decoded first
            many = run_forward(B, torch.cat([y, y.new_zeros(64, B.K)]), act)[:M]
            want, bound = forward_reference(B, y, act)
            assert ((h.double() - many.double()).abs().cpu() <= 2 * bound).all()
