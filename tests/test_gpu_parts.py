"""A library whose kernel of sums in parts came out with fewer registers than its warps share out: that kernel is
left out, and what it is one way of computing, and all that has nothing to do with it, is computed as ever."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import bf16, status, usual, within, workspace
from test_gpu_distill import leaning, reference, run, teacher
from test_gpu_gated import Block, inputs, run_grad

pytestmark = pytest.mark.gpu


@pytest.fixture
def part_registers():
    yield ans._set_part_registers
    ans._set_part_registers(0)


@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8])
def test_other_registers_than_asked_for(cuda, part_registers, dtype):
    rng = np.random.default_rng(3)
    L = usual(dtype, 4096, 2048, seed=3)  # (32 x 3 tiles of 128 tokens: wide ones, whose sums come in parts)
    M, vocab = 300, 4000
    ids, logits = teacher(rng, M, vocab, 5)
    x = leaning(L, rng, M, ids)
    a, b, c = reference(L, x, vocab, 1.0, ids, logits)
    dy = bf16(rng, M, 4096, scale=0.1).cuda()
    size = ans.ans_gemm_grad_workspace(L.layout, M, L.kind)

    def gradient():
        dx, st = torch.empty(M, 2048, dtype=torch.bfloat16, device="cuda"), status()
        ans.ans_gemm_grad(dy, M, *L.args, dx, workspace(size), size, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return dx
    usual_loss, usual_grad = run(L, x, vocab, 1.0, ids, logits, grad=False), gradient()
    for least in (256, 0):
        part_registers(least)
        loss, lse, _ = run(L, x, vocab, 1.0, ids, logits, grad=False)
        within(loss, *a, f"loss {least}")
        within(lse, *b, f"lse {least}")
        assert torch.equal(loss, usual_loss[0]) == (least == 0)  # (in one accumulator, or in parts again)
        assert torch.equal(gradient(), usual_grad)
        within(run(L, x, vocab, 1.0, ids, logits)[2], *c, f"dx {least}")
    B = Block(dtype, 256, 128)
    x, dh = inputs(B, 40, 1)
    want = run_grad(B, x, dh, ans.ACT_SILU)
    part_registers(256)
    assert all(torch.equal(p, q) for p, q in zip(run_grad(B, x, dh, ans.ACT_SILU), want))
