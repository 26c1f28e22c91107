"""ans_distill on lists at their ends: a teacher that has nothing above -infinity, and one that lists everything."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import BF16, Layer, sum_eps, usual, within
from test_gpu_distill import leaning, reference, run, teacher

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8])
@pytest.mark.parametrize("nothing", [-np.inf, np.nan, np.inf])
def test_a_teacher_with_nothing_above_minus_infinity(cuda, dtype, nothing):
    """A masked row's logits are all -infinity, and so is their lse (or it is NaN): nothing is listed."""
    rng = np.random.default_rng(4)
    L = usual(dtype, 512, 64, seed=13)
    M, vocab = 30, 500
    ids, logits = teacher(rng, M, vocab, 6)
    ids[2], logits[2] = torch.arange(6, dtype=torch.int32), -torch.inf
    ids[9] = torch.tensor([5, -1, 5, 400, -1, 7], dtype=torch.int32)
    logits[9] = -torch.inf
    x = leaning(L, rng, M, ids)
    held = torch.logsumexp(logits.double().masked_fill(ids < 0, -torch.inf), 1) + 0.3
    held = torch.where(torch.isfinite(held), held, 0.0).float()
    a, b, c = reference(L, x, vocab, 1.0, ids, logits, held)
    held[2] = held[9] = nothing
    for grad in (True, False):
        loss, lse, dx = run(L, x, vocab, 1.0, ids, logits, held, grad=grad)
        assert (loss[[2, 9]] == 0).all()
        within(loss, *a, "loss")
        within(lse, *b, "lse")
        if grad:
            assert not dx[[2, 9]].any()
            within(dx, *c, "dx")


@pytest.mark.parametrize("dtype", [ans.INT8, ans.FP4_E2M1, ans.BF16_SPLIT])
@pytest.mark.parametrize("step", [2.0 ** -20, 2.0 ** -12, 0.5])
def test_a_wholly_listed_vocabulary_that_has_been_learnt(cuda, dtype, step):
    """No others, and coefficients S p - t of 1e-8: they are rounded relative to the largest of them.

    Weights are small whole numbers (or halves) times 2^-6 and x sixteenths, so that logits are exact in fp32; the
    teacher's differ by a few steps that fp32 holds beside them.  What is left is 64-bit arithmetic (as in the
    other tests' reference), the roundings to 16 bits, the product's sums and dX's own rounding."""
    rng = np.random.default_rng([dtype, int(1 / step)])
    L = Layer(dtype, 256, 64, 128, 64, ans.SCALE_NONE if dtype == ans.BF16_SPLIT else ans.SCALE_ROW_F32, 0, 17)
    if dtype == ans.BF16_SPLIT:
        L.w = (L.w * 640).round() / 64
        codes = L.w.bfloat16()
        assert (codes.double() == L.w).all()
        L.layer = ans.CompressedLayer.from_weights(codes.view(torch.int16).numpy().view(np.uint16).reshape(-1), L.layout)
        L.tiles = L.layer.tiles
    else:
        L.w = (L.w / L.scales.cpu().double()[:, None]).round(decimals=1) / 64
        L.scales.fill_(1 / 64)
    M, vocab = 20, 200
    x = torch.from_numpy(rng.integers(-4, 5, (M, 64)) / 16.0).bfloat16()
    z = x.double() @ L.w[:vocab].T
    ids = torch.from_numpy(np.stack([rng.permutation(vocab) for _ in range(M)]).astype(np.int32))
    v = z.gather(1, ids.long()) + step * torch.from_numpy(rng.integers(-3, 4, (M, vocab)).astype(np.float64))
    v[7] = z[7].gather(0, ids[7].long())  # (this student is its teacher)
    logits = v.float()
    assert (logits.double() == v).all() and z.abs().max() < 8
    p = torch.softmax(z, 1)
    t = torch.zeros_like(p).scatter_(1, ids.long(), torch.softmax(v, 1))
    coef = p - t
    wide = (z.abs().amax(1) + v.abs().amax(1) + 20)[:, None]
    per = (L.factor_eps + sum_eps(vocab) + 2.0 ** -22) * coef.abs() + 2.0 ** -51 * wide * (p + t)
    w = L.w[:vocab]
    want = coef @ w
    inner = per @ w.abs() + 2.0 ** -37 * coef.abs().amax(1, keepdim=True) * w.abs().sum(0)[None, :]
    _, _, dx = run(L, x, vocab, 1.0, ids, logits)
    within(dx, want, inner + BF16 * (want.abs() + inner) + 2.0 ** -133, "dx")
    # a vocabulary that is all but listed: the row that is not carries what its probability is
    _, _, part = run(L, x, vocab, 1.0, ids[:, :-1].contiguous(), logits[:, :-1].contiguous())
    assert torch.isfinite(part).all()
