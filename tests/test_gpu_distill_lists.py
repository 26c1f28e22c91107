"""ans_distill on lists at their ends: a teacher that has nothing above -infinity, and one that lists everything."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import BF16, F16, Layer, sum_eps, usual, within
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
