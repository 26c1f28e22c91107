"""Infinities and NaN in adapters, activations and gradients: where the formulas in
64 bits give an infinity or NaN, the operators give the same, and the rest holds the
bounds of finite inputs."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import bf16, usual
from test_gpu_grad_lora import Adapters, lora_grad_reference, lora_reference, run_lora, run_lora_grad

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def same(got, want, bound, what):
    got, fin = got.detach().cpu().double(), torch.isfinite(want)
    assert fin.any() and not fin.all()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)]), what
    assert ((got - want).abs() <= bound)[fin].all(), what


def adapters(L, n, rank, **at):
    A = Adapters(L, n, rank, scale=False)
    for name, values in at.items():
        for place, v in values.items():
            getattr(A, name)[place] = v
    A.dev = ans.LoraAdapters(A.a.cuda(), A.b.cuda())
    A.lora = A.dev.lora
    return A


def inputs(L, M, n):
    """Random tokens, every third one with a single 1: what an adapter makes of it
    is a bf16 number, whose second part is 0."""
    rng = np.random.default_rng(M)
    x, dy = bf16(rng, M, L.K), bf16(rng, M, L.N)
    for m in range(0, M, 3):
        x[m] = 0
        x[m, m % L.K] = 1.0
    return x, dy, torch.from_numpy(rng.integers(-1, n, M).astype(np.int32))


@pytest.mark.parametrize("rank", [8, 24, 40, 72])
@pytest.mark.parametrize("M", [7, 40, 300])
def test_adapters_that_are_not_finite(cuda, M, rank):
    L = usual(ans.BF16_SPLIT, 384, 208, seed=rank)
    A = adapters(L, 4, rank, a={(0, 2, 7): INF, (3, 1, 200): NAN}, b={(1, 3, 5): INF, (1, 77, 0): -INF, (1, 300, 7): NAN, (0, 9, 2): INF})
    x, _, ids = inputs(L, M, 4)
    ids[:4] = torch.tensor([0, 1, 2, 1], dtype=torch.int32)
    y, st = run_lora(L, A, x, ids)
    assert st == 0
    same(y, *lora_reference(L, A, x, ids), "y")


@pytest.mark.parametrize("rank", [8, 24, 40, 72])
@pytest.mark.parametrize("M", [7, 40, 300])
def test_gradients_that_are_not_finite(cuda, M, rank):
    L = usual(ans.BF16_SPLIT, 384, 208, seed=rank)
    A = adapters(L, 4, rank)
    x, dy, ids = inputs(L, M, 4)
    ids[:7] = torch.tensor([0, 0, 1, 2, 3, 1, 2], dtype=torch.int32)
    dy[0, 100], dy[1, 5], dy[1, 383], dy[2, 0] = INF, -INF, NAN, -INF
    x[4, 33], x[5, 207] = -INF, NAN
    dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
    assert st == 0
    for name, got, ref in zip(("dx", "da", "db"), (dx, da, db), lora_grad_reference(L, A, x, dy, ids)):
        same(got, *ref, name)
    _, da2, db2, _ = run_lora_grad(L, A, x, dy, ids, want_dx=False)
    assert torch.equal(da.view(torch.int32), da2.view(torch.int32)) and torch.equal(db.view(torch.int32), db2.view(torch.int32))


@pytest.mark.parametrize("M", [7, 300])
def test_gradients_of_adapters_that_are_not_finite(cuda, M):
    L = usual(ans.INT8, 256, 320, seed=3)
    A = adapters(L, 4, 16, a={(0, 2, 7): INF}, b={(1, 3, 5): INF, (3, 255, 15): NAN})
    x, dy, ids = inputs(L, M, 4)
    ids[:4] = torch.tensor([0, 1, 2, 1], dtype=torch.int32)
    dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
    assert st == 0
    for name, got, ref in zip(("dx", "da", "db"), (dx, da, db), lora_grad_reference(L, A, x, dy, ids)):
        same(got, *ref, name)
