"""ans_xent where probabilities are small: what they leave in dX.

The bounds here scale with 1 - p_t.  A probability's rounding counts against the
others' sum alone: half a step of the format (2^-11 of it in f16, 2^-8 in bf16),
and what f16 cannot hold of it.  Stored as e s_n 2^k with the largest scale times
2^k at 2^8 or more, and the others' largest e at 1/2 or more, a rounding below
f16's normal range is off by at most 2^-25 2^-8 = 2^-33 of the largest scale, which
is 2^-32 of (1 - p_t) s_max; a block that is rescaled is rounded twice: 2^-31."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import BF16, status, sum_eps, usual, within, workspace

pytestmark = pytest.mark.gpu

FORMATS = [ans.INT8, ans.FP8_E4M3, ans.INT4_PAIRS, ans.FP4_E2M1, ans.BF16_SPLIT]


def reference(L, x, targets, vocab, weight=None):
    """(loss, lse, dx) in 64 bits with the bounds of right results, and 1 - p_t."""
    x64, w = x.double(), L.w[:vocab]
    z = x64 @ w.T
    has = targets >= 0
    at = targets.clamp_min(0).long()[:, None]
    zt = z.gather(1, at)[:, 0]
    others = torch.logsumexp(z.scatter(1, at, -torch.inf), 1)
    lse = torch.logaddexp(others, zt)
    loss = torch.where(has, torch.logaddexp(torch.zeros_like(zt), others - zt), 0.0)
    # a logit is an fp32 sum, times its factors and log2(e): 2^-22 more of it
    zerr = (sum_eps(L.K) * (x64.abs() @ w.abs().T)).amax(1) + 2.0 ** -22 * z.abs().amax(1)
    lse_b = zerr + 2.0 ** -19 + 2.0 ** -23 * lse.abs()
    # log(1 + e^d): relative to itself, the error of d and of the exponentials' sum
    loss_b = torch.where(has, loss * (torch.expm1(2 * zerr) + 2.0 ** -18), 0.0)
    g = torch.ones(len(x), dtype=torch.float64) if weight is None else weight.double()
    g = torch.where(has, g, 0.0)
    p = torch.exp(z.scatter(1, at, -torch.inf) - lse[:, None])
    rest = p.sum(1)
    dx = g[:, None] * (p @ w - rest[:, None] * w[at[:, 0]])
    mass = p @ w.abs() + rest[:, None] * w[at[:, 0]].abs()
    inner = g.abs()[:, None] * (L.factor_eps + sum_eps(L.N) + torch.expm1(4 * zerr)[:, None] + 2.0 ** -18) * mass
    if L.dtype != ans.BF16_SPLIT:
        s = L.scales[:vocab].cpu().double().abs() if L.kind in (ans.SCALE_ROW_BF16, ans.SCALE_ROW_F32) else torch.ones(vocab).double()
        inner = inner + (g.abs() * rest)[:, None] * 2.0 ** -31 * ((s.max() / s)[:, None] * w.abs()).sum(0)[None, :]
    return (loss, loss_b), (lse, lse_b), (dx, inner + BF16 * (dx.abs() + inner)), rest


def run(L, x, targets, vocab, weight=None, grad=True):
    M = x.shape[0]
    ws = workspace(ans.ans_xent_workspace(L.layout, M, L.kind, grad))
    loss, lse = (torch.full((M,), float("nan"), device="cuda") for _ in range(2))
    dx = torch.full((M, L.K), float("nan"), dtype=torch.bfloat16, device="cuda") if grad else None
    st = status()
    ans.ans_xent(x.cuda(), M, *L.args, vocab, targets.cuda(), loss, lse, None if weight is None else weight.cuda(), dx,
                 ws, ws.numel(), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return loss, lse, dx


def put(L, codes, values):
    """Other codes (as stored) and their values in the layer L."""
    L.codes = np.ascontiguousarray(codes)
    L.layer = ans.CompressedLayer.from_weights(L.codes.reshape(-1), L.layout)
    L.tiles = L.layer.tiles
    if L.kind in (ans.SCALE_ROW_F32, ans.SCALE_ROW_BF16):
        values = values * L.scales.cpu().double().numpy()[:, None]
    elif L.kind == ans.SCALE_GROUP_BF16:
        values = values * np.repeat(L.scales.cpu().double().numpy(), L.group_k, axis=1)
    L.w = torch.from_numpy(np.ascontiguousarray(values))


@pytest.mark.parametrize("N,vocab", [(256, 256), (24832, 24800)])
@pytest.mark.parametrize("dtype", FORMATS)
def test_rows_far_below_the_largest(cuda, dtype, N, vocab):
    # rows whose columns are theirs alone, 2^-18 to 2^-28 of the largest and in other
    # blocks than it: a column of dX is one probability times one weight
    L = usual(dtype, N, 64, seed=9)
    rows = [0, 40, 70, 100, 140, 170, 200, 255]
    below = np.array([0, 18, 20, 22, 24, 25, 26.5, 28])
    v = np.zeros((N, 64))
    for i, r in enumerate(rows):
        v[r, 8 * i:8 * i + 8] = 4.0
    if dtype == ans.INT8:
        put(L, v.astype(np.uint8), v)
    elif dtype == ans.FP8_E4M3:
        put(L, torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy(), v)
    elif dtype == ans.BF16_SPLIT:
        put(L, torch.from_numpy(v).bfloat16().view(torch.int16).numpy().view(np.uint16), v)
    else:
        nib = np.where(v > 0, 4 if dtype == ans.INT4_PAIRS else 6, 0).astype(np.uint8)
        put(L, nib[:, 0::2] | (nib[:, 1::2] << 4), v)
    z = torch.from_numpy(60 - np.log(2) * below)
    x = torch.cat([z[i].expand(8) / (8 * L.w[r, 8 * i]) for i, r in enumerate(rows)])
    x = torch.stack([x, x.flip(0)]).float().bfloat16()
    _, _, dx = run(L, x, torch.tensor([130, 130], dtype=torch.int32), vocab)
    _, _, want, _ = reference(L, x, torch.tensor([130, 130], dtype=torch.int32), vocab)
    within(dx, *want, "dx")
