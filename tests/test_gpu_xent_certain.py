"""ans_xent for tokens that are all but certain of their target: heads whose rows
share a mean, one row beside the target, and targets far above or alone.

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

from _ops_util import BF16, E2M1, bf16, status, sum_eps, usual, within, workspace

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


def check(L, x, targets, vocab, weight=None):
    loss, lse, dx = run(L, x, targets, vocab, weight)
    a, b, c, rest = reference(L, x, targets, vocab, weight)
    within(loss, *a, "loss")
    within(lse, *b, "lse")
    within(dx, *c, "dx")
    loss, lse, _ = run(L, x, targets, vocab, grad=False)
    within(loss, *a, "loss alone")
    within(lse, *b, "lse alone")
    return rest


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


def with_a_mean(L, seed):
    """Rows with a mean of their own size in every column, as a trained head's have."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((L.N, L.K)).astype(np.float32) + rng.standard_normal((1, L.K)).astype(np.float32)
    if L.dtype == ans.INT8:
        q = np.clip(np.rint(30 * v), -127, 127).astype(np.int8)
        put(L, q.view(np.uint8), q.astype(np.float64))
    elif L.dtype == ans.FP8_E4M3:
        t = torch.from_numpy(20 * v).to(torch.float8_e4m3fn)
        put(L, t.view(torch.uint8).numpy(), t.double().numpy())
    elif L.dtype == ans.BF16_SPLIT:
        t = torch.from_numpy(0.05 * v).bfloat16()
        put(L, t.view(torch.int16).numpy().view(np.uint16), t.double().numpy())
    elif L.dtype == ans.INT4_PAIRS:
        q = np.clip(np.rint(2 * v), -8, 7).astype(np.int64)
        nib = (q & 15).astype(np.uint8)
        put(L, nib[:, 0::2] | (nib[:, 1::2] << 4), q.astype(np.float64))
    else:
        nib = np.abs(np.abs(2 * v)[..., None] - E2M1[:8]).argmin(-1).astype(np.uint8)
        nib = np.where((v < 0) & (nib > 0), nib | 8, nib).astype(np.uint8)
        put(L, nib[:, 0::2] | (nib[:, 1::2] << 4), E2M1[nib])


def leaning(L, targets, vocab, wanted):
    """Hidden states along their target's row less the mean row, as long as they
    have to be for each 1 - p_t wanted."""
    w = L.w[:vocab]
    out = []
    for t, rest in zip(targets, wanted):
        d = w[t] - w.mean(0)
        z = w @ d
        low, high = 0.0, 400.0 / float(d @ d)
        for _ in range(60):
            b = 0.5 * (low + high)
            e = b * z
            e[t] = -torch.inf
            gap = float(b * z[t] - torch.logsumexp(e, 0))
            low, high = (b, high) if gap < np.log((1 - rest) / rest) else (low, b)
        out.append(low * d)
    return torch.stack(out).float().bfloat16()


REST = [0.3, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6, 1e-7]


@pytest.mark.parametrize("place", ["first", "last"])
@pytest.mark.parametrize("dtype", FORMATS)
def test_a_head_whose_rows_share_a_mean(cuda, dtype, place):
    N, vocab = 32000, 31990
    L = usual(dtype, N, 256, seed=1)
    with_a_mean(L, 2)
    start = 40 if place == "first" else vocab - 700
    targets = torch.arange(start, start + 97 * len(REST), 97, dtype=torch.int32)
    x = leaning(L, targets.tolist(), vocab, REST)
    rest = check(L, x, targets, vocab)
    assert rest.min() < 1e-6 and rest.max() > 0.1


@pytest.mark.parametrize("dtype", [ans.INT8, ans.FP8_E4M3, ans.FP4_E2M1])
def test_one_row_of_a_larger_scale(cuda, dtype):
    N = vocab = 32000
    L = usual(dtype, N, 128, seed=3)
    L.scales[777] = 8 * L.scales.max()
    with_a_mean(L, 4)
    targets = torch.arange(5, 5 + 4001 * len(REST), 4001, dtype=torch.int32)
    check(L, leaning(L, targets.tolist(), vocab, REST), targets, vocab)


def beside(L, pairs, gaps):
    """Hidden states under which row t of each pair stands first and row r the given
    number of nats below it (60 in all; the other rows are far lower)."""
    out = []
    for (t, r), gap in zip(pairs, gaps):
        rows = L.w[[t, r]]
        out.append(torch.linalg.lstsq(rows, torch.tensor([60.0, 60.0 - gap]).double()[:, None], driver="gelsd").solution[:, 0])
    return torch.stack(out).float().bfloat16()


# the runner-up in the target's block of 32, in another block, in another row block
@pytest.mark.parametrize("t,r", [(3, 30), (30, 3), (3, 40), (40, 3), (100, 255), (255, 0)])
@pytest.mark.parametrize("dtype", FORMATS)
def test_one_row_beside_the_target(cuda, dtype, t, r):
    L = usual(dtype, 256, 256, seed=5)
    gaps = [6.0, 10.0, 14.0, 16.0, 18.0, 20.0, 22.0]
    x = beside(L, [(t, r)] * len(gaps), gaps)
    check(L, x, torch.full((len(gaps),), t, dtype=torch.int32), 256)


# and in an earlier and a later piece of the vocabulary
@pytest.mark.parametrize("t,r", [(5, 24000), (24000, 5), (18900, 18990), (24600, 24570)])
@pytest.mark.parametrize("dtype", FORMATS)
def test_one_row_in_another_piece(cuda, dtype, t, r):
    L = usual(dtype, 24832, 256, seed=6)
    gaps = [14.0, 16.0, 18.0, 20.0, 22.0]
    x = beside(L, [(t, r)] * len(gaps), gaps)
    check(L, x, torch.full((len(gaps),), t, dtype=torch.int32), 24800, torch.tensor([1.0, -3.0, 1e5, 1e8, 0.5]))


@pytest.mark.parametrize("dtype", [ans.INT8, ans.BF16_SPLIT])
def test_targets_beyond_the_range_of_exponentials(cuda, dtype):
    # the target 100 to 5,000 nats above or below all others (its loss or its
    # probability is then nothing at all), and a vocabulary of the target alone
    L = usual(dtype, 256, 64, seed=7)
    rng = np.random.default_rng(8)
    d = L.w[9] / (L.w[9] @ L.w[9])
    x = (d[None, :] * torch.tensor([200., 2000., 10000., -200., -2000., -10000.])[:, None]).float().bfloat16()
    t = torch.full((6,), 9, dtype=torch.int32)
    a, b, c, rest = reference(L, x, t, 256)
    loss, lse, dx = run(L, x, t, 256)
    assert rest[0] < 1e-15 and rest[5] == 1
    # a loss below fp32's normal numbers may be flushed to 0, and so may what is left of dX
    within(loss, a[0], a[1] + 2.0 ** -126, "loss")
    within(lse, *b, "lse")
    within(dx, c[0], c[1] + 2.0 ** -120, "dx")
    x = bf16(rng, 5, 64, scale=300.0)
    t = torch.tensor([0, 0, -1, 0, 0], dtype=torch.int32)
    loss, lse, dx = run(L, x, t, 1)
    z = x.double() @ L.w[0]
    within(lse, z, sum_eps(64) * (x.double().abs() @ L.w[0].abs()) + 2.0 ** -22 * z.abs(), "lse of one row")
    assert not loss.any() and not dx.any()


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
