"""ans_xent against the definition in 64 bits: one piece of the vocabulary and
several, one chunk of tokens and several, padding, and values at the borders."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import ALL, BF16, Layer, bf16, status, sum_eps, usual, within, workspace

pytestmark = pytest.mark.gpu


def reference(L, x, targets, vocab, weight=None):
    """(loss, lse, dx) in 64 bits with the bounds of right results."""
    x64, w = x.double(), L.w[:vocab]
    z = x64 @ w.T
    lse = torch.logsumexp(z, 1)
    has = targets >= 0
    at = targets.clamp_min(0).long()
    zt = z.gather(1, at[:, None])[:, 0]
    loss = torch.where(has, lse - zt, 0.0)
    # a logit is an fp32 sum; the exponential's and the sum's rounding come to 2^-19 of the sum at most
    zerr = (sum_eps(L.K) * (x64.abs() @ w.abs().T)).amax(1) + 2.0 ** -23 * z.abs().amax(1)
    lse_b = zerr + 2.0 ** -19 + 2.0 ** -23 * lse.abs()
    loss_b = torch.where(has, 2 * zerr + 2.0 ** -19 + 2.0 ** -23 * loss, 0.0)
    g = torch.ones(len(x), dtype=torch.float64) if weight is None else weight.double()
    g = torch.where(has, g, 0.0)
    p = torch.exp(z - lse[:, None])
    others = p.scatter(1, at[:, None], 0.0)
    rest = others.sum(1)
    dx = g[:, None] * (others @ w - rest[:, None] * w[at])
    mass = others @ w.abs() + rest[:, None] * w[at].abs()
    inner = g.abs()[:, None] * (L.factor_eps + sum_eps(L.N) + 4 * zerr[:, None] + 2.0 ** -18) * mass
    # what f16 drops of the smallest terms: 2^-38 of the largest, V times
    inner = inner + g.abs()[:, None] * 2.0 ** -38 * vocab * w.abs().amax(0)[None, :]
    return (loss, loss_b), (lse, lse_b), (dx, inner + BF16 * (dx.abs() + inner))


def run(L, x, targets, vocab, weight=None, grad=True, ws=None):
    M = x.shape[0]
    size = ans.ans_xent_workspace(L.layout, M, L.kind, grad)
    ws = workspace(size) if ws is None else ws
    loss, lse = (torch.full((M,), float("nan"), device="cuda") for _ in range(2))
    dx = torch.full((M, L.K), float("nan"), dtype=torch.bfloat16, device="cuda") if grad else None
    st = status()
    ans.ans_xent(x.cuda(), M, *L.args, vocab, targets.cuda(), loss, lse, None if weight is None else weight.cuda(), dx,
                 ws, size, st)
    torch.cuda.synchronize()
    return loss, lse, dx, int(st.item())


def check(L, x, targets, vocab, weight=None, grad=True):
    loss, lse, dx, st = run(L, x, targets, vocab, weight, grad)
    assert st == 0
    a, b, c = reference(L, x, targets, vocab, weight)
    within(loss, *a, "loss")
    within(lse, *b, "lse")
    if grad:
        within(dx, *c, "dx")


def some_targets(rng, M, vocab):
    t = torch.from_numpy(rng.integers(0, vocab, M).astype(np.int32))
    t[torch.from_numpy(rng.random(M) < 0.1)] = -100
    return t


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("M", [1, 16, 33, 300])
@pytest.mark.parametrize("dtype", ALL)
def test_every_format(cuda, dtype, M, grad):
    L = usual(dtype, 512, 192, seed=M)
    rng = np.random.default_rng([dtype, M])
    x = bf16(rng, M, 192)
    weight = torch.from_numpy(rng.standard_normal(M).astype(np.float32))
    check(L, x, some_targets(rng, M, 500), 500, weight, grad)


# vocab of one, whole tiles, part of a tile, pieces that end in padding; several
# pieces, the last short; several chunks of tokens
@pytest.mark.parametrize("N,K,vocab,M", [(128, 16, 1, 3), (128, 16, 128, 40), (384, 80, 257, 65), (8192, 16, 8192, 20),
                                         (8320, 32, 8300, 50), (16384, 16, 8192, 9), (16512, 16, 16385, 260),
                                         (24704, 48, 24577, 129), (8320, 16, 8320, 4200), (512, 1040, 500, 700)])
@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8])
def test_pieces_and_chunks(cuda, dtype, N, K, vocab, M):
    L = usual(dtype, N, K, seed=N)
    rng = np.random.default_rng([N, M])
    check(L, bf16(rng, M, K), some_targets(rng, M, vocab), vocab)


@pytest.mark.parametrize("state_bits", [32, 64])
@pytest.mark.parametrize("dtype,kind", [(ans.BF16_SPLIT, ans.SCALE_ROW_BF16), (ans.INT4, ans.SCALE_ROW_F32),
                                        (ans.FP4_PAIRS, ans.SCALE_NONE), (ans.FP8_E4M3, ans.SCALE_ROW_BF16)])
def test_scale_kinds(cuda, dtype, kind, state_bits):
    L = Layer(dtype, 256, 128, 128, 32, kind, 0, seed=5, state_bits=state_bits)
    rng = np.random.default_rng(9)
    check(L, bf16(rng, 50, 128, scale=0.1), some_targets(rng, 50, 250), 250)


@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.FP8_E4M3])
def test_logits_far_apart(cuda, dtype):
    # tokens that are all but certain of their target, or of another, and rows
    # whose largest logit comes in the last piece, or in the first
    L = usual(dtype, 8448, 64, seed=3)
    rng = np.random.default_rng(4)
    targets = torch.tensor([5, 8400, 17, 8441, 100, 8300, 3, 8447], dtype=torch.int32)
    lean = torch.tensor([8400, 5, 17, 8441, 100, 8300, 8440, 2])
    rows = L.w[lean]
    x = (rows / rows.norm(dim=1, keepdim=True) * torch.tensor([30., 30., 30., 60., 200., 500., 400., 900.])[:, None]
         + torch.from_numpy(rng.standard_normal((8, 64))) * 0.1)
    check(L, x.float().bfloat16(), targets, 8442 + 6)


def test_padding_of_the_vocabulary_counts_for_nothing(cuda):
    # the rows from vocab on hold values that would win every softmax
    L = usual(ans.BF16_SPLIT, 384, 64, seed=8)
    codes = L.codes.copy()
    codes[300:] = 0x4380                       # 256
    layer = ans.CompressedLayer.from_weights(codes.reshape(-1), L.layout)
    L.w[300:] = 256.0
    L.layer, L.tiles = layer, layer.tiles
    rng = np.random.default_rng(2)
    check(L, bf16(rng, 30, 64).abs(), some_targets(rng, 30, 300), 300)


@pytest.mark.parametrize("code", [0x7F80, 0x7FC0])
@pytest.mark.parametrize("N,vocab", [(384, 300), (16512, 8200), (16512, 16400)])
def test_padding_may_hold_infinities_and_nan(cuda, N, vocab, code):
    L = usual(ans.BF16_SPLIT, N, 64, seed=8)
    codes = L.codes.copy()
    codes[vocab:] = code
    L.layer = ans.CompressedLayer.from_weights(codes.reshape(-1), L.layout)
    L.tiles = L.layer.tiles
    rng = np.random.default_rng(2)
    check(L, bf16(rng, 30, 64), some_targets(rng, 30, vocab), vocab)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30, 0.0])
@pytest.mark.parametrize("N,vocab", [(384, 299), (8320, 8200)])
@pytest.mark.parametrize("dtype,kind", [(ans.INT8, ans.SCALE_ROW_F32), (ans.FP8_E4M3, ans.SCALE_ROW_BF16),
                                        (ans.BF16_SPLIT, ans.SCALE_ROW_F32), (ans.INT4, ans.SCALE_GROUP_BF16)])
def test_padding_may_have_any_scale(cuda, dtype, kind, N, vocab, value):
    L = Layer(dtype, N, 64, 128, 64, kind, 64 if kind == ans.SCALE_GROUP_BF16 else 0, seed=12)
    L.scales[vocab:] = value
    L.w[vocab:] = 0.0
    rng = np.random.default_rng(2)
    check(L, bf16(rng, 30, 64, scale=0.1), some_targets(rng, 30, vocab), vocab)


def test_targets_out_of_range(cuda):
    L = usual(ans.INT8, 256, 64, seed=8)
    rng = np.random.default_rng(2)
    x = bf16(rng, 5, 64)
    targets = torch.tensor([3, 250, -1, 2 ** 31 - 1, 249], dtype=torch.int32)
    loss, lse, dx, st = run(L, x, targets, 250)
    assert st == ans.STATUS_BAD_INDEX
    a, b, c = reference(L, x, torch.where(targets >= 250, -1, targets), 250)
    within(loss, *a)
    within(lse, *b)
    within(dx, *c)
    assert not dx[1].any() and not dx[2].any() and not dx[3].any()


def test_infinities_and_nan_stay_in_their_rows(cuda):
    L = usual(ans.BF16_SPLIT, 256, 64, seed=8)
    rng = np.random.default_rng(2)
    x = bf16(rng, 6, 64)
    targets = torch.tensor([3, 4, 5, -1, 7, 8], dtype=torch.int32)
    x[1, 0], x[3, 2], x[4, 1] = float("nan"), float("nan"), float("inf")
    loss, lse, dx, st = run(L, x, targets, 256)
    good = [0, 2, 5]
    a, b, c = reference(L, x[good], targets[good], 256)
    within(loss[good], *a)
    within(lse[good], *b)
    within(dx[good], *c)
    assert torch.isnan(loss[1]) and torch.isnan(dx[1]).all()
    assert loss[3] == 0 and not dx[3].any() and torch.isnan(lse[3])     # no target: nothing to lose
    assert torch.isinf(lse[4]) or torch.isnan(lse[4])


def test_gradient_against_differences(cuda):
    # d(sum g loss) along a direction, by central differences of the 64-bit loss
    # and against the operator's dX
    L = usual(ans.BF16_SPLIT, 512, 64, seed=1)
    rng = np.random.default_rng(6)
    x, targets = bf16(rng, 4, 64), torch.tensor([0, 511, 77, 300], dtype=torch.int32)
    weight = torch.tensor([1.0, -2.0, 0.5, 3.0])
    _, _, dx, st = run(L, x, targets, 512, weight)
    assert st == 0
    v = torch.from_numpy(rng.standard_normal((4, 64)))

    def total(h):
        z = (x.double() + h * v) @ L.w.T
        return (weight.double() * (torch.logsumexp(z, 1) - z.gather(1, targets.long()[:, None])[:, 0])).sum()
    h = 1e-4
    slope = ((total(h) - total(-h)) / (2 * h)).item()
    _, _, (want, bound) = reference(L, x, targets, 512, weight)
    assert abs((dx.cpu().double() * v).sum().item() - slope) <= (bound * v.abs()).sum().item() + 1e-6 * abs(slope) + 1e-6


def test_loss_alone_is_the_loss_with_gradient(cuda):
    for M in (7, 100):
        L = usual(ans.FP4_PAIRS, 8448, 64, seed=1)
        rng = np.random.default_rng(6)
        x, t = bf16(rng, M, 64), some_targets(rng, M, 8448)
        a = run(L, x, t, 8448, grad=True)
        b = run(L, x, t, 8448, grad=False)
        want = reference(L, x, t, 8448)
        for k in range(2):
            assert (a[k] - b[k]).abs().max().item() <= 2 * want[k][1].max().item()


def test_workspace_streams_and_graphs(cuda):
    L = usual(ans.INT4_PAIRS, 8448, 128, seed=1)
    rng = np.random.default_rng(6)
    M = 90
    runs = []
    for _ in range(2):
        x, t = bf16(rng, M, 128), some_targets(rng, M, 8400)
        want = run(L, x, t, 8400)
        ws = torch.zeros(ans.ans_xent_workspace(L.layout, M, L.kind, True) + 256, dtype=torch.uint8, device="cuda")
        ws[-256:] = 0x5A
        out = [torch.zeros_like(v) for v in want[:3]]
        runs.append((x.cuda(), t.cuda(), ws, out, want[:3], status(), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def call(r):
        x, t, ws, (loss, lse, dx), _, st, stream = r
        ans.ans_xent(x, M, *L.args, 8400, t, loss, lse, None, dx, ws, ws.numel() - 256, st, stream)

    def same():
        torch.cuda.synchronize()
        for r in runs:
            assert int(r[5].item()) == 0 and (r[2][-256:] == 0x5A).all()
            for got, want in zip(r[3], r[4]):
                assert torch.equal(got, want)
                got.zero_()
        torch.cuda.synchronize()
    for _ in range(2):
        for r in runs:
            call(r)
    same()
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=r[6]):
            call(r)
        graphs.append((g, r[6]))
    for _ in range(2):
        for g, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    same()


def test_a_training_step_of_adapters_under_a_compressed_head(cuda):
    # the operators as they are used together: hidden = x + lora(x), loss on the
    # head, its gradient back through the head and the projection
    proj, head = usual(ans.INT8, 256, 256, seed=1), usual(ans.BF16_SPLIT, 1024, 256, seed=2)
    rng = np.random.default_rng(3)
    M, n, rank = 75, 3, 16
    a, b = bf16(rng, n, rank, 256, scale=256 ** -0.5), bf16(rng, n, 256, rank, scale=0.05)
    A = ans.LoraAdapters(a.cuda(), b.cuda())
    x, ids = bf16(rng, M, 256), torch.from_numpy(rng.integers(-1, n, M).astype(np.int32))
    t = some_targets(rng, M, 1000)
    weight = (t >= 0).float() / (t >= 0).sum()
    st = status()
    y = torch.empty(M, 256, device="cuda")
    ws = workspace(ans.ans_gemm_lora_workspace(proj.layout, M, proj.kind, A.lora))
    ans.ans_gemm_lora(x.cuda(), M, *proj.args, A.lora, ids.cuda(), y, ws, ws.numel(), st)
    hidden = y.bfloat16()
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dh = torch.empty(M, 256, dtype=torch.bfloat16, device="cuda")
    ws = workspace(ans.ans_xent_workspace(head.layout, M, head.kind, True))
    ans.ans_xent(hidden, M, *head.args, 1000, t.cuda(), loss, lse, weight.cuda(), dh, ws, ws.numel(), st)
    dx = torch.empty(M, 256, dtype=torch.bfloat16, device="cuda")
    da, db = torch.empty(a.shape, device="cuda"), torch.empty(b.shape, device="cuda")
    ws = workspace(ans.ans_gemm_lora_grad_workspace(proj.layout, M, proj.kind, A.lora))
    ans.ans_gemm_lora_grad(x.cuda(), dh, M, *proj.args, A.lora, ids.cuda(), dx, da, db, ws, ws.numel(), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # the whole step by automatic differentiation in 64 bits
    x64, a64, b64 = (v.double().requires_grad_() for v in (x, a, b))
    mine = (torch.arange(n)[None, :] == ids[:, None]).double()
    low = torch.einsum("mk,nrk,mn->mnr", x64, a64, mine)
    out = x64 @ proj.w.T + torch.einsum("mnr,ncr->mc", low, b64)
    z = out @ head.w[:1000].T
    total = (weight.double() * (torch.logsumexp(z, 1) - z.gather(1, t.clamp_min(0).long()[:, None])[:, 0])).sum()
    total.backward()
    assert abs((weight.double() * loss.cpu().double()).sum().item() - total.item()) <= 0.02 * abs(total.item())
    # bf16 activations between the operators (2^-8 each, twice) and bf16 dX: 2^-6 of each gradient's norm
    for got, want in ((dx, x64.grad), (da, a64.grad), (db, b64.grad)):
        off = (got.cpu().double() - want).norm() / want.norm()
        assert off <= 2.0 ** -6, off.item()
