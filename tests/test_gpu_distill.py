"""ans_distill against the definition in 64 bits.

Bounds.  A logit is an fp32 sum (zerr); the others' exponentials and their sum are right to 2^-19.
p_j = 1 / (1 + rest / e_j) takes an error d of the logits as p_j (1 - p_j) 2 d at most.  Listed
coefficients and the others' probabilities are rounded once to the operands' 16 bits
(factor_eps), the product sums in fp32.  Below f16's normal range (2^-14, where the largest of the
others is stored at 1/2 or more of what its row's scale is of the largest, here a quarter or more;
where a listed coefficient passes 2^14 it is that which the range hangs on) a value is off by
2^-25 of the unit: 4 (2^-24 of the largest other and 2^-39 of the largest coefficient)."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import ALL, BF16, bf16, status, sum_eps, usual, within, workspace

pytestmark = pytest.mark.gpu


def reference(L, x, vocab, per_t, ids, logits, teacher_lse=None, weight=None):
    x64, w = x.double(), L.w[:vocab]
    z = x64 @ w.T * per_t
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    zerr = (sum_eps(L.K) * per_t * (x64.abs() @ w.abs().T)).amax(1) + 2.0 ** -23 * z.abs().amax(1)
    has = (ids >= 0) & (ids < vocab)
    at = torch.where(has, ids, 0).long()
    v = (logits.double() * per_t).masked_fill(~has, -torch.inf)
    some = has.any(1) & (v > -torch.inf).any(1)
    norm = torch.logsumexp(v, 1) if teacher_lse is None else teacher_lse.double()
    log_t = torch.where(has, v - torch.where(some, norm, 0.0)[:, None], -torch.inf)
    t = log_t.exp()
    S = t.sum(1)
    log_p = z.gather(1, at) - lse[:, None]
    loss = torch.where(t > 0, t * (log_t - log_p), 0.0).sum(1)
    lse_b = zerr + 2.0 ** -19 + 2.0 ** -23 * lse.abs()
    loss_b = S * (2 * zerr + 2.0 ** -18) + 2.0 ** -23 * loss.abs()
    g = (torch.ones(len(x), dtype=torch.float64) if weight is None else weight.double()) * per_t
    dense_t = torch.zeros_like(p).scatter_add_(1, at, t)
    listed = torch.zeros_like(p).scatter_add_(1, at, has.double()) > 0
    coef = S[:, None] * p - dense_t
    dx = g[:, None] * (coef @ w)
    off = 2 * zerr[:, None] + 2.0 ** -19
    per = (L.factor_eps + sum_eps(vocab) + 2.0 ** -22) * coef.abs()
    per = per + S[:, None] * p * off * torch.where(listed, 1 - p, 1.0)
    # 64 bits, here and there: an exponent of |a| is rounded by 2^-53 |a|, which its power takes as
    # it is, so that S p and t, and their difference, are off by some 2^-52 (|z| + |v| + |lse| + 8)
    # of each (a certain student and teacher's S p - t of 1e-15 is that much; the reference's own
    # difference from 80-bit numbers came to 55 times the bound without this term)
    wide = z.abs().amax(1) + torch.where(has, v, 0.0).nan_to_num(0, 0, 0).abs().amax(1) + lse.abs() + 8
    per = per + 2.0 ** -51 * wide[:, None] * torch.where(listed, S[:, None] * p + dense_t, 0.0)
    most_other = torch.where(listed, 0.0, S[:, None] * p).amax(1)
    most_listed = torch.where(listed, coef.abs(), 0.0).amax(1)
    floor = 4 * (2.0 ** -24 * most_other + 2.0 ** -39 * most_listed)
    inner = g.abs()[:, None] * (per @ w.abs() + floor[:, None] * w.abs().sum(0)[None, :])
    return (loss, loss_b), (lse, lse_b), (dx, inner + BF16 * (dx.abs() + inner) + 2.0 ** -133)


def run(L, x, vocab, per_t, ids, logits, teacher_lse=None, weight=None, grad=True, ws=None, want_status=0):
    M, top = ids.shape
    size = ans.ans_distill_workspace(L.layout, M, L.kind, top, grad)
    ws = workspace(size) if ws is None else ws
    loss, lse = (torch.full((M + 1,), float("nan"), device="cuda") for _ in range(2))
    dx = torch.full((M + 1, L.K), float("nan"), dtype=torch.bfloat16, device="cuda") if grad else None
    st = status()
    dev = lambda t: None if t is None else t.cuda().contiguous()  # noqa: E731
    ans.ans_distill(dev(x), M, *L.args, vocab, per_t, top, dev(ids), dev(logits), dev(teacher_lse), loss, lse, dev(weight),
                    dx, ws, size, st)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    assert torch.isnan(loss[M:]).all() and torch.isnan(lse[M:]).all() and (dx is None or torch.isnan(dx[M:]).all())
    return loss[:M], lse[:M], (dx[:M] if grad else None)


def check(L, x, vocab, per_t, ids, logits, teacher_lse=None, weight=None, want_status=0):
    a, b, c = reference(L, x, vocab, per_t, ids, logits, teacher_lse, weight)
    loss, lse, dx = run(L, x, vocab, per_t, ids, logits, teacher_lse, weight, want_status=want_status)
    within(loss, *a, "loss")
    within(lse, *b, "lse")
    within(dx, *c, "dx")
    loss, lse, _ = run(L, x, vocab, per_t, ids, logits, teacher_lse, None, grad=False, want_status=want_status)
    within(loss, *a, "loss alone")
    within(lse, *b, "lse alone")


def teacher(rng, M, vocab, top, part=0.9):
    """Lists in no order, of different lengths, some empty."""
    ids = np.full((M, top), -1, np.int32)
    for m in range(M):
        n = min(top, vocab) if m % 3 else int(rng.integers(0, min(top, vocab) + 1))
        ids[m, rng.permutation(top)[:n]] = rng.permutation(vocab)[:n]
    logits = (2 * rng.standard_normal((M, top))).astype(np.float32)
    return torch.from_numpy(ids), torch.from_numpy(logits)


def leaning(L, rng, M, ids, size=1.0):
    """Hidden states that lean towards what is listed."""
    x = rng.standard_normal((M, L.K)) * 0.3
    w = L.w.numpy()
    for m in range(M):
        for j in range(min(3, ids.shape[1])):
            if ids[m, j] >= 0:
                row = w[int(ids[m, j])]
                x[m] += size * rng.uniform(0, 6) * row / max(np.linalg.norm(row) ** 2, 1e-9)
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("M,top", [(1, 1), (9, 20), (70, 64)])
def test_every_format(cuda, dtype, M, top):
    L = usual(dtype, 768, 128, seed=dtype)
    rng = np.random.default_rng([dtype, M])
    for vocab in (768, 700, 513):
        ids, logits = teacher(rng, M, vocab, top)
        x = leaning(L, rng, M, ids)
        weight = torch.from_numpy(rng.uniform(0, 2, M).astype(np.float32))
        check(L, x, vocab, 1.0, ids, logits, None, weight)


@pytest.mark.parametrize("per_t", [0.25, 1.0, 3.0])
def test_temperatures_and_mass_elsewhere(cuda, per_t):
    rng = np.random.default_rng(5)
    for dtype in (ans.BF16_SPLIT, ans.FP8_E4M3):
        L = usual(dtype, 1024, 192, seed=2)
        ids, logits = teacher(rng, 40, 1000, 16)
        x = leaning(L, rng, 40, ids)
        held = torch.from_numpy(rng.uniform(0.3, 0.99, 40))
        lse = torch.logsumexp((logits.double() * per_t).masked_fill(ids < 0, -torch.inf), 1) - held.log()
        lse = torch.where(torch.isfinite(lse), lse, 0.0).float()
        check(L, x, 1000, per_t, ids, logits, lse)
        check(L, x, 1000, per_t, ids, logits, None)


@pytest.mark.parametrize("top", [1, 31, 33, 127, 129, 256])
def test_lengths_of_lists(cuda, top):
    L = usual(ans.INT8, 512, 64, seed=4)
    rng = np.random.default_rng(top)
    ids, logits = teacher(rng, 33, 500, top)
    check(L, leaning(L, rng, 33, ids), 500, 1.0, ids, logits)


def test_all_of_a_vocabulary_is_listed(cuda):
    """No others at all; and a vocabulary of one row."""
    rng = np.random.default_rng(6)
    for dtype in (ans.BF16_SPLIT, ans.INT8):
        L = usual(dtype, 256, 64, seed=5)
        for vocab in (200, 33, 1):
            ids = torch.from_numpy(np.stack([rng.permutation(vocab) for _ in range(12)]).astype(np.int32))
            logits = torch.from_numpy(rng.standard_normal((12, vocab)).astype(np.float32))
            check(L, leaning(L, rng, 12, ids), vocab, 1.0, ids, logits)


def test_a_row_listed_twice(cuda):
    rng = np.random.default_rng(7)
    L = usual(ans.BF16_SPLIT, 384, 64, seed=6)
    ids, logits = teacher(rng, 20, 380, 12)
    ids[:, 5] = ids[:, 2]
    ids[3] = 77
    ids[4, ::2] = 379
    check(L, leaning(L, rng, 20, ids), 380, 1.0, ids, logits)


def test_entries_of_no_mass_and_far_logits(cuda):
    rng = np.random.default_rng(8)
    L = usual(ans.FP8_E4M3, 384, 64, seed=7)
    ids, logits = teacher(rng, 24, 384, 10)
    logits[:, 3] = -torch.inf
    logits[1] = -torch.inf
    ids[2, 0] = 5
    logits[2, 1:] = -1e30
    logits[5] += 3e4
    logits[6] = torch.finfo(torch.float32).min
    ids[6, 0], logits[6, 0] = 9, 0.0
    rest = torch.full((24,), 1.0)
    x = leaning(L, rng, 24, ids)
    ids[1] = -1
    check(L, x, 384, 1.0, ids, logits)
    logits[5] -= 3e4
    ids[1, 4] = 7
    logits[1] = -torch.inf
    check(L, x, 384, 1.0, ids, logits, rest)
    # nothing above -infinity: nothing is listed, with the teacher's lse and without
    for lse in (rest, None):
        loss, _, dx = run(L, x, 384, 1.0, ids, logits, lse)
        assert loss[1] == 0 and not dx[1].any()


@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8, ans.FP4_PAIRS])
@pytest.mark.parametrize("size", [1.0, 4.0, 8.0])
def test_a_student_that_has_learnt_its_teacher(cuda, dtype, size):
    """Certain students and teachers that all but agree: S p - t is a difference of like numbers."""
    rng = np.random.default_rng([dtype, int(size)])
    L = usual(dtype, 640, 128, seed=8)
    M, top, vocab = 40, 8, 600
    ids = torch.from_numpy(np.stack([rng.permutation(vocab)[:top] for _ in range(M)]).astype(np.int32))
    x = leaning(L, rng, M, ids, size)
    z = x.double() @ L.w[:vocab].T
    for off in (0.0, 1e-4, 1e-2):
        listed = z.gather(1, ids.long()) + off * torch.from_numpy(rng.standard_normal((M, top)))
        lse = torch.logsumexp(z, 1)
        check(L, x, vocab, 1.0, ids, listed.float(), lse.float())
        check(L, x, vocab, 1.0, ids, listed.float())


def test_pieces_and_chunks(cuda):
    """A first piece that serves the others' references, tokens in several chunks, and many tiles."""
    rng = np.random.default_rng(9)
    L = usual(ans.BF16_SPLIT, 16384, 64, seed=9)
    ids, logits = teacher(rng, 1400, 16300, 6)
    check(L, leaning(L, rng, 1400, ids), 16300, 1.0, ids, logits)
    L = usual(ans.INT8, 4096, 32, seed=9)
    ids, logits = teacher(rng, 4500, 4096, 4)
    check(L, leaning(L, rng, 4500, ids), 4096, 1.0, ids, logits)


def test_workspace_is_for_any_vocabulary(cuda):
    """A vocabulary far below the layer's rows, in a workspace that is used again."""
    rng = np.random.default_rng(10)
    L = usual(ans.INT4_PAIRS, 2048, 128, seed=10)
    M, top = 50, 5
    ws = workspace(ans.ans_distill_workspace(L.layout, M, L.kind, top, True))
    for vocab in (2048, 3, 130, 1025):
        ids, logits = teacher(rng, M, vocab, top)
        x = leaning(L, rng, M, ids)
        a, b, c = reference(L, x, vocab, 1.0, ids, logits)
        loss, lse, dx = run(L, x, vocab, 1.0, ids, logits, ws=ws)
        within(loss, *a, "loss")
        within(lse, *b, "lse")
        within(dx, *c, "dx")


def test_indexes_outside(cuda):
    rng = np.random.default_rng(11)
    L = usual(ans.BF16_SPLIT, 256, 64, seed=11)
    ids, logits = teacher(rng, 9, 250, 6)
    x = leaning(L, rng, 9, ids)
    ids[2, 3] = 250
    ids[7, 0] = 2 ** 31 - 1
    ids[8, 1] = -2 ** 31
    check(L, x, 250, 1.0, ids, logits, want_status=ans.STATUS_BAD_INDEX)


def test_not_finite_stays_with_its_token(cuda):
    rng = np.random.default_rng(12)
    for dtype in (ans.BF16_SPLIT, ans.INT8):
        L = usual(dtype, 512, 64, seed=12)
        M = 40
        ids, logits = teacher(rng, M, 512, 6)
        ids[[3, 4], 0] = 7
        ids[5] = -1
        x = leaning(L, rng, M, ids)
        loss, lse, dx = run(L, x, 512, 1.0, ids, logits)
        x2 = x.clone()
        x2[3, 1], x2[4, 2], x2[5, 3] = float("nan"), float("inf"), float("nan")
        loss2, lse2, dx2 = run(L, x2, 512, 1.0, ids, logits)
        rest = [m for m in range(M) if m not in (3, 4, 5)]
        for a, b in ((loss, loss2), (lse, lse2), (dx, dx2)):
            assert torch.equal(a[rest], b[rest])
        assert torch.isnan(dx2[[3, 4]]).all() and torch.isnan(lse2[[3, 5]]).all()
        assert (dx2[5] == 0).all() and loss2[5] == 0
        # rows of padding behind the vocabulary may hold anything
        if dtype == ans.BF16_SPLIT:
            L.codes[500:] = 0x7F80
            L.layer = ans.CompressedLayer.from_weights(L.codes.reshape(-1), L.layout)
            L.tiles = L.layer.tiles
            ids = torch.where(ids < 500, ids, -1)
            check(L, x, 500, 1.0, ids, logits)


@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8])
@pytest.mark.parametrize("M", [300, 1000])
def test_wide_tiles_of_long_sums(cuda, dtype, M):
    """Tokens in tiles of 128 and 256, whose sums of K = 4160 come in several parts where there is no gradient."""
    rng = np.random.default_rng(22)
    L = usual(dtype, 4096, 4160, seed=22)
    ids, logits = teacher(rng, M, 4090, 5)
    x = leaning(L, rng, M, ids)
    check(L, x, 4090, 1.0, ids, logits)
    # the same bits again
    a, b = run(L, x, 4090, 1.0, ids, logits, grad=False), run(L, x, 4090, 1.0, ids, logits, grad=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("M", [3, 300])
def test_nothing_listed_beside_infinite_weights(cuda, M):
    """A token that lists nothing has a zero gradient whatever the rows of W hold."""
    rng = np.random.default_rng(21)
    L = usual(ans.BF16_SPLIT, 256, 64, seed=21)
    L.codes[17, 5] = 0x7F80
    L.layer = ans.CompressedLayer.from_weights(L.codes.reshape(-1), L.layout)
    L.tiles = L.layer.tiles
    ids, logits = teacher(rng, M, 256, 4)
    x = leaning(usual(ans.BF16_SPLIT, 256, 64, seed=21), rng, M, ids)
    ids[0, 0], ids[1] = 7, -1
    loss, lse, dx = run(L, x, 256, 1.0, ids, logits)
    assert loss[1] == 0 and (dx[1] == 0).all()
    assert torch.isnan(dx[0, 5])


def test_same_bits_and_capture(cuda):
    rng = np.random.default_rng(13)
    L = usual(ans.FP8_E4M3, 1024, 128, seed=13)
    M, top, vocab = 60, 12, 1000
    st = status()
    size = ans.ans_distill_workspace(L.layout, M, L.kind, top, True)
    ws = workspace(size)
    sets = []
    for _ in range(3):
        ids, logits = teacher(rng, M, vocab, top)
        sets.append((leaning(L, rng, M, ids), ids, logits))
    buf = [t.cuda() for t in sets[0]]
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dx = torch.empty(M, L.K, dtype=torch.bfloat16, device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()

    def call():
        ans.ans_distill(buf[0], M, *L.args, vocab, 0.5, top, buf[1], buf[2], None, loss, lse, None, dx, ws, size, st)
    with torch.cuda.stream(side):
        for _ in range(3):
            call()
        graph.capture_begin()
        call()
        graph.capture_end()
    for x, ids, logits in sets:
        for a, b in zip(buf, (x, ids, logits)):
            a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = run(L, x, vocab, 0.5, ids, logits)
        assert all(torch.equal(a, b) for a, b in zip((loss, lse, dx), want))
        # in another order, the same lists are the same
        order = torch.from_numpy(rng.permutation(top))
        again = run(L, x, vocab, 0.5, ids[:, order], logits[:, order])
        assert torch.equal(want[1], again[1])
    assert int(st.item()) == 0


def test_gradient_against_differences(cuda):
    rng = np.random.default_rng(14)
    L = usual(ans.BF16_SPLIT, 512, 64, seed=14)
    ids, logits = teacher(rng, 20, 500, 8)
    x = leaning(L, rng, 20, ids)
    _, _, dx = run(L, x, 500, 0.7, ids, logits)
    v = torch.from_numpy(rng.standard_normal(x.shape))
    has = ids >= 0
    t = torch.softmax((logits.double() * 0.7).masked_fill(~has, -torch.inf), 1).nan_to_num(0.0)

    def loss(y):
        log_p = torch.log_softmax(y @ L.w[:500].T * 0.7, 1).gather(1, ids.clamp_min(0).long())
        return -(t * torch.where(has, log_p, 0.0)).sum()
    step = 1e-5
    slope = ((loss(x.double() + step * v) - loss(x.double() - step * v)) / (2 * step)).item()
    dx = dx.cpu().double()
    assert abs((dx * v).sum().item() - slope) <= 4 * BF16 * (dx.abs() * v.abs()).sum().item()


def test_the_cross_entropy_of_one_listed_row(cuda):
    """A teacher that lists one row is a target: loss and gradient are ans_xent's."""
    rng = np.random.default_rng(15)
    L = usual(ans.INT8, 512, 128, seed=15)
    M = 50
    targets = torch.from_numpy(rng.integers(-1, 500, M).astype(np.int32))
    x = leaning(L, rng, M, targets[:, None])
    loss, lse, dx = run(L, x, 500, 1.0, targets[:, None].contiguous(), torch.zeros(M, 1))
    size = ans.ans_xent_workspace(L.layout, M, L.kind, True)
    xl, xs = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    xd, st = torch.empty(M, L.K, dtype=torch.bfloat16, device="cuda"), status()
    ans.ans_xent(x.cuda(), M, *L.args, 500, targets.cuda(), xl, xs, None, xd, workspace(size), size, st)
    torch.cuda.synchronize()
    # the same fp32 logits: only sums of exponentials and roundings differ
    assert (lse - xs).abs().max() <= 2.0 ** -18 + 2.0 ** -22 * xs.abs().max()
    assert (loss - xl).abs().max() <= 2.0 ** -17 + 2.0 ** -21 * xl.abs().max() + 2.0 ** -22 * xs.abs().max()
    a, b = dx.double(), xd.double()
    assert ((a - b).norm(dim=1) <= 2 * BF16 * b.norm(dim=1) + 1e-30).all()
