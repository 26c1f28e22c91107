"""ans_verify of two models that agree but for a constant: p = q, and nothing is left over to draw from.

Logits are multiples of 2^-12 and the constants too, so that they add exactly: p and q are then equal as
real numbers.  Where the drafted token has none of either (or lies outside the vocabulary) it is refused, the
mass of max(0, p - q) is 0 but for what arithmetic leaves, and the next token is drawn from p."""
import numpy as np
import pytest

from rans_decode_gemm_b200 import ans

from test_gpu_verify import check, distribution

pytestmark = pytest.mark.gpu

SHIFTS = (0.0, 0.25, 1.0, 2.0, 3.5, -0.75, 17.000244140625)


def grid(rng, rows, vocab, size=1.5):
    return (np.rint(size * rng.standard_normal((rows, vocab)) * 4096) / 4096).astype(np.float32)


@pytest.mark.parametrize("vocab", [5, 500, 4099, 32000, 130001])
@pytest.mark.parametrize("t", [1.0, 0.7, 3.0])
def test_the_next_token_is_drawn_from_p(cuda, vocab, t):
    rng = np.random.default_rng(vocab)
    masked = vocab // 3
    values = np.array([0.0, 0.03, 0.25, 0.5, 0.77, 0.9, 0.999], np.float32)
    n = len(values)
    for shift in SHIFTS if vocab < 100000 else SHIFTS[1:4]:
        target = grid(rng, 1, vocab).repeat(2 * n, 0)
        target[:, masked] = -np.inf
        draft = target[:n] + np.float32(shift)
        finite = np.isfinite(draft)
        assert (draft.astype(np.float64) == target[:n].astype(np.float64) + shift)[finite].all()
        left = np.maximum(distribution(target[0], t) - distribution(draft[0], t), 0).sum()
        assert left <= 2.0 ** -40, left
        tokens = np.full(n, masked)
        check([1] * n, vocab, target, draft, tokens, np.full(n, 0.2, np.float32), values, [t] * n)


def test_a_token_outside_the_vocabulary(cuda):
    rng = np.random.default_rng(1)
    vocab, n = 32000, 5
    target = grid(rng, 2 * n, vocab)
    where = 2 * np.arange(n)
    for shift in (0.25, 2.0):
        draft = target[where] + np.float32(shift)
        check([1] * n, vocab, target, draft, np.full(n, -1), np.full(n, 0.2, np.float32),
              np.linspace(0.05, 0.95, n).astype(np.float32), None, want_status=ans.STATUS_BAD_INDEX)


@pytest.mark.parametrize("size", [3e5, 1e7])
def test_far_logits(cuda, size):
    """The same where a row's reference is past 2^30 in units of log 2 (T = 1e-5), and exponents are not near it."""
    rng = np.random.default_rng(2)
    vocab, n = 3001, 4
    target = np.rint(grid(rng, 1, vocab) * 2 + size).astype(np.float32).repeat(2 * n, 0)
    target[:, 7] = -np.inf
    for t in (1e-5, 4.0):
        draft = target[:n] + np.float32(64.0)
        assert (draft[np.isfinite(draft)] - target[:n][np.isfinite(draft)] == 64.0).all()
        check([1] * n, vocab, target, draft, np.full(n, 7), np.full(n, 0.3, np.float32),
              np.array([0.1, 0.4, 0.6, 0.95], np.float32), [t] * n)


def test_a_little_is_left(cuda):
    """One token in place of the constant: what p has more of is drawn, however small a part of p it is."""
    rng = np.random.default_rng(3)
    vocab = 5000
    values = np.array([0.0, 0.3, 0.6, 0.99], np.float32)
    target = grid(rng, 1, vocab).repeat(8, 0)
    target[:, 11] = -np.inf
    target[:, 4321] = -14.0
    draft = target[:4] + np.float32(1.0)
    draft[:, 4321] = -15.0
    p, q = distribution(target[0], 1.0), distribution(draft[0], 1.0)
    w = np.maximum(p - q, 0)
    assert 2.0 ** -40 < w.sum() < 1e-9 and w[4321] == w.sum()
    _, out = check([1] * 4, vocab, target, draft, np.full(4, 11), np.full(4, 0.5, np.float32), values, None)
    assert out[::2] == [4321] * 4
