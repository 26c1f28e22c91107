"""ans_verify against the definition, sequence by sequence in 64 bits.

What comes out are whole numbers and have to be equal.  The kernel's probabilities are off by
some 2^-42 of their value, so a random number decides otherwise than here with a chance of about
2^-40 a border; inputs that sit on a border on purpose do so in numbers that both hold exactly."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

pytestmark = pytest.mark.gpu


def distribution(logits, t):
    """p of one row, or None where it has none."""
    z = logits.astype(np.float64)
    if np.isnan(z).any() or (z == np.inf).any() or not (z > -np.inf).any():
        return None
    if not t > 0:
        p = np.zeros(len(z))
        p[int(np.argmax(z))] = 1.0
        return p
    t = np.float64(min(np.float32(t), np.float32(1e30)))
    top = z.max()
    e = np.exp((z - top) / t)
    return e / e.sum()


def sequence(target, draft, tokens, u, v, t, vocab):
    """(accepted, tokens out) of one sequence: target [n + 1, vocab], draft [n, vocab] or None."""
    out = []
    for i, x in enumerate(tokens):
        p = distribution(target[i], t)
        inside = 0 <= x < vocab
        if draft is None:
            q = np.zeros(vocab)
            if inside:
                q[x] = 1.0
        else:
            q = distribution(draft[i], t) if t > 0 else np.zeros(vocab)
        if p is None or q is None:
            return i, out + [-1] * (len(tokens) - i + 1)
        if t > 0:
            keep = inside and np.float64(u[i]) * q[x] < p[x]
        else:
            keep = inside and p[x] > 0
        if keep:
            out.append(int(x))
            continue
        w = np.maximum(p - q, 0.0) if t > 0 else p
        if w.sum() <= 2.0 ** -40:
            w = p
        return i, out + [draw(w, v)] + [-1] * (len(tokens) - i)
    p = distribution(target[len(tokens)], t)
    return len(tokens), out + [-1 if p is None else draw(p, v)]


def draw(w, v):
    run = np.cumsum(w)
    past = np.nonzero((run > np.float64(v) * run[-1]) & (w > 0))[0]
    return int(past[0]) if len(past) else int(np.nonzero(w > 0)[0][-1])


def check(counts, vocab, target, draft, tokens, u, v, temperature, t_stride=None, d_stride=None, shift=0, want_status=0):
    """Runs a batch (rows on strides and `shift` logits off a 16-byte boundary) and compares."""
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n, b = int(starts[-1]), len(counts)

    def rows(a, stride):
        stride = stride or vocab
        flat = torch.full((len(a) * stride + shift + 8,), float("nan"), device="cuda")
        view = flat[shift:shift + len(a) * stride].view(len(a), stride)
        view[:, :vocab] = torch.from_numpy(np.ascontiguousarray(a)).cuda()
        return view, stride
    dt, ts = rows(target, t_stride)
    dd, ds = rows(draft, d_stride) if draft is not None and n else (None, vocab)
    dev = lambda a, kind: torch.from_numpy(np.asarray(a, kind)).cuda()  # noqa: E731
    accepted = torch.full((b + 2,), -7, dtype=torch.int32, device="cuda")
    out = torch.full((n + b + 2,), -7, dtype=torch.int32, device="cuda")
    size = ans.ans_verify_workspace(b, n, vocab)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ans.ans_verify(dt, ts, dd, ds, b, n, vocab, dev(starts, np.int32), dev(tokens, np.int32), dev(u, np.float32),
                   dev(v, np.float32), None if temperature is None else dev(temperature, np.float32), accepted, out, ws,
                   size, st)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    want_a, want_o = [], []
    for k in range(b):
        s0, s1 = starts[k], starts[k + 1]
        a, o = sequence(target[s0 + k:s1 + k + 1], None if draft is None else draft[s0:s1], tokens[s0:s1], u[s0:s1],
                        v[k], 1.0 if temperature is None else temperature[k], vocab)
        want_a.append(a)
        want_o += o
    assert accepted.cpu().tolist() == want_a + [-7, -7]
    assert out.cpu().tolist() == want_o + [-7, -7]
    return want_a, want_o


def batch(rng, counts, vocab, agree=0.7, peaks=4):
    """Logits of two models that mostly agree, drafts drawn from the second's."""
    n, b = int(np.sum(counts)), len(counts)
    target = (1.5 * rng.standard_normal((n + b, vocab))).astype(np.float32)
    for r in target:
        r[rng.integers(0, vocab, peaks)] += rng.uniform(5, 12)
    where = np.arange(n) + np.repeat(np.arange(b), counts)
    draft = (target[where] + agree * rng.standard_normal((n, vocab))).astype(np.float32)
    p = np.exp(draft.astype(np.float64) - draft.max(axis=1, keepdims=True, initial=-1e9))
    tokens = np.array([rng.choice(vocab, p=row / row.sum()) for row in p], np.int64)
    return target, draft, tokens, rng.random(n, np.float32), rng.random(b, np.float32)


@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 257, 1000, 4099, 32000, 65499])
@pytest.mark.parametrize("looked_up", [False, True])
def test_batches(cuda, vocab, looked_up):
    rng = np.random.default_rng([vocab, looked_up])
    counts = [4, 0, 1, 7, 3, 0, 9]
    target, draft, tokens, u, v = batch(rng, counts, vocab)
    temperature = [1.0, 0.7, 0.0, 1.5, 0.0, 0.3, 0.9]
    check(counts, vocab, target, None if looked_up else draft, tokens, u, v, temperature)
    check(counts, vocab, target, None if looked_up else draft, tokens, u, v, None)


@pytest.mark.parametrize("shift,extra", [(1, 0), (2, 3), (3, 5), (0, 64)])
def test_strides_and_alignment(cuda, shift, extra):
    rng = np.random.default_rng(shift)
    counts = [3, 5]
    a = batch(rng, counts, 5003)
    check(counts, 5003, *a, [0.8, 0.0], t_stride=5003 + extra, d_stride=5003 + 2 * extra, shift=shift)


@pytest.mark.parametrize("counts", [[0], [1], [40], [0, 0, 0], [2] * 70, [0, 300, 0]])
def test_counts(cuda, counts):
    rng = np.random.default_rng(len(counts))
    a = batch(rng, counts, 700, agree=0.1)
    check(counts, 700, *a, None)


def test_one_row_of_a_large_vocabulary(cuda):
    rng = np.random.default_rng(3)
    for vocab in (131072, 262147):
        a = batch(rng, [2], vocab)
        check([2], vocab, *a, [1.0])


def test_the_last_and_the_first_token(cuda):
    """v = 0 takes the first token of any weight, the largest v below 1 the last that has some."""
    rng = np.random.default_rng(4)
    vocab = 2000
    for v, token in ((0.0, 5), (np.float32(1 - 2.0 ** -24), 1990)):
        target = rng.standard_normal((1, vocab)).astype(np.float32)
        target[:, :5] = -np.inf
        target[:, 1991:] = -np.inf
        target[0, token] = 3.0
        _, out = check([0], vocab, target, None, np.zeros(0, np.int64), np.zeros(0, np.float32), np.array([v], np.float32), None)
        assert out[0] == token


def test_masks_and_lowest_values(cuda):
    rng = np.random.default_rng(5)
    counts, vocab = [3, 3, 3], 3001
    target, draft, tokens, u, v = batch(rng, counts, vocab)
    lowest = np.finfo(np.float32).min
    keep = np.zeros(vocab, bool)
    keep[rng.integers(0, vocab, 9)] = True
    keep[tokens] = True
    target[:, ~keep] = -np.inf
    draft[:, ~keep] = -np.inf
    check(counts, vocab, target, draft, tokens, u, v, [1.0, 0.5, 0.0])
    target[:, ~keep] = lowest
    draft[:, ~keep] = lowest
    check(counts, vocab, target, draft, tokens, u, v, [1.0, 0.5, 0.0])
    # a drafted token that the target rules out
    target[:, tokens] = -np.inf
    check(counts, vocab, target, draft, tokens, u, v, [1.0, 0.5, 0.0])


def test_logits_of_any_size(cuda):
    """A reference moves within a part, within a thread and between parts; far logits count as 0."""
    rng = np.random.default_rng(6)
    counts, vocab = [2, 2], 40000
    for size in (1e3, 1e6, 1e30):
        target, draft, tokens, u, v = batch(rng, counts, vocab)
        target *= np.float32(size)
        draft *= np.float32(size)
        check(counts, vocab, target, draft, tokens, u, v, [1.0, 1e-3])
    target = np.linspace(-3e4, 3e4, vocab, dtype=np.float32)[None, :].repeat(4, 0) + np.zeros((6, 1), np.float32)[:4]
    target = np.concatenate([target, target[:2]])
    draft = target[:4].copy()
    tokens = np.array([vocab - 1, vocab - 2, vocab - 3, vocab - 1])
    u = np.array([0.5, 0.9, 0.3, 0.99], np.float32)
    check(counts, vocab, target, draft, tokens, u, np.array([0.3, 0.6], np.float32), [1.0, 30.0])
    check(counts, vocab, target[:, ::-1].copy(), draft[:, ::-1].copy(), vocab - 1 - tokens, u, np.array([0.3, 0.6], np.float32),
          [1.0, 1e30])


def test_rows_without_a_distribution(cuda):
    rng = np.random.default_rng(7)
    counts, vocab = [3, 3, 3, 3, 3, 3], 900
    target, draft, tokens, u, v = batch(rng, counts, vocab, agree=0.0)
    where = np.concatenate([np.arange(3) + 4 * b for b in range(6)])
    assert (draft == target[where]).all()      # the models agree: all drafts are accepted
    check(counts, vocab, target, draft, tokens, u, v, None)
    target[1, 17] = np.nan             # a draft's row of the target
    target[4 + 3, 5] = np.inf          # the row behind the drafts
    target[8 + 0, :] = -np.inf
    draft[9 + 2, 899] = np.nan         # a draft model's row
    draft[12 + 1, 0] = np.inf
    a, o = check(counts, vocab, target, draft, tokens, u, v, None)
    assert a[:5] == [1, 3, 0, 2, 1] and o[1] == -1 and o[7] == -1
    # a greedy sequence does not look at the draft model's
    a, _ = check(counts, vocab, target, draft, tokens, u, v, [1, 1, 1, 0, 0, 0])
    # one behind the stop changes nothing
    target, draft, tokens, u, v = batch(rng, [2], vocab)
    target[0, tokens[0]] = -np.inf
    target[1:, :] = np.nan
    draft[1:, :] = np.nan
    a, o = check([2], vocab, target, draft, tokens, u, v, None)
    assert a == [0] and o[0] >= 0 and o[1:] == [-1, -1]


def test_greedy_ties_go_to_the_first(cuda):
    vocab = 30000
    target = np.zeros((3, vocab), np.float32)
    target[0, [29000, 70, 8000]] = 2.0
    target[1, [123, 29999]] = 1.0
    tokens = np.array([70, 29999])
    a, o = check([2], vocab, target, None, tokens, np.zeros(2, np.float32), np.zeros(1, np.float32), [0.0])
    assert a == [1] and o == [70, 123, -1]


def test_nothing_left_over(cuda):
    """p = q, and the drafted token has none of either: the next token is drawn from p."""
    vocab = 500
    rng = np.random.default_rng(8)
    target = rng.standard_normal((2, vocab)).astype(np.float32)
    target[:, 33] = -np.inf
    draft = target[:1] + np.float32(2.0)   # the same distribution, other sums
    check([1], vocab, target, draft, np.array([33]), np.array([0.2], np.float32), np.array([0.77], np.float32), None)
    # looked up: all of p is on the drafted token's neighbour, or on the token itself
    target[:] = -np.inf
    target[:, 4] = 0.0
    for x in (3, 4):
        check([1], vocab, target, None, np.array([x]), np.array([0.99], np.float32), np.array([0.5], np.float32), None)


def test_tokens_outside_and_starts_that_fall(cuda):
    rng = np.random.default_rng(9)
    counts, vocab = [2, 2], 300
    target, draft, tokens, u, v = batch(rng, counts, vocab, agree=0.0)
    for bad in (-1, 300, 2 ** 31 - 1):
        t = tokens.copy()
        t[1] = bad
        check(counts, vocab, target, draft, t, u, v, None, want_status=ans.STATUS_BAD_INDEX)
        check(counts, vocab, target, None, t, u, v, [0.0, 1.0], want_status=ans.STATUS_BAD_INDEX)
    # starts within the rows whatever they say: flagged, and nothing else is written
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    for starts in ([0, 5, 4], [0, -3, 4], [1, 2, 4], [0, 2, 9], [2 ** 31 - 1, -2 ** 31, 7]):
        out = torch.full((8,), -7, dtype=torch.int32, device="cuda")
        accepted = torch.full((3,), -7, dtype=torch.int32, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        size = ans.ans_verify_workspace(2, 4, vocab)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        ans.ans_verify(dev(target), vocab, dev(draft), vocab, 2, 4, vocab, dev(np.array(starts, np.int32)),
                       dev(tokens.astype(np.int32)), dev(u), dev(v), None, accepted, out, ws, size, st)
        torch.cuda.synchronize()
        assert int(st.item()) == ans.STATUS_BAD_INDEX
        assert out[6:].tolist() == [-7, -7] and accepted[2] == -7


@pytest.mark.parametrize("starts", [[0, 5, 4, 6], [0, 4, 2, 6], [3, 0, 6, 6], [0, -3, 9, 1], [6, 6, 6, 6]])
@pytest.mark.parametrize("temperature", [[0.0, 1.0, 0.0], [1.0, 0.0, 0.5], [0.0, 0.0, 2.0]])
def test_wrong_starts_of_greedy_and_other_sequences(cuda, starts, temperature):
    """Rows that the starts give to two sequences: flagged, and what comes out is a token or -1."""
    rng = np.random.default_rng(12)
    vocab = 700
    target, draft, tokens, u, v = batch(rng, [2, 2, 2], vocab)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    size = ans.ans_verify_workspace(3, 6, vocab)
    for lookup in (False, True):
        for fill in (0, 0x7E):
            out = torch.full((9,), -1, dtype=torch.int32, device="cuda")
            accepted = torch.zeros(3, dtype=torch.int32, device="cuda")
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
            ans.ans_verify(dev(target), vocab, None if lookup else dev(draft), vocab, 3, 6, vocab,
                           dev(np.array(starts, np.int32)), dev(tokens.astype(np.int32)), dev(u), dev(v),
                           dev(np.array(temperature, np.float32)), accepted, out, ws, size, st)
            torch.cuda.synchronize()
            assert int(st.item()) == ans.STATUS_BAD_INDEX
            assert out.min() >= -1 and out.max() < vocab
            assert accepted.min() >= 0 and accepted.max() <= 6


def test_what_comes_out_is_distributed_as_the_target(cuda):
    """Over a grid of u and v and all drafts with their chances, the first token's distribution is p."""
    vocab, grid = 5, 64
    rng = np.random.default_rng(10)
    target = rng.standard_normal((2, vocab)).astype(np.float32)
    draft = rng.standard_normal((1, vocab)).astype(np.float32)
    p, q = distribution(target[0], 1.0), distribution(draft[0], 1.0)
    points = ((np.arange(grid) + 0.5) / grid).astype(np.float32)
    b = vocab * grid * grid
    tokens = np.repeat(np.arange(vocab), grid * grid).astype(np.int32)
    u, v = np.tile(np.repeat(points, grid), vocab), np.tile(points, vocab * grid)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    size = ans.ans_verify_workspace(b, b, vocab)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    accepted = torch.empty(b, dtype=torch.int32, device="cuda")
    out = torch.empty(2 * b, dtype=torch.int32, device="cuda")
    ans.ans_verify(dev(np.tile(target, (b, 1))), vocab, dev(np.tile(draft, (b, 1))), vocab, b, b, vocab,
                   dev(np.arange(b + 1, dtype=np.int32)), dev(tokens), dev(u), dev(v), None, accepted, out, ws, size, st)
    first = out.view(b, 2)[:, 0].cpu().numpy()
    assert int(st.item()) == 0
    got = np.zeros(vocab)
    np.add.at(got, first, q[tokens] / (grid * grid))
    # the grid holds each of the two chances to within one point of it
    assert np.abs(got - p).max() <= 2 * vocab / grid


def test_captured_and_on_another_stream(cuda):
    rng = np.random.default_rng(11)
    counts, vocab = [3, 2, 4], 9000
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n, b = 9, 3
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    size = ans.ans_verify_workspace(b, n, vocab)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a = batch(rng, counts, vocab)
    buf = [dev(a[0]), dev(a[1]), dev(a[2].astype(np.int32)), dev(a[3]), dev(a[4])]
    d_starts = dev(starts)
    accepted = torch.empty(b, dtype=torch.int32, device="cuda")
    out = torch.empty(n + b, dtype=torch.int32, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call(stream):
        ans.ans_verify(buf[0], vocab, buf[1], vocab, b, n, vocab, d_starts, buf[2], buf[3], buf[4], None, accepted, out, ws,
                       size, st, stream)
    with torch.cuda.stream(side):
        call(side)
        graph.capture_begin()
        call(side)
        graph.capture_end()
    for _ in range(3):
        a = batch(rng, counts, vocab)
        for t, v in zip(buf, (a[0], a[1], a[2].astype(np.int32), a[3], a[4])):
            t.copy_(dev(v))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = check(counts, vocab, *a, None)
        assert (accepted.tolist(), out.tolist()) == (want[0], want[1])
    assert int(st.item()) == 0
