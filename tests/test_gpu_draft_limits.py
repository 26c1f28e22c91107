"""The gated block, distillation and verification at their limits: workspaces that are too
small, waits that run out, offsets past 32 bits, calls side by side, and one draft model's
training step and one verification as they follow one another."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import BF16, bf16, status, usual, within, workspace
from test_gpu_distill import leaning, reference as distill_reference, run as run_distill, teacher
from test_gpu_gated import Block, forward_reference, inputs, run_forward, run_grad
from test_gpu_verify import batch, check as check_verify, sequence

pytestmark = pytest.mark.gpu


@pytest.fixture
def wait_budget():
    yield ans._set_wait_budget
    ans._set_wait_budget(0)


def test_workspaces_one_byte_short_are_refused_and_untouched(cuda):
    B = Block(ans.INT8, 256, 128)
    L = B.gate
    rng = np.random.default_rng(1)
    st = status()
    for M in (20, 300):
        x, dh = (t.cuda() for t in inputs(B, M, 1))
        ids, logits = (t.cuda() for t in teacher(rng, M, 250, 6))
        h, dg, du = (torch.zeros(M, 256, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        dx, loss = torch.zeros_like(x), torch.zeros(M, device="cuda")
        calls = [
            (ans.ans_gated_workspace(L.layout, M, L.kind), lambda ws, n: ans.ans_gated(x, M, *B.args(0), h, ws, n, st)),
            (ans.ans_gated_grad_workspace(L.layout, M, L.kind),
             lambda ws, n: ans.ans_gated_grad(x, dh, M, *B.args(0), dx, dg, du, ws, n, st)),
            (ans.ans_distill_workspace(L.layout, M, L.kind, 6, True),
             lambda ws, n: ans.ans_distill(x, M, *L.args, 250, 1.0, 6, ids, logits, None, loss, loss, None, dx, ws, n, st)),
            (ans.ans_distill_workspace(L.layout, M, L.kind, 6, False),
             lambda ws, n: ans.ans_distill(x, M, *L.args, 250, 1.0, 6, ids, logits, None, loss, loss, None, None, ws, n, st))]
        for size, fn in calls:
            ws = torch.full((size,), 0x33, dtype=torch.uint8, device="cuda")
            with pytest.raises(ans.AnsError) as e:
                fn(ws, size - 1)
            assert e.value.status == 4
            torch.cuda.synchronize()
            assert (ws == 0x33).all()
        for out in (h, dg, du, dx, loss):
            assert not out.any()
    z = torch.zeros(8, 300, device="cuda")
    whole = torch.zeros(9, dtype=torch.int32, device="cuda")
    size = ans.ans_verify_workspace(2, 5, 300)
    with pytest.raises(ans.AnsError) as e:
        ans.ans_verify(z, 300, z, 300, 2, 5, 300, whole, whole, z, z, None, whole, whole, workspace(size), size - 1, st)
    assert e.value.status == 4


@pytest.mark.parametrize("M", [20, 300])
def test_short_waits_are_exact_or_flagged_and_the_next_call_is_exact(cuda, wait_budget, M):
    # (as for the gradient and the loss: a wait that runs out says so)
    B = Block(ans.BF16_SPLIT, 1024, 2048, seed=1)
    L = B.up
    rng = np.random.default_rng(1)
    x, dh = inputs(B, M, 3)
    ids, logits = teacher(rng, M, 1000, 8)
    want_h = forward_reference(B, x, ans.ACT_SILU)
    y = bf16(rng, M, 2048, scale=0.1)
    want = distill_reference(L, y, 1000, 1.0, ids, logits)
    xc, yc, dhc, ic, lc = (t.cuda() for t in (x, y, dh, ids, logits))
    h_ws = workspace(ans.ans_gated_workspace(B.layout, M, 0))
    g_ws = workspace(ans.ans_gated_grad_workspace(B.layout, M, 0))
    d_ws = workspace(ans.ans_distill_workspace(L.layout, M, 0, 8, True))
    clean = run_grad(B, x, dh, ans.ACT_SILU)
    for budget in (1, 1000, 0):
        torch.cuda.synchronize()
        wait_budget(budget)
        h = torch.zeros(M, 1024, dtype=torch.bfloat16, device="cuda")
        dg, du, dx = torch.zeros_like(h), torch.zeros_like(h), torch.zeros(M, 2048, dtype=torch.bfloat16, device="cuda")
        loss, lse = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda")
        flags = []
        for call in (lambda st: ans.ans_gated(xc, M, *B.args(0), h, h_ws, h_ws.numel(), st),
                     lambda st: ans.ans_gated_grad(xc, dhc, M, *B.args(0), dx, dg, du, g_ws, g_ws.numel(), st),
                     lambda st: ans.ans_distill(yc, M, *L.args, 1000, 1.0, 8, ic, lc, None, loss, lse, None, None, d_ws,
                                                d_ws.numel(), st)):
            st = status()
            call(st)
            torch.cuda.synchronize()
            flags.append(int(st.item()))
            assert flags[-1] == 0 or (budget and flags[-1] & ans.STATUS_TIMEOUT)
        if flags[0] == 0:
            within(h, *want_h, "h")
        else:
            h_ws.zero_()  # (after a run that set the status)
        if flags[1] == 0:
            assert all(torch.equal(a, b) for a, b in zip((dx, dg, du), clean))
        if flags[2] == 0:
            within(loss, *want[0], "loss")
            within(lse, *want[1], "lse")


def test_offsets_past_32_bits(cuda):
    # more than 2^31 values in H, dH, dG and the kept probabilities; the rows looked at are the last and some between
    N, K, M = 33024, 64, 66000
    B = Block(ans.BF16_SPLIT, N, K, seed=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, 30000, 65029, 65030, 65537, M - 2, M - 1])
    st = status()
    h = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = workspace(ans.ans_gated_workspace(B.layout, M, 0))
    ans.ans_gated(x, M, *B.args(ans.ACT_SILU), h, ws, ws.numel(), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    few = x[rows.cuda()].cpu()
    within(h[rows.cuda()], *forward_reference(B, few, ans.ACT_SILU), "h")
    dh = h  # (any gradient will do)
    want = run_grad(B, few, dh[rows.cuda()].cpu(), ans.ACT_SILU)
    dg, du = torch.empty_like(h), torch.empty_like(h)
    dx = torch.empty_like(x)
    ws = workspace(ans.ans_gated_grad_workspace(B.layout, M, 0))
    ans.ans_gated_grad(x, dh, M, *B.args(ans.ACT_SILU), dx, dg, du, ws, ws.numel(), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # dG and dU are a token's alone, whatever the batch; dX is cut into other sums
    assert torch.equal(dg[rows.cuda()], want[1]) and torch.equal(du[rows.cuda()], want[2])
    a, b = dx[rows.cuda()].double(), want[0].double()
    assert ((a - b).norm(dim=1) <= 2 * BF16 * b.norm(dim=1)).all()


def test_kept_probabilities_past_32_bits(cuda):
    # 4,096 tokens of 540,672 rows at a time: 2.2e9 values; the tokens looked at are the last and some between
    N, K, M, top = 540672, 32, 4096, 5
    L = usual(ans.BF16_SPLIT, N, K, seed=2)
    rng = np.random.default_rng(4)
    rows = torch.tensor([0, 1, 2000, 3971, 3972, 4094, 4095])
    ids = torch.full((M, top), -1, dtype=torch.int32)
    logits = torch.zeros(M, top)
    some, v = teacher(rng, len(rows), N, top)
    some[:, 0] = torch.tensor([N - 1, 0, 5, N - 2, 31, 32, N - 1], dtype=torch.int32)
    some[:, 1:] = torch.where(some[:, 1:] == some[:, :1], -1, some[:, 1:])
    ids[rows], logits[rows] = some, v
    x = bf16(rng, M, K)
    loss, lse, dx = run_distill(L, x, N, 1.0, ids, logits)
    a, b, c = distill_reference(L, x[rows], N, 1.0, some, v)
    within(loss[rows.cuda()], *a, "loss")
    within(lse[rows.cuda()], *b, "lse")
    within(dx[rows.cuda()], *c, "dx")
    rest = torch.ones(M, dtype=torch.bool)
    rest[rows] = False
    assert not dx[rest.cuda()].any() and not loss[rest.cuda()].any()


def test_verification_of_rows_far_apart(cuda):
    """Rows whose offsets pass 2^31 logits."""
    vocab, stride = 1000, 700_000_000
    rng = np.random.default_rng(2)
    target, draft, tokens, u, v = batch(rng, [2], vocab)
    far = torch.zeros(2 * stride + vocab + 64, device="cuda")
    for r in range(3):
        far[r * stride:r * stride + vocab] = torch.from_numpy(target[r]).cuda()
    for r in range(2):
        far[r * stride + 100_000:r * stride + 100_000 + vocab] = torch.from_numpy(draft[r]).cuda()
    dev = lambda a, kind: torch.from_numpy(np.asarray(a, kind)).cuda()  # noqa: E731
    accepted, out = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    size = ans.ans_verify_workspace(1, 2, vocab)
    st = status()
    ans.ans_verify(far, stride, far[100_000:], stride, 1, 2, vocab, dev([0, 2], np.int32), dev(tokens, np.int32),
                   dev(u, np.float32), dev(v, np.float32), None, accepted, out, workspace(size), size, st)
    torch.cuda.synchronize()
    a, o = sequence(target, draft, tokens, u, v[0], 1.0, vocab)
    assert (accepted.tolist(), out.tolist(), int(st.item())) == ([a], o, 0)


def test_two_calls_side_by_side(cuda):
    """A workspace each, on two streams at once: the bits of calls alone."""
    B = Block(ans.INT4_PAIRS, 1024, 512, seed=2)
    L = usual(ans.FP8_E4M3, 2048, 512, seed=3)
    rng = np.random.default_rng(3)
    M = 150
    x, dh = inputs(B, M, 4)
    ids, logits = teacher(rng, M, 2000, 8)
    y = leaning(L, rng, M, ids)
    alone_g, alone_d = run_grad(B, x, dh, ans.ACT_GELU), run_distill(L, y, 2000, 1.0, ids, logits)
    xc, dhc, yc, ic, lc = (t.cuda() for t in (x, dh, y, ids, logits))
    dx, dg, du = torch.empty_like(xc), torch.empty_like(dhc), torch.empty_like(dhc)
    loss, lse, dy = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty_like(yc)
    g_ws = workspace(ans.ans_gated_grad_workspace(B.layout, M, B.kind))
    d_ws = workspace(ans.ans_distill_workspace(L.layout, M, L.kind, 8, True))
    st, st2 = status(), status()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        ans.ans_gated_grad(xc, dhc, M, *B.args(ans.ACT_GELU), dx, dg, du, g_ws, g_ws.numel(), st, a)
        ans.ans_distill(yc, M, *L.args, 2000, 1.0, 8, ic, lc, None, loss, lse, None, dy, d_ws, d_ws.numel(), st2, b)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and int(st2.item()) == 0
    assert all(torch.equal(p, q) for p, q in zip((dx, dg, du), alone_g))
    assert all(torch.equal(p, q) for p, q in zip((loss, lse, dy), alone_d))


def test_a_corrupt_layer_is_flagged(cuda):
    B = Block(ans.BF16_SPLIT, 256, 128, seed=4)
    x, dh = inputs(B, 40, 5)
    L = B.up
    good = L.layer.d_stream.clone()
    L.layer.d_stream[200:260] ^= 0x5A
    st = status()
    h = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
    for M in (8, 40):
        ws = workspace(ans.ans_gated_workspace(B.layout, M, 0))
        st.zero_()
        ans.ans_gated(x.cuda(), M, *B.args(0), h, ws, ws.numel(), st)
        torch.cuda.synchronize()
        assert int(st.item()) & ans.STATUS_CORRUPT
    L.layer.d_stream.copy_(good)
    within(run_forward(B, x, ans.ACT_SILU), *forward_reference(B, x, ans.ACT_SILU), "h")


def test_a_draft_model_is_trained_and_checked(cuda):
    """The operators together: a block and a head give logits; a teacher's top logits train them; drafts
    drawn from the head are verified against a target head's logits, as ans_gemm leaves them."""
    K, N, V, vocab, M = 128, 256, 1024, 1000, 12
    B = Block(ans.BF16_SPLIT, N, K, seed=5)
    down, head, target = usual(ans.BF16_SPLIT, K, N, seed=6), usual(ans.INT8, V, K, seed=7), usual(ans.FP8_E4M3, V, K, seed=8)
    rng = np.random.default_rng(9)
    x = bf16(rng, M, K)
    st = status()

    def gemm(L, t):
        y = torch.empty(M, L.N, device="cuda")
        ws = workspace(ans.ans_gemm_workspace(L.layout, M, L.kind))
        ans.ans_gemm(t, M, *L.args, y, ws, ws.numel(), st)
        return y
    h = run_forward(B, x, ans.ACT_SILU)
    hidden = (x.cuda().float() + gemm(down, h)).bfloat16()
    student, teacher_z = gemm(head, hidden), gemm(target, x.cuda())
    top = torch.topk(teacher_z[:, :vocab], 16)
    lse = torch.logsumexp(teacher_z[:, :vocab].double(), 1).float()
    ids, logits = top.indices.to(torch.int32), top.values.contiguous()
    loss, slse, d_hidden = run_distill(head, hidden.cpu(), vocab, 1.0, ids.cpu(), logits.cpu(), lse.cpu())
    want = distill_reference(head, hidden.cpu(), vocab, 1.0, ids.cpu(), logits.cpu(), lse.cpu())
    within(loss, *want[0], "loss")
    within(d_hidden, *want[2], "d_hidden")
    # back through the block: the down projection's input gradient, then the block's
    dh = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    ws = workspace(ans.ans_gemm_grad_workspace(down.layout, M, down.kind))
    ans.ans_gemm_grad(d_hidden, M, *down.args, dh, ws, ws.numel(), st)
    dx, _, _ = run_grad(B, x, dh.cpu(), ans.ACT_SILU)
    # the same in 64 bits, of the hidden states as rounded; each stage rounds once more
    leaf = x.double().requires_grad_()
    hh = torch.nn.functional.silu(leaf @ B.gate.w.T) * (leaf @ B.up.w.T)
    (want_dx,) = torch.autograd.grad(hh @ down.w.T, leaf, want[2][0])
    assert ((dx.cpu().double() - want_dx).norm() / want_dx.norm()).item() <= 3 * BF16
    # drafts: each row's likeliest token of the student but one, and a check of every three
    counts = [3, 3, 2]
    rows = np.concatenate([np.arange(4) + 4 * k for k in range(3)])[:11]
    drafts = np.concatenate([rows[0:3], rows[4:7], rows[8:10]])
    z, y = teacher_z[:11].cpu().numpy(), student.cpu().numpy()
    tokens = np.array([int(np.argsort(-y[r, :vocab])[k % 2]) for k, r in enumerate(drafts)])
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    check_verify(counts, vocab, z[rows][:, :vocab].copy(), y[drafts][:, :vocab].copy(), tokens,
                 rng.random(8, np.float32), rng.random(3, np.float32), [1.0, 0.6, 0.0], t_stride=V, d_stride=V)
