"""The adapter, gradient and loss operators at their limits: workspaces that are
too small, waits that run out, offsets past 32 bits, and layers of the sizes that
the library is measured on (sampled rows)."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import bf16, status, usual, within, workspace
from test_gpu_grad_lora import Adapters, grad_reference, lora_grad_reference, lora_reference, run_grad, some_ids
from test_gpu_xent import reference, run, some_targets

pytestmark = pytest.mark.gpu


@pytest.fixture
def wait_budget():
    yield ans._set_wait_budget
    ans._set_wait_budget(0)


def test_workspaces_one_byte_short_are_refused_and_untouched(cuda):
    L = usual(ans.INT8, 256, 128, seed=1)
    A = Adapters(L, 3, 16)
    rng = np.random.default_rng(1)
    for M in (20, 300):
        x, dy, ids, t = bf16(rng, M, 128).cuda(), bf16(rng, M, 256).cuda(), some_ids(rng, M, 3).cuda(), some_targets(rng, M, 256).cuda()
        y, loss = torch.zeros(M, 256, device="cuda"), torch.zeros(M, device="cuda")
        dx, da, db = torch.zeros_like(x), torch.zeros(A.a.shape, device="cuda"), torch.zeros(A.b.shape, device="cuda")
        st = status()
        calls = [
            (ans.ans_gemm_lora_workspace(L.layout, M, L.kind, A.lora),
             lambda ws, n: ans.ans_gemm_lora(x, M, *L.args, A.lora, ids, y, ws, n, st)),
            (ans.ans_gemm_grad_workspace(L.layout, M, L.kind), lambda ws, n: ans.ans_gemm_grad(dy, M, *L.args, dx, ws, n, st)),
            (ans.ans_gemm_lora_grad_workspace(L.layout, M, L.kind, A.lora),
             lambda ws, n: ans.ans_gemm_lora_grad(x, dy, M, *L.args, A.lora, ids, dx, da, db, ws, n, st)),
            (ans.ans_xent_workspace(L.layout, M, L.kind, True),
             lambda ws, n: ans.ans_xent(x, M, *L.args, 256, t, loss, loss, None, dx, ws, n, st)),
            (ans.ans_xent_workspace(L.layout, M, L.kind, False),
             lambda ws, n: ans.ans_xent(x, M, *L.args, 256, t, loss, loss, None, None, ws, n, st))]
        for size, fn in calls:
            ws = torch.full((size,), 0x33, dtype=torch.uint8, device="cuda")
            with pytest.raises(ans.AnsError) as e:
                fn(ws, size - 1)
            assert e.value.status == 4
            torch.cuda.synchronize()
            assert (ws == 0x33).all()
        for out in (y, loss, dx, da, db):
            assert not out.any()


@pytest.mark.parametrize("M", [20, 300])
def test_short_waits_are_exact_or_flagged_and_the_next_call_is_exact(cuda, wait_budget, M):
    # most waits end inside the barrier test's own suspend window, whatever the
    # budget; a wait that does run out says so, and nothing is wrong without that
    L = usual(ans.BF16_SPLIT, 1024, 2048, seed=1)
    rng = np.random.default_rng(1)
    dy, x, t = bf16(rng, M, 1024), bf16(rng, M, 2048, scale=0.1), some_targets(rng, M, 1000)
    want_dx, want = grad_reference(L, dy), reference(L, x, t, 1000)
    dyc, xc, tc = dy.cuda(), x.cuda(), t.cuda()
    g_ws = workspace(ans.ans_gemm_grad_workspace(L.layout, M, 0))
    x_ws = workspace(ans.ans_xent_workspace(L.layout, M, 0, True))
    for budget in (1, 1000, 0):
        torch.cuda.synchronize()
        wait_budget(budget)
        dx, st = torch.zeros(M, 2048, dtype=torch.bfloat16, device="cuda"), status()
        ans.ans_gemm_grad(dyc, M, *L.args, dx, g_ws, g_ws.numel(), st)
        torch.cuda.synchronize()
        flags = int(st.item())
        assert flags == 0 or (budget and flags & ans.STATUS_TIMEOUT)
        if flags == 0:
            within(dx, *want_dx, "dx")
        st = status()
        loss, lse = torch.zeros(M, device="cuda"), torch.zeros(M, device="cuda")
        ans.ans_xent(xc, M, *L.args, 1000, tc, loss, lse, None, dx, x_ws, x_ws.numel(), st)
        torch.cuda.synchronize()
        flags = int(st.item())
        assert flags == 0 or (budget and flags & ans.STATUS_TIMEOUT)
        if flags == 0:
            for a, b in zip((loss, lse, dx), want):
                within(a, *b)


def test_products_whose_offsets_pass_32_bits(cuda):
    # more than 2^31 values in dY and Y; the rows looked at are the last and some between
    N, K, M = 33024, 64, 66000
    L = usual(ans.BF16_SPLIT, N, K, seed=1)
    A = Adapters(L, 3, 8)
    rng = np.random.default_rng(1)
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(M, N, generator=g, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    # few tokens of an adapter, so that the sums over them can be formed here
    rows = torch.tensor([0, 1, 30000, 65029, 65030, 65537, M - 2, M - 1])
    ids = torch.full((M,), -1, dtype=torch.int32)
    ids[rows] = torch.tensor([0, 1, 2, 0, 1, 2, 1, 2], dtype=torch.int32)
    some, dy_s, x_s = ids[rows], dy[rows.cuda()].cpu(), x[rows.cuda()].cpu()
    dx, st = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), status()
    da, db = torch.empty(A.a.shape, device="cuda"), torch.empty(A.b.shape, device="cuda")
    ws = workspace(ans.ans_gemm_lora_grad_workspace(L.layout, M, 0, A.lora))
    ans.ans_gemm_lora_grad(x, dy, M, *L.args, A.lora, ids.cuda(), dx, da, db, ws, ws.numel(), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for got, want in zip((dx[rows.cuda()], da, db), lora_grad_reference(L, A, x_s, dy_s, some)):
        within(got, *want)
    del dy, ws, dx
    y = torch.empty(M, N, device="cuda")
    ws = workspace(ans.ans_gemm_lora_workspace(L.layout, M, 0, A.lora))
    ans.ans_gemm_lora(x, M, *L.args, A.lora, ids.cuda(), y, ws, ws.numel(), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    within(y[rows.cuda()], *lora_reference(L, A, x_s, some), "y")


@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8])
def test_loss_whose_offsets_pass_32_bits(cuda, dtype):
    N, K, M = 128, 16400, 131100
    L = usual(dtype, N, K, seed=1)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = 0.02 * torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    t = torch.randint(0, 128, (M,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dx, st = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), status()
    ws = workspace(ans.ans_xent_workspace(L.layout, M, L.kind, True))
    ans.ans_xent(x, M, *L.args, 128, t, loss, lse, None, dx, ws, ws.numel(), st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    rows = torch.tensor([0, 4095, 4096, 65000, 130948, 130949, M - 1], device="cuda")
    want = reference(L, x[rows].cpu(), t[rows].cpu(), 128)
    for got, w in zip((loss, lse, dx), want):
        within(got[rows], *w)


@pytest.mark.parametrize("dtype,N,K,M", [(ans.FP8_E4M3, 28672, 8192, 257), (ans.INT4_PAIRS, 14336, 4096, 1030)])
def test_layers_of_the_measured_sizes(cuda, dtype, N, K, M):
    L = usual(dtype, N, K, seed=2)
    rng = np.random.default_rng(2)
    rows = torch.tensor([0, 1, 128, 255, 256, M - 1])
    dy = torch.randn(M, N, device="cuda", dtype=torch.bfloat16)
    dx = run_grad(L, dy)
    within(dx[rows.cuda()], *grad_reference(L, dy[rows.cuda()].cpu()), "dx")
    x, t = bf16(rng, M, K, scale=0.02), some_targets(rng, M, N - 5)
    loss, lse, dx, st = run(L, x, t, N - 5)
    assert st == 0
    for got, w in zip((loss, lse, dx), reference(L, x[rows], t[rows], N - 5)):
        within(got[rows.cuda()], *w)


@pytest.mark.parametrize("dtype,M", [(ans.INT8, 16500), (ans.INT8, 70), (ans.BF16_SPLIT, 300)])
def test_loss_alone_over_pieces_and_chunks(cuda, dtype, M):
    # more than one piece of the vocabulary; the first size also has two chunks of tokens.  A piece's
    # last blocks are joined while the next piece is decoded
    N, K, vocab = 24832, 2064, 24820
    L = usual(dtype, N, K, seed=3)
    rng = np.random.default_rng(M)
    x, t = bf16(rng, M, K, scale=0.02), some_targets(rng, M, vocab)
    rows = torch.unique(torch.tensor([0, 1, M // 2, min(M - 1, 8447), min(M - 1, 8448), M - 2, M - 1]))
    ws = workspace(ans.ans_xent_workspace(L.layout, M, L.kind, False))
    loss, lse, _, st = run(L, x, t, vocab, grad=False, ws=ws)
    assert st == 0
    want = reference(L, x[rows], t[rows], vocab)
    within(loss[rows.cuda()], *want[0], "loss")
    within(lse[rows.cuda()], *want[1], "lse")
    for _ in range(3):
        again = run(L, x, t, vocab, grad=False, ws=ws)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype,M", [(ans.INT8, 600), (ans.BF16_SPLIT, 200), (ans.INT4_PAIRS, 2100)])
def test_calls_one_behind_another_share_a_workspace(cuda, dtype, M, graph):
    # kernels run beside the one before them: calls on other inputs, one behind another without a
    # pause and in one workspace an operator, give what each gives by itself
    L = usual(dtype, 4096, 2048, seed=4)
    A = Adapters(L, 3, 64)
    rng = np.random.default_rng(M)
    sets = [(bf16(rng, M, L.K, scale=0.1).cuda(), bf16(rng, M, L.N, scale=0.1).cuda(), some_ids(rng, M, 3).cuda(),
             some_targets(rng, M, 4000).cuda()) for _ in range(3)]
    g_ws, b_ws, x_ws, l_ws = (workspace(n) for n in (
        ans.ans_gemm_grad_workspace(L.layout, M, L.kind), ans.ans_gemm_lora_grad_workspace(L.layout, M, L.kind, A.lora),
        ans.ans_xent_workspace(L.layout, M, L.kind, True), ans.ans_xent_workspace(L.layout, M, L.kind, False)))
    st = status()

    def new():
        dx = [torch.zeros(M, L.K, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        return (*dx, torch.zeros(A.a.shape, device="cuda"), torch.zeros(A.b.shape, device="cuda"),
                *(torch.zeros(M, device="cuda") for _ in range(4)))

    def calls(s, o):
        x, dy, ids, t = s
        stream = torch.cuda.current_stream()
        yield lambda: ans.ans_gemm_grad(dy, M, *L.args, o[0], g_ws, g_ws.numel(), st, stream)
        yield lambda: ans.ans_gemm_lora_grad(x, dy, M, *L.args, A.lora, ids, o[1], o[3], o[4], b_ws, b_ws.numel(), st, stream)
        yield lambda: ans.ans_xent(x, M, *L.args, 4000, t, o[5], o[6], None, o[2], x_ws, x_ws.numel(), st, stream)
        yield lambda: ans.ans_xent(x, M, *L.args, 4000, t, o[7], o[8], None, None, l_ws, l_ws.numel(), st, stream)

    want, got = [new() for _ in sets], [new() for _ in sets]
    for s, o in zip(sets, want):
        for call in calls(s, o):
            call()
            torch.cuda.synchronize()

    def all_of_them():
        for each in zip(*(list(calls(s, o)) for s, o in zip(sets, got))):   # the same operator behind itself
            for call in each:
                call()
        for s, o in zip(sets, got):                                         # and behind the others
            for call in calls(s, o):
                call()

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_of_them()
        for _ in range(3):
            g.replay()
    else:
        all_of_them()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for a, b in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)
