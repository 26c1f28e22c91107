"""ans_gemm_grad, ans_gemm_lora and ans_gemm_lora_grad against their formulas in
64 bits, at the sizes where their kernels change course."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import ALL, BF16, Layer, bf16, status, sum_eps, usual, within, workspace

pytestmark = pytest.mark.gpu


# ---- plain forms and bounds ------------------------------------------------------
def grad_reference(L, dy):
    """dY W, and how far a right result may be: a rounded factor, fp32 sums, bf16 out."""
    want = dy.double() @ L.w
    mass = dy.double().abs() @ L.w.abs()
    rounded = 0.0 if L.dtype == ans.BF16_SPLIT and L.kind == ans.SCALE_NONE else L.factor_eps
    # what f16 drops below 2^-39 of the row's largest counts against that value
    floor = 2.0 ** -38 * (dy.double().abs().amax(1, keepdim=True) * L.w.abs().amax(0, keepdim=True) * L.N)
    inner = (rounded + sum_eps(L.N)) * mass + floor
    return want, BF16 * (want.abs() + inner) + inner


def run_grad(L, dy, ws=None):
    M = dy.shape[0]
    size = ans.ans_gemm_grad_workspace(L.layout, M, L.kind)
    ws = workspace(size) if ws is None else ws
    dx = torch.full((M, L.K), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = status()
    ans.ans_gemm_grad(dy.cuda(), M, *L.args, dx, ws, size, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return dx


class Adapters:
    def __init__(self, L, n, rank, seed=0, scale=True):
        rng = np.random.default_rng([seed, n, rank])
        self.a, self.b = bf16(rng, n, rank, L.K, scale=L.K ** -0.5), bf16(rng, n, L.N, rank, scale=0.05)
        self.s = torch.from_numpy(rng.uniform(0.5, 2.0, n).astype(np.float32)) if scale else None
        self.dev = ans.LoraAdapters(self.a.cuda(), self.b.cuda(), self.s.cuda() if scale else None)
        self.lora, self.n, self.rank = self.dev.lora, n, rank

    def scale(self, i):
        return float(self.s[i]) if self.s is not None else 1.0


def lora_reference(L, A, x, ids):
    x64 = x.double()
    want, bound = x64 @ L.w.T, sum_eps(L.K) * (x64.abs() @ L.w.abs().T)
    for i in range(A.n):
        at = (ids == i).nonzero()[:, 0]
        a, b, s = A.a[i].double(), A.b[i].double(), A.scale(i)
        h, mass = x64[at] @ a.T, x64[at].abs() @ a.abs().T
        want[at] += s * (h @ b.T)
        # h's sum, its two bf16 parts (2^-16 of it at most), the second sum
        bound[at] += s * (((sum_eps(L.K) + 2.0 ** -16 + sum_eps(A.rank)) * mass) @ b.abs().T)
    return want, bound + 2.0 ** -23 * want.abs()


def run_lora(L, A, x, ids, ws=None):
    M = x.shape[0]
    size = ans.ans_gemm_lora_workspace(L.layout, M, L.kind, A.lora)
    ws = workspace(size) if ws is None else ws
    y = torch.full((M, L.N), float("nan"), device="cuda")
    st = status()
    ans.ans_gemm_lora(x.cuda(), M, *L.args, A.lora, ids.cuda(), y, ws, size, st)
    torch.cuda.synchronize()
    return y, int(st.item())


def lora_grad_reference(L, A, x, dy, ids):
    dx, dx_bound = grad_reference(L, dy)
    x64, dy64 = x.double(), dy.double()
    da, db = torch.zeros(A.a.shape, dtype=torch.float64), torch.zeros(A.b.shape, dtype=torch.float64)
    da_b, db_b = torch.zeros_like(da), torch.zeros_like(db)
    for i in range(A.n):
        at = (ids == i).nonzero()[:, 0]
        a, b, s = A.a[i].double(), A.b[i].double(), A.scale(i)
        h, h_mass = s * (x64[at] @ a.T), s * (x64[at].abs() @ a.abs().T)
        g, g_mass = s * (dy64[at] @ b), s * (dy64[at].abs() @ b.abs())
        dx[at] += g @ a
        e_g = sum_eps(L.N) + 2.0 ** -16 + 2.0 ** -23
        # dH is rounded to bf16 once on its way into dX: half a step, 2^-8 of it
        inner = (e_g + BF16 + sum_eps(A.rank)) * (g_mass @ a.abs())
        dx_bound[at] += (1 + BF16) * inner + BF16 * (g @ a).abs()
        da[i], db[i] = g.T @ x64[at], dy64[at].T @ h
        n = len(at)
        da_b[i] = (e_g + sum_eps(n)) * (g_mass.T @ x64[at].abs()) + 2.0 ** -23 * da[i].abs()
        db_b[i] = (sum_eps(L.K) + 2.0 ** -16 + 2.0 ** -23 + sum_eps(n)) * (dy64[at].abs().T @ h_mass) \
            + 2.0 ** -23 * db[i].abs()
    return (dx, dx_bound), (da, da_b), (db, db_b)


def run_lora_grad(L, A, x, dy, ids, want_dx=True, ws=None):
    M = dy.shape[0]
    size = ans.ans_gemm_lora_grad_workspace(L.layout, M, L.kind, A.lora)
    ws = workspace(size) if ws is None else ws
    dx = torch.full((M, L.K), float("nan"), dtype=torch.bfloat16, device="cuda") if want_dx else None
    da = torch.full(A.a.shape, float("nan"), device="cuda")
    db = torch.full(A.b.shape, float("nan"), device="cuda")
    st = status()
    ans.ans_gemm_lora_grad(x.cuda(), dy.cuda(), M, *L.args, A.lora, ids.cuda(), dx, da, db, ws, size, st)
    torch.cuda.synchronize()
    return dx, da, db, int(st.item())


def some_ids(rng, M, n):
    return torch.from_numpy(rng.integers(-1, n, M).astype(np.int32))


# ---- ans_gemm_grad ---------------------------------------------------------------
@pytest.mark.parametrize("M", [1, 16, 33, 300])
@pytest.mark.parametrize("dtype", ALL)
def test_grad_of_every_format(cuda, dtype, M):
    L = usual(dtype, 512, 192, seed=M)
    dy = bf16(np.random.default_rng(M), M, L.N, scale=1e-3)
    within(run_grad(L, dy), *grad_reference(L, dy), "dx")


# N and K that fill no tile; every token tile width, whole and ragged; a sum in ranges and in one
@pytest.mark.parametrize("N,K,M", [(128, 16, 1), (128, 16, 31), (384, 80, 65), (128, 144, 257), (640, 1040, 129),
                                   (8192, 128, 5), (4096, 256, 64), (2432, 2064, 700), (512, 2048, 2049)])
@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8])
def test_grad_of_odd_sizes(cuda, dtype, N, K, M):
    L = usual(dtype, N, K, seed=N + K)
    dy = bf16(np.random.default_rng(M), M, N)
    within(run_grad(L, dy), *grad_reference(L, dy), "dx")


# sums that are cut into 16, 8 and 9 parts (these of uneven lengths), with ragged tiles; and
# more tiles than a round of the SMs, one to three rounds
@pytest.mark.parametrize("N,K,M", [(10240, 128, 40), (4096, 400, 300), (14336, 1040, 300), (1024, 4112, 1290),
                                   (2048, 4096, 1280), (640, 16384, 600)])
@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.FP8_E4M3])
def test_grad_where_sums_are_cut(cuda, dtype, N, K, M):
    L = usual(dtype, N, K, seed=N + K)
    dy = bf16(np.random.default_rng(M), M, N)
    ws = workspace(ans.ans_gemm_grad_workspace(L.layout, M, L.kind))
    first = run_grad(L, dy, ws)
    within(first, *grad_reference(L, dy), "dx")
    ws.fill_(0xFF)                                # every part is written before it is read
    assert torch.equal(run_grad(L, dy, ws), first)


@pytest.mark.parametrize("state_bits", [32, 64])
@pytest.mark.parametrize("dtype,kind,group", [
    (ans.BF16_SPLIT, ans.SCALE_ROW_F32, 0), (ans.BF16_SPLIT, ans.SCALE_ROW_BF16, 0), (ans.INT4, ans.SCALE_NONE, 0),
    (ans.INT4, ans.SCALE_ROW_F32, 0), (ans.INT4_PAIRS, ans.SCALE_GROUP_BF16, 128), (ans.FP8_E4M3, ans.SCALE_NONE, 0),
    (ans.FP8_E4M3, ans.SCALE_ROW_BF16, 0), (ans.INT8, ans.SCALE_ROW_BF16, 0), (ans.FP4_PAIRS, ans.SCALE_NONE, 0)])
def test_grad_of_every_scale_kind(cuda, dtype, kind, group, state_bits):
    L = Layer(dtype, 256, 256, 128, 32, kind, group, seed=7, state_bits=state_bits)
    dy = bf16(np.random.default_rng(3), 40, L.N)
    within(run_grad(L, dy), *grad_reference(L, dy), "dx")


def test_grad_keeps_rows_of_any_size(cuda):
    # rows from the smallest normal numbers to the largest, a zero row, and one
    # row whose values span 20 binary orders; rows do not touch one another
    L = usual(ans.FP8_E4M3, 256, 128, seed=1)
    rng = np.random.default_rng(5)
    sizes = torch.tensor([1e-30, 1e-12, 1.0, 1e20, 0.0, 1.0]).double()
    dy = torch.from_numpy(rng.standard_normal((6, 256)))
    dy[5] *= torch.from_numpy(2.0 ** -rng.integers(0, 20, 256).astype(np.float64))
    dy = (dy * sizes[:, None]).float().bfloat16()
    within(run_grad(L, dy), *grad_reference(L, dy), "dx")


@pytest.mark.parametrize("dtype", [ans.BF16_SPLIT, ans.INT8])
def test_grad_keeps_infinities_and_nan_to_their_rows(cuda, dtype):
    L = usual(dtype, 256, 128, seed=2)
    dy = bf16(np.random.default_rng(6), 5, 256)
    dy[1, 7] = float("inf")
    dy[3, 200] = float("nan")
    dx = run_grad(L, dy).cpu()
    want, bound = grad_reference(L, dy[[0, 2, 4]])
    within(dx[[0, 2, 4]], want, bound, "dx")
    assert not torch.isfinite(dx[1]).any() and torch.isnan(dx[3]).all()
    seen = L.w[7] != 0
    assert torch.equal(dx[1][seen].sign().double(), L.w[7][seen].sign())


def test_grad_against_differences(cuda):
    # the gradient of sum(Y * G) by differences of ans_gemm itself.  Y is linear
    # in X, so a difference has no truncation error, only the sums' rounding.
    L = usual(ans.BF16_SPLIT, 256, 128, seed=4)
    rng = np.random.default_rng(8)
    g, x = bf16(rng, 3, 256), bf16(rng, 3, 128)
    dx = run_grad(L, g).cpu().double()
    ws = workspace(ans.ans_gemm_workspace(L.layout, 3, 0))

    def loss(v):
        y, st = torch.empty(3, 256, device="cuda"), status()
        ans.ans_gemm(v.cuda(), 3, *L.args, y, ws, ws.numel(), st)
        return (y.cpu().double() * g.double()).sum().item()
    base = loss(x)
    for m, k in [(0, 0), (1, 77), (2, 127)]:
        moved = x.clone()
        moved[m, k] = x[m, k] + 1.0
        step = float(moved[m, k].double() - x[m, k].double())
        mass = (L.w[:, k].abs() @ g[m].double().abs()).item()
        all_mass = ((x.double().abs() + 2) @ L.w.abs().T * g.double().abs()).sum().item()
        bound = BF16 * mass + 2 * sum_eps(128) * all_mass / step
        assert abs((loss(moved) - base) / step - dx[m, k].item()) <= bound


# ---- ans_gemm_lora ---------------------------------------------------------------
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 72, 128])
@pytest.mark.parametrize("M", [1, 17, 290])
def test_lora_of_every_rank(cuda, rank, M):
    L = usual(ans.BF16_SPLIT, 384, 208, seed=rank)
    A = Adapters(L, 5, rank)
    rng = np.random.default_rng([rank, M])
    x, ids = bf16(rng, M, L.K), some_ids(rng, M, 5)
    y, st = run_lora(L, A, x, ids)
    assert st == 0
    within(y, *lora_reference(L, A, x, ids), "y")


@pytest.mark.parametrize("M", [3, 40, 600])
@pytest.mark.parametrize("dtype", ALL)
def test_lora_beside_every_format(cuda, dtype, M):
    L = usual(dtype, 256, 320, seed=M)
    A = Adapters(L, 3, 16, scale=dtype % 2 == 0)
    rng = np.random.default_rng(M)
    x, ids = bf16(rng, M, L.K), some_ids(rng, M, 3)
    y, st = run_lora(L, A, x, ids)
    assert st == 0
    within(y, *lora_reference(L, A, x, ids), "y")


@pytest.mark.parametrize("M,n", [(1, 1), (16, 256), (256, 1), (257, 1), (257, 256), (1500, 200), (4099, 2)])
@pytest.mark.parametrize("K", [16, 2064])
def test_lora_of_many_and_few_adapters(cuda, M, n, K):
    L = usual(ans.BF16_SPLIT, 128, K, seed=M)
    A = Adapters(L, n, 8)
    rng = np.random.default_rng([M, n])
    x, ids = bf16(rng, M, K), some_ids(rng, M, n)
    y, st = run_lora(L, A, x, ids)
    assert st == 0
    within(y, *lora_reference(L, A, x, ids), "y")


@pytest.mark.parametrize("M", [63, 64, 65, 256])
def test_lora_where_the_grouping_changes(cuda, M):
    # one adapter for all, an adapter for each, and every 16th token
    L = usual(ans.INT8, 256, 192, seed=M)
    A = Adapters(L, 64, 16)
    rng = np.random.default_rng(M)
    x = bf16(rng, M, L.K)
    for ids in (torch.full((M,), 5), torch.arange(M) % 64, torch.where(torch.arange(M) % 16 == 3, 63, -1)):
        ids = ids.to(torch.int32)
        y, st = run_lora(L, A, x, ids)
        assert st == 0
        within(y, *lora_reference(L, A, x, ids), "y")


def test_lora_tokens_without_an_adapter_are_the_product_itself(cuda):
    L = usual(ans.INT8, 256, 256, seed=9)
    A = Adapters(L, 4, 16)
    rng = np.random.default_rng(1)
    for M in (5, 100, 700):
        x = bf16(rng, M, 256)
        ws = workspace(ans.ans_gemm_workspace(L.layout, M, L.kind))
        base, st = torch.empty(M, 256, device="cuda"), status()
        ans.ans_gemm(x.cuda(), M, *L.args, base, ws, ws.numel(), st)
        ids = some_ids(rng, M, 4)
        ids[ids == 2] = -7
        y, s = run_lora(L, A, x, ids)
        assert s == 0
        assert torch.equal(y[(ids < 0).cuda()], base[(ids < 0).cuda()])
        y, s = run_lora(L, A, x, torch.full((M,), -1, dtype=torch.int32))
        assert s == 0 and torch.equal(y, base)


def test_an_index_past_the_adapters_is_reported_and_taken_as_none(cuda):
    L = usual(ans.BF16_SPLIT, 128, 128, seed=3)
    A = Adapters(L, 4, 8)
    rng = np.random.default_rng(2)
    x, dy = bf16(rng, 6, 128), bf16(rng, 6, 128)
    ids = torch.tensor([0, 4, 3, 2 ** 31 - 1, -2 ** 31, 1], dtype=torch.int32)
    y, st = run_lora(L, A, x, ids)
    assert st == ans.STATUS_BAD_INDEX
    as_none = torch.where(ids >= 4, -1, ids)
    within(y, *lora_reference(L, A, x, as_none), "y")
    dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
    assert st == ans.STATUS_BAD_INDEX
    for got, ref in zip((dx, da, db), lora_grad_reference(L, A, x, dy, as_none)):
        within(got, *ref)


def test_lora_keeps_infinities_and_nan_to_their_tokens(cuda):
    L = usual(ans.BF16_SPLIT, 128, 128, seed=5)
    A = Adapters(L, 2, 16)
    rng = np.random.default_rng(4)
    x = bf16(rng, 20, 128)
    ids = torch.zeros(20, dtype=torch.int32)
    x[3, 5], x[11, 6] = float("inf"), float("nan")
    y, _ = run_lora(L, A, x, ids)
    good = [i for i in range(20) if i not in (3, 11)]
    want, bound = lora_reference(L, A, x[good], ids[good])
    within(y[good], want, bound, "y")
    assert torch.isnan(y[11]).all()


def test_a_broken_adapter_reaches_its_own_tokens_alone(cuda):
    # infinities in one adapter's A and NaN in another's B, as a slot that was never
    # loaded may hold: the other adapters' tokens and gradients are what they are
    L = usual(ans.BF16_SPLIT, 256, 128, seed=5)
    for M in (40, 300):
        rng = np.random.default_rng(M)
        A = Adapters(L, 4, 16)
        A.a[1], A.b[2] = float("inf"), float("nan")
        A.dev = ans.LoraAdapters(A.a.cuda(), A.b.cuda(), A.s.cuda())
        A.lora = A.dev.lora
        x, dy, ids = bf16(rng, M, 128), bf16(rng, M, 256), some_ids(rng, M, 4)
        good = (ids != 1) & (ids != 2)
        y, st = run_lora(L, A, x, ids)
        assert st == 0
        want, bound = lora_reference(L, A, x, ids)
        within(y.cpu()[good], want[good], bound[good], "y")
        dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
        assert st == 0
        (wx, bx), (wa, ba), (wb, bb) = lora_grad_reference(L, A, x, dy, ids)
        within(dx.cpu()[good], wx[good], bx[good], "dx")
        for i in (0, 3):
            within(da[i], wa[i], ba[i], "da")
            within(db[i], wb[i], bb[i], "db")
        within(da[1], wa[1], ba[1], "da of the adapter whose A is infinite")


# ---- ans_gemm_lora_grad ----------------------------------------------------------
@pytest.mark.parametrize("rank", [8, 16, 24, 40, 72, 104, 128])
@pytest.mark.parametrize("M", [1, 33, 300])
def test_lora_grad_of_every_rank(cuda, rank, M):
    L = usual(ans.BF16_SPLIT, 384, 208, seed=rank)
    A = Adapters(L, 3, rank)
    rng = np.random.default_rng([rank, M])
    x, dy, ids = bf16(rng, M, L.K), bf16(rng, M, L.N, scale=1e-2), some_ids(rng, M, 3)
    dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
    assert st == 0
    for name, got, ref in zip(("dx", "da", "db"), (dx, da, db), lora_grad_reference(L, A, x, dy, ids)):
        within(got, *ref, name)


@pytest.mark.parametrize("dtype", ALL)
def test_lora_grad_beside_every_format(cuda, dtype):
    L = usual(dtype, 512, 320, seed=1)
    A = Adapters(L, 6, 32, scale=dtype % 2 == 0)
    rng = np.random.default_rng(dtype)
    x, dy, ids = bf16(rng, 400, L.K), bf16(rng, 400, L.N, scale=1e-2), some_ids(rng, 400, 6)
    ids[ids == 4] = 5            # an adapter without tokens has gradients of zero
    dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
    assert st == 0
    for name, got, ref in zip(("dx", "da", "db"), (dx, da, db), lora_grad_reference(L, A, x, dy, ids)):
        within(got, *ref, name)
    assert not da[4].any() and not db[4].any()
    # without dX, the adapters' gradients are the same bits
    _, da2, db2, st = run_lora_grad(L, A, x, dy, ids, want_dx=False)
    assert st == 0 and torch.equal(da, da2) and torch.equal(db, db2)


@pytest.mark.parametrize("M,n,N,K", [(1, 256, 128, 16), (2051, 1, 128, 2064), (900, 100, 1152, 16), (128, 2, 2048, 512)])
def test_lora_grad_of_odd_sizes(cuda, M, n, N, K):
    L = usual(ans.BF16_SPLIT, N, K, seed=M)
    A = Adapters(L, n, 16)
    rng = np.random.default_rng([M, n])
    x, dy, ids = bf16(rng, M, K), bf16(rng, M, N, scale=1e-2), some_ids(rng, M, n)
    dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
    assert st == 0
    for name, got, ref in zip(("dx", "da", "db"), (dx, da, db), lora_grad_reference(L, A, x, dy, ids)):
        within(got, *ref, name)


def test_without_tokens_gradients_are_zero_and_the_rest_is_untouched(cuda):
    L = usual(ans.BF16_SPLIT, 128, 128, seed=6)
    A = Adapters(L, 2, 8)
    none = torch.empty(0, dtype=torch.int32)
    _, da, db, st = run_lora_grad(L, A, bf16(np.random.default_rng(0), 0, 128), bf16(np.random.default_rng(0), 0, 128), none)
    assert st == 0 and not da.any() and not db.any()
    y, st = run_lora(L, A, bf16(np.random.default_rng(0), 0, 128), none)
    assert st == 0
    # every token without an adapter: the gradients are written all the same
    ids = torch.full((9,), -1, dtype=torch.int32)
    rng = np.random.default_rng(1)
    x, dy = bf16(rng, 9, 128), bf16(rng, 9, 128)
    dx, da, db, st = run_lora_grad(L, A, x, dy, ids)
    assert st == 0 and not da.any() and not db.any()
    within(dx, *grad_reference(L, dy), "dx")


def test_outputs_end_where_they_end(cuda):
    # guards behind every output keep their bytes
    L = usual(ans.INT8, 384, 208, seed=6)
    A = Adapters(L, 3, 24)
    rng = np.random.default_rng(3)
    for M in (5, 300):
        x, dy, ids = bf16(rng, M, L.K).cuda(), bf16(rng, M, L.N).cuda(), some_ids(rng, M, 3).cuda()

        def guarded(n, dtype):
            t = torch.full((n + 64,), -77.0, dtype=dtype, device="cuda")
            return t, t[:n]
        (y_all, y), (dx_all, dx) = guarded(M * L.N, torch.float32), guarded(M * L.K, torch.bfloat16)
        (da_all, da), (db_all, db) = guarded(A.a.numel(), torch.float32), guarded(A.b.numel(), torch.float32)
        st = status()
        ws = workspace(ans.ans_gemm_lora_workspace(L.layout, M, L.kind, A.lora))
        ans.ans_gemm_lora(x, M, *L.args, A.lora, ids, y, ws, ws.numel(), st)
        size = ans.ans_gemm_lora_grad_workspace(L.layout, M, L.kind, A.lora)
        ws2 = torch.full((size + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        ans.ans_gemm_lora_grad(x, dy, M, *L.args, A.lora, ids, dx, da, db, ws2, size, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        for t in (y_all, dx_all, da_all, db_all):
            assert (t[-64:] == -77.0).all() and not (t[:-64] == -77.0).any()
        assert (ws2[-256:] == 0x5A).all()


def test_results_do_not_depend_on_what_ran_before(cuda):
    # one workspace for calls of different ids and tokens, and again the first
    L = usual(ans.INT4_PAIRS, 512, 256, seed=6)
    A = Adapters(L, 8, 32)
    rng = np.random.default_rng(3)
    M = 333
    ws = workspace(ans.ans_gemm_lora_grad_workspace(L.layout, M, L.kind, A.lora))
    x, dy, ids = bf16(rng, M, L.K), bf16(rng, M, L.N), some_ids(rng, M, 8)
    first = run_lora_grad(L, A, x, dy, ids, ws=ws)
    run_lora_grad(L, A, bf16(rng, M, L.K), bf16(rng, M, L.N), some_ids(rng, M, 3), ws=ws)
    again = run_lora_grad(L, A, x, dy, ids, ws=ws)
    for a, b in zip(first[:3], again[:3]):
        assert torch.equal(a, b)


def test_streams_graphs_and_two_calls_at_once(cuda):
    L = usual(ans.BF16_SPLIT, 1024, 512, seed=2)
    A = Adapters(L, 4, 16)
    rng = np.random.default_rng(5)
    M = 70
    runs = []
    for _ in range(2):
        x, dy, ids = bf16(rng, M, L.K), bf16(rng, M, L.N), some_ids(rng, M, 4)
        want = run_lora(L, A, x, ids)[0], *run_lora_grad(L, A, x, dy, ids)[:3]
        fwd = workspace(ans.ans_gemm_lora_workspace(L.layout, M, L.kind, A.lora))
        bwd = workspace(ans.ans_gemm_lora_grad_workspace(L.layout, M, L.kind, A.lora))
        out = [torch.zeros_like(t) for t in want]
        runs.append((x.cuda(), dy.cuda(), ids.cuda(), fwd, bwd, out, want, status(), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def both(r):
        x, dy, ids, fwd, bwd, out, _, st, stream = r
        ans.ans_gemm_lora(x, M, *L.args, A.lora, ids, out[0], fwd, fwd.numel(), st, stream)
        ans.ans_gemm_lora_grad(x, dy, M, *L.args, A.lora, ids, *out[1:], bwd, bwd.numel(), st, stream)

    def check():
        torch.cuda.synchronize()
        for r in runs:
            assert int(r[7].item()) == 0
            for got, want in zip(r[5], r[6]):
                assert torch.equal(got, want)
                got.zero_()
        torch.cuda.synchronize()
    for _ in range(3):
        for r in runs:
            both(r)
    check()
    graphs = []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=r[8]):
            both(r)
        graphs.append((g, r[8]))
    for _ in range(3):
        for g, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
    check()


def test_a_corrupt_layer_is_reported(cuda):
    L = usual(ans.INT8, 256, 256, seed=2)
    bad = L.layer.h_stream.copy()
    bad[400] ^= 0x20
    broken = ans.CompressedLayer(L.layout, L.layer.codebook, bad, L.layer.h_offsets, L.layer.h_raw)
    dy = bf16(np.random.default_rng(1), 20, 256).cuda()
    dx, st = torch.zeros(20, 256, dtype=torch.bfloat16, device="cuda"), status()
    size = ans.ans_gemm_grad_workspace(L.layout, 20, L.kind)
    ws = workspace(size)
    ans.ans_gemm_grad(dy, 20, broken.tiles, L.kind, L.scales, 0, dx, ws, size, st)
    torch.cuda.synchronize()
    assert int(st.item()) & ans.STATUS_CORRUPT
    offsets = L.layer.h_offsets.copy()
    offsets[2] += 8
    broken = ans.CompressedLayer(L.layout, L.layer.codebook, L.layer.h_stream, offsets, L.layer.h_raw)
    st = status()
    ans.ans_gemm_grad(dy, 20, broken.tiles, L.kind, L.scales, 0, dx, ws, size, st)
    torch.cuda.synchronize()
    assert int(st.item()) & ans.STATUS_BAD_OFFSETS


@pytest.mark.parametrize("dtype", [ans.INT4, ans.BF16_SPLIT, ans.FP8_E4M3])
def test_grad_of_a_layer_of_one_symbol(cuda, dtype):
    N, K = 128, 64
    L = usual(dtype, N, K, seed=1)
    codes = np.full_like(L.codes, {ans.INT4: 0x33, ans.BF16_SPLIT: 0x3F80, ans.FP8_E4M3: 0x38}[dtype])
    layer = ans.CompressedLayer.from_weights(codes.reshape(-1), L.layout)
    value = {ans.INT4: 3.0, ans.BF16_SPLIT: 1.0, ans.FP8_E4M3: 1.0}[dtype]
    L.layer, L.tiles, L.kind, L.scales, L.group_k = layer, layer.tiles, ans.SCALE_NONE, None, 0
    L.w = torch.full((N, K), value, dtype=torch.float64)
    dy = bf16(np.random.default_rng(1), 20, N)
    within(run_grad(L, dy), *grad_reference(L, dy), "dx")
