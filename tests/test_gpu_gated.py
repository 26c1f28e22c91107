"""ans_gated and ans_gated_grad against the definition in 64 bits.

Bounds.  G and U are fp32 sums of exact products (sum_eps of the sum of magnitudes; X in f16 may
lose 2^-25 of the largest of a row).  Every activation's first two derivatives are below 1.2 and
0.9 in magnitude, so that an error of G enters act(G) and act'(G) at most 1.2 and 0.9 times; the
activations' own evaluation is right to 2^-18 of the value (of 1, for derivatives).  Results are
rounded to bf16 once."""
import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

from _ops_util import ALL, BF16, Layer, bf16, status, sum_eps, usual, within, workspace

pytestmark = pytest.mark.gpu

ACTS = {
    ans.ACT_SILU: torch.nn.functional.silu,
    ans.ACT_GELU: torch.nn.functional.gelu,
    ans.ACT_GELU_TANH: lambda g: torch.nn.functional.gelu(g, approximate="tanh"),
    ans.ACT_RELU: torch.nn.functional.relu,
}


class Block:
    """A gate and an up layer of one layout."""

    def __init__(self, dtype, N, K, seed=0, **kw):
        self.gate, self.up = usual(dtype, N, K, 2 * seed, **kw), usual(dtype, N, K, 2 * seed + 1, **kw)
        self.N, self.K, self.layout, self.kind = N, K, self.gate.layout, self.gate.kind

    def args(self, act):
        return (self.gate.tiles, self.up.tiles, self.kind, self.gate.scales, self.up.scales, self.gate.group_k, act)


def products(B, x):
    """G, U and bounds of their fp32 values."""
    x64 = x.double()
    loss = 2.0 ** -25 * x64.abs().amax(1, keepdim=True)
    out = []
    for w in (B.gate.w, B.up.w):
        out += [x64 @ w.T, sum_eps(B.K) * (x64.abs() @ w.abs().T) + loss * w.abs().sum(1)[None, :]]
    return out


def forward_reference(B, x, act):
    g, ge, u, ue = products(B, x)
    a = ACTS[act](g)
    h = a * u
    ae = 1.2 * ge + 2.0 ** -18 * a.abs()
    inner = ae * u.abs() + a.abs() * ue + ae * ue + 2.0 ** -23 * h.abs()
    return h, inner + BF16 * (h.abs() + inner)


def run_forward(B, x, act, stream=None):
    M = len(x)
    size = ans.ans_gated_workspace(B.layout, M, B.kind)
    h = torch.full((M + 1, B.N), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = status()
    ans.ans_gated(x.cuda(), M, *B.args(act), h, workspace(size), size, st, stream)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.isnan(h[M:]).all()
    return h[:M]


def run_grad(B, x, dh, act, with_dx=True):
    M = len(x)
    size = ans.ans_gated_grad_workspace(B.layout, M, B.kind)
    dx = torch.full((M + 1, B.K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg, du = (torch.full((M + 1, B.N), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st = status()
    ans.ans_gated_grad(x.cuda(), dh.cuda(), M, *B.args(act), dx if with_dx else None, dg, du, workspace(size), size, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and all(torch.isnan(t[M:]).all() for t in (dx, dg, du))
    return (dx[:M] if with_dx else None), dg[:M], du[:M]


def check_grad(B, x, dh, act):
    dx, dg, du = run_grad(B, x, dh, act)
    g, ge, u, ue = products(B, x)
    d = dh.double()
    leaf_g, leaf_u = g.clone().requires_grad_(), u.clone().requires_grad_()
    want_g, want_u = torch.autograd.grad(ACTS[act](leaf_g) * leaf_u, (leaf_g, leaf_u), d)
    a = ACTS[act](g)
    slope_e = 0.9 * ge + 2.0 ** -18
    if act == ans.ACT_RELU:
        slope_e = torch.where(g.abs() <= ge, 1.0, slope_e)
    ig = d.abs() * ((1.2 + slope_e) * ue + slope_e * u.abs()) + 2.0 ** -22 * want_g.abs()
    iu = d.abs() * (1.2 * ge + 2.0 ** -18 * a.abs()) + 2.0 ** -22 * want_u.abs()
    # (bf16 values below its normal range keep fewer bits)
    bg = ig + BF16 * (want_g.abs() + ig) + 2.0 ** -133
    bu = iu + BF16 * (want_u.abs() + iu) + 2.0 ** -133
    within(dg, want_g, bg, "dg")
    within(du, want_u, bu, "du")
    wg, wu = B.gate.w, B.up.w
    if B.gate.dtype == ans.BF16_SPLIT:
        # dX of dG and dU as they came back, or, under row scales, of those times the scales, rounded once
        g64, u64 = dg.cpu().double(), du.cpu().double()
        eg, eu, eps = 0.0, 0.0, 0.0
        if B.kind != ans.SCALE_NONE:
            g64, u64, eg, eu, eps = want_g, want_u, ig, iu, BF16
        floor = 0.0
    else:
        # of the values before they are rounded, in f16 under the token's bound: 11 bits, and 2^-25 of
        # the unit below its normal range, 2^-39 of the bound (2^-38: its power of two)
        g64, u64, eg, eu, eps = want_g, want_u, ig, iu, 2.0 ** -11
        code = {ans.INT8: 128, ans.FP8_E4M3: 448, ans.INT4: 8, ans.INT4_PAIRS: 8}.get(B.gate.dtype, 6)
        rowed = B.kind in (ans.SCALE_ROW_BF16, ans.SCALE_ROW_F32)
        tops = [1.0 if L.scales is None else L.scales.double().max().item() for L in (B.gate, B.up)]
        bound = 1.14 * d.abs().amax(1) * x.double().norm(dim=1) * B.K ** 0.5 * code * max(tops) ** (2 if rowed else 1)
        codes = [L.w.abs() / (L.scales.cpu().double()[:, None] if rowed else 1.0) for L in (B.gate, B.up)]
        floor = 2.0 ** -38 * bound[:, None] * (codes[0].sum(0) + codes[1].sum(0))[None, :]
    mass = g64.abs() @ wg.abs() + u64.abs() @ wu.abs()
    inner = (eps + sum_eps(2 * B.N)) * mass + floor
    if B.gate.dtype != ans.BF16_SPLIT or B.kind != ans.SCALE_NONE:
        inner = inner + (1 + eps) * (eg @ wg.abs() + eu @ wu.abs())
    want = g64 @ wg + u64 @ wu
    within(dx, want, inner + BF16 * (want.abs() + inner) + 2.0 ** -133, "dx")
    # and, beside weights in bf16, of the formula's own
    want = want_g @ wg + want_u @ wu
    inner = inner + bg @ wg.abs() + bu @ wu.abs()
    within(dx, want, inner + BF16 * (want.abs() + inner) + 2.0 ** -133, "dx of exact dG and dU")


def inputs(B, M, seed, size=1.0):
    rng = np.random.default_rng([seed, M, B.N, B.K])
    return bf16(rng, M, B.K, scale=size), bf16(rng, M, B.N, scale=0.01)


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("M", [1, 17, 40, 130])
def test_every_format(cuda, dtype, M):
    B = Block(dtype, 256, 192, seed=dtype)
    x, dh = inputs(B, M, dtype)
    for act in (ans.ACT_SILU, ans.ACT_GELU):
        within(run_forward(B, x, act), *forward_reference(B, x, act), f"h {act}")
        check_grad(B, x, dh, act)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,N,K", [(ans.BF16_SPLIT, 128, 16), (ans.INT8, 384, 80), (ans.FP8_E4M3, 640, 208),
                                       (ans.INT4_PAIRS, 512, 1024)])
def test_shapes(cuda, act, dtype, N, K):
    B = Block(dtype, N, K, seed=3)
    for M in (2, 16, 32, 33, 64, 127, 129, 257):
        x, dh = inputs(B, M, act)
        within(run_forward(B, x, act), *forward_reference(B, x, act), f"h M {M}")
        if M in (2, 33, 129):
            check_grad(B, x, dh, act)


@pytest.mark.parametrize("state_bits", [32, 64])
@pytest.mark.parametrize("dtype,kind,group", [(ans.BF16_SPLIT, ans.SCALE_ROW_BF16, 0), (ans.BF16_SPLIT, ans.SCALE_ROW_F32, 0),
                                              (ans.INT4, ans.SCALE_GROUP_BF16, 64), (ans.INT8, ans.SCALE_NONE, 0),
                                              (ans.FP4_PAIRS, ans.SCALE_ROW_BF16, 0), (ans.INT4_PAIRS, ans.SCALE_ROW_F32, 0)])
def test_scales_and_streams(cuda, dtype, kind, group, state_bits):
    B = Block(ans.BF16_SPLIT, 128, 128)
    tile = 256 if group else 128
    B.gate, B.up = (Layer(dtype, 512, 128, tile, 64, kind, group, seed, state_bits) for seed in (0, 1))
    B.N, B.K, B.layout, B.kind = 512, 128, B.gate.layout, kind
    size = 0.01 if kind == ans.SCALE_NONE else 1.0
    for M in (5, 70):
        x, dh = inputs(B, M, 1, size)
        within(run_forward(B, x, ans.ACT_SILU), *forward_reference(B, x, ans.ACT_SILU), "h")
        check_grad(B, x, dh, ans.ACT_SILU)


def test_rounds_of_tiles(cuda):
    """More tiles than SMs, and sums of several ranges."""
    B = Block(ans.BF16_SPLIT, 1280, 512)
    for M in (1100, 2500):
        x, dh = inputs(B, M, 0)
        within(run_forward(B, x, ans.ACT_GELU_TANH), *forward_reference(B, x, ans.ACT_GELU_TANH), "h")
        check_grad(B, x, dh, ans.ACT_GELU_TANH)


def test_same_bits_and_without_dx(cuda):
    B = Block(ans.INT8, 512, 256)
    for M in (8, 200):
        x, dh = inputs(B, M, 2)
        assert torch.equal(run_forward(B, x, ans.ACT_SILU), run_forward(B, x, ans.ACT_SILU))
        a, b = run_grad(B, x, dh, ans.ACT_SILU), run_grad(B, x, dh, ans.ACT_SILU, with_dx=False)
        assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
        assert all(torch.equal(p, q) for p, q in zip(a, run_grad(B, x, dh, ans.ACT_SILU)))


def test_large_and_small_values(cuda):
    """Saturated activations: far to either side, at 0, and gradients of every size."""
    B = Block(ans.BF16_SPLIT, 256, 128)
    for size in (1e-6, 30.0, 1000.0):
        for M in (9, 60):
            x, dh = inputs(B, M, 5, size)
            x[1] = 0
            dh[0] *= 1e-20
            dh[2] *= 1e10
            for act in ACTS:
                g, ge, u, ue = products(B, x)
                h = run_forward(B, x, act)
                want, bound = forward_reference(B, x, act)
                within(h, want, bound + 2.0 ** -100, f"h {size} {act}")
                # where a wide G passes through the activations' knees, its error is a value's
                if size < 100:
                    check_grad(B, x, dh, act)
                else:
                    assert all(torch.isfinite(t).all() for t in run_grad(B, x, dh, act))


@pytest.mark.parametrize("M", [6, 50])
def test_slopes_far_out(cuda, M):
    """G of 1e13 to 1e20 either way: the activations are g or 0 there, and their slopes 1 or 0."""
    B = Block(ans.BF16_SPLIT, 128, 16, seed=9)
    x, dh = inputs(B, M, 9)
    for size in (1e15, 1e18, 1e20):
        big = (x.float() * size).bfloat16()
        small = (dh.float() * 1e-20).bfloat16()
        for act in ACTS:
            _, dg, du = run_grad(B, big, small, act)
            g, u = big.double() @ B.gate.w.T, big.double() @ B.up.w.T
            d = small.double()
            clear = g.abs() > size * 0.02   # (away from 0, whose slopes are between)
            rel = 2 * BF16
            for got, want in ((dg, torch.where(g > 0, d * u, 0.0)), (du, torch.where(g > 0, d * g, 0.0))):
                got = got.cpu().double()
                assert torch.isfinite(got).all()
                off = (got - want).abs()
                # G and U: fp32 sums of 16 products
                assert (off <= rel * want.abs() + d.abs() * size * 2.0 ** -16)[clear].all()


@pytest.mark.parametrize("M", [6, 50])
def test_not_finite_stays_with_its_token(cuda, M):
    B = Block(ans.FP8_E4M3, 256, 128)
    x, dh = inputs(B, M, 6)
    h = run_forward(B, x, ans.ACT_SILU)
    dx, dg, du = run_grad(B, x, dh, ans.ACT_SILU)
    x2, dh2 = x.clone(), dh.clone()
    x2[3, 5] = float("nan")
    x2[4, 7] = float("inf")
    dh2[1, 9] = float("inf")
    h2 = run_forward(B, x2, ans.ACT_SILU)
    dx2, dg2, du2 = run_grad(B, x2, dh2, ans.ACT_SILU)
    rest = [m for m in range(M) if m not in (3, 4)]
    assert torch.equal(h[rest], h2[rest]) and torch.isnan(h2[3]).all()
    rest = [m for m in range(M) if m not in (1, 3, 4)]
    for a, b in ((dx, dx2), (dg, dg2), (du, du2)):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(dg2[3]).all() and torch.isinf(du2[1, 9])
    keep = [n for n in range(256) if n != 9]
    assert torch.equal(du[1, keep], du2[1, keep])


def test_gradient_against_differences(cuda):
    """d(sum(dH * H)) along a direction of X, by differences of the 64-bit definition, against dX."""
    B = Block(ans.BF16_SPLIT, 256, 64, seed=1)
    x, dh = inputs(B, 40, 7)
    for act in (ans.ACT_SILU, ans.ACT_GELU, ans.ACT_GELU_TANH):
        dx = run_grad(B, x, dh, act)[0].cpu().double()
        v = torch.from_numpy(np.random.default_rng(1).standard_normal(x.shape))
        f = lambda t: (dh.double() * ACTS[act](t @ B.gate.w.T) * (t @ B.up.w.T)).sum()  # noqa: E731
        step = 1e-5
        slope = ((f(x.double() + step * v) - f(x.double() - step * v)) / (2 * step)).item()
        got = (dx * v).sum().item()
        # dX is off by 2^-8 of itself and of dG and dU, independently: a sum of 40 x 64 such
        size = (dx.abs() * v.abs()).sum().item()
        assert abs(got - slope) <= 4 * BF16 * size


def test_one_workspace_call_after_call_streams_and_capture(cuda):
    B = Block(ans.INT4_PAIRS, 512, 256)
    for M in (4, 90):
        size = max(ans.ans_gated_workspace(B.layout, M, B.kind), 1)
        ws, st = workspace(size), status()
        gsize = ans.ans_gated_grad_workspace(B.layout, M, B.kind)
        gws = workspace(gsize)
        x, dh = (t.cuda() for t in inputs(B, M, 8))
        h = torch.empty(M, B.N, dtype=torch.bfloat16, device="cuda")
        dx = torch.empty(M, B.K, dtype=torch.bfloat16, device="cuda")
        dg, du = torch.empty_like(h), torch.empty_like(h)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()

        def call():
            ans.ans_gated(x, M, *B.args(ans.ACT_SILU), h, ws, size, st)
            ans.ans_gated_grad(x, dh, M, *B.args(ans.ACT_SILU), dx, dg, du, gws, gsize, st)
        with torch.cuda.stream(side):
            for _ in range(3):
                call()
            graph.capture_begin()
            call()
            graph.capture_end()
        for seed in (1, 2, 3):
            nx, nd = inputs(B, M, 80 + seed)
            x.copy_(nx)
            dh.copy_(nd)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert int(st.item()) == 0
            assert torch.equal(h, run_forward(B, nx, ans.ACT_SILU))
            a = run_grad(B, nx, nd, ans.ACT_SILU)
            assert torch.equal(dx, a[0]) and torch.equal(dg, a[1]) and torch.equal(du, a[2])


def test_with_the_down_projection_and_adapters(cuda):
    """A block as it is used: H into the down projection; back through it, and into the gate's adapters."""
    N, K, M, rank = 512, 256, 60, 8
    B = Block(ans.INT8, N, K, seed=2)
    down = usual(ans.INT8, K, N, seed=9)
    rng = np.random.default_rng(12)
    x, dy = bf16(rng, M, K), bf16(rng, M, K, scale=0.01)
    A = ans.LoraAdapters(bf16(rng, 2, rank, K).cuda(), bf16(rng, 2, N, rank).cuda())
    ids = torch.from_numpy(rng.integers(-1, 2, M).astype(np.int32)).cuda()
    st = status()
    h = run_forward(B, x, ans.ACT_SILU)
    y = torch.empty(M, K, device="cuda")
    size = ans.ans_gemm_workspace(down.layout, M, down.kind)
    ans.ans_gemm(h, M, down.tiles, down.kind, down.scales, down.group_k, y, workspace(size), size, st)
    dh = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    size = ans.ans_gemm_grad_workspace(down.layout, M, down.kind)
    ans.ans_gemm_grad(dy.cuda(), M, *down.args, dh, workspace(size), size, st)
    dx, dg, du = run_grad(B, x, dh.cpu(), ans.ACT_SILU)
    da = torch.empty(2, rank, K, device="cuda")
    db = torch.empty(2, N, rank, device="cuda")
    size = ans.ans_gemm_lora_grad_workspace(B.layout, M, B.kind, A.lora)
    ans.ans_gemm_lora_grad(x.cuda(), dg, M, *B.gate.args, A.lora, ids, None, da, db, workspace(size), size, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # the same in 64 bits; every stage rounds to bf16 (2^-9 of a value on average less), three in a row
    leaf = x.double().requires_grad_()
    hh = ACTS[ans.ACT_SILU](leaf @ B.gate.w.T) * (leaf @ B.up.w.T)
    yy = hh @ down.w.T
    (want_dx,) = torch.autograd.grad(yy, leaf, dy.double())
    rel = lambda a, b: ((a.cpu().double() - b).norm() / b.norm()).item()  # noqa: E731
    assert rel(y, yy.detach()) <= BF16
    assert rel(dx, want_dx) <= 3 * BF16
    g64 = dg.cpu().double()
    for a in range(2):
        at = (ids.cpu() == a).nonzero()[:, 0]
        dh_a = g64[at] @ A.B[a].cpu().double()
        assert rel(da[a], dh_a.T @ x.double()[at]) <= 2.0 ** -12
