"""The adapter, gradient and loss operators on compressed layers, as they are measured.

Each case is one pass through one operator of ``rans_decode_gemm_b200.ans``:

  lora       ans_gemm_lora: Y = X W^T + s_a (X A_a^T) B_a^T, a the adapter of each token
  grad       ans_gemm_grad: dX = dY W
  lora_grad  ans_gemm_lora_grad: dX, dA and dB of the first
  xent       ans_xent: loss and log-sum-exp of softmax(X W^T) per token, with dX where asked

With ``own`` false the same values come from elementary torch operations in 32 bits on the
weights' original codes; with ``own`` true the weights are held compressed.
"""
import math

import torch

own = False

# Per format: the tile the weights are coded in, bits a weight as coded, and how scales are held.
FORMATS = {
    "bf16": {"tile": (128, 64), "bits": 10.72, "scales": None},
    "fp8": {"tile": (128, 128), "bits": 6.59, "scales": "row"},
    "int8": {"tile": (128, 64), "bits": 7.30, "scales": "row"},
    "fp4": {"tile": (128, 64), "bits": 3.69, "scales": "row"},
    "int4": {"tile": (256, 64), "bits": 2.45, "scales": "group"},
}
GROUP = 128  # columns of one int4 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of one request through one projection: what a decoding step waits for
        {"name": "lora bf16 4096x4096 m1", "op": "lora", "format": "bf16", "n": 4096, "k": 4096, "m": 1, "adapters": 8, "rank": 16},
        # a decoding batch, a request a token, some without an adapter
        {"name": "lora int8 14336x4096 m32", "op": "lora", "format": "int8", "n": 14336, "k": 4096, "m": 32, "adapters": 16, "rank": 16},
        # prompts of several requests in one pass, ragged
        {"name": "lora int4 28672x8192 m601", "op": "lora", "format": "int4", "n": 28672, "k": 8192, "m": 601, "adapters": 5, "rank": 64},
        # the gradient that leaves a frozen projection: a short batch, and a long one
        {"name": "grad bf16 4096x4096 m200", "op": "grad", "format": "bf16", "n": 4096, "k": 4096, "m": 200},
        {"name": "grad int8 14336x4096 m2048", "op": "grad", "format": "int8", "n": 14336, "k": 4096, "m": 2048},
        # a training step's projection with the adapters of several tenants, in three sizes and formats
        {"name": "lora_grad bf16 4096x4096 m500", "op": "lora_grad", "format": "bf16", "n": 4096, "k": 4096, "m": 500, "adapters": 4, "rank": 16},
        {"name": "lora_grad int4 14336x4096 m2048", "op": "lora_grad", "format": "int4", "n": 14336, "k": 4096, "m": 2048, "adapters": 8, "rank": 32},
        {"name": "lora_grad fp8 4096x14336 m4096", "op": "lora_grad", "format": "fp8", "n": 4096, "k": 14336, "m": 4096, "adapters": 2, "rank": 64},
        # log-probabilities of a decoding batch, and of a document that is scored
        {"name": "xent bf16 32000x4096 m16", "op": "xent", "format": "bf16", "n": 32000, "k": 4096, "m": 16, "vocab": 32000, "with_grad": False},
        {"name": "xent int8 65536x2048 m1000", "op": "xent", "format": "int8", "n": 65536, "k": 2048, "m": 1000, "vocab": 65499, "with_grad": False},
        # the loss of a training step with the gradient of the last hidden states
        {"name": "xent+grad bf16 32000x4096 m2048", "op": "xent", "format": "bf16", "n": 32000, "k": 4096, "m": 2048, "vocab": 32000, "with_grad": True},
        {"name": "xent+grad fp8 131072x4096 m4096", "op": "xent", "format": "fp8", "n": 131072, "k": 4096, "m": 4096, "vocab": 130001, "with_grad": True},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["lora", "grad", "lora_grad", "xent"])
    fmt = rng.choice(sorted(FORMATS))
    step = FORMATS[fmt]["tile"][0]
    n = step * _log_uniform(rng, 2, (65536 if op == "xent" else 28672) // step)
    k = 128 * _log_uniform(rng, 4, min(112, 120_000_000 // n // 128))
    m = _log_uniform(rng, 1, 4096)
    case = {"op": op, "format": fmt, "n": n, "k": k, "m": m}
    if op.startswith("lora"):
        case |= {"adapters": rng.randint(1, 24), "rank": 8 * _log_uniform(rng, 1, 16)}
    if op == "xent":
        case |= {"vocab": n - rng.randint(0, 127), "with_grad": rng.random() < 0.5}
    return case


# ---- inputs ----------------------------------------------------------------------------
def _weights(fmt, n, k, g):
    """Codes in the format's storage and their scales, drawn as a trained layer's are."""
    if fmt == "int4":
        u = torch.rand(n, k, generator=g, device="cuda") - 0.5
        codes = (-0.9 * u.sign() * (1 - 2 * u.abs()).clamp_min(1e-7).log()).round().clamp(-8, 7).to(torch.int8)
        scales = (0.003 + 0.027 * torch.rand(n, k // GROUP, generator=g, device="cuda")).bfloat16()
        low = codes.view(torch.uint8) & 15
        return low[:, 0::2] | (low[:, 1::2] << 4), scales
    w = torch.randn(n, k, generator=g, device="cuda").mul_(0.02)
    if fmt == "bf16":
        return w.bfloat16(), None
    top = w.abs().amax(dim=1)
    if fmt == "fp8":
        s = top / 448
        return (w / s[:, None]).to(torch.float8_e4m3fn), s
    if fmt == "int8":
        s = top / 127
        return (w / s[:, None]).round().clamp(-127, 127).to(torch.int8), s
    s = top / 6
    grid = torch.tensor(E2M1, device="cuda")
    code = torch.bucketize((w / s[:, None]).abs(), (grid[1:] + grid[:-1]) / 2).to(torch.uint8)
    code = torch.where((w < 0) & (code > 0), code | 8, code)
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def _requests(case, g):
    """The adapter of every token: runs of a request each, -1 for those without one."""
    m, count = case["m"], case["adapters"]
    each = 1 if m <= 64 else max(1, m // (2 * count))
    of_run = torch.randint(-1, count, (m,), generator=g, device="cuda", dtype=torch.int32)
    starts = torch.rand(m, generator=g, device="cuda") < 1.0 / each
    return of_run[starts.long().cumsum(0).clamp_max(m - 1)].contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, fmt, n, k, m = case["op"], case["format"], case["n"], case["k"], case["m"]
    codes, scales = _weights(fmt, n, k, g)
    s = {"case": dict(case), "codes": codes, "scales": scales}
    x = torch.randn(m, k, generator=g, device="cuda")
    if op == "xent":
        # hidden states that lean towards their next token, some much, some not; a few tokens are
        # padding, which has no target
        targets = torch.randint(0, case["vocab"], (m,), generator=g, device="cuda", dtype=torch.int32)
        rows = _values(s, targets.long())
        lean = 10 * torch.rand(m, 1, generator=g, device="cuda")
        x += lean * rows / rows.norm(dim=1, keepdim=True)
        left_out = torch.rand(m, generator=g, device="cuda") < (0.05 if m > 1 else 0.0)
        s["targets"] = torch.where(left_out, torch.full_like(targets, -1), targets)
        s["weight"] = (s["targets"] >= 0).float() / (s["targets"] >= 0).sum().clamp_min(1)
    if op in ("grad", "lora_grad"):
        size = 1e-3 * torch.exp(torch.randn(m, 1, generator=g, device="cuda"))
        s["dy"] = (size * torch.randn(m, n, generator=g, device="cuda")).bfloat16()
    if op.startswith("lora"):
        count, rank = case["adapters"], case["rank"]
        s["a"] = (torch.randn(count, rank, k, generator=g, device="cuda") / math.sqrt(k)).bfloat16()
        s["b"] = (0.02 * torch.randn(count, n, rank, generator=g, device="cuda")).bfloat16()
        s["alpha"] = 0.5 + 1.5 * torch.rand(count, generator=g, device="cuda")
        s["ids"] = _requests(case, g)
    s["x"] = x.bfloat16()
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a user's program keeps for the calls: the compressed layer, the adapters' plan, a
    workspace, a status word and the output buffers."""
    import numpy as np

    from rans_decode_gemm_b200 import ans

    c = s["case"]
    op, fmt, n, k, m = c["op"], c["format"], c["n"], c["k"], c["m"]
    kind = {"bf16": ans.BF16_SPLIT, "fp8": ans.FP8_E4M3, "int8": ans.INT8, "fp4": ans.FP4_PAIRS, "int4": ans.INT4_PAIRS}[fmt]
    layout = ans.make_layout(kind, n, k, *FORMATS[fmt]["tile"], 64)
    host = s.pop("codes").view(torch.int16 if fmt == "bf16" else torch.uint8).reshape(-1).cpu().numpy()
    s["layer"] = ans.CompressedLayer.from_weights(host.view(np.uint16) if fmt == "bf16" else host, layout)
    s["kind"] = {None: ans.SCALE_NONE, "row": ans.SCALE_ROW_F32, "group": ans.SCALE_GROUP_BF16}[FORMATS[fmt]["scales"]]
    s["group"] = GROUP if fmt == "int4" else 0
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op.startswith("lora"):
        s["lora"] = ans.LoraAdapters(s["a"], s["b"], s["alpha"])
    if op == "lora":
        size = ans.ans_gemm_lora_workspace(layout, m, s["kind"], s["lora"].lora)
        s["y"] = new(m, n)
    elif op == "grad":
        size = ans.ans_gemm_grad_workspace(layout, m, s["kind"])
        s["dx"] = new(m, k, dtype=torch.bfloat16)
    elif op == "lora_grad":
        size = ans.ans_gemm_lora_grad_workspace(layout, m, s["kind"], s["lora"].lora)
        s["dx"], s["da"], s["db"] = new(m, k, dtype=torch.bfloat16), new(*s["a"].shape), new(*s["b"].shape)
    else:
        size = ans.ans_xent_workspace(layout, m, s["kind"], c["with_grad"])
        s["loss"], s["lse"] = new(m), new(m)
        s["dx"] = new(m, k, dtype=torch.bfloat16) if c["with_grad"] else None
    s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- one pass --------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from rans_decode_gemm_b200 import ans

    c, w = s["case"], (s["layer"].tiles, s["kind"], s["scales"], s["group"])
    rest = (s["ws"], s["ws"].numel(), s["status"])
    if c["op"] == "lora":
        ans.ans_gemm_lora(s["x"], c["m"], *w, s["lora"].lora, s["ids"], s["y"], *rest)
        return {"y": s["y"]}
    if c["op"] == "grad":
        ans.ans_gemm_grad(s["dy"], c["m"], *w, s["dx"], *rest)
        return {"dx": s["dx"]}
    if c["op"] == "lora_grad":
        ans.ans_gemm_lora_grad(s["x"], s["dy"], c["m"], *w, s["lora"].lora, s["ids"], s["dx"], s["da"], s["db"], *rest)
        return {"dx": s["dx"], "da": s["da"], "db": s["db"]}
    ans.ans_xent(s["x"], c["m"], *w, c["vocab"], s["targets"], s["loss"], s["lse"], s["weight"] if c["with_grad"] else None, s["dx"], *rest)
    return {"loss": s["loss"], "lse": s["lse"]} | ({"dx": s["dx"]} if c["with_grad"] else {})


def _values(s, rows=None, dtype=torch.float32):
    """The weights' values, of all rows or of those asked for."""
    fmt, codes, scales = s["case"]["format"], s["codes"], s["scales"]
    if rows is not None:
        codes = codes.view(torch.uint8)[rows].view(codes.dtype) if fmt == "fp8" else codes[rows]
        scales = None if scales is None else scales[rows]
    if fmt in ("int4", "fp4"):
        nibbles = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(1)
        if fmt == "int4":
            values = nibbles.to(dtype)
            values = values - 16 * (values > 7)
            return values * scales.to(dtype).repeat_interleave(GROUP, dim=1)
        grid = torch.tensor([*E2M1, *(-v for v in E2M1)], dtype=dtype, device="cuda")
        return grid[nibbles.int()] * scales.to(dtype)[:, None]
    values = codes.to(dtype)
    return values if scales is None else values * scales.to(dtype)[:, None]


def _run_plain(s):
    c, x, w = s["case"], s["x"].float(), _values(s)
    if c["op"] == "grad":
        return {"dx": (s["dy"].float() @ w).bfloat16()}
    if c["op"] == "xent":
        return _xent_plain(c, s, x, w)
    # every token meets every adapter, and its own is kept
    count, rank = c["adapters"], c["rank"]
    mine = torch.arange(count, device="cuda")[None, :] == s["ids"][:, None]
    mine = (mine * s["alpha"][None, :]).repeat_interleave(rank, dim=1)
    a = s["a"].float().flatten(0, 1)
    b = s["b"].float().transpose(1, 2).reshape(count * rank, c["n"])
    h = (x @ a.T) * mine
    if c["op"] == "lora":
        return {"y": x @ w.T + h @ b}
    dy = s["dy"].float()
    dh = (dy @ b.T) * mine
    return {
        "dx": (dy @ w + dh @ a).bfloat16(),
        "da": (dh.T @ x).reshape(count, rank, c["k"]),
        "db": (h.T @ dy).reshape(count, rank, c["n"]).transpose(1, 2).contiguous(),
    }


def _xent_plain(c, s, x, w):
    w = w[: c["vocab"]]
    z = x @ w.T
    top = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (total.log() + top)[:, 0]
    has = s["targets"] >= 0
    at = s["targets"].clamp_min(0).long()[:, None]
    out = {"loss": torch.where(has, lse - z.gather(1, at)[:, 0], 0.0), "lse": lse}
    if c["with_grad"]:
        e /= total
        # p - 1 of the target, from what the others hold: 1 - p loses it where p is near 1
        others = e.scatter(1, at, 0.0)
        p = others.scatter(1, at, -others.sum(dim=1, keepdim=True))
        out["dx"] = ((p * s["weight"][:, None]) @ w).bfloat16()
    return out


# ---- the floor of a pass ---------------------------------------------------------------
def work(case):
    n, k, m = case["n"], case["k"], case["m"]
    weights = n * k * FORMATS[case["format"]]["bits"] / 8
    weights += {None: 0, "row": 4 * n, "group": 2 * n * k / GROUP}[FORMATS[case["format"]]["scales"]]
    product = 2 * m * n * k
    if case["op"] == "grad":
        return {"bytes": weights + 2 * m * n + 2 * m * k, "flops": product}
    if case["op"] == "xent":
        grad = case["with_grad"]
        return {"bytes": weights + 2 * m * k + 12 * m + (2 * m * k + 4 * m if grad else 0), "flops": product * (2 if grad else 1)}
    # a decoding batch may not meet every adapter
    used, rank = min(case["adapters"], m), case["rank"]
    adapters = 2 * used * rank * (n + k)
    if case["op"] == "lora":
        return {"bytes": weights + adapters + 2 * m * k + 4 * m * n + 4 * m, "flops": product + 2 * m * rank * (n + k)}
    grads = 4 * case["adapters"] * rank * (n + k)
    return {"bytes": weights + adapters + grads + 4 * m * k + 2 * m * n + 4 * m, "flops": product + 6 * m * rank * (n + k)}


# ---- the same values in 64 bits, from the definitions ----------------------------------
def _blocks(s):
    """Row blocks of the weights in 64 bits."""
    n, step = s["case"]["n"], 4096
    for r in range(0, n, step):
        yield r, _values(s, torch.arange(r, min(n, r + step), device="cuda"), torch.float64)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_xent(s) if case["op"] == "xent" else _exact_linear(s)


def _exact_linear(s):
    c, x = s["case"], s["x"].double()
    op, n, m = c["op"], c["n"], c["m"]
    y, dx = torch.zeros(m, n, dtype=torch.float64, device="cuda"), torch.zeros_like(x)
    dy = s["dy"].double() if op != "lora" else None
    for r, w in _blocks(s):
        if op == "lora":
            y[:, r:r + len(w)] = torch.einsum("mk,nk->mn", x, w)
        else:
            dx += torch.einsum("mn,nk->mk", dy[:, r:r + len(w)], w)
    if op == "grad":
        return {"dx": dx}
    da = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    for i in range(c["adapters"]):
        at = (s["ids"] == i).nonzero()[:, 0]
        a, b, alpha = s["a"][i].double(), s["b"][i].double(), s["alpha"][i].double()
        if op == "lora":
            y[at] += alpha * torch.einsum("mr,nr->mn", torch.einsum("mk,rk->mr", x[at], a), b)
        else:
            back = alpha * torch.einsum("mn,nr->mr", dy[at], b)
            dx[at] += torch.einsum("mr,rk->mk", back, a)
            da[i] = torch.einsum("mr,mk->rk", back, x[at])
            db[i] = alpha * torch.einsum("mn,mr->nr", dy[at], torch.einsum("mk,rk->mr", x[at], a))
    return {"y": y} if op == "lora" else {"dx": dx, "da": da, "db": db}


def _exact_xent(s):
    c, x = s["case"], s["x"].double()
    vocab, targets = c["vocab"], s["targets"].long()
    has = targets >= 0
    parts = []
    for r, w in _blocks(s):
        parts.append(torch.logsumexp(x @ w[: max(0, vocab - r)].T, dim=1))
    lse = torch.logsumexp(torch.stack(parts), dim=0)
    aim = _values(s, targets.clamp_min(0), torch.float64)
    z = (x * aim).sum(dim=1)
    out = {"loss": torch.where(has, lse - z, 0.0), "lse": lse}
    if c["with_grad"]:
        dx, rest = torch.zeros_like(x), torch.zeros_like(lse)
        for r, w in _blocks(s):
            w = w[: max(0, vocab - r)]
            p = torch.exp(x @ w.T - lse[:, None])
            p[torch.arange(r, r + len(w), device="cuda")[None, :] == targets[:, None]] = 0
            rest += p.sum(dim=1)
            dx += p @ w
        out["dx"] = s["weight"].double()[:, None] * (dx - rest[:, None] * aim)
    return out
