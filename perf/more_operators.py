"""The gated block, distillation and draft verification, as they are measured.

Each case is one pass through one operator of ``rans_decode_gemm_b200.ans``:

  gated       ans_gated: H = act(X Wg^T) * (X Wu^T), both projections compressed
  gated_grad  ans_gated_grad: dX, and the gradients dG and dU that reach the projections
  distill     ans_distill: KL divergence from a teacher's top logits to softmax(X W^T / T) of
              a compressed vocabulary head per token, with dX where asked
  verify      ans_verify: which drafted tokens the target's logits accept, and the token that
              follows them

With ``own`` false the same values come from elementary torch operations on the weights'
original codes; with ``own`` true the weights are held compressed.
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
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def listed():
    return [
        # one token through a block's gate and up projections: what a decoding step waits for
        {"name": "gated bf16 14336x4096 m1", "op": "gated", "format": "bf16", "n": 14336, "k": 4096, "m": 1, "act": "silu"},
        # a decoding batch
        {"name": "gated int8 14336x4096 m24", "op": "gated", "format": "int8", "n": 14336, "k": 4096, "m": 24, "act": "silu"},
        # a short prompt, ragged
        {"name": "gated int4 14336x4096 m301", "op": "gated", "format": "int4", "n": 14336, "k": 4096, "m": 301, "act": "gelu_tanh"},
        # a long prompt, or the forward pass of a training step
        {"name": "gated fp8 14336x4096 m2048", "op": "gated", "format": "fp8", "n": 14336, "k": 4096, "m": 2048, "act": "silu"},
        # the backward pass through a frozen block: a short batch of a small model, and a long one
        {"name": "gated_grad bf16 4096x4096 m200", "op": "gated_grad", "format": "bf16", "n": 4096, "k": 4096, "m": 200, "act": "gelu"},
        {"name": "gated_grad int8 14336x4096 m2048", "op": "gated_grad", "format": "int8", "n": 14336, "k": 4096, "m": 2048, "act": "silu"},
        # how far a batch of a draft model's tokens is from its teacher
        {"name": "distill bf16 32000x4096 m16 top8", "op": "distill", "format": "bf16", "n": 32000, "k": 4096, "m": 16, "vocab": 32000, "top": 8, "rest": False, "temperature": 1.0, "with_grad": False},
        # training steps of a draft model: many listed logits, all the teacher's mass on them
        {"name": "distill+grad bf16 32000x4096 m2048 top64", "op": "distill", "format": "bf16", "n": 32000, "k": 4096, "m": 2048, "vocab": 32000, "top": 64, "rest": False, "temperature": 2.0, "with_grad": True},
        # a large vocabulary, few listed logits, some of the mass elsewhere
        {"name": "distill+grad fp8 65536x4096 m3001 top20", "op": "distill", "format": "fp8", "n": 65536, "k": 4096, "m": 3001, "vocab": 65499, "top": 20, "rest": True, "temperature": 1.0, "with_grad": True},
        # one user's drafted tokens
        {"name": "verify 1x5 of 32000", "op": "verify", "seqs": 1, "drafted": 5, "vocab": 32000, "stride": 32000},
        # a batch without a draft model's logits: drafts looked up in the prompt
        {"name": "verify 16x4 of 65499, looked up", "op": "verify", "seqs": 16, "drafted": 4, "vocab": 65499, "stride": 65536, "looked_up": True},
        # a large batch of a large vocabulary
        {"name": "verify 64x8 of 130001", "op": "verify", "seqs": 64, "drafted": 8, "vocab": 130001, "stride": 131072},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["gated", "gated_grad", "distill", "verify"])
    if op == "verify":
        vocab = _log_uniform(rng, 1000, 131072)
        return {"op": op, "seqs": _log_uniform(rng, 1, 64), "drafted": rng.randint(1, 8), "vocab": vocab,
                "stride": vocab + rng.randint(0, 127), "looked_up": rng.random() < 0.3}
    fmt = rng.choice(sorted(FORMATS))
    step = FORMATS[fmt]["tile"][0]
    if op == "distill":
        n = step * _log_uniform(rng, 2, 65536 // step)
        k = 128 * _log_uniform(rng, 4, min(64, 120_000_000 // n // 128))
        m = min(_log_uniform(rng, 1, 3000), 400_000_000_000 // (n * k))
        return {"op": op, "format": fmt, "n": n, "k": k, "m": max(m, 1), "vocab": n - rng.randint(0, 127), "top": _log_uniform(rng, 1, 64),
                "rest": rng.random() < 0.5, "temperature": rng.choice([0.5, 1.0, 2.0]), "with_grad": rng.random() < 0.7}
    n = step * _log_uniform(rng, 2, 14336 // step)
    k = 128 * _log_uniform(rng, 4, min(64, 60_000_000 // n // 128))
    return {"op": op, "format": fmt, "n": n, "k": k, "m": _log_uniform(rng, 1, 2048), "act": rng.choice(ACTS)}


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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": dict(case)}
    if case["op"] == "verify":
        _prepare_verify(s, g)
        return s
    fmt, n, k, m = case["format"], case["n"], case["k"], case["m"]
    s["layers"] = [_weights(fmt, n, k, g) for _ in range(1 if case["op"] == "distill" else 2)]
    x = torch.randn(m, k, generator=g, device="cuda")
    if case["op"] == "distill":
        _prepare_teacher(s, x, g)
    elif case["op"] == "gated_grad":
        size = 1e-3 * torch.exp(torch.randn(m, 1, generator=g, device="cuda"))
        s["dh"] = (size * torch.randn(m, n, generator=g, device="cuda")).bfloat16()
    s["x"] = x.bfloat16()
    if own:
        _prepare_own(s)
    return s


def _prepare_teacher(s, x, g):
    """A teacher's top logits, and hidden states whose own logits lean towards the first of
    them, some much, some not.  Some tokens have fewer listed logits than others, and a few
    are padding, which has none."""
    c = s["case"]
    m, top, vocab = c["m"], min(c["top"], c["vocab"]), c["vocab"]
    c["top"] = top
    j = torch.arange(top, device="cuda")
    first = torch.randint(0, vocab, (m, 1), generator=g, device="cuda")
    step = torch.randint(1, max(2, vocab // top), (m, 1), generator=g, device="cuda")
    ids = (first + j * step) % vocab  # all of a token's are different
    fall = 0.5 + 2.5 * torch.rand(m, 1, generator=g, device="cuda")
    logits = 15 - fall * torch.log1p(j.float()) - 0.2 * torch.rand(m, top, generator=g, device="cuda")
    for i in range(min(3, top)):
        rows = _values(s, 0, ids[:, i])
        lean = (8.0, 4.0, 2.0)[i] * torch.rand(m, 1, generator=g, device="cuda")
        x += lean * rows / rows.norm(dim=1, keepdim=True)
    count = torch.randint(max(1, top // 2), top + 1, (m, 1), generator=g, device="cuda")
    if m > 1:
        count[torch.rand(m, 1, generator=g, device="cuda") < 0.05] = 0
    ids = torch.where(j < count, ids, -1)
    s["ids"], s["logits"] = ids.to(torch.int32).contiguous(), logits.contiguous()
    s["teacher_lse"] = None
    if c["rest"]:
        # what the teacher has on all its vocabulary: the listed logits hold 80 to 99 % of it
        listed_part = torch.logsumexp((logits / c["temperature"]).masked_fill(j >= count, -math.inf), dim=1)
        held = 0.8 + 0.19 * torch.rand(m, generator=g, device="cuda")
        s["teacher_lse"] = torch.where(count[:, 0] > 0, listed_part - held.log(), 0.0)
    s["weight"] = (count[:, 0] > 0).float() / (count > 0).sum().clamp_min(1)


def _drafts_of(most, b):
    """How many tokens the b-th sequence drafts, in some order: up to two fewer than the most."""
    return max(0, most - b % 3)


def _prepare_verify(s, g):
    """Logits of a target and of a draft model that mostly agree, drafts drawn from the draft
    model's, or guessed without one; some sequences draft fewer tokens, some decode greedily."""
    c = s["case"]
    seqs, most, vocab, stride = c["seqs"], c["drafted"], c["vocab"], c["stride"]
    count = torch.tensor([_drafts_of(most, b) for b in range(seqs)], device="cuda")[torch.randperm(seqs, generator=g, device="cuda")]
    starts = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    starts[1:] = count.cumsum(0)
    drafted = int(starts[-1])
    z = 1.5 * torch.randn(drafted + seqs, stride, generator=g, device="cuda")
    lead = torch.randint(0, vocab, (drafted + seqs, 6), generator=g, device="cuda")
    z.scatter_add_(1, lead, 9 + 4 * torch.rand(drafted + seqs, 6, generator=g, device="cuda"))
    of_draft = torch.repeat_interleave(torch.arange(seqs, device="cuda"), count)
    temperature = 0.5 + torch.rand(seqs, generator=g, device="cuda")
    temperature[torch.rand(seqs, generator=g, device="cuda") < 0.1] = 0
    rows = torch.arange(drafted, device="cuda") + of_draft
    y = z[rows] + 0.7 * torch.randn(drafted, stride, generator=g, device="cuda")
    hot = temperature[of_draft].clamp_min(1e-3)[:, None]
    noise = -torch.log(-torch.log(torch.rand(drafted, vocab, generator=g, device="cuda").clamp(1e-9, 1 - 1e-6)))
    tokens = (y[:, :vocab] / hot + noise * (temperature[of_draft] > 0)[:, None]).argmax(dim=1)
    s["target"], s["draft"] = z, None if c.get("looked_up") else y
    s["starts"], s["tokens"], s["temperature"] = starts, tokens.to(torch.int32), temperature
    s["u"] = torch.rand(drafted, generator=g, device="cuda")
    s["v"] = torch.rand(seqs, generator=g, device="cuda")
    s["drafted"], s["of_draft"], s["rows"] = drafted, of_draft, rows
    if own:
        from rans_decode_gemm_b200 import ans

        s["ws"] = torch.zeros(ans.ans_verify_workspace(seqs, drafted, vocab), dtype=torch.uint8, device="cuda")
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["accepted"] = torch.empty(seqs, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(drafted + seqs, dtype=torch.int32, device="cuda")


def _prepare_own(s):
    """What a user's program keeps for the calls: the compressed layers, a workspace, a status
    word and the output buffers."""
    import numpy as np

    from rans_decode_gemm_b200 import ans

    c = s["case"]
    op, fmt, n, k, m = c["op"], c["format"], c["n"], c["k"], c["m"]
    code = {"bf16": ans.BF16_SPLIT, "fp8": ans.FP8_E4M3, "int8": ans.INT8, "fp4": ans.FP4_PAIRS, "int4": ans.INT4_PAIRS}[fmt]
    layout = ans.make_layout(code, n, k, *FORMATS[fmt]["tile"], 64)
    s["scales"], s["compressed"] = [scales for _, scales in s["layers"]], []
    for codes, _ in s.pop("layers"):
        host = codes.view(torch.int16 if fmt == "bf16" else torch.uint8).reshape(-1).cpu().numpy()
        s["compressed"].append(ans.CompressedLayer.from_weights(host.view(np.uint16) if fmt == "bf16" else host, layout))
    s["kind"] = {None: ans.SCALE_NONE, "row": ans.SCALE_ROW_F32, "group": ans.SCALE_GROUP_BF16}[FORMATS[fmt]["scales"]]
    s["group"] = GROUP if fmt == "int4" else 0
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op == "gated":
        size = ans.ans_gated_workspace(layout, m, s["kind"])
        s["h"] = new(m, n, dtype=torch.bfloat16)
    elif op == "gated_grad":
        size = ans.ans_gated_grad_workspace(layout, m, s["kind"])
        s["dx"] = new(m, k, dtype=torch.bfloat16)
        s["dg"], s["du"] = new(m, n, dtype=torch.bfloat16), new(m, n, dtype=torch.bfloat16)
    else:
        size = ans.ans_distill_workspace(layout, m, s["kind"], c["top"], c["with_grad"])
        s["loss"], s["lse"] = new(m), new(m)
        s["dx"] = new(m, k, dtype=torch.bfloat16) if c["with_grad"] else None
    if op != "distill":
        s["act"] = {"silu": ans.ACT_SILU, "gelu": ans.ACT_GELU, "gelu_tanh": ans.ACT_GELU_TANH, "relu": ans.ACT_RELU}[c["act"]]
    s["ws"] = torch.zeros(size, dtype=torch.uint8, device="cuda")
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")


# ---- one pass --------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from rans_decode_gemm_b200 import ans

    c, rest = s["case"], (s["ws"], s["ws"].numel(), s["status"])
    if c["op"] == "verify":
        ans.ans_verify(s["target"], c["stride"], s["draft"], c["stride"], c["seqs"], s["drafted"], c["vocab"], s["starts"],
                       s["tokens"], s["u"], s["v"], s["temperature"], s["accepted"], s["out"], *rest)
        return {"accepted": s["accepted"], "tokens": s["out"]}
    if c["op"] == "distill":
        ans.ans_distill(s["x"], c["m"], s["compressed"][0].tiles, s["kind"], s["scales"][0], s["group"], c["vocab"],
                        1.0 / c["temperature"], c["top"], s["ids"], s["logits"], s["teacher_lse"], s["loss"], s["lse"],
                        s["weight"] if c["with_grad"] else None, s["dx"], *rest)
        return {"loss": s["loss"], "lse": s["lse"]} | ({"dx": s["dx"]} if c["with_grad"] else {})
    gate, up = (layer.tiles for layer in s["compressed"])
    w = (gate, up, s["kind"], *s["scales"], s["group"], s["act"])
    if c["op"] == "gated":
        ans.ans_gated(s["x"], c["m"], *w, s["h"], *rest)
        return {"h": s["h"]}
    ans.ans_gated_grad(s["x"], s["dh"], c["m"], *w, s["dx"], s["dg"], s["du"], *rest)
    return {"dx": s["dx"], "dg": s["dg"], "du": s["du"]}


def _values(s, layer, rows=None, dtype=torch.float32):
    """A layer's values, of all rows or of those asked for."""
    fmt, (codes, scales) = s["case"]["format"], s["layers"][layer]
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


def _activation(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * 0.044715 * g * g)
    return g.clamp_min(0), (g > 0).to(g.dtype)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "verify":
        return _verify_plain(c, s)
    if c["op"] == "distill":
        return _distill_plain(c, s)
    x, wg, wu = s["x"].float(), _values(s, 0), _values(s, 1)
    u = x @ wu.T
    value, slope = _activation(c["act"], x @ wg.T)
    if c["op"] == "gated":
        return {"h": (value * u).bfloat16()}
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * value
    return {"dx": (dg @ wg + du @ wu).bfloat16(), "dg": dg.bfloat16(), "du": du.bfloat16()}


def _distill_plain(c, s):
    w = _values(s, 0)[: c["vocab"]]
    z = (s["x"].float() @ w.T) / c["temperature"]
    peak = z.amax(dim=1, keepdim=True)
    p = torch.exp(z - peak)
    total = p.sum(dim=1, keepdim=True)
    lse = total.log() + peak
    has = s["ids"] >= 0
    at = s["ids"].clamp_min(0).long()
    v = (s["logits"] / c["temperature"]).masked_fill(~has, -math.inf)
    some = has.any(dim=1, keepdim=True)
    if s["teacher_lse"] is None:
        most = torch.where(some, v.amax(dim=1, keepdim=True), 0.0)
        all_of_it = torch.exp(v - most).sum(dim=1, keepdim=True).log() + most
    else:
        all_of_it = s["teacher_lse"][:, None]
    log_t = torch.where(has, v - torch.where(some, all_of_it, 0.0), 0.0)
    t = torch.where(has, log_t.exp(), 0.0)
    log_p = z.gather(1, at) - lse
    out = {"loss": (t * (log_t - log_p)).sum(dim=1), "lse": lse[:, 0]}
    if c["with_grad"]:
        p *= t.sum(dim=1, keepdim=True) / total
        p.scatter_add_(1, at, -t)
        p *= s["weight"][:, None] / c["temperature"]
        out["dx"] = (p @ w).bfloat16()
    return out


def _verify_plain(c, s):
    # (in 64 bits: a running sum of small probabilities meets a random number)
    seqs, vocab = c["seqs"], c["vocab"]
    z, of_draft, rows = s["target"][:, :vocab], s["of_draft"], s["rows"]
    of_row = torch.empty(len(z), dtype=torch.long, device="cuda")
    of_row[rows] = of_draft
    ends = s["starts"][1:].long() + torch.arange(seqs, device="cuda")
    of_row[ends] = torch.arange(seqs, device="cuda")

    def probabilities(logits, temperature):
        greedy = temperature == 0
        t = torch.where(greedy, 1.0, temperature.double())[:, None]
        a = logits.double() / t
        e = torch.exp(a - a.amax(dim=1, keepdim=True))
        e = e / e.sum(dim=1, keepdim=True)
        # greedy: all of it on the first of the largest
        best = (logits == logits.amax(dim=1, keepdim=True)).int().argmax(dim=1)
        point = torch.zeros_like(e).scatter_(1, best[:, None], 1.0)
        return torch.where(greedy[:, None], point, e)

    p = probabilities(z, s["temperature"][of_row])
    at = s["tokens"].long()[:, None]
    px = p[rows].gather(1, at)[:, 0]
    if s["draft"] is None:
        qx = torch.ones_like(px)
    else:
        q = probabilities(s["draft"][:, :vocab], s["temperature"][of_draft])
        qx = q.gather(1, at)[:, 0]
    accept = s["u"].double() * qx < px
    # a sequence's first refused draft, or its number of drafts
    index = torch.arange(s["drafted"], device="cuda")
    first = torch.full((seqs,), s["drafted"], device="cuda").scatter_reduce_(0, of_draft, torch.where(accept, s["drafted"], index), "amin")
    starts, stops = s["starts"][:-1].long(), s["starts"][1:].long()
    stop = torch.minimum(first, stops)
    row = stop + torch.arange(seqs, device="cuda")
    last = p[row]
    refused = stop < stops
    if len(index):
        d = stop.clamp_max(s["drafted"] - 1)
        other = torch.zeros_like(last).scatter_(1, at[d], 1.0) if s["draft"] is None else q[d]
        if s["draft"] is None:
            over = torch.where(other > 0, 0.0, last)
        else:
            over = (last - other).clamp_min(0)
        use = refused & (over.sum(dim=1) > 2.0 ** -40)
        last = torch.where(use[:, None], over, last)
    run_sum = last.cumsum(dim=1)
    token = (run_sum > s["v"].double()[:, None] * run_sum[:, -1:]).int().argmax(dim=1)
    out = torch.full((len(z),), -1, device="cuda")
    kept = index < stop[of_draft]
    out[rows] = torch.where(kept, at[:, 0], -1)
    out[row] = token
    return {"accepted": (stop - starts).to(torch.int32), "tokens": out.to(torch.int32)}


# ---- the floor of a pass ---------------------------------------------------------------
def work(case):
    if case["op"] == "verify":
        # every drafted token's row of both, and each sequence's last row
        seqs = case["seqs"]
        drafted = sum(_drafts_of(case["drafted"], b) for b in range(seqs))
        logits = case["vocab"] * (seqs + drafted * (1 if case.get("looked_up") else 2))
        return {"bytes": 4 * logits + 12 * drafted + 20 * seqs, "flops": 3 * logits}
    n, k, m = case["n"], case["k"], case["m"]
    layer = n * k * FORMATS[case["format"]]["bits"] / 8
    layer += {None: 0, "row": 4 * n, "group": 2 * n * k / GROUP}[FORMATS[case["format"]]["scales"]]
    product = 2 * m * n * k
    if case["op"] == "gated":
        return {"bytes": 2 * layer + 2 * m * k + 2 * m * n, "flops": 2 * product}
    if case["op"] == "gated_grad":
        return {"bytes": 2 * layer + 4 * m * k + 6 * m * n, "flops": 4 * product}
    grad = case["with_grad"]
    small = 8 * m * case["top"] + 8 * m + (4 * m if case["rest"] else 0)
    return {"bytes": layer + 2 * m * k + small + (2 * m * k + 4 * m if grad else 0), "flops": product * (2 if grad else 1)}


# ---- the same values in 64 bits, from the definitions ----------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "verify":
        return _exact_verify(s)
    return _exact_distill(s) if case["op"] == "distill" else _exact_gated(s)


def _exact_gated(s):
    c, x = s["case"], s["x"].double()
    n, m = c["n"], c["m"]
    act = {
        "silu": torch.nn.functional.silu,
        "gelu": torch.nn.functional.gelu,
        "gelu_tanh": lambda g: torch.nn.functional.gelu(g, approximate="tanh"),
        "relu": torch.nn.functional.relu,
    }[c["act"]]
    h = torch.empty(m, n, dtype=torch.float64, device="cuda")
    dg, du, dx = torch.empty_like(h), torch.empty_like(h), torch.zeros_like(x)
    for r in range(0, n, 2048):
        rows = torch.arange(r, min(n, r + 2048), device="cuda")
        wg, wu = _values(s, 0, rows, torch.float64), _values(s, 1, rows, torch.float64)
        g = torch.einsum("mk,nk->mn", x, wg).requires_grad_()
        u = torch.einsum("mk,nk->mn", x, wu).requires_grad_()
        with torch.enable_grad():
            part = act(g) * u
        h[:, rows] = part.detach()
        if c["op"] == "gated_grad":
            dg[:, rows], du[:, rows] = torch.autograd.grad(part, (g, u), s["dh"][:, rows].double())
            dx += torch.einsum("mn,nk->mk", dg[:, rows], wg) + torch.einsum("mn,nk->mk", du[:, rows], wu)
    return {"h": h} if c["op"] == "gated" else {"dx": dx, "dg": dg, "du": du}


def _exact_distill(s):
    c, x = s["case"], s["x"].double()
    n, m, vocab, hot = c["n"], c["m"], c["vocab"], c["temperature"]
    blocks = [torch.arange(r, min(vocab, r + 4096), device="cuda") for r in range(0, vocab, 4096)]
    lse = torch.stack([torch.logsumexp(x @ _values(s, 0, rows, torch.float64).T / hot, dim=1) for rows in blocks]).logsumexp(dim=0)
    teacher = torch.full((m, n), -math.inf, dtype=torch.float64, device="cuda")
    for j in range(c["top"]):
        has = (s["ids"][:, j] >= 0).nonzero()[:, 0]
        teacher[has, s["ids"][has, j].long()] = s["logits"][has, j].double() / hot
    some = torch.isfinite(teacher).any(dim=1)
    norm = teacher.logsumexp(dim=1) if s["teacher_lse"] is None else s["teacher_lse"].double()
    teacher -= torch.where(some, norm, 0.0)[:, None]
    held = teacher.exp().sum(dim=1)
    loss, dx = torch.zeros(m, dtype=torch.float64, device="cuda"), torch.zeros_like(x)
    for rows in blocks:
        w = _values(s, 0, rows, torch.float64)
        log_p = x @ w.T / hot - lse[:, None]
        t = teacher[:, rows].exp()
        loss += torch.where(t > 0, t * (teacher[:, rows] - log_p), 0.0).sum(dim=1)
        if c["with_grad"]:
            dx += (held[:, None] * log_p.exp() - t) @ w
    out = {"loss": loss, "lse": lse}
    if c["with_grad"]:
        out["dx"] = dx * (s["weight"].double() / hot)[:, None]
    return out


def _exact_verify(s):
    c = s["case"]
    vocab, starts, v = c["vocab"], s["starts"].tolist(), s["v"].double()
    accepted, tokens = [], []

    def distribution(logits, hot):
        logits = logits[:vocab].double()
        if hot == 0:
            best = int((logits == logits.max()).nonzero()[0, 0])
            return torch.nn.functional.one_hot(torch.tensor(best, device="cuda"), vocab).double()
        return torch.softmax(logits / hot, dim=0)

    for b in range(c["seqs"]):
        hot, kept, after = s["temperature"][b].double(), 0, None
        hot = hot.item()
        for i in range(starts[b], starts[b + 1]):
            x = int(s["tokens"][i])
            p = distribution(s["target"][i + b], hot)
            if s["draft"] is None:
                q = torch.nn.functional.one_hot(torch.tensor(x, device="cuda"), vocab).double()
            else:
                q = distribution(s["draft"][i], hot)
            if bool(s["u"][i].double() * q[x] < p[x]):
                kept += 1
                continue
            after = (p - q).clamp_min(0)
            if float(after.sum()) <= 2.0 ** -40:
                after = p
            break
        if after is None:
            after = distribution(s["target"][starts[b + 1] + b], hot)
        below = torch.cumsum(after, dim=0)
        token = int((below > v[b] * below[-1]).nonzero()[0, 0])
        accepted.append(kept)
        drafts = s["tokens"][starts[b]: starts[b] + kept].tolist()
        tokens += drafts + [token] + [-1] * (starts[b + 1] - starts[b] - kept)
    whole = lambda values: torch.tensor(values, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"accepted": whole(accepted), "tokens": whole(tokens)}
