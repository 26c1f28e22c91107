"""What ans_gated, ans_gated_grad, ans_distill and ans_verify refuse, and in which words:
every check comes before any device work, so none of this needs a GPU (the pointers below
are never read)."""
import ctypes as C

import numpy as np
import pytest

from rans_decode_gemm_b200 import ans

ARG, SHAPE, ALPHABET, UNSUPPORTED = 1, 2, 3, 8
P = 1 << 20   # stands for a device pointer, aligned to anything asked for


def layer(dtype=ans.FP8_E4M3, N=256, K=128, tile_n=128, tile_k=32, state_bits=32):
    lay = ans.make_layout(dtype, N, K, tile_n, tile_k, state_bits)
    cb = ans.ans_build_codebook(np.arange(1, ans.ALPHABET[dtype] + 1), ans.ALPHABET[dtype])
    return ans.AnsTiles(lay, cb, P, 4096, P, P)


def ref(x):
    return C.byref(x) if x is not None else None


def call(name, **over):
    """The call with good arguments, but for those given by name."""
    L = ans.load()
    W, W2 = over.pop("W", None) or layer(), over.pop("W2", None)
    W2 = W2 or layer(W.layout.dtype, W.layout.N, W.layout.K, W.layout.tile_n, W.layout.tile_k, W.layout.state_bits)
    v = {"X": P, "M": 8, "kind": ans.SCALE_ROW_F32, "scales": P, "scales2": P, "group": 0, "act": ans.ACT_SILU, "H": P, "dH": P,
         "dX": P, "dG": P, "dU": P, "ws": P, "bytes": 1 << 40, "status": P, "vocab": 256, "per_t": 1.0, "top": 4, "ids": P,
         "logits": P, "teacher": P, "loss": P, "lse": P, "weight": P, "target": P, "t_stride": 300, "draft": P, "d_stride": 300,
         "seqs": 2, "drafted": 5, "starts": P, "tokens": P, "u": P, "v": P, "temperature": P, "accepted": P, "out": P} | over
    end = (v["ws"], v["bytes"], v["status"], None)
    both = (ref(W), ref(W2), v["kind"], v["scales"], v["scales2"], v["group"], v["act"])
    if name == "ans_gated":
        return L.ans_gated(v["X"], v["M"], *both, v["H"], *end)
    if name == "ans_gated_grad":
        return L.ans_gated_grad(v["X"], v["dH"], v["M"], *both, v["dX"], v["dG"], v["dU"], *end)
    if name == "ans_distill":
        return L.ans_distill(v["X"], v["M"], ref(W), v["kind"], v["scales"], v["group"], v["vocab"], v["per_t"], v["top"],
                             v["ids"], v["logits"], v["teacher"], v["loss"], v["lse"], v["weight"], v["dX"], *end)
    return L.ans_verify(v["target"], v["t_stride"], v["draft"], v["d_stride"], v["seqs"], v["drafted"], v["vocab"], v["starts"],
                        v["tokens"], v["u"], v["v"], v["temperature"], v["accepted"], v["out"], *end)


LAYERED = ["ans_gated", "ans_gated_grad", "ans_distill"]
NEEDS = {"ans_gated": ["X", "H", "ws", "status", "scales", "scales2"],
         "ans_gated_grad": ["X", "dH", "dG", "dU", "ws", "status", "scales", "scales2"],
         "ans_distill": ["X", "ids", "logits", "loss", "lse", "ws", "status", "scales"],
         "ans_verify": ["target", "starts", "tokens", "u", "v", "accepted", "out", "ws", "status"]}
ALIGNED = {"ans_gated": ["X", "H", "scales", "scales2"], "ans_gated_grad": ["X", "dH", "dX", "dG", "dU", "scales", "scales2"],
           "ans_distill": ["X", "dX", "scales"], "ans_verify": []}
WORDS = {"ans_gated": [], "ans_gated_grad": [], "ans_distill": ["ids", "logits", "teacher", "loss", "lse", "weight"],
         "ans_verify": ["target", "draft", "starts", "tokens", "u", "v", "temperature", "accepted", "out", "status"]}


@pytest.mark.parametrize("name", list(NEEDS))
def test_missing_and_misaligned_pointers(ans_lib, name):
    for arg in NEEDS[name]:
        assert call(name, **{arg: None}) == ARG, arg
    for arg in ALIGNED[name]:
        assert call(name, **{arg: P + 8}) == ARG, arg
    for arg in WORDS[name]:
        assert call(name, **{arg: P + 2}) == ARG, arg
    assert call(name, ws=P + 128) == ARG


@pytest.mark.parametrize("name", LAYERED)
def test_layers_and_scales(ans_lib, name):
    assert call(name, W=layer(tile_k=48)) == SHAPE
    broken = layer()
    broken.codebook.freq[3] += 1
    assert call(name, W=broken) == ALPHABET
    whole = layer()
    whole.layout.dtype = ans.BF16_WHOLE
    assert call(name, W=whole, W2=layer()) == ARG
    no_raw = layer(ans.BF16_SPLIT)
    no_raw.raw = None
    assert call(name, W=no_raw, kind=ans.SCALE_NONE) == ARG
    assert call(name, kind=7) == ARG
    assert call(name, kind=ans.SCALE_GROUP_BF16, group=32) == ARG           # group scales are int4's
    assert call(name, W=layer(ans.INT4), kind=ans.SCALE_GROUP_BF16, group=40) == ARG
    assert call(name, W=layer(ans.INT4), kind=ans.SCALE_GROUP_BF16, group=16) == UNSUPPORTED
    assert call(name, M=(1 << 24) + 1) == UNSUPPORTED
    assert call(name, M=0) == 0
    assert call(name, M=0, ws=None, bytes=0, X=None) == 0


@pytest.mark.parametrize("name", ["ans_gated", "ans_gated_grad"])
def test_two_layers_of_one_layout(ans_lib, name):
    for other in (layer(N=384), layer(K=256), layer(tile_n=256), layer(tile_k=64), layer(ans.INT8), layer(state_bits=64)):
        assert call(name, W2=other) == SHAPE
    broken = layer()
    broken.codebook.cdf[3] += 1
    assert call(name, W2=broken) == ALPHABET
    no_stream = layer()
    no_stream.stream = None
    assert call(name, W2=no_stream) == ARG
    for act in (-1, 4, 100):
        assert call(name, act=act) == ARG


def test_distillation_arguments(ans_lib):
    assert call("ans_distill", vocab=0) == SHAPE
    assert call("ans_distill", vocab=257) == SHAPE
    assert call("ans_distill", top=0) == SHAPE
    assert call("ans_distill", top=257) == UNSUPPORTED
    for per_t in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** -41, 2.0 ** 41):
        assert call("ans_distill", per_t=per_t) == ARG


def test_verification_arguments(ans_lib):
    assert call("ans_verify", vocab=0) == SHAPE
    assert call("ans_verify", vocab=301) == SHAPE             # past a row's stride
    assert call("ans_verify", t_stride=255) == SHAPE
    assert call("ans_verify", d_stride=255) == SHAPE
    assert call("ans_verify", t_stride=(1 << 40) + 1) == SHAPE
    assert call("ans_verify", vocab=(1 << 24) + 1, t_stride=1 << 25, d_stride=1 << 25) == UNSUPPORTED
    assert call("ans_verify", seqs=1 << 20, drafted=1) == UNSUPPORTED
    assert call("ans_verify", seqs=1, drafted=1 << 20) == UNSUPPORTED
    assert call("ans_verify", seqs=2 ** 32 - 1, drafted=2) == UNSUPPORTED
    assert call("ans_verify", seqs=0, drafted=5) == SHAPE
    assert call("ans_verify", seqs=0, drafted=0) == 0
    assert call("ans_verify", seqs=0, drafted=0, target=None, out=None, ws=None, bytes=0) == 0


def test_workspace_queries(ans_lib):
    L, lay = ans.load(), ans.make_layout(ans.FP8_E4M3, 256, 128, 128, 32)
    out = C.c_size_t(7)
    queries = {
        "ans_gated_workspace": lambda lay, M, kind, out: L.ans_gated_workspace(lay, M, kind, out),
        "ans_gated_grad_workspace": lambda lay, M, kind, out: L.ans_gated_grad_workspace(lay, M, kind, out),
        "ans_distill_workspace": lambda lay, M, kind, out: L.ans_distill_workspace(lay, M, kind, 5, 1, out),
    }
    for name, q in queries.items():
        out.value = 7
        assert q(ref(lay), 0, 0, ref(out)) == 0 and out.value == 0, name
        assert q(ref(lay), 8, 0, None) == ARG, name
        assert q(None, 8, 0, ref(out)) == ARG, name
        assert q(ref(lay), 8, 9, ref(out)) == ARG, name
        assert q(ref(lay), 8, ans.SCALE_GROUP_BF16, ref(out)) == ARG, name
        assert q(ref(ans.make_layout(ans.FP8_E4M3, 256, 130, 128, 32)), 8, 0, ref(out)) == SHAPE, name
        assert q(ref(lay), (1 << 24) + 1, 0, ref(out)) == UNSUPPORTED, name
    assert L.ans_distill_workspace(ref(lay), 8, 0, 0, 1, ref(out)) == SHAPE
    assert L.ans_distill_workspace(ref(lay), 8, 0, 257, 1, ref(out)) == UNSUPPORTED
    assert L.ans_verify_workspace(2, 5, 256, None) == ARG
    assert L.ans_verify_workspace(2, 5, 0, ref(out)) == SHAPE
    assert L.ans_verify_workspace(0, 5, 256, ref(out)) == SHAPE
    assert L.ans_verify_workspace(2, 1 << 20, 256, ref(out)) == UNSUPPORTED
    assert L.ans_verify_workspace(0, 0, 256, ref(out)) == 0 and out.value == 0


def test_verification_workspaces_grow_with_what_they_hold(ans_lib):
    """At least a part a row, and no more than 64, whatever the vocabulary."""
    for vocab in (1, 255, 1024, 32000, 131072, 1 << 24):
        for seqs, drafted in ((1, 0), (1, 5), (64, 448), (1000, 3)):
            rows = seqs + 2 * drafted
            assert 16 * rows <= ans.ans_verify_workspace(seqs, drafted, vocab) <= 64 * 16 * rows
