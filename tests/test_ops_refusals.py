"""What ans_gemm_lora, ans_gemm_grad, ans_gemm_lora_grad and ans_xent refuse, and
in which words: every check comes before any device work, so none of this needs
a GPU (the pointers below are never read)."""
import ctypes as C

import numpy as np
import pytest
import torch

from rans_decode_gemm_b200 import ans

ARG, SHAPE, ALPHABET, UNSUPPORTED = 1, 2, 3, 8
P = 1 << 20   # stands for a device pointer, aligned to anything asked for


def layer(dtype=ans.FP8_E4M3, N=256, K=128, tile_n=128, tile_k=32):
    lay = ans.make_layout(dtype, N, K, tile_n, tile_k)
    cb = ans.ans_build_codebook(np.arange(1, ans.ALPHABET[dtype] + 1), ans.ALPHABET[dtype])
    return ans.AnsTiles(lay, cb, P, 4096, P, P)


def adapters(n=4, rank=16, a=P, b=P, scale=P):
    return ans.AnsLora(n, rank, a, b, scale)


def ref(x):
    return C.byref(x) if x is not None else None


def call(name, **over):
    """The call with good arguments, but for those given by name."""
    L = ans.load()
    W = over.pop("W", None) or layer()
    v = {"X": P, "dY": P, "M": 8, "kind": ans.SCALE_ROW_F32, "scales": P, "group": 0, "lora": adapters(), "ids": P, "Y": P,
         "dX": P, "dA": P, "dB": P, "ws": P, "bytes": 1 << 40, "status": P, "vocab": 256, "targets": P, "loss": P,
         "lse": P, "weight": P} | over
    w = (ref(W), v["kind"], v["scales"], v["group"])
    end = (v["ws"], v["bytes"], v["status"], None)
    if name == "ans_gemm_lora":
        return L.ans_gemm_lora(v["X"], v["M"], *w, ref(v["lora"]), v["ids"], v["Y"], *end)
    if name == "ans_gemm_grad":
        return L.ans_gemm_grad(v["dY"], v["M"], *w, v["dX"], *end)
    if name == "ans_gemm_lora_grad":
        return L.ans_gemm_lora_grad(v["X"], v["dY"], v["M"], *w, ref(v["lora"]), v["ids"], v["dX"], v["dA"], v["dB"], *end)
    return L.ans_xent(v["X"], v["M"], *w, v["vocab"], v["targets"], v["loss"], v["lse"], v["weight"], v["dX"], *end)


NAMES = ["ans_gemm_lora", "ans_gemm_grad", "ans_gemm_lora_grad", "ans_xent"]
NEEDS = {"ans_gemm_lora": ["X", "ids", "Y", "ws", "status", "scales", "lora"],
         "ans_gemm_grad": ["dY", "dX", "ws", "status", "scales"],
         "ans_gemm_lora_grad": ["X", "dY", "ids", "dA", "dB", "ws", "status", "scales", "lora"],
         "ans_xent": ["X", "targets", "loss", "lse", "ws", "status", "scales"]}
ALIGNED = {"ans_gemm_lora": ["X", "Y", "scales"], "ans_gemm_grad": ["dY", "dX", "scales"],
           "ans_gemm_lora_grad": ["X", "dY", "dX", "dA", "dB", "scales"], "ans_xent": ["X", "dX", "scales"]}
WORDS = {"ans_gemm_lora": ["ids"], "ans_gemm_grad": [], "ans_gemm_lora_grad": ["ids"],
         "ans_xent": ["targets", "loss", "lse", "weight"]}


@pytest.mark.parametrize("name", NAMES)
def test_missing_and_misaligned_pointers(ans_lib, name):
    for arg in NEEDS[name]:
        assert call(name, **{arg: None}) == ARG, arg
    for arg in ALIGNED[name]:
        assert call(name, **{arg: P + 8}) == ARG, arg
    for arg in WORDS[name]:
        assert call(name, **{arg: P + 2}) == ARG, arg
    assert call(name, ws=P + 128) == ARG


@pytest.mark.parametrize("name", NAMES)
def test_layers_and_scales(ans_lib, name):
    assert call(name, W=layer(tile_k=48)) == SHAPE
    broken = layer()
    broken.codebook.freq[3] += 1
    assert call(name, W=broken) == ALPHABET
    whole = layer()
    whole.layout.dtype = ans.BF16_WHOLE
    assert call(name, W=whole) == ARG
    no_raw = layer(ans.BF16_SPLIT)
    no_raw.raw = None
    assert call(name, W=no_raw, kind=ans.SCALE_NONE) == ARG
    assert call(name, kind=7) == ARG
    assert call(name, kind=ans.SCALE_GROUP_BF16, group=32) == ARG           # group scales are int4's
    assert call(name, W=layer(ans.INT4), kind=ans.SCALE_GROUP_BF16, group=40) == ARG
    assert call(name, W=layer(ans.INT4), kind=ans.SCALE_GROUP_BF16, group=16) == UNSUPPORTED


@pytest.mark.parametrize("name", ["ans_gemm_lora", "ans_gemm_lora_grad"])
def test_adapters(ans_lib, name):
    assert call(name, lora=adapters(n=0)) == ARG
    assert call(name, lora=adapters(rank=0)) == ARG
    assert call(name, lora=adapters(n=257)) == UNSUPPORTED
    assert call(name, lora=adapters(rank=136)) == UNSUPPORTED
    assert call(name, lora=adapters(rank=20)) == UNSUPPORTED
    for bad in ({"a": None}, {"b": None}, {"a": P + 8}, {"b": P + 8}, {"scale": P + 2}):
        assert call(name, lora=adapters(**bad)) == ARG, bad


@pytest.mark.parametrize("name", NAMES)
def test_token_counts(ans_lib, name):
    assert call(name, M=(1 << 24) + 1) == UNSUPPORTED
    if name != "ans_gemm_lora_grad":      # there, without tokens, gradients of zero are written
        assert call(name, M=0) == 0
        assert call(name, M=0, ws=None, bytes=0) == 0


def test_vocabularies(ans_lib):
    assert call("ans_xent", vocab=0) == SHAPE
    assert call("ans_xent", vocab=257) == SHAPE


def test_workspace_queries(ans_lib):
    L, lay = ans.load(), ans.make_layout(ans.FP8_E4M3, 256, 128, 128, 32)
    out = C.c_size_t(7)
    queries = {
        "ans_gemm_lora_workspace": lambda lay, M, kind, out: L.ans_gemm_lora_workspace(lay, M, kind, ref(adapters(a=None, b=None)), out),
        "ans_gemm_grad_workspace": lambda lay, M, kind, out: L.ans_gemm_grad_workspace(lay, M, kind, out),
        "ans_gemm_lora_grad_workspace": lambda lay, M, kind, out: L.ans_gemm_lora_grad_workspace(lay, M, kind, ref(adapters(a=None, b=None)), out),
        "ans_xent_workspace": lambda lay, M, kind, out: L.ans_xent_workspace(lay, M, kind, 1, out),
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
    for bad, want in ((adapters(n=300), UNSUPPORTED), (adapters(rank=12), UNSUPPORTED), (adapters(rank=0), ARG), (None, ARG)):
        assert L.ans_gemm_lora_workspace(ref(lay), 8, 0, ref(bad), ref(out)) == want
        assert L.ans_gemm_lora_grad_workspace(ref(lay), 8, 0, ref(bad), ref(out)) == want


def test_adapter_tensors(ans_lib):
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 128, 8, dtype=torch.bfloat16)
    s = torch.ones(2)
    assert ans.LoraAdapters(a, b, s).lora.rank == 8
    for bad in ((a, b[:1], s), (a, torch.zeros(2, 128, 16, dtype=torch.bfloat16), s), (a, b, torch.ones(3)),
                (a.float(), b, s), (a, b, s.double()), (a.transpose(1, 2), b, s),
                (a, b.expand(2, 128, 8).transpose(0, 0).flip(0)[:, ::2], s)):
        with pytest.raises(ans.AnsError):
            ans.LoraAdapters(*bad)


def test_adapters_of_another_projection_or_device(ans_lib):
    # the struct carries neither N nor K: a set made for another layer would be read past its end
    def of(N, K, device="cpu"):
        return ans.LoraAdapters(torch.zeros(2, 8, K, dtype=torch.bfloat16, device=device),
                                torch.zeros(2, N, 8, dtype=torch.bfloat16, device=device)).lora
    W, x = layer(), torch.zeros(8, 128, dtype=torch.bfloat16)
    calls = [
        lambda lora: ans.ans_gemm_lora(x, 8, W, 0, None, 0, lora, x, x, x, 1 << 40, x),
        lambda lora: ans.ans_gemm_lora_grad(x, x, 8, W, 0, None, 0, lora, x, x, x, x, x, 1 << 40, x),
        lambda lora: ans.ans_gemm_lora_workspace(W.layout, 8, 0, lora),
        lambda lora: ans.ans_gemm_lora_grad_workspace(W.layout, 8, 0, lora)]
    for fn in calls:
        for N, K in ((256, 64), (256, 256), (128, 128), (384, 128), (128, 256)):
            with pytest.raises(ans.AnsError) as e:
                fn(of(N, K))
            assert e.value.status == SHAPE
    for fn in calls[:2]:
        for device in ("cpu", "meta"):
            with pytest.raises(ans.AnsError) as e:
                fn(of(256, 128, device))
            assert e.value.status == ARG
    with pytest.raises(ans.AnsError):
        ans.LoraAdapters(torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 128, 8, dtype=torch.bfloat16, device="meta"))
    with pytest.raises(ans.AnsError):
        ans.LoraAdapters(torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(2, 128, 8, dtype=torch.bfloat16))


def test_the_struct_holds_the_adapters(ans_lib):
    import gc
    import weakref
    a, b = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 128, 8, dtype=torch.bfloat16)
    held = weakref.ref(a)
    lora = ans.LoraAdapters(a, b).lora
    del a, b
    gc.collect()
    assert held() is not None and lora.d_A == held().data_ptr()
