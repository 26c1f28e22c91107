"""One workspace for calls of changing token counts, each with the bits of a fresh one."""
import pytest
import torch

from rans_decode_gemm_b200 import ans
from rans_decode_gemm_b200 import workloads as WL

from _gpu_util import scales_dev, status_tensor, x_dev

pytestmark = pytest.mark.gpu


def _layer(name, N, K, tile_n, tile_k, j=0):
    base = WL.CONFIGS[name]
    cfg = WL.Config(**{**base.__dict__, "seed": base.seed + 1000 * j, "tile_n": tile_n, "tile_k": tile_k})
    d = WL.make_weights(cfg, 0, N=N, K=K)
    lay = ans.make_layout(cfg.dtype, N, K, tile_n, tile_k)
    return cfg, scales_dev(cfg, d), lay, ans.CompressedLayer.from_weights(d["w"], lay, device="cuda")


@pytest.mark.parametrize("name,N,K,tile_k", [("bf16_4096", 16384, 80, 16), ("fp8_405b", 8192, 1040, 16),
                                             ("bf16_4096", 1024, 1024, 64)])
def test_gemm_of_one_pass_and_of_several(cuda, name, N, K, tile_k):
    """K = 80 and 1040 are no multiples of 64: more tokens than a pass take several on the same schedule."""
    cfg, sc, lay, layer = _layer(name, N, K, 128, tile_k)
    order = (1, 1100, 40, 17, 700, 1, 600, 3)
    size = max(ans.ans_gemm_workspace(lay, M, cfg.scale_kind) for M in order)
    ws, st = torch.zeros(size, dtype=torch.uint8, device="cuda"), status_tensor()
    for turn, M in enumerate(order):
        x = x_dev(WL.make_x(cfg, M, K, stream=turn))
        y, want = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        ans.ans_gemm(x, M, layer.tiles, cfg.scale_kind, sc, cfg.group_k, y, ws, size, st)
        fresh = torch.zeros(size, dtype=torch.uint8, device="cuda")
        ans.ans_gemm(x, M, layer.tiles, cfg.scale_kind, sc, cfg.group_k, want, fresh, size, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        same = torch.equal(y, want)
        assert same, f"M {M}, turn {turn}"


@pytest.mark.parametrize("name,tile_n,shapes", [("bf16_4096", 128, [(1024, 1024), (512, 2048), (1024, 512)]),
                                                ("int4_70b", 256, [(1024, 1024), (1024, 1024)]),
                                                ("fp8_405b", 128, [(512, 1040), (8192, 80)])])
def test_batched_layers(cuda, name, tile_n, shapes):
    layers = [_layer(name, N, K, tile_n, 64 if K % 64 == 0 else 16, j) for j, (N, K) in enumerate(shapes)]
    cfg = layers[0][0]
    st = status_tensor()

    def call(M, turn, ws):
        jobs = [(x_dev(WL.make_x(c, M, lay.K, stream=turn)), layer.tiles, sc, torch.empty(M, lay.N, device="cuda"))
                for c, sc, lay, layer in layers]
        size = ans.ans_gemm_batched_workspace(jobs, M, cfg.scale_kind)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda") if ws is None else ws
        ans.ans_gemm_batched(jobs, M, cfg.scale_kind, cfg.group_k, ws, ws.numel(), st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return size, [job[3] for job in jobs]
    order = (8, 20, 300, 1, 1100, 32, 5, 300, 17)
    want = [call(M, turn, None) for turn, M in enumerate(order)]
    ws = torch.zeros(max(size for size, _ in want), dtype=torch.uint8, device="cuda")
    for turn, M in enumerate(order):
        same = all(torch.equal(a, b) for a, b in zip(call(M, turn, ws)[1], want[turn][1]))
        assert same, f"M {M}, turn {turn}"


@pytest.mark.parametrize("K", [1024, 1040])
def test_adapters(cuda, K):
    N, rank = 8192, 16
    cfg, sc, lay, layer = _layer("fp8_405b", N, K, 128, 64 if K % 64 == 0 else 16)
    g = torch.Generator(device="cuda").manual_seed(1)
    A = ans.LoraAdapters(torch.randn(3, rank, K, generator=g, device="cuda").bfloat16(),
                         torch.randn(3, N, rank, generator=g, device="cuda").bfloat16())
    order = (1, 1100, 40, 200, 1, 700, 5)
    size = max(ans.ans_gemm_lora_workspace(lay, M, cfg.scale_kind, A.lora) for M in order)
    ws, st = torch.zeros(size, dtype=torch.uint8, device="cuda"), status_tensor()
    for turn, M in enumerate(order):
        x = x_dev(WL.make_x(cfg, M, K, stream=turn))
        ids = torch.randint(-1, 3, (M,), generator=g, device="cuda", dtype=torch.int32)
        y, want = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        for to, buf in ((y, ws), (want, torch.zeros(size, dtype=torch.uint8, device="cuda"))):
            ans.ans_gemm_lora(x, M, layer.tiles, cfg.scale_kind, sc, cfg.group_k, A.lora, ids, to, buf, size, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        same = torch.equal(y, want)
        assert same, f"M {M}, turn {turn}"
