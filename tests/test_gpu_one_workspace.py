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
