"""Shared helpers for the tests of the adapter, gradient and loss operators:
random layers of every coded format, with their weights in 64 bits."""
import numpy as np
import torch

from rans_decode_gemm_b200 import ans

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
NIBBLES = (ans.INT4, ans.INT4_PAIRS, ans.FP4_E2M1, ans.FP4_PAIRS)
ALL = [ans.INT4, ans.BF16_SPLIT, ans.FP8_E4M3, ans.INT4_PAIRS, ans.INT8, ans.FP4_E2M1, ans.FP4_PAIRS]

# Unit steps of the roundings that the operators make: half a step relative to
# the value.  fp32 sums on the tensor cores: at most a step of 2^-23 for each
# block of 16 products (they may truncate), and some for joining partial sums.
BF16, F16 = 2.0 ** -8, 2.0 ** -11


def sum_eps(terms):
    return (terms / 16 + 32) * 2.0 ** -23


class Layer:
    """codes, scales and the layer on the device; w: the weights' values in 64 bits."""

    def __init__(self, dtype, N, K, tile_n, tile_k, scale_kind=ans.SCALE_NONE, group_k=0, seed=0, state_bits=64,
                 device="cuda"):
        rng = np.random.default_rng([seed, dtype, N, K])
        self.dtype, self.N, self.K, self.kind, self.group_k = dtype, N, K, scale_kind, group_k
        if dtype in NIBBLES:
            # skewed, so that the codebook has short and long symbols
            nib = (rng.integers(0, 16, (N, K)) & rng.integers(0, 16, (N, K))).astype(np.uint8)
            if dtype in (ans.INT4, ans.INT4_PAIRS):
                v = nib.astype(np.float64) - 16.0 * (nib > 7)
            else:
                v = E2M1[nib]
            self.codes = (nib[:, 0::2] | (nib[:, 1::2] << 4)).astype(np.uint8)
        elif dtype == ans.BF16_SPLIT:
            t = torch.from_numpy((rng.standard_normal((N, K)) * 0.05).astype(np.float32)).bfloat16()
            self.codes = t.view(torch.int16).numpy().view(np.uint16)
            v = t.double().numpy()
        elif dtype == ans.FP8_E4M3:
            t = torch.from_numpy((rng.standard_normal((N, K)) * 20).astype(np.float32)).to(torch.float8_e4m3fn)
            self.codes = t.view(torch.uint8).numpy()
            v = t.double().numpy()
        else:
            q = np.clip(np.rint(rng.standard_normal((N, K)) * 30), -128, 127).astype(np.int8)
            self.codes = q.view(np.uint8)
            v = q.astype(np.float64)
        self.scales = None
        if scale_kind == ans.SCALE_ROW_F32:
            s = rng.uniform(1e-3, 4e-3, N).astype(np.float32)
            v = v * s.astype(np.float64)[:, None]
            self.scales = torch.from_numpy(s).to(device)
        elif scale_kind == ans.SCALE_ROW_BF16:
            s = torch.from_numpy(rng.uniform(5e-3, 2e-2, N).astype(np.float32)).bfloat16()
            v = v * s.double().numpy()[:, None]
            self.scales = s.to(device)
        elif scale_kind == ans.SCALE_GROUP_BF16:
            s = torch.from_numpy(rng.uniform(3e-3, 3e-2, (N, K // group_k)).astype(np.float32)).bfloat16()
            v = v * np.repeat(s.double().numpy(), group_k, axis=1)
            self.scales = s.to(device)
        self.w = torch.from_numpy(np.ascontiguousarray(v))
        self.layout = ans.make_layout(dtype, N, K, tile_n, tile_k, state_bits)
        self.layer = ans.CompressedLayer.from_weights(np.ascontiguousarray(self.codes).reshape(-1), self.layout,
                                                      device=device)
        self.tiles = self.layer.tiles

    @property
    def args(self):
        return self.tiles, self.kind, self.scales, self.group_k

    # rounding of a computed factor that meets these weights in a product
    @property
    def factor_eps(self):
        return BF16 if self.dtype == ans.BF16_SPLIT else F16


def usual(dtype, N, K, seed=0, **kw):
    """A layer with the scales its format is used with."""
    if dtype in (ans.INT4, ans.INT4_PAIRS):
        kind, group = (ans.SCALE_GROUP_BF16, 64) if K % 64 == 0 else (ans.SCALE_ROW_BF16, 0)
    elif dtype == ans.BF16_SPLIT:
        kind, group = ans.SCALE_NONE, 0
    else:
        kind, group = ans.SCALE_ROW_F32, 0
    return Layer(dtype, N, K, 256 if N % 256 == 0 and dtype in NIBBLES else 128, 64 if K % 64 == 0 else 16, kind, group,
                 seed, **kw)


def bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16()


def workspace(nbytes):
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device="cuda")


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def within(got, want, bound, what=""):
    """Every element of got within bound of want (64 bits, CPU)."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    off = (got - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (off / bound.clamp_min(1e-300)).max().item() if off.numel() else 0.0
    assert (off <= bound).all(), f"{what}: {worst:.3g} of the bound"
    return worst
