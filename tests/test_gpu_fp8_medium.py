"""FP8 experts of some dozens of rows (tiles of 64 columns, whose weight ring has three slots), with a
last step of one block, whose copy is the shorter one and can land before the step in front of it."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
from parity import REL_TOL
from test_tile_rule import tile_width

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("N,K", [(94, 3408), (300, 3408), (1000, 1408), (640, 5120), (128, 384), (2048, 1104)])
@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_ragged_experts(fmt, N, K):
    E, T = 200, 6000
    g = torch.Generator(device=DEV).manual_seed(N + K)
    rng = np.random.default_rng(N + K)
    while E * N * K > 6e8:
        E, T = E // 2, T // 2
    share = rng.gamma(1.0, size=E) + 1e-3
    off = np.concatenate([[0], np.cumsum(rng.multinomial(T, share / share.sum()))]).astype(np.int32)
    for workspace in (0, 1):
        assert tile_width(int(fmt == "fp8"), T, K, N, E, 0, workspace, 148) == 64
    x = torch.randn((T, K), generator=g, device=DEV).half()
    scale = torch.rand((E, N), generator=g, device=DEV) + 0.5
    if fmt == "fp8":
        codes = (torch.randn((E, N, K), generator=g, device=DEV) * 90).clamp_(-448, 448).to(torch.float8_e4m3fn)
        w = sk.PackedExpertsFP8.from_logical(codes.view(torch.uint8), scale)
        weight = lambda e: codes[e].double() * scale[e].double()[:, None]
    else:
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        block = torch.randint(0x18, 0x59, (E, N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
        w = sk.PackedExpertsNVFP4.from_logical(codes, block, scale[:, 0].contiguous())
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
        table = torch.cat((table, -table))

        def weight(e):
            c = torch.stack((codes[e] & 15, codes[e] >> 4), -1).view(N, K).int()
            return table[c] * block[e].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * scale[e, 0].double()

    ref = torch.empty((T, N), dtype=torch.float64, device=DEV)
    bound = torch.empty_like(ref)
    for e in range(E):
        rows = slice(int(off[e]), int(off[e + 1]))
        v, xe = weight(e), x[rows].double()
        ref[rows], bound[rows] = xe @ v.T, xe.abs() @ v.abs().T
    offsets = torch.from_numpy(off).to(DEV)
    for ws in (None, sk.make_experts_workspace(), None):
        for _ in range(5):
            y = sk.gemm_experts(x, w, offsets, torch.float32, workspace=ws)
            torch.cuda.synchronize()
            assert sk.tile_device_error(clear=True) == 0
            assert bool(((y.double() - ref).abs() <= REL_TOL * bound).all())
