"""8-bit integer quantisation and products, bit for bit against numpy in 64 bits."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk

pytestmark = pytest.mark.gpu

DEV = "cuda"


def done():
    torch.cuda.synchronize()
    assert sk.tile_device_error(clear=True) == 0


def quantized(x):
    """(q, scale) by the definition: the scale an FP32 quotient, q the nearest whole number of the exact quotient."""
    top = np.abs(x.astype(np.float32)).max(axis=1)
    bad = ~np.isfinite(top)
    scale = (np.where(bad, 0, top) / np.float32(127)).astype(np.float32)
    safe = np.where(scale > 0, scale, 1).astype(np.float64)
    q = np.clip(np.rint(np.where(bad[:, None], 0, x).astype(np.float64) / safe[:, None]), -127, 127)
    q = np.where((scale > 0)[:, None], q, 0).astype(np.int8)
    return q, np.where(bad, np.float32(np.nan), scale).astype(np.float32)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 5120), (3, 48), (7, 1040), (513, 272), (600, 5120), (2, 17408),
                                 (520, 40000)])
def test_quantize(M, K, dtype):
    rng = np.random.default_rng(M * K)
    x = (rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))).astype(dtype)
    q, scale = sk.quantize_int8(torch.from_numpy(x).to(DEV))
    done()
    rq, rs = quantized(x)
    assert np.array_equal(scale.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quantize_ties_zeros_and_extremes():
    x = np.zeros((9, 32), np.float32)
    x[1] = np.arange(32) - 15.5                       # half-way quotients once the scale is 1/2 ...
    x[1, 0] = 63.5                                    # ... which this maximum makes it
    x[2, 0], x[2, 1:] = 127, np.arange(31) + 0.5      # scale 1: x.5 goes to the even side
    x[3, 5] = np.float32(1e-45)                       # the scale underflows to 0
    x[4] = np.float32(1e-42) * np.arange(32)          # a subnormal scale
    x[5, 3] = np.inf
    x[6, 4] = np.nan
    x[7] = np.float32(3e38) * np.linspace(-1, 1, 32, dtype=np.float32)
    x[8] = np.float32(1.5) * 3 * (np.arange(32) % 7)
    x[8, 0] = 381                                     # scale 3
    q, scale = sk.quantize_int8(torch.from_numpy(x).to(DEV))
    done()
    rq, rs = quantized(x)
    assert np.array_equal(scale.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)


def product(q, rs, c, cs, out):
    acc = q.astype(np.float64) @ c.astype(np.float64).T          # exact: below 2^53
    y = acc.astype(np.float32) * rs[:, None] * cs[None]          # FP32, in this order
    return y if out == torch.float32 else y.astype(np.float16)


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("out", [torch.float32, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 1, 16), (3, 129, 48), (8, 5120, 1040), (17, 300, 5120),
                                   (33, 640, 272), (61, 1000, 640), (129, 257, 144), (256, 512, 512),
                                   (300, 1100, 400), (700, 130, 2064), (513, 20000, 272), (100, 30001, 144)])
def test_product(M, N, K, out, split):
    rng = np.random.default_rng(M + N + K)
    q, c = rng.integers(-128, 128, (M, K), dtype=np.int8), rng.integers(-128, 128, (N, K), dtype=np.int8)
    rs, cs = (rng.uniform(0.5, 1.5, n).astype(np.float32) / 1000 for n in (M, N))
    w = sk.WeightInt8(torch.from_numpy(c).to(DEV), torch.from_numpy(cs).to(DEV))
    y = sk.gemm_int8(torch.from_numpy(q).to(DEV), torch.from_numpy(rs).to(DEV), w, out,
                     workspace=sk.make_int8_workspace() if split else None)
    done()
    assert np.array_equal(y.cpu().numpy(), product(q, rs, c, cs, out))


@pytest.mark.parametrize("M,N,K", [(20, 300, 5120), (61, 300, 5120), (61, 19000, 5120), (100, 19200, 5120),
                                   (300, 6400, 16384), (1020, 5120, 16384)])
def test_split_tiles_of_every_width(M, N, K):
    """Products whose last tiles are split along K (with 148 SMs), from 32 to 256 tokens wide."""
    rng = np.random.default_rng(M + N + K)
    q, c = rng.integers(-128, 128, (M, K), dtype=np.int8), rng.integers(-128, 128, (N, K), dtype=np.int8)
    rs, cs = (rng.uniform(0.5, 1.5, n).astype(np.float32) / 1000 for n in (M, N))
    d = lambda a: torch.from_numpy(a).to(DEV)
    w, dq, drs = sk.WeightInt8(d(c), d(cs)), d(q), d(rs)
    acc = dq.double() @ d(c).double().T                            # exact: below 2^53
    expected = acc.float() * drs[:, None] * d(cs)[None]
    for ws in (sk.make_int8_workspace(), None):
        assert torch.equal(sk.gemm_int8(dq, drs, w, torch.float32, workspace=ws), expected)
        if ws is not None:                                         # the flags are free again
            assert not ws[-32 * torch.cuda.get_device_properties(0).multi_processor_count:].any()
    done()


def test_largest_sums_do_not_wrap():
    K = 131056
    q = np.full((2, K), -128, np.int8)
    c = np.full((3, K), -128, np.int8)
    c[1] = 127
    one = lambda n: torch.ones(n, device=DEV)
    y = sk.gemm_int8(torch.from_numpy(q).to(DEV), one(2), sk.WeightInt8(torch.from_numpy(c).to(DEV), one(3)),
                     torch.float32, workspace=sk.make_int8_workspace())
    done()
    assert np.array_equal(y.cpu().numpy(), product(q, np.ones(2, np.float32), c, np.ones(3, np.float32), torch.float32))


def test_a_row_that_is_not_finite_comes_out_nan():
    x = np.random.default_rng(0).standard_normal((4, 256)).astype(np.float16)
    x[2, 9] = np.inf
    c = np.random.default_rng(1).integers(-127, 128, (40, 256), dtype=np.int8)
    w = sk.WeightInt8(torch.from_numpy(c).to(DEV), torch.ones(40, device=DEV))
    y = sk.gemm_int8(*sk.quantize_int8(torch.from_numpy(x).to(DEV)), w, torch.float32).cpu().numpy()
    assert np.isnan(y[2]).all() and np.isfinite(y[[0, 1, 3]]).all()
    done()


def test_workspace_serves_experts_and_int8_in_turn_and_in_graphs():
    """One workspace, calls of unlike shape back to back, captured and replayed."""
    rng = np.random.default_rng(5)
    ws = sk.make_int8_workspace()
    calls = []
    for M, N, K in ((1, 5120, 1024), (40, 300, 640), (3, 129, 272)):
        q, c = rng.integers(-128, 128, (M, K), dtype=np.int8), rng.integers(-128, 128, (N, K), dtype=np.int8)
        w = sk.WeightInt8(torch.from_numpy(c).to(DEV), torch.ones(N, device=DEV))
        y = torch.zeros((M, N), device=DEV)
        calls.append((y, torch.from_numpy(q).to(DEV), torch.ones(M, device=DEV), w, product(
            q, np.ones(M, np.float32), c, np.ones(N, np.float32), torch.float32)))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            for y, q, rs, w, _ in calls:
                sk.gemm_int8_into(y, q, rs, w, workspace=ws)
    for _ in range(3):
        for graph in graphs:
            for y, *_ in calls:
                y.zero_()
            graph.replay()
            done()
            for y, *_, ref in calls:
                assert np.array_equal(y.cpu().numpy(), ref)


def test_no_rows():
    w = sk.WeightInt8(torch.zeros((16, 32), dtype=torch.int8, device=DEV), torch.ones(16, device=DEV))
    q, rs = sk.quantize_int8(torch.empty((0, 32), dtype=torch.float16, device=DEV))
    assert sk.gemm_int8(q, rs, w).shape == (0, 16)
    done()
