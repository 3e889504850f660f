"""Kernels that read what the library's kernel just before them writes, in a replayed CUDA
graph, where the two launches overlap (programmatic dependent launch): each replay gives what
the same calls give one by one."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
import synthetic_inputs as si

pytestmark = pytest.mark.gpu

DEV = "cuda"
IN = 512


def dev(a):
    return torch.from_numpy(a).to(DEV)


def producer(kind, M, N, dtype):
    """A call that fills y [M, N] from an input, and that input's tensor."""
    y = torch.zeros((M, N), dtype=dtype, device=DEV)
    if kind == "int8":
        x = torch.zeros((M, IN), dtype=torch.int8, device=DEV)
        c = torch.randint(-127, 128, (N, IN), device=DEV).to(torch.int8)
        w, one = sk.WeightInt8(c, torch.full((N,), 1e-3, device=DEV)), torch.ones(M, device=DEV)
        ws = sk.make_int8_workspace()
        return (lambda: sk.gemm_int8_into(y, x, one, w, workspace=ws)), x, y
    x = torch.zeros((M, IN), dtype=torch.float16, device=DEV)
    if kind == "skinny":
        w = sk.PackedNVFP4.from_logical(*si.nvfp4_weights(N, IN, seed=1), 1 / 448)
        ws = sk.make_workspace(sk.FMT_NVFP4, M, N, IN)
        return (lambda: sk.gemm_into(y, x, w, workspace=ws)), x, y
    parts = [si.nvfp4_weights(N, IN, seed=1, tensor_id=2 * e) for e in range(2)]
    w = sk.PackedExpertsNVFP4.from_logical(np.stack([c for c, _ in parts]), np.stack([s for _, s in parts]),
                                           np.full(2, 1 / 448, np.float32))
    off, ws = dev(np.array([0, M // 2, M], np.int32)), sk.make_experts_workspace()
    return (lambda: sk.gemm_experts_into(y, x, w, off, workspace=ws)), x, y


def refill(x):
    x.copy_(torch.randint(-127, 128, x.shape, device=DEV) if x.dtype == torch.int8 else torch.randn(x.shape, device=DEV))


def check(steps, x, outputs):
    """`steps` in one replayed graph against `steps` with a synchronisation after each."""
    for step in steps:
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for step in steps:
            step()
    for _ in range(8):
        refill(x)
        for t in outputs:
            t.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outputs]
        for step in steps:
            step()
            torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, outputs))
    assert sk.tile_device_error(clear=True) == 0 and sk.device_error(clear=True) == 0


# 1040 columns stay in registers, 40000 are read twice
@pytest.mark.parametrize("N", [1040, 40000])
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("kind", ["skinny", "experts", "int8"])
@pytest.mark.parametrize("M", [2, 12])
def test_quantize_reads_what_a_product_wrote(M, kind, dtype, N):
    call, x, y = producer(kind, M, N, dtype)
    q, scale = torch.zeros((M, N), dtype=torch.int8, device=DEV), torch.zeros(M, device=DEV)
    check([call, lambda: sk.quantize_int8_into(q, scale, y)], x, [y, q, scale])


@pytest.mark.parametrize("kind", ["skinny", "experts", "int8"])
def test_verify_reads_what_a_product_wrote(kind):
    B, S, V = 2, 3, 5000
    call, x, y = producer(kind, B * (S + 1), V, torch.float32)
    drafted = torch.randint(0, V, (B, S), device=DEV, dtype=torch.int32)
    u = torch.full((B, S + 1), 0.5, device=DEV)
    tokens = torch.zeros((B, S + 1), dtype=torch.int32, device=DEV)
    accepted = torch.zeros(B, dtype=torch.int32, device=DEV)
    check([call, lambda: sk.verify_draft_into(tokens, accepted, y.view(B, S + 1, V), None, drafted, u)], x,
          [y, tokens, accepted])


@pytest.mark.parametrize("kind", ["skinny", "experts"])
def test_int8_product_reads_what_quantize_wrote_of_a_product(kind):
    M, N, out = 12, 1040, 700
    call, x, y = producer(kind, M, N, torch.float16)
    q, scale = torch.zeros((M, N), dtype=torch.int8, device=DEV), torch.zeros(M, device=DEV)
    w = sk.WeightInt8(torch.randint(-127, 128, (out, N), device=DEV).to(torch.int8), torch.ones(out, device=DEV))
    z, ws = torch.zeros((M, out), device=DEV), sk.make_int8_workspace()
    check([call, lambda: sk.quantize_int8_into(q, scale, y), lambda: sk.gemm_int8_into(z, q, scale, w, workspace=ws)], x,
          [y, q, scale, z])
