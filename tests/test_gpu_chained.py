"""A GEMM whose activations the kernel just before it on the stream writes, in
a replayed CUDA graph, where the two launches overlap (programmatic dependent
launch): the second has to see what the first wrote."""
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
import synthetic_inputs as si

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("M", [1, 4, 12])
def test_graph_replay_of_a_gemm_that_reads_the_previous_gemms_output(M):
    K, F, N = 1024, 1024, 1000
    wg = sk.PackedGateUp.from_logical(*si.nvfp4_weights(2 * F, K, seed=1), 1 / 448)
    wd = sk.PackedNVFP4.from_logical(*si.nvfp4_weights(N, F, seed=2), 1 / 448)
    q, s = si.fp8_weights(F, F, seed=3)
    wf = sk.PackedFP8.from_logical(q, s)
    ws = [sk.make_workspace(fmt, M, n, F) for fmt, n in ((sk.FMT_NVFP4, 2 * F), (sk.FMT_FP8, F), (sk.FMT_NVFP4, N))]
    x = torch.randn((M, K), device=DEV).half()
    h, h2 = (torch.zeros((M, F), dtype=torch.float16, device=DEV) for _ in range(2))
    y = torch.zeros((M, N), device=DEV)

    def run():
        sk.gemm_silu_mul_into(h, x, wg, workspace=ws[0])
        sk.gemm_into(h2, h, wf, workspace=ws[1])
        sk.gemm_into(y, h2, wd, workspace=ws[2])

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(10):
        x.copy_(torch.randn((M, K), device=DEV))
        h.fill_(7.0)
        h2.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        one_by_one = [t.clone() for t in (h, h2, y)]
        for step in (lambda: sk.gemm_silu_mul_into(h, x, wg, workspace=ws[0]),
                     lambda: sk.gemm_into(h2, h, wf, workspace=ws[1]), lambda: sk.gemm_into(y, h2, wd, workspace=ws[2])):
            step()
            torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(one_by_one, (h, h2, y)))
    assert sk.device_error(clear=True) == 0
