"""The skinny calls that allocate their outputs, with a stream other than the current one."""
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
import synthetic_inputs as si
from test_gpu_streams import stream_of, tensors

pytestmark = pytest.mark.gpu

DEV = "cuda"


def calls():
    M, N, K = 8, 65536, 128
    codes, scales = si.nvfp4_weights(N, K, seed=1)
    w, gu = sk.PackedNVFP4.from_logical(codes, scales, 1 / 448), sk.PackedGateUp.from_logical(codes, scales, 1 / 448)
    w8 = sk.PackedFP8.from_logical(*si.fp8_weights(N, K, seed=2))
    x = torch.randn((M, K), device=DEV).half()
    ws = sk.make_workspace(sk.FMT_NVFP4, M, N, K)
    return {
        "gemm": lambda s: sk.gemm(x, w, torch.float32, workspace=ws, stream=s),
        "gemm_fp8": lambda s: sk.gemm(x, w8, stream=s),
        "gemm_silu_mul": lambda s: sk.gemm_silu_mul(x, gu, workspace=ws, stream=s),
        "gemm_argmax": lambda s: sk.gemm_argmax(x, w, ws, stream=s),
    }


@pytest.mark.parametrize("name", ["gemm", "gemm_fp8", "gemm_silu_mul", "gemm_argmax"])
def test_outputs_belong_to_the_calls_stream(name):
    call, side = calls()[name], torch.cuda.Stream()
    expected = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    out = tensors(call(side))
    torch.cuda.synchronize()
    assert all(stream_of(t) == side.cuda_stream for t in out)
    assert all(torch.equal(a, b) for a, b in zip(out, expected))
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert all(stream_of(t) == 0 for t in tensors(call(None)))
    assert sk.device_error(clear=True) == 0
