"""Calls with a stream other than the current one: what they allocate belongs to that stream."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk

pytestmark = pytest.mark.gpu

DEV = "cuda"


def calls():
    """name -> a call of `stream` that allocates its outputs, about 2 MB each."""
    E, N, K = 2, 2048, 128
    codes, scales = (torch.randint(0, 100, (E, N, n), dtype=torch.uint8) for n in (K // 2, K // 16))
    one = torch.ones(E)
    plain, gate_up = (sk.PackedExpertsNVFP4.from_logical(codes, scales, one, gate_up=g) for g in (False, True))
    x = torch.randn((512, K), device=DEV).half()
    off = torch.tensor([0, 200, 512], dtype=torch.int32, device=DEV)
    w8 = sk.WeightInt8(torch.randint(-127, 128, (N, K), device=DEV).to(torch.int8), torch.ones(N, device=DEV))
    q, rs = sk.quantize_int8(x)
    wide = torch.randn((512, 4096), device=DEV).half()
    B, S = 1024, 511                    # tokens [B, S + 1]: 2 MB
    p = torch.rand((1, 1, 4), device=DEV).expand(B, S + 1, 4)
    drafted, u = torch.zeros((B, S), dtype=torch.int32, device=DEV), torch.rand((B, S + 1), device=DEV)
    ws = sk.make_experts_workspace()
    return {
        "experts": lambda s: sk.gemm_experts(x, plain, off, workspace=ws, stream=s),
        "experts_silu_mul": lambda s: sk.gemm_experts_silu_mul(x, gate_up, off, torch.float32, workspace=ws, stream=s),
        "quantize": lambda s: sk.quantize_int8(wide, stream=s),
        "int8": lambda s: sk.gemm_int8(q, rs, w8, workspace=ws, stream=s),
        "verify": lambda s: sk.verify_draft(p, None, drafted, u, stream=s),
    }


NAMES = ["experts", "experts_silu_mul", "quantize", "int8", "verify"]


def stream_of(t):
    """The stream whose memory a tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


def tensors(out):
    return out if isinstance(out, tuple) else (out,)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_calls_stream(name):
    call, side = calls()[name], torch.cuda.Stream()
    torch.cuda.synchronize()
    expected = [t.clone() for t in tensors(call(None))]
    assert all(stream_of(t) == torch.cuda.current_stream().cuda_stream for t in tensors(call(None)))
    torch.cuda.synchronize()
    out = tensors(call(side))
    torch.cuda.synchronize()
    assert all(stream_of(t) == side.cuda_stream for t in out)
    assert all(torch.equal(a, b) for a, b in zip(out, expected))
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with torch.cuda.stream(side):       # the current one, if none is given
        assert all(stream_of(t) == side.cuda_stream for t in tensors(call(None)))
    torch.cuda.synchronize()
    assert all(stream_of(t) == 0 for t in tensors(call(torch.cuda.default_stream())))


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads_is_left_alone(name):
    call, side = calls()[name], torch.cuda.Stream()
    big = torch.randn((4096, 4096), device=DEV)
    shapes = [(t.shape, t.dtype) for t in tensors(call(None))]
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.ones(s, dtype=t, device=DEV) for s, t in shapes]
        for _ in range(10):
            big @ big                   # keeps the current stream busy
        sums = [h.double().sum() for h in held]
        del held                        # free for this stream's next allocation, while the sums wait
        out = call(side)
        torch.cuda.synchronize()
        assert [int(s) for s in sums] == [int(np.prod(s)) for s, _ in shapes]
        del out


def test_a_stream_that_is_none_is_refused():
    for name, call in calls().items():
        with pytest.raises(ValueError, match="stream must be"):
            call(17)
