"""Weights and workspaces that the kernels would read past are refused by the compiled binding.
Its checks of the weights come before the one of the device, so they run here."""
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk

BYTES = 9216          # of one packed NVFP4 block of 128 x 128


def nvfp4(**kw):
    a = dict(data=torch.zeros(2 * BYTES, dtype=torch.uint8), scale=torch.ones(2), E=2, N=128, K=128, gate_up=False)
    return sk.PackedExpertsNVFP4(**{**a, **kw})


def fp8(**kw):
    a = dict(data=torch.zeros(2 * 16384, dtype=torch.uint8), scale=torch.ones(2, 128), E=2, N=128, K=128, gate_up=False)
    return sk.PackedExpertsFP8(**{**a, **kw})


def run(w):
    call = sk.gemm_experts_silu_mul if w.gate_up else sk.gemm_experts
    call(torch.zeros((3, w.K), dtype=torch.float16), w, torch.zeros(w.E + 1, dtype=torch.int32))


def test_good_experts_come_as_far_as_the_device():
    for w in (nvfp4(), fp8(), nvfp4(gate_up=True, N=128), fp8(gate_up=True, N=128)):
        with pytest.raises(ValueError, match="CUDA device"):
            run(w)


@pytest.mark.parametrize("w,what", [
    (nvfp4(data=torch.zeros(2 * BYTES - 1, dtype=torch.uint8)), "data"),
    (nvfp4(data=torch.zeros(4 * BYTES, dtype=torch.uint8)[::2]), "data"),
    (nvfp4(data=torch.zeros(2 * BYTES, dtype=torch.int8)), "data"),
    (nvfp4(N=129), "data"),
    (nvfp4(K=144), "data"),
    (nvfp4(E=3), "data"),
    (nvfp4(N=256, gate_up=True), "data"),
    (nvfp4(scale=torch.ones(1)), "scale"),
    (nvfp4(scale=torch.ones(2).double()), "scale"),
    (nvfp4(scale=torch.ones(1).expand(2)), "scale"),
    (fp8(data=torch.zeros(2 * BYTES, dtype=torch.uint8)), "data"),
    (fp8(scale=torch.ones(2)), "scale"),
    (fp8(scale=torch.ones(2, 127)), "scale"),
    (fp8(scale=torch.ones(128, 2).T), "scale"),
])
def test_experts_that_do_not_fit_their_sizes(w, what):
    with pytest.raises(ValueError, match="^%s must be" % what):
        run(w)


def test_experts_of_no_shape():
    for w in (nvfp4(K=24), nvfp4(N=0), nvfp4(N=1, gate_up=True)):
        with pytest.raises(sk.SkinnyError):
            run(w)


def test_int8_weights_changed_after_they_were_checked():
    q, one = torch.zeros((2, 16), dtype=torch.int8), torch.ones(2)
    w = sk.WeightInt8(torch.zeros((4, 16), dtype=torch.int8), torch.ones(4))
    with pytest.raises(ValueError, match="CUDA device"):
        sk.gemm_int8(q, one, w)
    for codes, scale, what in ((torch.zeros(4, dtype=torch.int8), torch.ones(4), "codes"),
                               (torch.zeros((4, 16), dtype=torch.uint8), torch.ones(4), "codes"),
                               (torch.zeros((4, 32), dtype=torch.int8)[:, ::2], torch.ones(4), "codes"),
                               (torch.zeros((4, 16), dtype=torch.int8), torch.ones(3), "channel_scale"),
                               (torch.zeros((4, 16), dtype=torch.int8), torch.ones(4).half(), "channel_scale"),
                               (torch.zeros((4, 16), dtype=torch.int8), torch.ones(1).expand(4), "channel_scale")):
        w.codes, w.channel_scale = codes, scale
        with pytest.raises(ValueError, match="^%s must be" % what):
            sk.gemm_int8(q, one, w)


@pytest.mark.gpu
def test_a_workspace_with_gaps_is_refused():
    dev = "cuda"
    w = sk.WeightInt8(torch.zeros((64, 64), dtype=torch.int8, device=dev), torch.ones(64, device=dev))
    q, one = torch.zeros((1, 64), dtype=torch.int8, device=dev), torch.ones(1, device=dev)
    n = sk.tile_workspace_bytes()
    experts = nvfp4(data=torch.zeros(2 * BYTES, dtype=torch.uint8, device=dev), scale=torch.ones(2, device=dev))
    x, off = torch.zeros((3, 128), dtype=torch.float16, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    for ws in (torch.zeros(1, dtype=torch.uint8, device=dev).expand(n), torch.zeros(2 * n, dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            sk.gemm_int8(q, one, w, workspace=ws)
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            sk.gemm_experts(x, experts, off, workspace=ws)
