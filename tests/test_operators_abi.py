"""Argument checks of the expert-grouped, int8 and verification calls that run before any CUDA call."""
import ctypes

import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk

ALIGNED = 1 << 20  # a fake address: never dereferenced by these checks
BIG = 1 << 40


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), sk.ERR_INVALID_ARG),
    (dict(fmt=-1), sk.ERR_INVALID_ARG),
    (dict(T=-1), sk.ERR_INVALID_ARG),
    (dict(K=40), sk.ERR_INVALID_ARG),
    (dict(K=0), sk.ERR_INVALID_ARG),
    (dict(N=0), sk.ERR_INVALID_ARG),
    (dict(N=-(1 << 62)), sk.ERR_INVALID_ARG),
    (dict(E=0), sk.ERR_INVALID_ARG),
    (dict(out=5), sk.ERR_INVALID_ARG),
    (dict(x=None), sk.ERR_INVALID_ARG),
    (dict(off=None), sk.ERR_INVALID_ARG),
    (dict(w=None), sk.ERR_INVALID_ARG),
    (dict(s=None), sk.ERR_INVALID_ARG),
    (dict(y=None), sk.ERR_INVALID_ARG),
    (dict(E=513), sk.ERR_UNSUPPORTED),
    (dict(T=BIG), sk.ERR_UNSUPPORTED),
    (dict(K=1 << 21), sk.ERR_UNSUPPORTED),
    (dict(T=1 << 24, N=1 << 23, K=16), sk.ERR_UNSUPPORTED),      # more tiles than 31 bits count
    (dict(x=ALIGNED + 8), sk.ERR_ALIGNMENT),
    (dict(off=ALIGNED + 2), sk.ERR_ALIGNMENT),
    (dict(w=ALIGNED + 4), sk.ERR_ALIGNMENT),
    (dict(y=ALIGNED + 1), sk.ERR_ALIGNMENT),
    (dict(y=ALIGNED + 2, out=1), sk.ERR_ALIGNMENT),
    (dict(ws=ALIGNED + 8), sk.ERR_ALIGNMENT),
    (dict(T=0, x=None), sk.OK),
])
def test_experts_argument_checks(kw, status, silu):
    a = dict(fmt=0, x=ALIGNED, T=3, K=64, off=ALIGNED, E=2, w=ALIGNED, s=ALIGNED, N=64, y=ALIGNED, out=0, ws=None)
    a.update(kw)
    fn = sk.library().skinny_gemm_experts_silu_mul if silu else sk.library().skinny_gemm_experts
    assert fn(a["fmt"], a["x"], a["T"], a["K"], a["off"], a["E"], a["w"], a["s"], a["N"], a["y"], a["out"], a["ws"],
              0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), sk.ERR_INVALID_ARG),
    (dict(K=24), sk.ERR_INVALID_ARG),
    (dict(N=0), sk.ERR_INVALID_ARG),
    (dict(out=2), sk.ERR_INVALID_ARG),
    (dict(q=None), sk.ERR_INVALID_ARG),
    (dict(rs=None), sk.ERR_INVALID_ARG),
    (dict(w=None), sk.ERR_INVALID_ARG),
    (dict(cs=None), sk.ERR_INVALID_ARG),
    (dict(y=None), sk.ERR_INVALID_ARG),
    (dict(K=131072), sk.ERR_UNSUPPORTED),                         # sums could pass 31 bits
    (dict(M=BIG), sk.ERR_UNSUPPORTED),
    (dict(q=ALIGNED + 8), sk.ERR_ALIGNMENT),
    (dict(w=ALIGNED + 8), sk.ERR_ALIGNMENT),
    (dict(rs=ALIGNED + 2), sk.ERR_ALIGNMENT),
    (dict(cs=ALIGNED + 2), sk.ERR_ALIGNMENT),
    (dict(ws=ALIGNED + 4), sk.ERR_ALIGNMENT),
    (dict(M=0, q=None), sk.OK),
])
def test_int8_argument_checks(kw, status):
    a = dict(q=ALIGNED, rs=ALIGNED, M=3, K=64, w=ALIGNED, cs=ALIGNED, N=64, y=ALIGNED, out=0, ws=None)
    a.update(kw)
    assert sk.library().skinny_int8_gemm(a["q"], a["rs"], a["M"], a["K"], a["w"], a["cs"], a["N"], a["y"], a["out"],
                                         a["ws"], 0, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), sk.ERR_INVALID_ARG),
    (dict(K=20), sk.ERR_INVALID_ARG),
    (dict(x=None), sk.ERR_INVALID_ARG),
    (dict(q=None), sk.ERR_INVALID_ARG),
    (dict(s=None), sk.ERR_INVALID_ARG),
    (dict(M=BIG), sk.ERR_UNSUPPORTED),
    (dict(x=ALIGNED + 8), sk.ERR_ALIGNMENT),
    (dict(q=ALIGNED + 8), sk.ERR_ALIGNMENT),
    (dict(M=0, x=None), sk.OK),
])
def test_quantize_argument_checks(kw, status):
    a = dict(x=ALIGNED, dt=0, M=3, K=64, q=ALIGNED, s=ALIGNED)
    a.update(kw)
    assert sk.library().skinny_quantize_int8(a["x"], a["dt"], a["M"], a["K"], a["q"], a["s"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dt=3), sk.ERR_INVALID_ARG),
    (dict(B=-1), sk.ERR_INVALID_ARG),
    (dict(S=-1), sk.ERR_INVALID_ARG),
    (dict(V=0), sk.ERR_INVALID_ARG),
    (dict(target=None), sk.ERR_INVALID_ARG),
    (dict(drafted=None), sk.ERR_INVALID_ARG),
    (dict(u=None), sk.ERR_INVALID_ARG),
    (dict(tokens=None), sk.ERR_INVALID_ARG),
    (dict(accepted=None), sk.ERR_INVALID_ARG),
    (dict(S=1025), sk.ERR_UNSUPPORTED),
    (dict(V=BIG), sk.ERR_UNSUPPORTED),
    (dict(B=BIG), sk.ERR_UNSUPPORTED),
    (dict(target=ALIGNED + 2), sk.ERR_ALIGNMENT),
    (dict(draft=ALIGNED + 1), sk.ERR_ALIGNMENT),
    (dict(tokens=ALIGNED + 1), sk.ERR_ALIGNMENT),
    (dict(B=0, target=None), sk.OK),
])
def test_verify_argument_checks(kw, status):
    a = dict(target=ALIGNED, draft=ALIGNED, dt=1, drafted=ALIGNED, u=ALIGNED, count=None, B=2, S=3, V=100,
             tokens=ALIGNED, accepted=ALIGNED)
    a.update(kw)
    assert sk.library().skinny_verify_draft(a["target"], 400, 100, a["draft"], 300, 100, a["dt"], a["drafted"], a["u"],
                                            a["count"], a["B"], a["S"], a["V"], a["tokens"], a["accepted"],
                                            None) == status


def test_packed_sizes_and_refusals():
    lib = sk.library()
    size = lib.skinny_experts_packed_bytes
    assert size(0, 3, 129, 144, 0) == 3 * 2 * 2 * 9216 and size(1, 3, 129, 144, 0) == 3 * 2 * 2 * 16384
    assert size(0, 1, 130, 128, 1) == 2 * 9216                    # 65 outputs: two tiles of 64
    for bad in ((2, 1, 128, 128, 0), (0, 0, 128, 128, 0), (0, 513, 128, 128, 0), (0, 1, 0, 128, 0), (0, 1, 128, 8, 0),
                (0, 1, 129, 128, 1), (0, 1, 1 << 25, 128, 0), (0, 1, 128, 1 << 21, 0)):
        assert size(*bad) == 0
    assert lib.skinny_pack_experts(0, None, ALIGNED, 1, 128, 128, 0, ALIGNED, None) == sk.ERR_INVALID_ARG
    assert lib.skinny_pack_experts(0, ALIGNED, None, 1, 128, 128, 0, ALIGNED, None) == sk.ERR_INVALID_ARG
    assert lib.skinny_pack_experts(0, ALIGNED, ALIGNED, 1, 128, 128, 0, ALIGNED + 4, None) == sk.ERR_ALIGNMENT
    assert lib.skinny_pack_experts(0, ALIGNED + 4, ALIGNED, 1, 128, 128, 0, ALIGNED, None) == sk.ERR_ALIGNMENT
    assert lib.skinny_tile_workspace_bytes(None) == sk.ERR_INVALID_ARG
    assert lib.skinny_tile_device_error(0, None) == sk.ERR_INVALID_ARG


def test_binding_refuses_bad_tensors():
    """The Python binding's own checks: no GPU, no launch."""
    half = lambda *s: torch.zeros(s, dtype=torch.float16)
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)
    w = sk.PackedExpertsNVFP4(torch.zeros(9216, dtype=torch.uint8), torch.ones(1), 1, 128, 128, False)
    for x, off, y, err in ((half(2, 128).float(), ints(2), half(2, 128), ValueError),
                           (half(2, 256)[:, ::2], ints(2), half(2, 128), ValueError),
                           (half(2, 64), ints(2), half(2, 128), ValueError),
                           (half(2, 128), ints(3), half(2, 128), ValueError),
                           (half(2, 128), ints(2).long(), half(2, 128), ValueError),
                           (half(2, 128), ints(2), half(3, 128), ValueError),
                           (half(2, 128), ints(2), half(2, 128).bfloat16(), ValueError),
                           (half(2, 128), ints(2), half(2, 128), ValueError)):      # the last one: not on a GPU
        with pytest.raises(err):
            sk.gemm_experts_into(y, x, w, off)
    with pytest.raises(TypeError):
        sk.gemm_experts_silu_mul_into(half(2, 64), half(2, 128), w, ints(2))
    with pytest.raises(ValueError):
        sk.WeightInt8(torch.zeros((4, 16)), torch.ones(4))
    with pytest.raises(ValueError):
        sk.WeightInt8(torch.zeros((4, 16), dtype=torch.int8), torch.ones(3))
    w8 = sk.WeightInt8(torch.zeros((4, 16), dtype=torch.int8), torch.ones(4))
    assert (w8.N, w8.K) == (4, 16)
    with pytest.raises(ValueError):
        sk.gemm_int8(torch.zeros((2, 32), dtype=torch.int8), torch.ones(2), w8)
    with pytest.raises(ValueError):
        sk.gemm_int8(torch.zeros((2, 16), dtype=torch.int8), torch.ones(3), w8)
    with pytest.raises(ValueError):
        sk.quantize_int8(torch.zeros((2, 16), dtype=torch.bfloat16))
    p = torch.zeros((2, 3, 10))
    good = dict(target=p, draft=p[:, :2], draft_tokens=ints(2, 2), uniform=torch.zeros(2, 3), num_drafts=None)
    for bad in (dict(target=p.double()), dict(target=p[0]), dict(target=p.transpose(1, 2)), dict(draft=p),
                dict(draft=p[:, :2].half()), dict(draft_tokens=ints(2, 3)), dict(draft_tokens=ints(2, 2).long()),
                dict(uniform=torch.zeros(2, 2)), dict(num_drafts=ints(3)), dict()):          # the last one: not on a GPU
        with pytest.raises(ValueError):
            sk.verify_draft(**{**good, **bad})
    with pytest.raises(ValueError):
        sk.PackedExpertsNVFP4.from_logical(torch.zeros((1, 4, 8), dtype=torch.uint8),
                                           torch.full((1, 4, 1), 0x7F, dtype=torch.uint8), torch.ones(1), device="cpu")
    with pytest.raises(ValueError):
        sk.PackedExpertsFP8.from_logical(torch.full((1, 4, 16), 0xFF, dtype=torch.uint8), torch.ones((1, 4)),
                                         device="cpu")
