"""Products of random sizes over the allowed range, between guard values, against torch in 64 bits."""
import math
import random

import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
from parity import REL_TOL

pytestmark = pytest.mark.gpu

DEV = "cuda"
E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6]


def log(r, lo, hi):
    return int(round(math.exp(r.uniform(math.log(lo), math.log(hi)))))


def guarded(shape, dtype):
    """A tensor of sevens inside a larger one."""
    n = math.prod(shape)
    buf = torch.full((n + 512,), 7.0, dtype=dtype, device=DEV)
    return buf, buf[256:256 + n].view(shape)


def done(buf):
    torch.cuda.synchronize()
    assert sk.tile_device_error(clear=True) == 0
    assert bool((buf[:256] == 7).all()) and bool((buf[-256:] == 7).all())


def f16_step(v):
    """At most half a step of FP16 at v (subnormals: half of 2^-24)."""
    return v.abs() * 2.0**-11 + 2.0**-25


@pytest.mark.parametrize("seed", range(60))
def test_experts(seed):
    r, g = random.Random(seed), torch.Generator(device=DEV).manual_seed(seed)
    fmt, silu, out = r.choice(["nvfp4", "fp8"]), r.random() < 0.5, r.choice([torch.float16, torch.float32])
    E, K, F, T = r.choice([1, 2, 3, 7, 16, 33, 64, 200, 512]), 16 * log(r, 1, 300), log(r, 1, 2500), log(r, 1, 8000)
    while E * F * K > 6e7:
        E, F = max(1, E // 2), max(1, 2 * F // 3)
    while T * max(K, F) > 2e7:
        T //= 2
    N = 2 * F if silu else F
    first, behind = (r.choice([0, 0, 4]), r.choice([0, 0, 3])) if T > 20 else (0, 0)
    rng = np.random.default_rng(seed)
    share = rng.gamma(r.choice([0.1, 1, 10]), size=E) + 1e-3
    off = np.concatenate([[0], np.cumsum(rng.multinomial(T - first - behind, share / share.sum()))]) + first
    x = torch.randn((T, K), generator=g, device=DEV).half()
    x[:first], x[T - behind:] = float("nan"), float("inf")
    if fmt == "nvfp4":
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        block = torch.randint(0, 0x7F, (E, N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
        scale = (torch.rand(E, generator=g, device=DEV) + 0.5) / 1e4
        w = sk.PackedExpertsNVFP4.from_logical(codes, block, scale, gate_up=silu)
        table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=DEV)
    else:
        codes = torch.randint(0, 256, (E, N, K), generator=g, device=DEV, dtype=torch.uint8)
        codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes)
        scale = (torch.rand((E, N), generator=g, device=DEV) + 0.5) / 1e4
        w = sk.PackedExpertsFP8.from_logical(codes, scale, gate_up=silu)
    buf, y = guarded((T, F), out)
    call = sk.gemm_experts_silu_mul_into if silu else sk.gemm_experts_into
    call(y, x, w, torch.from_numpy(off.astype(np.int32)).to(DEV), workspace=sk.make_experts_workspace() if r.random() < 0.7 else None)
    done(buf)
    assert bool((y[:first] == 7).all()) and bool((y[T - behind:] == 7).all())
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        if a == b:
            continue
        if fmt == "nvfp4":
            c = torch.stack((codes[e] & 15, codes[e] >> 4), -1).view(N, K).int()
            v = table[c] * block[e].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1) * scale[e].double()
        else:
            v = codes[e].view(torch.float8_e4m3fn).double() * scale[e].double()[:, None]
        xe = x[a:b].double()
        ref, tol = xe @ v.T, REL_TOL * (xe.abs() @ v.abs().T)
        if silu:
            # |d silu / dz| <= 1.1 and |silu(z)| <= |z|, then the activation's own FP32 steps
            gate, up = ref.chunk(2, 1)
            dg, du = tol.chunk(2, 1)
            ref = gate * torch.sigmoid(gate) * up
            tol = 1.1 * dg * (up.abs() + du) + gate.abs() * du + 1e-6 * ref.abs() + 1e-30
        if out == torch.float16:
            tol = tol + f16_step(ref.abs() + tol)
        got = y[a:b].double()
        fits = ref.abs() + tol < 65504 if out == torch.float16 else torch.ones_like(ref, dtype=torch.bool)
        assert bool(((got - ref).abs() <= tol)[fits].all()), (fmt, E, N, K, T, e)


@pytest.mark.parametrize("seed", range(30))
def test_int8(seed):
    r, g = random.Random(1000 + seed), torch.Generator(device=DEV).manual_seed(seed)
    M, N, K, out = log(r, 1, 6000), log(r, 1, 20000), 16 * log(r, 1, 500), r.choice([torch.float16, torch.float32])
    while N * max(M, K) > 4e7:
        N = max(1, N // 2)
    q, c = (torch.randint(-128, 128, (n, K), generator=g, device=DEV).to(torch.int8) for n in (M, N))
    rs, cs = torch.rand(M, generator=g, device=DEV) / 1000, torch.rand(N, generator=g, device=DEV)
    buf, y = guarded((M, N), out)
    sk.gemm_int8_into(y, q, rs, sk.WeightInt8(c, cs), workspace=sk.make_int8_workspace() if r.random() < 0.7 else None)
    done(buf)
    # the sum is exact (below 2^53), then FP32 steps in the documented order
    assert torch.equal(y, ((q.double() @ c.double().T).float() * rs[:, None] * cs[None]).to(out)), (M, N, K)
