"""The tile GEMM at the tile widths that the tests mean (of 148 SMs)."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
import oracle
from parity import REL_TOL, assert_parity, ulp16
from test_gpu_experts import dev, done, expected, make, offsets_of
from test_tile_rule import INT8_LAST_TILE, SILU_WIDE, STORE_WIDE, tile_width

pytestmark = pytest.mark.gpu

DEV = "cuda"


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def assert_width(width, *sizes):
    if sms() == 148:
        assert [tile_width(*sizes, workspace, 148) for workspace in (0, 1)] == [width, width]


def looked_at(off, every):
    """Rows to look at: one in `every`, the first and the last of each expert."""
    rows = set(range(0, int(off[-1]), every))
    for a, b in zip(off[:-1], off[1:]):
        rows |= {int(a), int(b) - 1} if a < b else set()
    return np.array(sorted(rows))


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("F,K,counts,width", SILU_WIDE)
@pytest.mark.parametrize("fmt", ["nvfp4", "fp8"])
def test_silu_mul(fmt, F, K, counts, width, out):
    off = offsets_of(counts)
    assert_width(width, int(fmt == "fp8"), int(off[-1]), K, 2 * F, len(counts), 1)
    logical, w, x = make(fmt, len(counts), 2 * F, K, int(off[-1]), gate_up=True)
    rows = looked_at(off, 11)
    ref, bound = expected(fmt, logical, x[rows], np.searchsorted(rows, off))
    h = oracle.silu_mul(ref)
    # as in test_gpu_experts.test_silu_mul: |d silu / dz| <= 1.1, |silu(z)| <= |z|, FP32 steps
    dg, du = REL_TOL * bound[:, :F], REL_TOL * bound[:, F:]
    tol = 1.1 * dg * (np.abs(ref[:, F:]) + du) + np.abs(ref[:, :F]) * du + 1e-6 * np.abs(h) + 1e-30
    if out == "f16":
        tol = tol + 0.5 * ulp16(np.abs(h) + tol)
    T = int(off[-1])
    for ws in (sk.make_experts_workspace(), None):
        y = torch.full((T + 1, F), 7.0, dtype=torch.float32 if out == "f32" else torch.float16, device=DEV)
        sk.gemm_experts_silu_mul_into(y[:T], dev(x), w, dev(off), workspace=ws)
        done()
        got = y[:T].double().cpu().numpy()[rows]
        assert np.all(np.abs(got - h) <= tol), np.max(np.abs(got - h) / tol)
        assert bool((y[T] == 7).all()) and bool(torch.isfinite(y).all())
        if ws is not None:
            assert not ws[-32 * sms():].any()       # the flags are free again


@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("fmt,N,K,counts,width", STORE_WIDE)
def test_store(fmt, N, K, counts, width, out):
    off = offsets_of(counts)
    assert_width(width, fmt, int(off[-1]), K, N, len(counts), 0)
    name = ("nvfp4", "fp8")[fmt]
    logical, w, x = make(name, len(counts), N, K, int(off[-1]))
    rows = looked_at(off, 11)
    ref, bound = expected(name, logical, x[rows], np.searchsorted(rows, off))
    for ws in (sk.make_experts_workspace(), None):
        y = sk.gemm_experts(dev(x), w, dev(off), torch.float32 if out == "f32" else torch.float16, workspace=ws)
        done()
        assert_parity(y.double().cpu().numpy()[rows], ref, bound, out, "%s %dx%d %s" % (name, N, K, counts))


@pytest.mark.parametrize("M,N,K", INT8_LAST_TILE)
def test_int8_last_tile_of_a_few_tokens(M, N, K):
    """A pair's last tile holds 1 to 4 tokens: the smallest matrix instruction of 256 rows."""
    assert_width(256, -1, M, K, N, 1, 0)
    rng = np.random.default_rng(M)
    d = lambda a: torch.from_numpy(a).to(DEV)
    q, c = (d(rng.integers(-128, 128, shape, dtype=np.int8)) for shape in ((M, K), (N, K)))
    rs, cs = (d(rng.uniform(0.5, 1.5, n).astype(np.float32) / 1000) for n in (M, N))
    w = sk.WeightInt8(c, cs)
    expected = (q.double() @ c.double().T).float() * rs[:, None] * cs[None]      # the sum is exact: below 2^53
    for ws in (sk.make_int8_workspace(), None):
        assert torch.equal(sk.gemm_int8(q, rs, w, torch.float32, workspace=ws), expected)
        done()
