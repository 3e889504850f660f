"""Products grouped by expert against the float64 oracle, expert by expert: row
counts from none to several tiles, odd sizes, both formats and epilogues."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
import oracle
import synthetic_inputs as si
from parity import REL_TOL, assert_parity, ulp16

pytestmark = pytest.mark.gpu

DEV = "cuda"


def make(fmt, E, N, K, T, seed=0, gate_up=False):
    """Logical weights of each expert, the packed experts, and x."""
    logical = []
    if fmt == "nvfp4":
        for e in range(E):
            logical.append(si.nvfp4_weights(N, K, seed=seed, cfg_id=300, tensor_id=2 * e))
        g = np.linspace(0.5, 1.5, E).astype(np.float32) / np.float32(448)
        w = sk.PackedExpertsNVFP4.from_logical(np.stack([c for c, _ in logical]), np.stack([s for _, s in logical]), g,
                                               gate_up=gate_up, device=DEV)
        logical = [(c, s, float(g[e])) for e, (c, s) in enumerate(logical)]
    else:
        for e in range(E):
            logical.append(si.fp8_weights(N, K, seed=seed, cfg_id=301, tensor_id=2 * e))
        w = sk.PackedExpertsFP8.from_logical(np.stack([q for q, _ in logical]), np.stack([s for _, s in logical]),
                                             gate_up=gate_up, device=DEV)
    x = si.activations(max(T, 1), K, seed=seed, cfg_id=302)[:T]
    return logical, w, x


def expected(fmt, logical, x, offsets):
    """y and sum |w x| of every row that has an expert (NaN elsewhere), in float64."""
    N = logical[0][0].shape[0]
    y = np.full((x.shape[0], N), np.nan)
    b = np.zeros((x.shape[0], N))
    for e, parts in enumerate(logical):
        r0, r1 = int(offsets[e]), int(offsets[e + 1])
        if r0 < r1:
            y[r0:r1], b[r0:r1] = (oracle.nvfp4_gemm if fmt == "nvfp4" else oracle.fp8_gemm)(x[r0:r1], *parts)
    return y, b


def offsets_of(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


def dev(a):
    return torch.from_numpy(a).to(DEV)


def done():
    torch.cuda.synchronize()
    assert sk.tile_device_error(clear=True) == 0


CASES = [
    # fmt, N, K, rows per expert
    ("nvfp4", 256, 512, [1]),                            # one row, one expert
    ("nvfp4", 128, 16, [1, 0, 1]),                       # one sixteenth of a block
    ("nvfp4", 1, 144, [0, 3, 0]),                        # one output; a second, partial block
    ("nvfp4", 129, 1040, [2, 0, 17, 16, 1, 0]),
    ("nvfp4", 300, 640, [0, 0, 0, 40, 0, 5]),
    ("nvfp4", 384, 256, [33, 65, 128, 129]),
    ("nvfp4", 200, 272, [300, 1, 0, 257]),               # several token tiles of an expert
    ("nvfp4", 640, 5120, [1, 1, 0, 2]),
    ("fp8", 256, 512, [1]),
    ("fp8", 131, 272, [0, 7, 0, 31, 2]),
    ("fp8", 128, 1408, [90, 0, 130]),
    ("fp8", 77, 400, [600, 3]),
    ("nvfp4", 129, 1040, [10, 20, 13]),
    ("fp8", 129, 272, [30, 40, 1]),
    ("nvfp4", 260, 1040, [60, 50, 70]),
    ("fp8", 260, 400, [60, 50, 70]),
    ("nvfp4", 2000, 400, [400, 390, 5, 7, 300]),         # whole tiles next to split ones
    ("nvfp4", 20000, 144, [200, 130, 70, 1, 260]),
    ("fp8", 10001, 272, [200, 130, 70, 1, 260]),
]


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("fmt,N,K,counts", CASES)
def test_store(fmt, N, K, counts, out, split):
    off = offsets_of(counts)
    logical, w, x = make(fmt, len(counts), N, K, int(off[-1]))
    ws = sk.make_experts_workspace() if split else None
    y = sk.gemm_experts(dev(x), w, dev(off), torch.float32 if out == "f32" else torch.float16, workspace=ws)
    done()
    ref, bound = expected(fmt, logical, x, off)
    assert_parity(y.double().cpu().numpy(), ref, bound, out, "%s %dx%d %s" % (fmt, N, K, counts))
    if ws is not None:    # the flags are free again
        assert not ws[-32 * torch.cuda.get_device_properties(0).multi_processor_count:].any()


@pytest.mark.parametrize("fmt,N,K,counts", [
    ("nvfp4", 260, 5120, [20]),
    ("fp8", 300, 5120, [20, 0, 25]),
    ("nvfp4", 1000, 5120, [33, 64, 1]),
    ("nvfp4", 19200, 5120, [100]),
    ("fp8", 6400, 16384, [570]),
])
def test_split_tiles_of_every_width(fmt, N, K, counts):
    """Products whose last tiles are split along K (with 148 SMs), from 32 to 192 tokens wide;
    of many tokens every thirteenth is looked at."""
    off = offsets_of(counts)
    logical, w, x = make(fmt, len(counts), N, K, int(off[-1]))
    seen = np.arange(0, len(x), 13 if len(x) > 99 else 1)
    seen_off = np.searchsorted(seen, off).astype(np.int32)
    ref, bound = expected(fmt, logical, x[seen], seen_off)
    for ws in (sk.make_experts_workspace(), None):
        y = sk.gemm_experts(dev(x), w, dev(off), torch.float32, workspace=ws)
        done()
        assert_parity(y.double().cpu().numpy()[seen], ref, bound, "f32", "%s %dx%d %s" % (fmt, N, K, counts))
        if ws is not None:
            assert not ws[-32 * torch.cuda.get_device_properties(0).multi_processor_count:].any()


@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("fmt,F,K,counts", [
    ("nvfp4", 64, 512, [1]),
    ("nvfp4", 1, 16, [2, 0, 1]),
    ("nvfp4", 65, 1040, [2, 0, 17]),
    ("nvfp4", 200, 272, [300, 1, 0, 40]),
    ("fp8", 100, 400, [5, 0, 140]),
])
def test_silu_mul(fmt, F, K, counts, out):
    off = offsets_of(counts)
    logical, w, x = make(fmt, len(counts), 2 * F, K, int(off[-1]), gate_up=True)
    y = sk.gemm_experts_silu_mul(dev(x), w, dev(off), torch.float32 if out == "f32" else torch.float16,
                                 workspace=sk.make_experts_workspace())
    done()
    ref, bound = expected(fmt, logical, x, off)
    h = oracle.silu_mul(ref)
    # |d silu / dz| <= 1.1 and |silu(z)| <= |z|: gate and up each off by the sums' tolerance, then
    # the activation's own FP32 steps (a few 2^-24 each, and the clamp of e^-z at the FP32 range)
    dg, du = REL_TOL * bound[:, :F], REL_TOL * bound[:, F:]
    tol = 1.1 * dg * (np.abs(ref[:, F:]) + du) + np.abs(ref[:, :F]) * du + 1e-6 * np.abs(h) + 1e-30
    got = y.double().cpu().numpy()
    if out == "f16":
        tol = tol + 0.5 * ulp16(np.abs(h) + tol)
    assert np.all(np.abs(got - h) <= tol), np.max(np.abs(got - h) / tol)


def test_rows_of_no_expert_are_left():
    counts = [3, 0, 20, 4]
    off = offsets_of(counts, first=5)
    T = int(off[-1]) + 9
    logical, w, x = make("nvfp4", 4, 200, 272, T)
    x[:5] = np.nan
    x[off[-1]:] = np.inf
    y = torch.full((T, 200), 7.0, dtype=torch.float32, device=DEV)
    sk.gemm_experts_into(y, dev(x), w, dev(off), workspace=sk.make_experts_workspace())
    done()
    got = y.double().cpu().numpy()
    assert np.all(got[:5] == 7) and np.all(got[off[-1]:] == 7)
    ref, bound = expected("nvfp4", logical, x, off)
    assert_parity(got[5:off[-1]], ref[5:off[-1]], bound[5:off[-1]], "f32")


def test_nan_and_infinite_rows_stay_in_their_rows():
    counts = [2, 3, 1]
    off = offsets_of(counts)
    logical, w, x = make("nvfp4", 3, 130, 272, 6)
    x[1, 7] = np.nan
    x[4] = np.inf
    y = sk.gemm_experts(dev(x), w, dev(off), torch.float32, workspace=sk.make_experts_workspace())
    done()
    got = y.double().cpu().numpy()
    assert np.all(np.isnan(got[1])) and not np.any(np.isfinite(got[4]))
    fine = [0, 2, 3, 5]
    ref, bound = expected("nvfp4", logical, x, off)
    assert_parity(got[fine], ref[fine], bound[fine], "f32")


@pytest.mark.parametrize("bad", [[0, 5, 3, 8], [-4, 2, 2, 8], [0, 2, 100, 100], [9, 9, 9, 9], [8, 0, 0, 0]])
def test_offsets_out_of_order_or_range_count_as_the_nearest_allowed(bad):
    logical, w, x = make("nvfp4", 3, 130, 272, 8)
    y = torch.full((8, 130), 7.0, dtype=torch.float32, device=DEV)
    sk.gemm_experts_into(y, dev(x), w, dev(np.array(bad, np.int32)), workspace=sk.make_experts_workspace())
    done()
    off = np.maximum.accumulate(np.clip(bad, 0, 8))
    ref, bound = expected("nvfp4", logical, x, off)
    ref = np.where(np.isnan(ref), 7.0, ref)
    assert_parity(y.double().cpu().numpy(), ref, bound, "f32")


def test_many_experts_and_reproducibility():
    """512 experts, a few rows each; the same call twice gives the same bits, on
    another stream and from a captured graph too."""
    rng = np.random.default_rng(3)
    counts = rng.integers(0, 4, 512)
    off = offsets_of(counts)
    logical, w, x = make("nvfp4", 512, 48, 144, int(off[-1]))
    ws = sk.make_experts_workspace()
    xd, od = dev(x), dev(off)
    y = sk.gemm_experts(xd, w, od, torch.float32, workspace=ws)
    done()
    ref, bound = expected("nvfp4", logical, x, off)
    assert_parity(y.double().cpu().numpy(), ref, bound, "f32")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = torch.zeros_like(y)
    with torch.cuda.stream(side):
        sk.gemm_experts_into(y2, xd, w, od, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    y3 = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sk.gemm_experts_into(y3, xd, w, od, workspace=ws)
    for _ in range(3):
        graph.replay()
    done()
    assert torch.equal(y, y2) and torch.equal(y, y3)


def test_a_graph_replays_with_new_offsets_and_rows():
    logical, w, x = make("nvfp4", 4, 300, 640, 64)
    ws = sk.make_experts_workspace()
    xd, od = dev(x), dev(offsets_of([64, 0, 0, 0]))
    y = torch.zeros((64, 300), dtype=torch.float32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    sk.gemm_experts_into(y, xd, w, od, workspace=ws)
    with torch.cuda.graph(graph):
        sk.gemm_experts_into(y, xd, w, od, workspace=ws)
    for seed, counts in enumerate(([1, 2, 3, 58], [16, 16, 16, 16], [0, 0, 64, 0])):
        x2 = si.activations(64, 640, seed=seed, cfg_id=303)
        off = offsets_of(counts)
        xd.copy_(dev(x2))
        od.copy_(dev(off))
        graph.replay()
        done()
        ref, bound = expected("nvfp4", logical, x2, off)
        assert_parity(y.double().cpu().numpy(), ref, bound, "f32")


def test_no_rows():
    _, w, _ = make("nvfp4", 2, 128, 128, 1)
    y = sk.gemm_experts(torch.empty((0, 128), dtype=torch.float16, device=DEV), w, dev(np.zeros(3, np.int32)))
    assert y.shape == (0, 128)
    done()
