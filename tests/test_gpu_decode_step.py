"""The operators of one verify round together, as a decode step calls them: experts' gate+up
and down projections of routed tokens, an 8-bit projection, the vocabulary projection, and the
verification of the drafts; each stage against its definition on the inputs it was given, then
the whole step captured into a CUDA graph and replayed."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk
import oracle
import synthetic_inputs as si
from parity import REL_TOL, assert_parity
from test_gpu_int8 import product, quantized
from test_gpu_verify import reference

pytestmark = pytest.mark.gpu

DEV = "cuda"
M, H, F, E, TOP, V = 8, 512, 96, 8, 2, 1000


class Step:
    def __init__(self):
        r = np.random.default_rng(4)
        self.gate_up = [si.nvfp4_weights(2 * F, H, seed=4, cfg_id=310, tensor_id=2 * e) for e in range(E)]
        self.g1 = np.full(E, 1 / 448, np.float32)
        self.w1 = sk.PackedExpertsNVFP4.from_logical(np.stack([c for c, _ in self.gate_up]),
                                                     np.stack([s for _, s in self.gate_up]), self.g1, gate_up=True)
        self.down = [si.fp8_weights(H, F, sigma=0.1, seed=4, cfg_id=311, tensor_id=2 * e) for e in range(E)]
        self.w2 = sk.PackedExpertsFP8.from_logical(np.stack([q for q, _ in self.down]),
                                                   np.stack([s for _, s in self.down]))
        self.c = r.integers(-127, 128, (H, H), dtype=np.int8)
        self.cs = r.uniform(0.5, 1.5, H).astype(np.float32) / (127 * 16)
        self.w3 = sk.WeightInt8(torch.from_numpy(self.c).to(DEV), torch.from_numpy(self.cs).to(DEV))
        self.head = si.nvfp4_weights(V, H, seed=4, cfg_id=312)
        self.w4 = sk.PackedNVFP4.from_logical(*self.head, 1 / 64, DEV)
        self.ws_tile, self.ws_head = sk.make_experts_workspace(), sk.make_workspace(sk.FMT_NVFP4, M, V, H)
        self.router = torch.from_numpy(r.standard_normal((E, H)).astype(np.float32)).to(DEV)
        self.draft = torch.softmax(torch.from_numpy(r.standard_normal((1, M - 1, V)).astype(np.float32)).to(DEV), -1)
        self.drafted = torch.from_numpy(r.integers(0, V, (1, M - 1)).astype(np.int32)).to(DEV)
        self.uniform = torch.from_numpy(r.random((1, M)).astype(np.float32)).to(DEV)

    def __call__(self, x):
        out = {}
        weight, expert = torch.softmax(x.float() @ self.router.T, -1).topk(TOP, -1)
        order = expert.flatten().argsort(stable=True)
        token = order // TOP
        counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, expert.flatten(),
                                                                           torch.ones_like(order))
        out["offsets"] = torch.cat((counts.new_zeros(1), counts.cumsum(0))).int()
        out["rows"] = x[token]
        out["act"] = sk.gemm_experts_silu_mul(out["rows"], self.w1, out["offsets"], workspace=self.ws_tile)
        out["mlp"] = sk.gemm_experts(out["act"], self.w2, out["offsets"], torch.float32, workspace=self.ws_tile)
        h = x.float().index_add(0, token, out["mlp"] * weight.flatten()[order][:, None])
        out["h"] = h.half()
        out["q"], out["scale"] = sk.quantize_int8(out["h"])
        out["proj"] = sk.gemm_int8(out["q"], out["scale"], self.w3, workspace=self.ws_tile)
        out["logits"] = sk.gemm(out["proj"], self.w4, torch.float32, workspace=self.ws_head)
        out["probs"] = torch.softmax(out["logits"] * 0.02, -1)[None]
        out["tokens"], out["accepted"] = sk.verify_draft(out["probs"], self.draft, self.drafted, self.uniform)
        return out


def test_stages_against_their_definitions_and_graph_replay():
    step = Step()
    x = torch.from_numpy(si.activations(M, H, seed=4, cfg_id=313)).to(DEV)
    with torch.cuda.stream(torch.cuda.Stream()):
        o = step(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g = step(x)
    for seed in (4, 5):
        x.copy_(torch.from_numpy(si.activations(M, H, seed=seed, cfg_id=313)))
        o = step(x)
        graph.replay()
        torch.cuda.synchronize()
        assert sk.tile_device_error(clear=True) == 0 and sk.device_error(clear=True) == 0
        for name in ("act", "mlp", "h", "q", "scale", "proj", "logits", "tokens", "accepted"):
            assert torch.equal(o[name], g[name]), name
        n = {k: v.cpu().numpy() for k, v in o.items()}
        off = n["offsets"]
        assert off[0] == 0 and off[-1] == M * TOP
        for e in range(E):
            rows = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            ref, b = oracle.nvfp4_gemm(n["rows"][rows], *self_scaled(step.gate_up[e], step.g1[e]))
            act = oracle.silu_mul(ref)
            du = REL_TOL * b
            tol = 1.1 * du[:, :F] * (np.abs(ref[:, F:]) + du[:, F:]) + np.abs(ref[:, :F]) * du[:, F:] + np.abs(act) / 1024 + 1e-7
            assert np.all(np.abs(n["act"][rows] - act) <= tol)
            ref, b = oracle.fp8_gemm(n["act"][rows], *step.down[e])
            assert_parity(n["mlp"][rows], ref, b, "f32")
        q, scale = quantized(n["h"])
        assert np.array_equal(n["q"], q) and np.array_equal(n["scale"], scale)
        assert np.array_equal(n["proj"], product(q, scale, step.c, step.cs, torch.float16))
        ref, b = oracle.nvfp4_gemm(n["proj"], *step.head, 1 / 64)
        assert_parity(n["logits"], ref, b, "f32")
        tokens, accepted = reference(n["probs"].astype(np.float64), step.draft.double().cpu().numpy(),
                                     step.drafted.cpu().numpy(), step.uniform.double().cpu().numpy(), [M - 1])
        assert np.array_equal(n["tokens"], tokens) and np.array_equal(n["accepted"], accepted)


def self_scaled(weights, g):
    return (*weights, float(g))


def test_two_streams_with_their_own_workspaces():
    """Calls that can overlap on the GPU, each with a workspace of its own, give what they give alone."""
    jobs = []
    for i, (m, n, k) in enumerate(((1, 5120, 2048), (40, 3000, 1040), (200, 1000, 528))):
        r = np.random.default_rng(i)
        q, c = r.integers(-127, 128, (m, k), dtype=np.int8), r.integers(-127, 128, (n, k), dtype=np.int8)
        w = sk.WeightInt8(torch.from_numpy(c).to(DEV), torch.ones(n, device=DEV))
        jobs.append((torch.from_numpy(q).to(DEV), torch.ones(m, device=DEV), w, sk.make_int8_workspace(),
                     torch.cuda.Stream(), torch.zeros((20, m, n), device=DEV),
                     product(q, np.ones(m, np.float32), c, np.ones(n, np.float32), torch.float32)))
    torch.cuda.synchronize()
    for i in range(20):
        for q, one, w, ws, stream, y, _ in jobs:
            sk.gemm_int8_into(y[i], q, one, w, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    assert sk.tile_device_error(clear=True) == 0
    for *_, y, ref in jobs:
        assert np.array_equal(y.cpu().numpy(), np.broadcast_to(ref, y.shape))


def test_operands_written_by_the_kernel_just_before():
    """Weights, activations and offsets that the previous kernel on the stream wrote are seen."""
    m, n, k = 4, 4096, 1024
    ws = sk.make_int8_workspace()
    codes = torch.zeros((n, k), dtype=torch.int8, device=DEV)
    q = torch.zeros((m, k), dtype=torch.int8, device=DEV)
    w = sk.WeightInt8(codes, torch.ones(n, device=DEV))
    one = torch.ones(m, device=DEV)
    for i in range(1, 30):
        q.fill_(1)
        codes.fill_(i)
        y = sk.gemm_int8(q, one, w, torch.float32, workspace=ws)
        assert bool((y == i * k).all())
    assert sk.tile_device_error(clear=True) == 0


def test_a_workspace_that_is_too_small_is_refused():
    w = sk.WeightInt8(torch.zeros((64, 64), dtype=torch.int8, device=DEV), torch.ones(64, device=DEV))
    q, one = torch.zeros((1, 64), dtype=torch.int8, device=DEV), torch.ones(1, device=DEV)
    with pytest.raises(sk.SkinnyError) as e:
        sk.gemm_int8(q, one, w, workspace=torch.zeros(1024, dtype=torch.uint8, device=DEV))
    assert e.value.status == sk.ERR_WORKSPACE
    with pytest.raises(ValueError):
        sk.gemm_int8(q, one.cpu(), w)
    with pytest.raises(ValueError):
        sk.gemm_int8_into(None, q, one, w)
