"""Operators of a decode step that drafts tokens and routes its MLP to experts:

  experts    y[r] = x[r] . W_e(r)^T over packed NVFP4 or FP8 experts, rows sorted by expert, ragged
             (optionally gate+up with SiLU*mul)
  int8       activations to 8-bit integers with a scale per token, then
             y[m, n] = (q[m] . c[n]) * row_scale[m] * channel_scale[n]
  verify     accept or reject drafted tokens against the target's probabilities and draw the next token

``listed()`` gives the cases, ``prepare`` their inputs, ``run`` one pass: the plain form in torch, or
with ``own`` the framework's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
VOCAB = 151936          # the vocabulary projection of synthetic_inputs.py
F16, F32 = "float16", "float32"


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one request, eight experts: the latency of a decode step's gate+up
        dict(name="experts_one_token", op="experts", fmt="nvfp4", silu=True, E=64, N=2816, K=2048, rows=8, out=F16),
        # a verify round of 8 tokens x 8 experts: most experts that are hit have one row
        dict(name="experts_verify_round", op="experts", fmt="nvfp4", silu=True, E=128, N=2816, K=5120, rows=64,
             out=F16),
        # the down projection of the same round, in FP8
        dict(name="experts_down_fp8", op="experts", fmt="fp8", silu=False, E=128, N=5120, K=1408, rows=64, out=F16),
        # a served batch: some dozens of rows for each expert, ragged, an odd number of outputs
        dict(name="experts_batch", op="experts", fmt="nvfp4", silu=False, E=32, N=2051, K=2048, rows=1003, out=F16),
        # prefill: hundreds to thousands of rows for each expert, bound by the tensor cores
        dict(name="experts_prefill", op="experts", fmt="nvfp4", silu=True, E=32, N=2816, K=5120, rows=16387, out=F16),
        # an attention projection of one token: bound by reading the weights
        dict(name="int8_one_token", op="int8", M=1, N=5120, K=5120, out=F16),
        # gate+up of a served batch of an odd number of tokens
        dict(name="int8_batch", op="int8", M=61, N=34816, K=5120, out=F16),
        # gate+up of a prefill chunk: bound by the tensor cores
        dict(name="int8_prefill", op="int8", M=2048, N=34816, K=5120, out=F16),
        # the vocabulary projection of a verify round, whose logits stay in 32 bits
        dict(name="int8_logits", op="int8", M=8, N=VOCAB, K=5120, out=F32),
        # a k=7 verify round of one request, and of a served batch
        dict(name="verify_one", op="verify", B=1, S=7, V=VOCAB, dtype=F32, draft=True),
        dict(name="verify_batch", op="verify", B=64, S=7, V=VOCAB, dtype=F32, draft=True),
        # drafts found by lookup in the text so far have no distribution of their own
        dict(name="verify_lookup", op="verify", B=8, S=4, V=VOCAB, dtype="bfloat16", draft=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("experts", "experts", "experts", "int8", "int8", "verify"))
    if op == "experts":
        silu = rng.random() < 0.5
        # gate+up packs outputs in pairs of 64 rows; otherwise any number of outputs
        n = 128 * rng.randint(2, 22) if silu else _log(rng, 256, 5120)
        return dict(op=op, fmt=rng.choice(("nvfp4", "nvfp4", "fp8")), silu=silu, E=rng.choice((4, 8, 16, 32, 60)),
                    N=n, K=16 * _log(rng, 16, 160), rows=_log(rng, 1, 12000), out=F16)
    if op == "int8":
        return dict(op=op, M=_log(rng, 1, 2000), N=_log(rng, 256, 20000), K=16 * _log(rng, 16, 320),
                    out=rng.choice((F16, F16, F32)))
    return dict(op=op, B=_log(rng, 1, 48), S=rng.randint(1, 7), V=_log(rng, 1000, VOCAB),
                dtype=rng.choice((F32, F32, F16, "bfloat16")), draft=rng.random() < 0.75)


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _expert_offsets(case, seed):
    """Row counts as a router leaves them: a few experts are popular, some get nothing."""
    r = np.random.default_rng(seed)
    share = r.gamma(1.0, size=case["E"]) + 0.02
    counts = r.multinomial(case["rows"], share / share.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    if case["op"] == "experts":
        E, N, K = case["E"], case["N"], case["K"]
        off = _expert_offsets(case, seed)
        s["most"] = max(1, int(np.diff(off).max()))
        s["offsets"] = torch.from_numpy(off).to(DEV)
        s["x"] = torch.randn((case["rows"], K), generator=g, device=DEV).half()
        if case["fmt"] == "nvfp4":
            # uniform codes, block scales uniform over the E4M3 values of [2^-4, 2^4], a scale per expert
            s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
            s["scales"] = torch.randint(0x18, 0x59, (E, N, K // 16), generator=g, device=DEV, dtype=torch.uint8)
            s["expert_scale"] = (torch.rand(E, generator=g, device=DEV) + 0.5) / 448
        else:
            w = torch.randn((E, N, K), generator=g, device=DEV)
            s["codes"] = (w * 90).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s["channel_scale"] = (torch.rand((E, N), generator=g, device=DEV) + 0.5) * (0.02 / 90)
            del w
        if own:
            import fp8_weight_only_w4a16_b200 as sk

            # packed once when the model is loaded; the workspace is the program's for all its calls
            if case["fmt"] == "nvfp4":
                s["w"] = sk.PackedExpertsNVFP4.from_logical(s["codes"], s["scales"], s["expert_scale"],
                                                            gate_up=case["silu"])
            else:
                s["w"] = sk.PackedExpertsFP8.from_logical(s["codes"], s["channel_scale"], gate_up=case["silu"])
            s["workspace"] = sk.make_experts_workspace()
    elif case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        # activations whose rows are of unlike size, as hidden states are; weights quantised when the model was made
        s["x"] = (torch.randn((M, K), generator=g, device=DEV) * torch.rand((M, 1), generator=g, device=DEV).add_(0.2)).half()
        s["c"] = torch.randn((N, K), generator=g, device=DEV).mul_(36).round_().clamp_(-127, 127).to(torch.int8)
        s["channel_scale"] = (torch.rand(N, generator=g, device=DEV) + 0.5) * (0.02 / 36)
        if own:
            import fp8_weight_only_w4a16_b200 as sk

            s["w"] = sk.WeightInt8(s["c"], s["channel_scale"])
            s["workspace"] = sk.make_int8_workspace()
    else:
        B, S, V = case["B"], case["S"], case["V"]
        dt = getattr(torch, case["dtype"])
        z = torch.randn((B, S + 1, V), generator=g, device=DEV).mul_(3)
        s["target"] = torch.softmax(z, -1).to(dt)
        z = z[:, :S]
        if case["draft"]:
            # the drafter's distribution is the target's with some noise; its tokens are drawn from it
            z = z.add_(torch.randn((B, S, V), generator=g, device=DEV).mul_(0.5))
            z = torch.softmax(z, -1)
            s["draft"] = z.to(dt)
        else:
            s["draft"] = None       # drafts by lookup: no distribution
            z = torch.softmax(z, -1)
        s["draft_tokens"] = torch.multinomial(z.reshape(B * S, V), 1, generator=g).reshape(B, S).int()
        s["num_drafts"] = torch.randint(S // 2, S + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        s["uniform"] = torch.rand((B, S + 1), generator=g, device=DEV)
        del z
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return {"experts": _experts, "int8": _int8, "verify": _verify}[s["op"]](s)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _experts(s):
    if own:
        import fp8_weight_only_w4a16_b200 as sk

        call = sk.gemm_experts_silu_mul if s["silu"] else sk.gemm_experts
        return call(s["x"], s["w"], s["offsets"], getattr(torch, s["out"]), workspace=s["workspace"])
    E, N, K, T, most = s["E"], s["N"], s["K"], s["rows"], s["most"]
    if s["fmt"] == "nvfp4":
        table = torch.tensor(_E2M1, device=DEV)
        w = torch.stack((table[(s["codes"] & 15).int()], table[(s["codes"] >> 4).int()]), -1).view(E, N, K // 16, 16)
        w = w * s["scales"].view(torch.float8_e4m3fn).float()[..., None]
        w = w.view(E, N, K)
        scale = s["expert_scale"][:, None, None]
    else:
        w = s["codes"].view(torch.float8_e4m3fn).float()
        scale = s["channel_scale"][:, None, :]
    # the rows of each expert side by side, padded to the longest
    off = s["offsets"].long()
    place = torch.arange(most, device=DEV)[None] + off[:-1, None]
    x = s["x"].float()[place.clamp(max=T - 1)]
    y = torch.bmm(x, w.transpose(1, 2)) * scale
    if s["silu"]:
        gate, up = y[..., : N // 2], y[..., N // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    row = torch.arange(T, device=DEV)
    e = torch.searchsorted(off[1:], row, right=True)
    return y[e, row - off[e]].to(getattr(torch, s["out"]))


def _int8(s):
    out = getattr(torch, s["out"])
    if own:
        import fp8_weight_only_w4a16_b200 as sk

        q, row_scale = sk.quantize_int8(s["x"])
        return sk.gemm_int8(q, row_scale, s["w"], out, workspace=s["workspace"])
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True)
    row_scale = top / torch.full_like(top, 127.0)
    # a quotient next to the middle between two whole numbers needs more than 32 bits
    q = torch.where(row_scale > 0, x.double() / row_scale.double(), 0.0).round().clamp(-127, 127)
    # sums of products of 8-bit integers pass 24 bits: 64
    y = torch.matmul(q, s["c"].double().T).float()
    return (y * row_scale * s["channel_scale"]).to(out)


def _verify(s):
    if own:
        import fp8_weight_only_w4a16_b200 as sk

        return sk.verify_draft(s["target"], s["draft"], s["draft_tokens"], s["uniform"], s["num_drafts"])
    B, S, V = s["B"], s["S"], s["V"]
    target, d, u = s["target"], s["draft_tokens"].long(), s["uniform"].double()
    place = torch.arange(S, device=DEV)
    p = target[:, :S].gather(2, d[..., None])[..., 0].double()
    q = s["draft"].gather(2, d[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(p)
    ok = (u[:, :S] * q < p) & (place < s["num_drafts"][:, None])
    n = ok.int().cumprod(1).sum(1)
    at = torch.arange(B, device=DEV)
    w = target[at, n].double()
    rejected = (n < s["num_drafts"])[:, None]
    i = n.clamp(max=S - 1)
    if s["draft"] is not None:
        less = s["draft"][at, i].double()
    else:
        less = torch.where(torch.arange(V, device=DEV) == d[at, i][:, None], torch.inf, 0.0)
    w = torch.where(rejected, (w - less).clamp(min=0), w)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, target[at, n].double())
    c = w.cumsum(1)
    token = ((c > u[:, S:] * c[:, -1:]) & (w > 0)).int().argmax(1)
    column = torch.arange(S + 1, device=DEV)
    tokens = torch.cat((d, torch.zeros_like(d[:, :1])), 1)
    tokens = torch.where(column == n[:, None], token[:, None], torch.where(column < n[:, None], tokens, -1))
    return tokens.int(), n.int()


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = {F16: 2, "bfloat16": 2, F32: 4}
    if case["op"] == "experts":
        E, N, K, T = case["E"], case["N"], case["K"], case["rows"]
        # the weights of the experts that get rows, whose number goes by the draw: its mean over draws
        r = random.Random(0)
        hit, trials = 0, 20
        for _ in range(trials):
            share = [r.gammavariate(1.0, 1.0) + 0.02 for _ in range(E)]
            total = sum(share)
            hit += sum(1 - (1 - v / total) ** T for v in share)
        hit = min(hit / trials, T)
        per = N * K * (0.5 + 1 / 16) + 4 if case["fmt"] == "nvfp4" else N * K + 4 * N
        outs = T * (N // 2 if case["silu"] else N)
        return {"bytes": int(hit * per + 2 * T * K + size[case["out"]] * outs + 4 * (E + 1)), "flops": 2 * T * N * K}
    if case["op"] == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * N + size[case["out"]] * M * N, "flops": 2 * M * N * K}
    # one row of the target's, and of the draft's where there is one, for each request
    rows = case["B"] * (2 if case["draft"] else 1)
    return {"bytes": rows * case["V"] * size[case["dtype"]] + case["B"] * (16 * case["S"] + 8),
            "flops": 3 * case["B"] * case["V"]}


# --------------------------------------------------------------------------- 64 bits

def _e2m1_64(n):
    """The value of an E2M1 code from its sign, exponent and mantissa bits."""
    e, m = (n >> 1) & 3, (n & 1).double()
    v = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    return torch.where(n >= 8, -v, v)


def _e4m3_64(b):
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m / 512, torch.exp2(e.double() - 7) * (1 + m / 8))
    return torch.where(b >= 128, -v, v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "experts":
        off = s["offsets"].tolist()
        y = torch.empty((case["rows"], case["N"]), dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            if off[e] == off[e + 1]:
                continue
            c = s["codes"][e].int()
            if case["fmt"] == "nvfp4":
                w = torch.empty((case["N"], case["K"]), dtype=torch.float64, device=DEV)
                w[:, 0::2], w[:, 1::2] = _e2m1_64(c & 15), _e2m1_64(c >> 4)
                w *= _e4m3_64(s["scales"][e].int()).repeat_interleave(16, 1) * s["expert_scale"][e].double()
            else:
                w = _e4m3_64(c) * s["channel_scale"][e].double()[:, None]
            y[off[e]:off[e + 1]] = s["x"][off[e]:off[e + 1]].double() @ w.T
        if case["silu"]:
            gate, up = y.chunk(2, 1)
            y = gate * torch.sigmoid(gate) * up
        return y
    if case["op"] == "int8":
        x = s["x"].double()
        step = (x.abs().max(1).values[:, None] / 127).float().double()     # the scale is a 32-bit number
        whole = torch.round(x / step)
        return torch.mm(whole, s["c"].double().t()) * step * s["channel_scale"].double()[None]
    tokens = np.full((case["B"], case["S"] + 1), -1, np.int32)
    accepted = np.zeros(case["B"], np.int32)
    u, drafted, count = s["uniform"].cpu().numpy().astype(np.float64), s["draft_tokens"].cpu().numpy(), s["num_drafts"].tolist()
    for b in range(case["B"]):
        n = 0
        while n < count[b]:
            token = int(drafted[b, n])
            q = float(s["draft"][b, n, token]) if case["draft"] else 1.0
            if not u[b, n] * q < float(s["target"][b, n, token]):
                break
            tokens[b, n] = token
            n += 1
        accepted[b] = n
        row = s["target"][b, n].double().cpu().numpy()
        left = row
        if n < count[b]:
            left = row.copy()
            if case["draft"]:
                left = np.maximum(row - s["draft"][b, n].double().cpu().numpy(), 0)
            else:
                left[drafted[b, n]] = 0
            left = left if left.sum() > 0 else row
        run_up = np.cumsum(left)
        tokens[b, n] = np.nonzero((run_up > u[b, -1] * run_up[-1]) & (left > 0))[0][0]
    return tokens, accepted


if __name__ == "__main__":
    for case in listed():
        print(case["name"], work(case))
