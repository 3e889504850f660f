"""Verification of drafted tokens against a plain float64 loop: tokens and counts are equal."""
import numpy as np
import pytest
import torch

import fp8_weight_only_w4a16_b200 as sk

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def reference(target, draft, drafted, uniform, count):
    """One request at a time, by the definition; arrays in float64 (the values the device holds)."""
    B, S1, V = target.shape
    tokens, accepted = np.full((B, S1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n, k = 0, min(max(int(count[b]), 0), S1 - 1)
        while n < k:
            d = int(drafted[b, n])
            if not 0 <= d < V:
                break
            q = draft[b, n, d] if draft is not None else 1.0
            if not uniform[b, n] * q < target[b, n, d]:
                break
            tokens[b, n] = d
            n += 1
        accepted[b] = n
        p = target[b, n]
        rows = [p]
        if n < k:
            less = draft[b, n] if draft is not None else np.where(np.arange(V) == drafted[b, n], p, 0)
            with np.errstate(invalid="ignore"):
                rows = [p - less, p]
        for w in rows:
            w = np.where(np.isfinite(w) & (w > 0), w, 0)
            if w.sum() > 0:
                run = np.cumsum(w)
                at = np.nonzero((run > uniform[b, -1] * run[-1]) & (w > 0))[0]
                tokens[b, n] = at[0] if at.size else np.nonzero(w)[0][-1]
                break
    return tokens, accepted


def check(target, draft, drafted, uniform, count=None, run=sk.verify_draft):
    B, S1, _ = target.shape
    tokens, accepted = run(target, draft, drafted, uniform, count)
    torch.cuda.synchronize()
    f = lambda t: t.double().cpu().numpy() if t is not None else None
    n = count.cpu().numpy() if count is not None else np.full(B, S1 - 1)
    rt, ra = reference(f(target), f(draft), drafted.cpu().numpy(), f(uniform), n)
    assert np.array_equal(accepted.cpu().numpy(), ra)
    assert np.array_equal(tokens.cpu().numpy(), rt)
    return rt, ra


def inputs(B, S, V, dtype, seed=0, noise=0.5, with_draft=True):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((B, S + 1, V), generator=g) * 2
    zq = z[:, :S] + noise * torch.randn((B, S, V), generator=g)
    q = torch.softmax(zq, -1)
    drafted = torch.multinomial(q.reshape(-1, V), 1, generator=g).reshape(B, S).int() if S else torch.zeros((B, 0)).int()
    u = torch.rand((B, S + 1), generator=g)
    target = torch.softmax(z, -1).to(TYPES[dtype]).to(DEV)
    return target, q.to(TYPES[dtype]).to(DEV) if with_draft else None, drafted.to(DEV), u.to(DEV)


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,S,V", [(1, 1, 1), (1, 7, 1000), (3, 0, 257), (5, 2, 33), (9, 4, 4099), (2, 7, 151936),
                                   (40, 3, 2050), (1, 40, 130)])
def test_matches_the_definition(B, S, V, dtype, with_draft):
    target, draft, drafted, u = inputs(B, S, V, dtype, seed=B * 1000 + S, with_draft=with_draft)
    check(target, draft, drafted, u)
    if S:
        count = torch.arange(B, dtype=torch.int32, device=DEV) % (S + 3) - 1     # out of range at both ends
        check(target, draft, drafted, u, count)


def test_the_drafters_tokens_follow_the_targets_distribution():
    """Each of 4 tokens comes out as often as its target probability says, whatever the draft was."""
    B, V = 40000, 4
    g = torch.Generator().manual_seed(1)
    p, q = torch.tensor([0.5, 0.2, 0.3, 0.0]), torch.tensor([0.1, 0.6, 0.1, 0.2])
    drafted = torch.multinomial(q, B, replacement=True, generator=g).int()[:, None].to(DEV)
    u = torch.rand((B, 2), generator=g).to(DEV)
    target = p.expand(B, 2, V).contiguous().to(DEV)
    tokens, _ = sk.verify_draft(target, q.expand(B, 1, V).contiguous().to(DEV), drafted, u)
    freq = np.bincount(tokens[:, 0].cpu().numpy(), minlength=V) / B
    # five standard deviations of a frequency over B draws
    assert np.all(np.abs(freq - p.numpy()) <= 5 * np.sqrt(p.numpy() * (1 - p.numpy()) / B))


def test_borders_of_the_draw():
    V = 600
    p = torch.zeros((6, 1, V))
    p[:, 0, 100], p[:, 0, 300], p[:, 0, 599] = 0.25, 0.25, 0.5
    u = torch.tensor([[0.0], [0.25], [0.5], [1 - 2**-24], [1.0], [float("nan")]])
    t, _ = check(p.to(DEV), None, torch.zeros((6, 0), dtype=torch.int32, device=DEV), u.to(DEV))
    assert t[:, 0].tolist() == [100, 300, 599, 599, 599, 599]


def test_rows_without_weight():
    """Equal rows that are rejected, rows of zeros, NaN and infinities, tokens out of range."""
    V = 5000
    g = torch.Generator().manual_seed(2)
    p = torch.softmax(torch.randn((6, 2, V), generator=g), -1)
    q = p[:, :1].clone()
    u = torch.full((6, 2), 0.4)
    u[0, 0] = 1.0                       # u q < p fails where p = q: the difference is empty
    p[1, 0] = 0                         # nothing to draw from at all
    p[2, 0, 1::2] = float("nan")
    q[2] = 0.5
    p[3, 0, 17] = float("inf")
    drafted = torch.tensor([[4], [5], [1], [17], [V], [-1]], dtype=torch.int32)
    t, n = check(p.to(DEV), q.to(DEV), drafted.to(DEV), u.to(DEV))
    assert n[0] == 0 and t[1, 0] == -1 and n[4] == n[5] == 0
    check(p.to(DEV), None, drafted.to(DEV), u.to(DEV))


def test_strides_and_odd_addresses():
    B, S, V = 3, 4, 1003
    target, draft, drafted, u = inputs(B, S, V, "f32")
    wide = torch.full((B, S + 3, V + 2), float("nan"), device=DEV)
    wide[:, 1:S + 2, 1:V + 1] = target
    wide_q = torch.full((S, B, V + 1), float("nan"), device=DEV)
    wide_q[:, :, :V] = draft.transpose(0, 1)
    check(wide[:, 1:S + 2, 1:V + 1], wide_q[:, :, :V].transpose(0, 1), drafted, u)
    same = torch.softmax(torch.randn((1, 1, V), device=DEV), -1).expand(B, S + 1, V)
    check(same, draft, drafted, u)


def test_streams_and_graphs():
    target, draft, drafted, u = inputs(4, 5, 3001, "f32", seed=8)
    tokens, accepted = torch.zeros((4, 6), dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    sk.verify_draft_into(tokens, accepted, target, draft, drafted, u)
    with torch.cuda.graph(graph):
        sk.verify_draft_into(tokens, accepted, target, draft, drafted, u)

    def replay(*_):
        tokens.zero_()
        graph.replay()
        return tokens, accepted

    for seed in (8, 9):
        new = inputs(4, 5, 3001, "f32", seed=seed)
        for old, t in zip((target, draft, drafted, u), new):
            old.copy_(t)
        check(target, draft, drafted, u, run=replay)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    check(target, draft, drafted, u, run=lambda *a: sk.verify_draft(*a, stream=side))


def test_no_requests():
    t, n = sk.verify_draft(torch.empty((0, 3, 10), device=DEV), None, torch.empty((0, 2), dtype=torch.int32, device=DEV),
                           torch.empty((0, 3), device=DEV))
    assert t.shape == (0, 3) and n.shape == (0,)
