"""Sampling and the acceptance of drafts over their whole declared range: what was drawn against the definition where
probabilities, residuals and weights are far from the ordinary ones. (The bars are those of test_gpu_sampling.)"""
import math

import numpy as np
import pytest
import torch

import mtp_speculative_draft_head_gb300 as m
from test_gpu_sampling import DEV, PROB, WIDEN, check, logits, params, sample, tensors

pytestmark = pytest.mark.gpu


def test_emitted_tokens_follow_the_target():
    """q = (1/2, 1/4, 1/4) drafts, p = (1/4, 1/4, 1/2) accepts: over a grid of the draw's, the acceptance's and the
    last token's numbers, each with each, the emitted token comes up exactly as often as p says. (One number for
    both the draw and the acceptance would emit token 0 in half of the cases: it is drawn and accepted for u < 1/2.)"""
    n = 32
    mid = (torch.arange(n, device=DEV) + 0.5) / n
    u_draw, u_accept, u_last = (t.reshape(-1).contiguous() for t in torch.meshgrid(mid, mid, mid, indexing="ij"))
    B = n ** 3
    p = torch.tensor([0.25, 0.25, 0.5], device=DEV).expand(B, 2, 3).contiguous()
    l = torch.log(torch.tensor([0.5, 0.25, 0.25], device=DEV)).expand(B, 3).contiguous()

    def emitted(u_acc):
        x = torch.empty(B, dtype=torch.int32, device=DEV)
        q = torch.empty(B, 3, device=DEV)
        m.mtp_head_sample(l, u_draw, x, probs=q)
        tokens, acc = torch.empty(B, 2, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
        m.mtp_head_verify(p, q[:, None].contiguous(), x[:, None].contiguous(), torch.stack((u_acc, u_last), 1), tokens, acc)
        return (torch.bincount(tokens[:, 0].long(), minlength=3) / B).tolist()
    assert emitted(u_accept) == [0.25, 0.25, 0.5]
    assert emitted(u_draw)[0] == 0.5


def test_verify_takes_probabilities_into_range_before_it_compares():
    """A draft is accepted while u q(x) < p(x) with both taken into [0, 1]; NaN p counts as 0, and a draft whose q is
    NaN is refused (nothing is known of how it was drawn: what is emitted then comes from p alone)."""
    nan, inf = float("nan"), float("inf")
    rows = [  # p(x), q(x), u, accepted
        (1.5, 2.0, 0.9, 1), (2.0, 1.0, 0.99, 1), (inf, inf, 0.5, 1), (0.6, inf, 0.5, 1), (0.4, inf, 0.5, 0),
        (0.0, -0.5, 0.5, 0), (-0.5, -2.0, 0.5, 0), (0.25, -1.0, 0.9, 1), (0.3, 0.0, 0.9, 1),
        (nan, 0.5, 0.0, 0), (nan, -0.5, 0.5, 0), (0.5, nan, 0.1, 0), (nan, nan, 0.0, 0), (0.5, 0.5, 0.999, 1)]
    B, V = len(rows), 4
    p, q = torch.full((B, 2, V), 0.25, device=DEV), torch.full((B, 1, V), 0.25, device=DEV)
    x, u = torch.full((B, 1), 2, dtype=torch.int32, device=DEV), torch.full((B, 2), 0.5, device=DEV)
    for b, (pv, qv, uv, _) in enumerate(rows):
        p[b, 0, 2], q[b, 0, 2], u[b, 0] = pv, qv, uv
    tokens = torch.zeros(B, 2, dtype=torch.int32, device=DEV)
    acc = torch.zeros(B, dtype=torch.int32, device=DEV)
    m.mtp_head_verify(p, q, x, u, tokens, acc)
    assert acc.tolist() == [r[3] for r in rows]
    for b, (pv, qv, _, a) in enumerate(rows):
        w = np.clip(np.nan_to_num(p[b, a].double().cpu().numpy(), nan=0.0, posinf=1.0), 0.0, 1.0)
        if a == 0:
            left = np.maximum(w - np.clip(np.nan_to_num(q[b, 0].double().cpu().numpy(), nan=0.0, posinf=1.0), 0.0, 1.0), 0.0)
            w = left if left.sum() > 0 else w
        assert int(tokens[b, a]) == int((np.cumsum(w) <= 0.5 * w.sum()).sum()), b


def drawn(w, u, token, prob):
    """The token drawn from the weights w (fp64, not normalised) by u, and its probability, are right."""
    c = np.cumsum(w) / w.sum()
    assert 0 <= token < w.size and w[token] > 0
    assert (c[token - 1] if token else 0.0) - WIDEN <= u < c[token] + WIDEN, (token, u, c[token])
    assert abs(prob - w[token] / w.sum()) <= 2.0 ** -20 * w[token] / w.sum()


def draw_from(p, q, x, u, n):
    """verify of one draft a sequence, with tokens, accepted and prob on the host."""
    B = x.shape[0]
    tokens = torch.zeros(B, 2, dtype=torch.int32, device=DEV)
    acc, prob = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, device=DEV)
    m.mtp_head_verify(p, q, x, u, tokens, acc, prob, draft_len=n)
    return tokens.tolist(), acc.tolist(), prob.tolist()


@pytest.mark.parametrize("V", [3, 700, 154880])
@pytest.mark.parametrize("scale", [0.9, 1e-3, 1e-10, 1e-20, 1e-30, 1e-38, 1e-41])
def test_verify_rows_far_below_one(V, scale):
    """Probabilities need not sum to one: a row scaled down draws as the row itself (as fp32 holds it), however
    little mass it has."""
    g = np.random.default_rng(V)
    w = np.exp(2.0 * g.standard_normal((4, 2, V)))
    p = (w / w.max(-1, keepdims=True) * scale).astype(np.float32)
    u = g.random((4, 2)).astype(np.float32)
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    n = torch.zeros(4, dtype=torch.int32, device=DEV)
    tokens, acc, prob = draw_from(up(p), None, torch.zeros(4, 1, dtype=torch.int32, device=DEV), up(u), n)
    for b in range(4):
        assert acc[b] == 0 and tokens[b][1] == -1
        drawn(p[b, 0].astype(np.float64), float(u[b, 1]), tokens[b][0], prob[b])


@pytest.mark.parametrize("V", [700, 154880])
@pytest.mark.parametrize("top", [1e-2, 1e-6, 1e-12, 1e-30])
def test_verify_small_residuals(V, top):
    """After a rejection little of the target is left: nearly all of it on the rejected token (greedy drafts), or a
    drafter that differs in the last bits only. The residual is drawn from all the same, not the target's row."""
    g = np.random.default_rng(V + 1)
    B, at = 6, V // 3
    w = np.exp(3.0 * g.standard_normal((B, V)))
    p = (w / w.max(-1, keepdims=True) * top / V).astype(np.float32)
    p[:, at] = np.float32(0.75)
    u = g.random((B, 2)).astype(np.float32)
    u[:, 0] = 0.875
    full = np.stack((p, p), 1)
    up = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    x = torch.full((B, 1), at, dtype=torch.int32, device=DEV)
    tokens, acc, prob = draw_from(up(full), None, x, up(u), None)
    rest = p.astype(np.float64)
    rest[:, at] = 0.0
    for b in range(B):
        assert acc[b] == 0
        drawn(rest[b], float(u[b, 1]), tokens[b][0], prob[b])
    # q one or two steps below p or above it, and all but certain of the draft
    q = (p * (1.0 + 2.0 ** -23 * g.integers(-2, 3, p.shape))).astype(np.float32)
    q[:, at] = 1.0
    tokens, acc, prob = draw_from(up(full), up(q[:, None].copy()), x, up(u), None)
    rest = np.maximum(p.astype(np.float64) - q.astype(np.float64), 0.0)
    for b in range(B):
        assert acc[b] == 0
        drawn(rest[b], float(u[b, 1]), tokens[b][0], prob[b])


def test_verify_long_rows():
    """2^28 tokens whose probabilities, 2^-28 and a little more, are in two halves that a step of 2^-34 would round
    apart: the draw crosses the middle where the exact halves do."""
    V, B = 2 ** 28, 3
    lo, hi = np.float32(2.0 ** -28 * (1 + 0.3 / 64)), np.float32(2.0 ** -28 * (1 + 0.6 / 64))
    p = torch.full((B, 2, V), float(lo), device=DEV)
    p[:, :, V // 2:] = float(hi)
    u = torch.tensor([[0.5, 0.25], [0.5, 0.4985], [0.5, 0.9]], device=DEV)
    n = torch.zeros(B, dtype=torch.int32, device=DEV)
    tokens, acc, prob = draw_from(p, None, torch.zeros(B, 1, dtype=torch.int32, device=DEV), u, n)
    z = (float(lo) + float(hi)) * (V // 2)
    for b in range(B):
        t = tokens[b][0]
        c = (min(t, V // 2) * float(lo) + max(t - V // 2, 0) * float(hi)) / z
        assert abs(c - float(u[b, 1])) <= WIDEN, (t, c)
        w = float(lo if t < V // 2 else hi) / z
        assert abs(prob[b] - w) <= 2.0 ** -20 * w


@pytest.mark.parametrize("V", [2 ** 20, 2 ** 20 + 1, 3_000_001])
@pytest.mark.parametrize("which", ["T", "Tp", "Tkp", "Tkpm"])
def test_rows_of_about_a_million(V, which):
    """Both sides of the length from which a row's masses are scaled by its sum."""
    for bf in (False, True):
        l = logits(2, V, V + bf, bf)
        u = np.random.default_rng(V + 1).random(2).astype(np.float32).tolist()
        par = params(2, V + 2, which)
        if which == "Tkp":
            par["k"] = [400000, 1000]
        check(l, sample(l, u, par), u, par)


@pytest.mark.parametrize("V,bits", [(2 ** 26 + 1, 37), (2 ** 28 + 3, 35), (2 ** 30 + 1, 33)])
def test_long_rows_keep_small_weights(V, bits):
    """One token of weight one and all the others just below 2^-bits of it: each less than half a step of a sum
    that has room for V ones, and together 2^-11 to 2^-3 of the mass."""
    l = torch.full((1, V), -(bits * math.log(2.0) + 0.1), device=DEV)
    w = math.exp(float(l[0, 1]))
    l[0, 0] = 0.0
    z = 1.0 + w * (V - 1)
    tail = (z - 1.0) / z
    assert tail > 2.0 ** -12
    t, pr, _ = sample(l, [0.5], probs=False)
    assert int(t) == 0 and abs(float(pr) * z - 1.0) <= PROB
    for f in (0.9, 0.5, 0.01):
        u = float(np.float32(1.0 - f * tail))
        t, pr, _ = sample(l, [u], probs=False)
        assert abs((1.0 + w * (int(t) - 1)) / z - u) <= WIDEN
        assert abs(float(pr) * z / w - 1.0) <= PROB
    # top_p cuts among the ties, at an index
    p = float(np.float32(1.0 - 0.5 * tail))
    _, pr, dist = sample(l, [0.0], dict(p=[p]))
    n = int((dist > 0).sum())
    assert abs((1.0 + w * (n - 1)) / z - p) <= WIDEN and bool((dist[0, :n] > 0).all())
    assert abs(float(pr) * (1.0 + w * (n - 1)) - 1.0) <= PROB


@pytest.mark.parametrize("k", [256, 512, 640, 800, 1024, 1025, 2048, 4096, 4097])
def test_top_k_around_the_length_of_the_list(k):
    """top_k up to, at and beyond what one sorted list holds, in clusters of 16 and of 4 and with single CTAs."""
    for R, V in ((2, 154880), (24, 50257), (160, 9000)):
        l = logits(R, V, k + R)
        u = np.random.default_rng(k).random(R).astype(np.float32).tolist()
        par = dict(k=[k] * R, p=[1.0 if r % 2 else 0.96875 for r in range(R)], T=[0.5 + r % 3 for r in range(R)])
        check(l, sample(l, u, par), u, par, rows=range(0, R, max(1, R // 6)))


def test_negative_zero_is_zero():
    """-0 as a random number, top_p, min_p or temperature is 0."""
    l = logits(6, 5000, 41)
    par = dict(T=[1.0, 0.0, 0.7, 1.0, 1.0, 1.0], p=[1.0, 1.0, 0.0, 0.0, 1.0, 0.9], k=[0, 0, 0, 40, 900, 0], mp=[0.0] * 6)
    neg = {n: [-0.0 if v == 0.0 and n != "k" else v for v in vs] for n, vs in par.items()}
    a, b = sample(l, [0.0] * 6, par), sample(l, [-0.0] * 6, neg)
    check(l, a, [0.0] * 6, par)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    p = torch.softmax(logits(4, 5000, 42), 1).view(2, 2, 5000).contiguous()
    x = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
    out = []
    for z in (0.0, -0.0):
        u = torch.full((2, 2), z, device=DEV)
        t, acc = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
        m.mtp_head_verify(p, p[:, :1].contiguous(), x, u, t, acc)
        out.append((t.tolist(), acc.tolist()))
    assert out[0] == out[1]


@pytest.mark.parametrize("R,V", [(3, 60000), (40, 20000), (200, 3000)])
def test_token_and_prob_in_the_place_of_parameters(R, V):
    l = logits(R, V, R)
    u = np.random.default_rng(R).random(R).astype(np.float32).tolist()
    par = params(R, R + 1)
    par["T"][R - 1] = -1.0  # a refused row among them
    token, prob, _ = sample(l, u, par, ok=False)
    for at in ("top_k", "u"):
        tp = tensors(par)
        ut = torch.tensor(u, dtype=torch.float32, device=DEV)
        t2 = tp["top_k"] if at == "top_k" else torch.zeros_like(token)
        p2 = ut if at == "u" else tp["min_p"]
        m.mtp_head_sample(l, ut, t2, p2, **tp)
        assert torch.equal(t2, token) and torch.equal(p2, prob)
