"""Sampling and the acceptance of drafts over their whole declared range: what was drawn against the definition where
probabilities, residuals and weights are far from the ordinary ones. (The bars are those of test_gpu_sampling.)"""
import math

import numpy as np
import pytest
import torch

import mtp_speculative_draft_head_gb300 as m
from test_gpu_sampling import DEV, PROB, WIDEN, check, logits, params, sample

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
