"""Plain 64-bit forms of the attention half's operators (torch, no library code), and what their results may be
off by. A rounding is off by at most half a step: eps / 2 relative (BF16 2^-8, f16 2^-11, fp32 2^-24)."""
import numpy as np
import torch

import fp4_helpers as ref

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def values(q, bs, rs):
    """fp64 values [..., D] of cached rows (host or device tensors)."""
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    lut = torch.cat((E2M1, -E2M1)).to(q.device)
    s = torch.from_numpy(np.append(ref.E4M3, np.nan)).to(q.device)[bs.long() & 127]
    return lut[c] * s.repeat_interleave(16, -1) * rs.double().unsqueeze(-1)


def quantize(rows: np.ndarray):
    """fp64 rows [n, D] -> packed codes [n, D/2], block scales [n, D/16], row scales [n], from the definition."""
    D = rows.shape[1]
    codes, sc, rs = ref.quantize(rows)
    return ref.pack(codes)[:, :D // 2], sc[:, :D // 16], rs


def attention(q, k, v, limits, scale):
    """Rows q [n, D] over keys and values [t, D], row i seeing the first limits[i] tokens: outputs [n, D], lse [n], and
    A = sum_j p_j |v_j| [n, D], E = scale max_j sum_d |q_d k_jd| [n], P = max_j p_j max_d |v_jd| [n] for the bounds. All fp64."""
    a = (q @ k.t()) * scale
    e = (q.abs() @ k.abs().t()) * scale
    seen = torch.arange(k.shape[0], device=q.device).view(1, -1) < limits.view(-1, 1)
    a = a.masked_fill(~seen, float("-inf"))
    e = e.masked_fill(~seen, 0.0)
    none = limits.view(-1) <= 0
    if k.shape[0] == 0 or bool(none.all()):
        z = torch.full((q.shape[0],), float("-inf"), dtype=torch.float64, device=q.device)
        o = torch.zeros_like(q)
        return o, z, o.clone(), torch.zeros_like(z), torch.zeros_like(z)
    z = torch.logsumexp(a, 1)
    p = torch.exp(a - torch.where(none, 0.0, z).view(-1, 1))
    clean = torch.where(seen.any(0).view(-1, 1), v, 0.0)
    big = (p * clean.abs().amax(1)).amax(1)
    return p @ clean, z, p @ clean.abs(), e.amax(1), big


def score_error(E, D):
    """How far a score may be off: its products are exact, their D / 16 partial sums and the four factors round by 2^-22
    of the sum of magnitudes each (twice what fp32 does); the largest score's own error comes on top."""
    return (D / 16 + 8) * 2.0 ** -22 * E + 2.0 ** -20


def bound_out(o, A, E, P, D, tokens, weight_eps, log_scale=0.0):
    """Outputs: their own rounding to BF16; the weights' rounding (weight_eps), the exponential (2^-22 and the score's
    error) and the fp32 sums (tokens / 16 additions of 2^-22) relative to A; weights below the 16-bit types' normal range
    are off by 2^-24 of the frame's largest (f16; nothing for BF16), whose value element may be any of a row's. log_scale:
    the largest |log2| of a value's row scale, which the weights' exponents carry: the logarithm is off by 2^-22 of itself
    and three fp32 sums of that size by 2^-24 each, times ln 2."""
    rel = weight_eps + 4.0 * score_error(E, D) + 2.0 ** -20 + (tokens / 16 + 16) * 2.0 ** -22 + log_scale * 2.0 ** -21
    small = tokens * 2.0 ** -24 * P if weight_eps < 2.0 ** -8 else torch.zeros_like(P)
    t = rel.view(-1, 1) * A + small.view(-1, 1)
    return t + 2.0 ** -8 * (o.abs() + t) + 2.0 ** -133


def bound_lse(z, E, D, tokens):
    return score_error(E, D) * 2.0 + (tokens / 32 + 32) * 2.0 ** -23 + 2.0 ** -22 * torch.nan_to_num(z, neginf=0.0).abs()
