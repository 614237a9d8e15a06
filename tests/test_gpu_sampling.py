"""Sampling and the acceptance of drafts, against fp64 references from the definitions.

Bars. A weight exp((l - m) / T) is formed in fp32 from an exact exponent: below 2^-22 relative (the
series' remainder 2^-27, a rounding of 2^-24 in each of the last Horner steps and one in the
exponent's product with ln 2), so probabilities are within 2^-21 + 2^-23 of exact. The cumulative
distribution is a sum of such weights over such a sum: within 2^-21 of exact, plus V roundings of the
fixed-point masses, 2^-62 V each against a total of at least one (V^2 2^-62 in all, below 2^-22 for
V < 2^20). A token is right when u lies in its interval widened by 2^-20."""
import math

import numpy as np
import pytest
import torch

import mtp_speculative_draft_head_gb300 as m

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
WIDEN = 2.0 ** -20
PROB = 2.0 ** -21 + 2.0 ** -23


def reference(l, T=1.0, k=0, p=1.0, mp=0.0):
    """The restricted distribution of one row in fp64 (its definition), or None without any mass."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    mx = l.max()
    if mx == -np.inf:
        return None
    if T == 0:
        T, k = 1.0, 1
    order = np.argsort(-l, kind="stable")
    v = l[order]
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        w = np.where(v == mx, 1.0, np.exp((v - mx) / T))
    w = np.where((v > -np.inf) & ((mx < np.inf) | (v == mx)), w, 0.0)
    keep = int(k) if 0 < k < l.size else l.size
    if p < 1.0:
        before = np.concatenate(([0.0], np.cumsum(w)[:-1]))[:keep]
        keep = max(1, int((before < p * w[:keep].sum()).sum()))
    if mp > 0:
        bound = mx + (T * math.log(mp) if mp < 1 else 0.0)
        keep = min(keep, int((v >= bound).sum()))
    out = np.zeros(l.size)
    out[order[:keep]] = w[:keep]
    return out / out.sum()


def check(l, got, u, par, rows=None):
    token, prob, probs = (None if t is None else t.cpu().numpy() for t in got)
    l = l.float().cpu().numpy()
    for r in (range(l.shape[0]) if rows is None else rows):
        want = reference(l[r], **{k: float(v[r]) for k, v in par.items()})
        if want is None:
            assert token[r] == -1 and prob[r] == 0 and (probs is None or not probs[r].any())
            continue
        t, ur = int(token[r]), float(u[r])
        assert 0 <= t < l.shape[1] and want[t] > 0, (r, t)
        c = np.cumsum(want)
        lo = c[t - 1] if t else 0.0
        assert lo - WIDEN <= ur < c[t] + WIDEN, (r, t, lo, ur, c[t])
        assert abs(prob[r] - want[t]) <= PROB * want[t] + 1e-37
        if probs is not None:
            assert np.all(np.abs(probs[r] - want) <= PROB * want + 1e-37), r


def tensors(par):
    name = dict(T=("temperature", torch.float32), k=("top_k", torch.int32), p=("top_p", torch.float32),
                mp=("min_p", torch.float32))
    return {name[k][0]: torch.tensor(v, dtype=name[k][1], device=DEV) for k, v in par.items()}


def sample(l, u, par=None, probs=True, ok=True, **kw):
    R, V = l.shape
    token = torch.full((R,), -9, dtype=torch.int32, device=DEV)
    prob = torch.full((R,), -9.0, device=DEV)
    dist = torch.full((R, V), -9.0, device=DEV) if probs else None
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mtp_head_sample(l, torch.tensor(u, dtype=torch.float32, device=DEV), token, prob, dist, status=st,
                      **tensors(par or {}), **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == (0 if ok else m.ERR_ARG)
    return token, prob, dist


def logits(R, V, seed, bf=False):
    g = np.random.default_rng(seed)
    l = g.standard_normal((R, V)) * 2.0
    for r in range(R):
        l[r, g.integers(0, V, min(V, 12))] += g.random(min(V, 12)) * 10
    t = torch.from_numpy(l.astype(np.float32)).to(DEV)
    return t.bfloat16() if bf else t


def params(R, seed, which="Tkpm"):
    g = np.random.default_rng(seed)
    par = {}
    if "T" in which:
        par["T"] = np.float32(0.3 + 1.2 * g.random(R)).tolist()
    if "k" in which:
        par["k"] = g.integers(1, 60, R).tolist()
    if "p" in which:
        par["p"] = np.float32(0.5 + 0.5 * g.random(R)).tolist()
    if "m" in which:
        par["mp"] = np.float32(0.2 * g.random(R)).tolist()
    return par


@pytest.mark.parametrize("V", [1, 2, 31, 32, 33, 511, 512, 513, 1000, 4097, 16385, 50257, 154880])
@pytest.mark.parametrize("which", ["", "T", "Tk", "Tp", "Tkp", "Tkpm", "m"])
def test_lengths_and_filters(V, which):
    R = 5
    l = logits(R, V, V)
    u = np.random.default_rng(V + 1).random(R).astype(np.float32).tolist()
    par = params(R, V + 2, which)
    check(l, sample(l, u, par), u, par)


@pytest.mark.parametrize("R,V,bf", [(1, 154880, False), (1, 154880, True), (16, 154880, True), (40, 32000, False),
                                    (100, 5000, True), (300, 1200, False), (160, 154880, False)])
def test_row_counts(R, V, bf):
    l = logits(R, V, R, bf)
    u = np.random.default_rng(R).random(R).astype(np.float32).tolist()
    par = params(R, R + 5)
    check(l, sample(l, u, par), u, par, rows=range(0, R, max(1, R // 12)))


def test_vocabulary_longer_than_the_cluster_holds():
    V = 1_200_000
    l = logits(2, V, 3)
    u, par = [0.3, 0.9], dict(T=[1.0, 0.8], k=[0, 70000], p=[0.95, 0.999])
    check(l, sample(l, u, par), u, par)


@pytest.mark.parametrize("u", [0.0, 0.25, 0.5, 1.0 - 2.0 ** -24])
def test_equal_logits(u):
    """Every entry ties: prefixes by index, and the draw is exact (equal weights)."""
    V = 40000
    l = torch.full((4, V), 1.5, device=DEV)
    par = dict(k=[0, 5, 0, 39000], p=[1.0, 1.0, 0.5, 0.25])
    t, pr, dist = sample(l, [u] * 4, par)
    kept = [V, 5, V // 2, 9750]
    for r, n in enumerate(kept):
        assert int((dist[r] > 0).sum()) == n and bool((dist[r, :n] > 0).all())
        assert int(t[r]) == min(n - 1, int(math.floor(u * n)))
    check(l, (t, pr, dist), [u] * 4, par)


def test_many_ties_at_the_cut():
    """BF16 logits on a coarse grid: thousands of entries share the cut's value, the lowest indices stay."""
    g = np.random.default_rng(1)
    l = torch.from_numpy(np.round(g.standard_normal((3, 120000)) * 2).astype(np.float32)).to(DEV).bfloat16()
    u, par = [0.1, 0.6, 0.99], dict(k=[30000, 2, 100000], p=[1.0, 0.9, 0.7])
    check(l, sample(l, u, par), u, par)


def test_masked_entries():
    inf, nan = float("inf"), float("nan")
    l = logits(8, 3000, 2)
    l[0] = -inf
    l[1] = nan
    l[2, ::2] = -inf
    l[3] = -inf
    l[3, 2999] = -5.0
    l[4, 100:] = nan
    l[5, 7] = l[5, 2000] = inf          # two infinities share the mass
    l[6] = torch.finfo(torch.float32).min
    l[6, 11] = l[6, 13] = 0.0
    l[7, 0] = 3e38
    l[7, 1] = -3e38
    par = params(8, 3)
    par["k"][5] = 40
    par["p"][5] = 0.9
    u = [0.3, 0.3, 0.7, 0.99, 0.5, 0.6, 0.75, 0.5]
    got = sample(l, u, par)
    check(l, got, u, par)
    assert int(got[0][0]) == -1 and int(got[0][3]) == 2999 and int(got[0][5]) == 2000


def test_row_of_only_lowest_values():
    l = torch.full((2, 700), torch.finfo(torch.float32).min, device=DEV)
    u, par = [0.5, 0.5], dict(k=[0, 3])
    check(l, sample(l, u, par), u, par)


@pytest.mark.parametrize("V", [5, 3000, 60000])
def test_greedy_is_the_lowest_argmax(V):
    l = logits(3, V, 9)
    l[1, V // 2] = l[1, V - 1] = 50.0
    t, pr, dist = sample(l, [0.999, 0.999, 0.0], dict(T=[0.0] * 3))
    assert t.tolist() == [int(torch.argmax(l[0])), V // 2, int(torch.argmax(l[2]))]
    assert pr.tolist() == [1.0] * 3 and bool((dist.sum(1) == 1).all())


def test_extreme_parameters():
    l = logits(8, 20000, 4)
    par = dict(T=[1e30, 1e-30, 1e-6, 3.0, 1.0, 1.0, 1.0, 0.7], p=[1.0, 0.5, 1.0, 0.0, 1e-7, 1.0, 1.0, 2.0],
               mp=[0.0, 0.0, 0.0, 0.0, 0.0, 1.0, 1e-30, 0.0], k=[0, 0, 0, 0, 0, 0, 20000, -3])
    u = [0.5] * 8
    got = sample(l, u, par)
    check(l, got, u, par)
    top = torch.argmax(l, 1).tolist()
    for r in (1, 3, 4, 5):
        assert int(got[0][r]) == top[r] and float(got[1][r]) == 1.0


def test_one_far_outlier():
    """One logit at 1e30: every other entry falls into the last bin of the first round."""
    l = logits(2, 30000, 6)
    l[:, 77] = 1e30
    u, par = [0.5, 0.9], dict(k=[500, 25000])
    t, pr, dist = sample(l, u, par)
    assert t.tolist() == [77, 77] and pr.tolist() == [1.0, 1.0]
    l[:, 77] = -1e30
    u, par = [0.5, 0.9], dict(k=[500, 25000], p=[0.9, 0.99])
    check(l, sample(l, u, par), u, par)


def test_bad_parameters_refuse_their_row_alone():
    nan, inf = float("nan"), float("inf")
    l = logits(8, 900, 5)
    T = [1.0, -1.0, nan, inf, 1.0, 1.0, 1.0, 1.0]
    p = [1.0, 1.0, 1.0, 1.0, nan, -0.1, 1.0, 1.0]
    mp = [0.0] * 6 + [1.5, nan]
    t, pr, dist = sample(l, [0.5] * 8, dict(T=T, p=p, mp=mp), ok=False)
    assert t[1:].tolist() == [-1] * 7 and not pr[1:].any() and not dist[1:].any()
    check(l, (t, pr, dist), [0.5] * 8, {}, rows=[0])
    t, pr, dist = sample(l, [1.0, -0.5, nan, 0.5, 0.5, 0.5, 0.5, 0.5], ok=False)
    assert t[:3].tolist() == [-1] * 3 and int(t[3]) >= 0


def test_strided_rows_and_partial_outputs():
    wide = logits(6, 2100, 8)
    l = wide[:, 3:2003]
    u = np.random.default_rng(1).random(6).astype(np.float32).tolist()
    par = params(6, 2)
    got = sample(l, u, par)
    check(l, got, u, par)
    ut = torch.tensor(u, device=DEV)
    token = torch.zeros(6, dtype=torch.int32, device=DEV)
    m.mtp_head_sample(l, ut, token, **tensors(par))
    assert torch.equal(token, got[0])
    dist = torch.zeros(6, 2000, device=DEV)
    m.mtp_head_sample(l, probs=dist, **tensors(par))
    assert torch.equal(dist, got[2])
    with pytest.raises(ValueError, match="overlap|contiguous"):
        m.mtp_head_sample(wide.t(), ut, token)
    with pytest.raises(m.MTPError):
        m.mtp_head_sample(l, None, token)


def test_same_token_whatever_the_grouping():
    """A row's result does not depend on how many rows are sampled with it (clusters of another size)."""
    l = logits(200, 70000, 13)
    u = np.random.default_rng(3).random(200).astype(np.float32).tolist()
    par = params(200, 4)
    a = sample(l, u, par)
    for r in (0, 57, 199):
        one = {k: [v[r]] for k, v in par.items()}
        b = sample(l[r:r + 1], [u[r]], one)
        assert torch.equal(b[0], a[0][r:r + 1]) and torch.equal(b[2], a[2][r:r + 1])


def test_sampled_frequencies():
    """Evenly spaced u: each token comes up as often as its probability says, to within one step."""
    n = 4096
    l = logits(1, 300, 21).expand(n, 300).contiguous()
    u = ((np.arange(n) + 0.5) / n).astype(np.float32).tolist()
    t, _, dist = sample(l, u, dict(T=[0.9] * n, k=[40] * n))
    counts = np.bincount(t.cpu().numpy(), minlength=300)
    assert np.all(np.abs(counts - n * dist[0].cpu().numpy()) <= 1.0 + n * 2 ** -20)


def test_graph_replay_with_new_numbers():
    l = logits(4, 33000, 30)
    u = torch.zeros(4, device=DEV)
    par = params(4, 7)
    tp = tensors(par)
    token = torch.zeros(4, dtype=torch.int32, device=DEV)
    prob = torch.zeros(4, device=DEV)
    g = m.MtpDraftHead.capture(lambda s: m.mtp_head_sample(l, u, token, prob, stream=s, **tp))
    for seed in range(3):
        u.copy_(torch.rand(4, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        check(l, (token, prob, None), u.tolist(), par)


@pytest.mark.parametrize("R", [14, 15, 18, 19, 36, 37, 39, 151, 152, 153])
@pytest.mark.parametrize("which", ["Tp", "Tkp"])
def test_cluster_borders(R, which):
    """Row counts on both sides of every change of the CTAs per row and of what shared memory holds."""
    V = 9001
    l = logits(R, V, R, R % 2 == 0)
    u = np.random.default_rng(R).random(R).astype(np.float32).tolist()
    par = params(R, R + 1, which)
    check(l, sample(l, u, par), u, par, rows=[0, R // 2, R - 1])


@pytest.mark.parametrize("R,V", [(2, 688127), (2, 688129), (20, 172031), (20, 172033), (40, 57343), (40, 57345),
                                 (40, 172033), (152, 43007), (152, 43009)])
def test_slice_borders(R, V):
    """Rows about as long as what the cluster's CTAs hold in shared memory, one by one or two on an SM."""
    l = logits(R, V, V)
    u = np.random.default_rng(V).random(R).astype(np.float32).tolist()
    par = params(R, V, "Tp")
    check(l, sample(l, u, par), u, par, rows=[0, R - 1])


def test_longest_row():
    """2^31 - 1 tokens: equal logits share evenly (every weight is one, so the token is floor(u V) exactly); a
    few planted ones, the last index among them, are found."""
    V = 2 ** 31 - 1
    l = torch.full((1, V), -2.0, dtype=torch.bfloat16, device=DEV)
    for u in (0.0, 0.3, 0.75, 1.0 - 2.0 ** -24):
        t, pr, _ = sample(l, [u], probs=False)
        assert int(t) == int(np.float32(u).astype(np.float64) * V)
        assert abs(float(pr) * V - 1) <= PROB
    at = [5, 2 ** 30 + 7, V - 1]
    l[0, at] = torch.tensor([3.0, 4.0, 3.5], dtype=torch.bfloat16, device=DEV)
    for par in (dict(k=[3]), dict(p=[1e-7]), dict(mp=[0.3])):
        want = np.exp(np.array([3.0, 4.0, 3.5]) - 4.0)
        if "p" in par:  # the mass of all: 2^31 weights of e^-6, so only the largest is before the limit
            want = np.array([0.0, 1.0, 0.0])
        want /= want.sum()
        for u in (0.0, 0.5, 0.999):
            t, pr, _ = sample(l, [u], par, probs=False)
            j = int((np.cumsum(want) <= u).sum())
            assert int(t) == at[j] and abs(float(pr) - want[j]) <= PROB * want[j]


def test_rows_past_32_bits():
    """Row offsets beyond 2^32 elements of logits, and beyond 2^31 of the distribution."""
    V, ld = 1000, 2 ** 31 - 1
    buf = torch.empty(2 * ld + V, dtype=torch.bfloat16, device=DEV)
    l = buf.as_strided((3, V), (ld, 1))
    l.copy_(logits(3, V, 50, True))
    u, par = [0.2, 0.6, 0.9], params(3, 51)
    check(l, sample(l, u, par), u, par)
    del buf, l
    R, V = 16384, 151936
    l = torch.randn(R, V, dtype=torch.bfloat16, device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    u = np.random.default_rng(9).random(R).astype(np.float32).tolist()
    par = dict(p=[0.9] * R, k=[50] * R)
    t, pr, dist = sample(l, u, par)
    rows = [0, 8191, 14133, 14134, 14135, R - 1]
    check(l[rows], (t[rows], pr[rows], dist[rows]), [u[r] for r in rows], {k: [v[r] for r in rows] for k, v in par.items()})
    assert int((t < 0).sum()) == 0


def test_calls_in_flight_together():
    """Calls on several streams at once, and two captured graphs replayed side by side: each gives the bits of
    its own plain call (the operators share nothing)."""
    ls = [logits(r, v, s) for r, v, s in ((1, 154880, 1), (20, 40000, 2), (90, 5000, 3))]
    us = [np.random.default_rng(s).random(l.shape[0]).astype(np.float32).tolist() for s, l in enumerate(ls)]
    pars = [params(l.shape[0], 7 + s) for s, l in enumerate(ls)]
    want = [sample(l, u, p) for l, u, p in zip(ls, us, pars)]
    uts = [torch.tensor(u, dtype=torch.float32, device=DEV) for u in us]
    tps = [tensors(p) for p in pars]
    out = [[torch.zeros_like(t) for t in w] for w in want]
    graphs = [m.MtpDraftHead.capture(lambda s, i=i: m.mtp_head_sample(ls[i], uts[i], *out[i], stream=s, **tps[i]))
              for i in range(3)]
    got = [[torch.zeros_like(t) for t in w] for w in want]
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(3):
            m.mtp_head_sample(ls[i], uts[i], *got[i], stream=streams[i], **tps[i])
            with torch.cuda.stream(streams[3 + i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for w, g, o in zip(want, got, out):
        for x, y, z in zip(w, g, o):
            assert torch.equal(x, y) and torch.equal(x, z)


# ---------------------------------------------------------------------------- acceptance
def accept_reference(p, q, x, u, n):
    """(accepted, distribution of the next token or None) of one sequence, fp64."""
    V = p.shape[1]
    c = lambda a: np.clip(np.where(np.isnan(a), 0.0, a), 0.0, 1.0)  # noqa: E731
    a = 0
    while a < n:
        t = int(x[a])
        if not 0 <= t < V or not float(u[a]) * (1.0 if q is None else float(q[a, t])) < float(p[a, t]):
            break
        a += 1
    w = c(p[a].astype(np.float64))
    if a < n:
        if q is None:
            other = np.zeros(V)
            if 0 <= x[a] < V:
                other[x[a]] = 1.0
        else:
            other = c(q[a].astype(np.float64))
        left = np.maximum(w - other, 0.0)
        w = left if left.sum() > 0 else w
    return a, (w / w.sum() if w.sum() > 0 else None)


def run_verify(p, q, x, u, n=None, want_status=0):
    B, D = x.shape
    tokens = torch.full((B, D + 1), -9, dtype=torch.int32, device=DEV)
    acc = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    prob = torch.full((B,), -9.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mtp_head_verify(p, q, x, u, tokens, acc, prob, draft_len=n, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == want_status
    return tokens.cpu().numpy(), acc.cpu().numpy(), prob.cpu().numpy()


def check_verify(p, q, x, u, n=None, want_status=0, skip=()):
    tokens, acc, prob = run_verify(p, q, x, u, n, want_status)
    ph, xh, uh = p.cpu().numpy(), x.cpu().numpy(), u.cpu().numpy()
    qh = None if q is None else q.cpu().numpy()
    B, D = xh.shape
    for b in range(B):
        if b in skip:
            assert acc[b] == 0 and (tokens[b] == -1).all() and prob[b] == 0
            continue
        nb = D if n is None else int(n[b])
        a, w = accept_reference(ph[b], None if qh is None else qh[b], xh[b], uh[b], nb)
        assert acc[b] == a, (b, acc[b], a)
        assert (tokens[b, :a] == xh[b, :a]).all() and (tokens[b, a + 1:] == -1).all()
        t = int(tokens[b, a])
        if w is None:
            assert t == -1 and prob[b] == 0
            continue
        assert 0 <= t < w.size and w[t] > 0
        c = np.cumsum(w)
        assert (c[t - 1] if t else 0.0) - WIDEN <= uh[b, D] < c[t] + WIDEN, (b, t)
        assert abs(prob[b] - w[t]) <= 2.0 ** -20 * w[t]


def distributions(B, D, V, seed, noise=0.5):
    g = np.random.default_rng(seed)
    l = g.standard_normal((B, D + 1, V)) * 2
    ql = l[:, :D] + noise * g.standard_normal((B, D, V))
    soft = lambda z: np.exp(z - z.max(-1, keepdims=True)) / np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
    p, q = soft(l).astype(np.float32), soft(ql).astype(np.float32)
    x = np.stack([[g.choice(V, p=q[b, i].astype(np.float64) / q[b, i].astype(np.float64).sum()) for i in range(D)]
                  for b in range(B)]).astype(np.int32)
    u = g.random((B, D + 1)).astype(np.float32)
    return tuple(torch.from_numpy(a).to(DEV) for a in (p, q, x, u))


@pytest.mark.parametrize("B,D,V", [(1, 1, 1), (1, 1, 2), (3, 2, 31), (2, 1, 512), (5, 4, 513), (16, 4, 4096),
                                   (7, 8, 1000), (2, 3, 50257), (40, 2, 3000), (2, 70, 300), (1, 4, 154880)])
@pytest.mark.parametrize("greedy", [False, True])
def test_verify(B, D, V, greedy):
    p, q, x, u = distributions(B, D, V, B + D + V)
    if greedy:
        x = q.argmax(2).to(torch.int32)
    check_verify(p, None if greedy else q, x, u)


@pytest.mark.parametrize("B", [4, 5, 9, 10, 19, 20, 38, 39, 76, 77, 200])
def test_verify_cluster_borders(B):
    p, q, x, u = distributions(B, 2, 9001, B)
    check_verify(p, q, x, u)


def test_verify_past_32_bits():
    """Distributions of more than 2^31 numbers. Equal shares of 2^-24 are exact: every draft is accepted and the
    token is floor(u V); in the last sequence the drafter knows the first half only, its draft is refused
    (0.75 * 2 > 1) and the token comes from the second half."""
    B, D, V = 16, 9, 1 << 24
    p = torch.full((B, D + 1, V), 2.0 ** -24, device=DEV)
    q = torch.full((B, D, V), 2.0 ** -24, device=DEV)
    q[B - 1, 0, : V // 2] = 2.0 ** -23
    q[B - 1, 0, V // 2:] = 0.0
    x = torch.full((B, D), 5, dtype=torch.int32, device=DEV)
    u = torch.rand(B, D + 1, generator=torch.Generator().manual_seed(2))
    u[B - 1, 0] = 0.75
    tokens, acc, prob = run_verify(p, q, x, u.to(DEV))
    assert acc.tolist() == [D] * (B - 1) + [0]
    last = (u[:, D].double() * V).floor().long()
    last[B - 1] = V // 2 + int((u[B - 1, D].double() * (V // 2)).floor())
    assert [int(tokens[b, a]) for b, a in enumerate(acc.tolist())] == last.tolist()
    assert prob.tolist() == [2.0 ** -24] * (B - 1) + [2.0 ** -23]


def test_verify_lengths():
    p, q, x, u = distributions(6, 4, 700, 3)
    n = torch.tensor([0, 1, 2, 3, 4, 4], dtype=torch.int32, device=DEV)
    check_verify(p, q, x, u, n)
    check_verify(p, None, x, u, n)


def test_verify_same_distribution_accepts_everything():
    p, q, x, u = distributions(5, 3, 900, 4)
    q = p[:, :3].contiguous()
    x = torch.stack([torch.stack([(q[b, i].double().cumsum(0) < 0.5).sum() for i in range(3)]) for b in range(5)])
    check_verify(p, q, x.to(torch.int32), u)


def test_verify_empty_residual_and_empty_rows():
    """p = q at a rejected draft (a probability of zero under both) falls back to p; rows without mass
    give -1; NaN and negative entries count as nothing."""
    p, q, x, u = distributions(5, 2, 600, 5)
    q[0] = p[0, :2]
    q[0, 0, 9] = p[0, 0, 9] = 0.0
    x[0, 0] = 9
    p[1] = 0.0
    p[2, :, 17] = float("nan")
    x[2, 0] = 17
    p[3, 0, 100:] = -1.0
    x[3, 0] = 300
    q[4, 0] = float("nan")
    check_verify(p, q, x, u)


def test_verify_bad_sequences():
    p, q, x, u = distributions(6, 3, 400, 6)
    x[0, 0] = 400
    x[1, 0] = -1
    u[2, 1] = 1.0
    u[3, 3] = float("nan")
    n = torch.tensor([3, 3, 3, 3, 4, 3], dtype=torch.int32, device=DEV)
    tokens, acc, prob = run_verify(p[:2].contiguous(), q[:2].contiguous(), x[:2].contiguous(), u[:2].contiguous(),
                                   want_status=m.ERR_TOKEN_RANGE)
    assert acc.tolist() == [0, 0] and (tokens[:, 0] >= 0).all()
    check_verify(p[:2].contiguous(), q[:2].contiguous(), x[:2].contiguous(), u[:2].contiguous(),
                 want_status=m.ERR_TOKEN_RANGE)
    check_verify(p[:2].contiguous(), None, x[:2].contiguous(), u[:2].contiguous(), want_status=m.ERR_TOKEN_RANGE)
    check_verify(p[2:].contiguous(), q[2:].contiguous(), x[2:].contiguous(), u[2:].contiguous(), n[2:].contiguous(),
                 want_status=m.ERR_ARG, skip=(0, 1, 2))


def test_verify_graph_replay():
    p, q, x, u = distributions(4, 3, 5000, 7)
    tokens = torch.zeros(4, 4, dtype=torch.int32, device=DEV)
    acc = torch.zeros(4, dtype=torch.int32, device=DEV)
    g = m.MtpDraftHead.capture(lambda s: m.mtp_head_verify(p, q, x, u, tokens, acc, stream=s))
    for seed in range(3):
        u.copy_(torch.rand(4, 4, generator=torch.Generator().manual_seed(seed)))
        g.replay()
        torch.cuda.synchronize()
        t2, a2, _ = run_verify(p, q, x, u)
        assert np.array_equal(tokens.cpu().numpy(), t2) and np.array_equal(acc.cpu().numpy(), a2)


def test_drafting_and_acceptance_together():
    """A speculative step as it is used: D sampled drafts per sequence over the head's FP4 copies, each
    fed into the next, then the acceptance against target distributions made by the same sampler. With
    the target equal to the drafter every draft is accepted; recorded as one graph it replays alike."""
    import synth
    H, V, B, D = 256, 4096, 5, 3
    w = synth.make_weights(H, V, 1, "cpu")
    g = {k: v.to(DEV) for k, v in w.as_dict().items()}
    head = m.MtpDraftHead(g["embed"], g["lm_head"], g["eh_proj"], g["enorm_w"], g["hnorm_w"], g["final_norm_w"],
                          max_batch=B)
    assert head.quantize_fp4() == 0
    tokens, hidden = (t.to(DEV) for t in synth.make_step_inputs(H, V, B, 2, "cpu"))
    u = torch.rand(B, D + 1, generator=torch.Generator().manual_seed(0)).to(DEV)
    T = torch.full((B,), 0.8, device=DEV)
    topk = torch.full((B,), 50, dtype=torch.int32, device=DEV)
    target = torch.softmax(torch.randn(B, D + 1, V, generator=torch.Generator().manual_seed(1)).to(DEV), 2)

    def step(tgt):
        tok, h, drafts, dists = tokens, hidden, [], []
        for i in range(D):
            x, lg, _ = head.forward(tok, h, fp4=True, logits=True)
            tok, _, dist = head.sample(lg, u[:, i].contiguous(), temperature=T, top_k=topk)
            drafts.append(tok)
            dists.append(dist)
            h = x
        x = torch.stack(drafts, 1)
        q = torch.stack(dists, 1)
        p = torch.cat([q, tgt[:, -1:]], 1) if tgt is target else tgt
        return x, q, p, head.verify(p, q, x, u)

    x, q, p, (out, acc) = step(target)
    torch.cuda.synchronize()
    assert acc.tolist() == [D] * B and torch.equal(out[:, :D], x) and bool((out[:, D] >= 0).all())
    for b in range(B):
        assert bool((q[b].gather(1, x[b].long()[:, None]) > 0).all())
    other = target.clone()
    x, q, p, (out, acc) = step(other)
    check_verify(p, q, x, u)
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        x2, q2, p2, (out2, acc2) = step(other)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x2, x) and torch.equal(q2, q) and torch.equal(out2, out) and torch.equal(acc2, acc)
