"""The FP4 copies and the stages over them, against fp64 references from the definitions."""
import numpy as np
import pytest
import torch

import fp4_helpers as ref
import mtp_speculative_draft_head_gb300 as m
import oracle
import synth
from gpu_helpers import context_band, lowest_argmax

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


def bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(oracle.f64_to_bf16(a).view(np.int16).copy()).view(torch.bfloat16).to(DEV)


def vals(t: torch.Tensor) -> np.ndarray:
    return oracle.bf16_to_f64(synth.bits(t))


def make_copy(w: torch.Tensor):
    w4 = m.fp4_empty(*w.shape, DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mtp_head_quantize_fp4(w, *w4, st)
    return w4, int(st.item())


def host(w4):
    return tuple(t.cpu().numpy() for t in w4)


def rng_matrix(V, H, seed, kind="normal"):
    r = np.random.default_rng(seed)
    w = r.standard_normal((V, H)) * 0.02
    if kind == "outliers":
        w[r.random((V, H)) < 0.01] *= 300.0
    elif kind == "ties":       # small multiples of a power of two: quotients on the rounding borders
        w = r.integers(-24, 25, (V, H)) * 0.25
        w[:, 0] = 2688.0 / 448.0
        w[: V // 2, H - 1] = 2688.0   # row scale 1: block scales and codes tie exactly
    elif kind == "tiny":
        w = r.standard_normal((V, H)) * 1e-38
        w[0] = 0.0
        w[1 % V] = 9.2e-41 * (r.random(H) < 0.5)
    elif kind == "huge":
        w = r.standard_normal((V, H)) * 5e37
    elif kind == "wide":       # blocks far below their row's maximum: scales underflow to zero
        w = r.standard_normal((V, H)) * 10.0 ** r.uniform(-9, 1, (V, H))
    elif kind == "signs":
        w = np.where(r.random((V, H)) < 0.5, -0.0, 0.0)
        w[:, H // 2] = -1.0
    return w


@pytest.mark.parametrize("V,H", [(1, 1), (3, 15), (5, 16), (2, 24), (2, 255), (7, 256), (4, 257), (300, 1000),
                                 (1300, 264), (9, 4100), (1, 131072), (1217, 33)])
def test_quantize_bits(V, H):
    w = bf16(rng_matrix(V, H, V * 7 + H))
    w4, st = make_copy(w)
    assert st == 0
    codes, sc, rs = ref.quantize(vals(w))
    q, bs, r = host(w4)
    assert np.array_equal(r.view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(bs, sc)
    assert np.array_equal(q, ref.pack(codes))


@pytest.mark.parametrize("V,H", [(20000, 40), (9800, 1536), (20, 1544), (5000, 2056), (20, 6144), (2600, 6152),
                                 (20, 12288), (1300, 12296), (3, 24576), (3, 24584), (1500, 1001)])
def test_quantize_and_back_on_both_sides_of_every_form(V, H):
    """Row lengths around the changes of threads per row, and more rows than run at once; sampled rows."""
    g = torch.Generator(DEV).manual_seed(V + H)
    w = (torch.randn(V, H, device=DEV, generator=g) * 0.02).bfloat16()
    w4, st = make_copy(w)
    assert st == 0
    rows = torch.cat([torch.arange(0, V, max(1, V // 9)), torch.tensor([V - 1])]).to(DEV)
    codes, sc, rs = ref.quantize(vals(w[rows]))
    q, bs, r = host(tuple(t[rows] for t in w4))
    assert np.array_equal(r.view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(bs, sc)
    assert np.array_equal(q, ref.pack(codes))
    out = torch.full((V, H), 7.0, dtype=torch.bfloat16, device=DEV)
    m.mtp_head_dequantize_fp4(*w4, out)
    v = torch.from_numpy((ref.E2M1[codes & 7] * np.where(codes > 7, -1.0, 1.0) *
                          np.repeat(ref.E4M3[bs], 16, axis=1))[:, :H].astype(np.float32) * r[:, None]).bfloat16()
    assert torch.equal(out[rows].cpu(), v)
    assert not bool((out == 7.0).any())


@pytest.mark.parametrize("kind", ["outliers", "ties", "tiny", "huge", "wide", "signs"])
@pytest.mark.parametrize("V,H", [(40, 272), (1300, 72), (13, 101)])
def test_quantize_bits_hard_rows(kind, V, H):
    w = bf16(rng_matrix(V, H, 5, kind))
    w4, st = make_copy(w)
    assert st == 0
    codes, sc, rs = ref.quantize(vals(w))
    q, bs, r = host(w4)
    assert np.array_equal(r.view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(bs, sc)
    assert np.array_equal(q, ref.pack(codes))


@pytest.mark.parametrize("V", [6, 1300])
def test_quantize_nonfinite_rows_become_zeros(V):
    w = rng_matrix(V, 80, 3)
    t = bf16(w)
    t[1, 7] = float("nan")
    t[V - 1, 79] = float("-inf")
    w4, st = make_copy(t)
    assert st == m.ERR_NONFINITE
    q, bs, r = host(w4)
    for row in (1, V - 1):
        assert r[row] == 0 and not q[row].any() and not bs[row].any()
    codes, sc, rs = ref.quantize(vals(t[2:3]))
    assert np.array_equal(q[2:3], ref.pack(codes)) and r[2] == rs[0]


@pytest.mark.parametrize("V,H", [(1, 1), (3, 8), (3, 17), (5, 24), (33, 256), (70, 1000), (4, 4099)])
@pytest.mark.parametrize("kind", ["normal", "wide", "huge"])
def test_dequantize(V, H, kind):
    w4, _ = make_copy(bf16(rng_matrix(V, H, 11, kind)))
    out = torch.full((V, H), 7.0, dtype=torch.bfloat16, device=DEV)
    m.mtp_head_dequantize_fp4(*w4, out)
    q, bs, rs = host(w4)
    c = ref.unpack(q)
    v = np.where(c > 7, -ref.E2M1[c & 7], ref.E2M1[c & 7]) * np.repeat(ref.E4M3[bs], 16, axis=1)
    want = (v[:, :H].astype(np.float32) * rs[:, None]).astype(np.float64)
    assert np.array_equal(vals(out), oracle.bf16_to_f64(oracle.f64_to_bf16(want)))


# ---------------------------------------------------------------------------- output stage
def sweep_band(H: int) -> float:
    """Bound of |logit - exact| over the sum of |products| (row scale applied): 16 chained MMAs of 16
    exact products at a time (each at most two roundings of 2^-23 of the running sum of magnitudes),
    the run totals added in fp32 (2^-24 each), two multiplications at the end, and the f16
    activations' underflow (2^-25 of 2^14, below 2^-38 of the largest, at most once per product)."""
    n = ref.padded(H) // 256
    return 16 * 2 * 2.0 ** -23 + (n + 2) * 2.0 ** -24


def run_sweep(x, fw, w4, logits=True, ws=None, B=None, **kw):
    B, H = x.shape
    V = w4[2].numel()
    ws = m.fp4_workspace(B, H, V, DEV) if ws is None else ws
    lg = torch.full((B, V), 1e30, dtype=torch.float32, device=DEV) if logits else None
    d = torch.full((B,), -7, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mtp_head_logits_argmax_fp4(x, fw, *w4, lg, d, ws, st, eps=EPS, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    return lg, d, ws


def sweep_inputs(B, H, V, seed):
    r = np.random.default_rng(seed)
    x = bf16(r.standard_normal((B, H)))
    fw = bf16(1.0 + 0.1 * r.standard_normal(H))
    w4, st = make_copy(bf16(rng_matrix(V, H, seed + 1)))
    assert st == 0
    return x, fw, w4


def check_sweep(x, fw, w4, lg, d):
    B, H = x.shape
    xhat = ref.norm(synth.bits(x), synth.bits(fw), EPS)
    w = ref.values(*host(w4), H)
    exact = xhat @ w.T
    tol = sweep_band(H) * (np.abs(xhat) @ np.abs(w).T) + 2.0 ** -38 * np.abs(xhat).max(1, keepdims=True) * np.abs(w).sum(1)
    got = lg.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - exact) <= tol), float((np.abs(got - exact) / tol).max())
    for b in range(B):
        assert int(d[b].item()) == lowest_argmax(got[b])


@pytest.mark.parametrize("B,H,V", [(1, 1, 1), (1, 64, 5), (2, 100, 300), (3, 255, 129), (1, 256, 4096), (8, 257, 1000),
                                   (9, 520, 777), (16, 1024, 2500), (5, 1, 40), (16, 16, 20000), (1, 6144, 3001),
                                   (13, 4097, 333), (4, 65536, 70)])
def test_sweep_against_fp64(B, H, V):
    x, fw, w4 = sweep_inputs(B, H, V, B + H + V)
    lg, d, ws = run_sweep(x, fw, w4)
    check_sweep(x, fw, w4, lg, d)
    # without logits: the same drafts; the workspace serves the next call and smaller batches
    _, d2, _ = run_sweep(x, fw, w4, logits=False, ws=ws)
    assert torch.equal(d, d2)
    lg3, d3, _ = run_sweep(x[:1].contiguous(), fw, w4, ws=ws)
    assert torch.equal(lg3[0], lg[0]) and int(d3[0]) == int(d[0])
    assert not ws[:2304].any()


def test_sweep_magnitudes():
    """Activations and weights far from one, rows of zeros, and eps that dominates."""
    x, fw, w4 = sweep_inputs(4, 512, 600, 21)
    x[0] *= 1e18
    x[1] *= 1e-18
    x[2] = 0.0
    w = bf16(rng_matrix(600, 512, 4) * 1e20)
    w[5] = 0.0
    w4, _ = make_copy(w)
    lg, d, _ = run_sweep(x, fw, w4)
    check_sweep(x, fw, w4, lg, d)
    assert int(d[2]) == 0 and not lg[2].any() and not lg[:, 5].any()


@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("scale", [1e-38, 1e-25, 1e-12, 1e18, 1e30, 3e37])
def test_sweep_rows_whose_squares_leave_fp32(scale, eps):
    x, fw, w4 = sweep_inputs(2, 300, 400, 22)
    x[1] = (x[1].double() * scale).bfloat16()
    V = 400
    lg = torch.zeros(2, V, device=DEV)
    d = torch.zeros(2, dtype=torch.int32, device=DEV)
    m.mtp_head_logits_argmax_fp4(x, fw, *w4, lg, d, m.fp4_workspace(2, 300, V, DEV), eps=eps)
    xhat = ref.norm(synth.bits(x), synth.bits(fw), float(np.float32(eps)))
    w = ref.values(*host(w4), 300)
    tol = sweep_band(300) * (np.abs(xhat) @ np.abs(w).T) + 2.0 ** -38 * np.abs(xhat).max(1, keepdims=True) * np.abs(w).sum(1)
    # below the fp32 range the logits round to its smallest step
    assert np.all(np.abs(lg.cpu().numpy() - xhat @ w.T) <= tol + 2.0 ** -148)


def test_sweep_ties_take_the_lowest_row():
    x, fw, _ = sweep_inputs(3, 256, 8, 2)
    w = bf16(rng_matrix(1500, 256, 9) * 0.01)
    big = torch.sign(x[0].float()).bfloat16()
    for r in (1499, 700, 130, 131):
        w[r] = big
    w4, _ = make_copy(w)
    lg, d, _ = run_sweep(x, fw, w4)
    check_sweep(x, fw, w4, lg, d)
    assert int(d[0]) == 130


def test_sweep_nan_sequence_drafts_minus_one():
    x, fw, w4 = sweep_inputs(2, 256, 500, 8)
    x[1, 3] = float("nan")
    lg, d, ws = run_sweep(x, fw, w4)
    assert int(d[1]) == -1 and bool(torch.isnan(lg[1]).all())
    assert int(d[0]) == lowest_argmax(lg[0].cpu().numpy().astype(np.float64))
    assert not ws[:2304].any()


@pytest.mark.parametrize("B", [1, 16])
@pytest.mark.parametrize("limit", [0, 200])
def test_sweep_wait_limit(B, limit):
    """Stage waits cut short report MTP_ERR_TIMEOUT or finish; the workspace serves the next call."""
    x, fw, w4 = sweep_inputs(B, 2048, 30000, 17)
    lg, d, ws = run_sweep(x, fw, w4)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    l2, d2 = torch.zeros_like(lg), torch.zeros_like(d)
    prev = m.mtp_head_set_wait_limit_ns(limit)
    try:
        m.mtp_head_logits_argmax_fp4(x, fw, *w4, l2, d2, ws, st, eps=EPS)
        torch.cuda.synchronize()
    finally:
        m.mtp_head_set_wait_limit_ns(prev)
    code = int(st.item())
    assert code == m.ERR_TIMEOUT if limit == 0 else code in (0, m.ERR_TIMEOUT)
    assert not ws[:2304].any()
    l3, d3, _ = run_sweep(x, fw, w4, ws=ws)
    assert torch.equal(l3, lg) and torch.equal(d3, d)


def test_sweep_graph_and_streams():
    """Two captured graphs with workspaces of their own, replayed on different streams together, and a
    call on a side stream: the bits of the plain call."""
    x, fw, w4 = sweep_inputs(16, 768, 9000, 31)
    lg, d, _ = run_sweep(x, fw, w4)
    outs, graphs = [], []
    for _ in range(2):
        ws = m.fp4_workspace(16, 768, 9000, DEV)
        l2, d2 = torch.zeros_like(lg), torch.zeros_like(d)
        graphs.append(m.MtpDraftHead.capture(
            lambda s, ws=ws, l2=l2, d2=d2: m.mtp_head_logits_argmax_fp4(x, fw, *w4, l2, d2, ws, eps=EPS, stream=s)))
        outs.append((l2, d2))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for l2, d2 in outs:
        assert torch.equal(l2, lg) and torch.equal(d2, d)
    s = torch.cuda.Stream()
    l3, d3 = torch.zeros_like(lg), torch.zeros_like(d)
    ws = m.fp4_workspace(16, 768, 9000, DEV)
    torch.cuda.synchronize()
    m.mtp_head_logits_argmax_fp4(x, fw, *w4, l3, d3, ws, eps=EPS, stream=s)
    s.synchronize()
    assert torch.equal(l3, lg) and torch.equal(d3, d)


# ---------------------------------------------------------------------------- linear
def check_linear(x, w4, y):
    R, K = x.shape
    codes, sc, rs = ref.quantize(vals(x))
    a = ref.values(ref.pack(codes), sc, rs, K)
    w = ref.values(*host(w4), K)
    exact = a @ w.T
    # the fp32 accumulation (context_band), two scale products, then one rounding to BF16
    e = (context_band(K) + 2.0 ** -22) * (np.abs(a) @ np.abs(w).T)
    tol = e + 2.0 ** -8 * (np.abs(exact) + e) + 1e-45
    got = vals(y)
    assert np.all(np.abs(got - exact) <= tol), float((np.abs(got - exact) / tol).max())


@pytest.mark.parametrize("R,N,K", [(1, 1, 1), (1, 64, 256), (2, 130, 100), (7, 33, 257), (8, 128, 512), (16, 300, 1024),
                                   (17, 257, 768), (32, 96, 320), (33, 512, 2048), (64, 700, 264), (100, 1000, 1000),
                                   (129, 128, 256), (300, 555, 777), (513, 264, 512), (1, 6144, 3000), (3, 40, 131072),
                                   (1000, 16, 64), (256, 256, 4096)])
def test_linear_against_fp64(R, N, K):
    r = np.random.default_rng(R + N + K)
    x = bf16(r.standard_normal((R, K)))
    w4, _ = make_copy(bf16(rng_matrix(N, K, R + 1)))
    ws = m.linear_fp4_workspace(R, N, K, DEV)
    ws.fill_(0xEE)  # no initialisation is needed
    y = torch.full((R, N), 1e30, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mtp_head_linear_fp4(x, *w4, y, ws, st)
    assert int(st.item()) == 0
    check_linear(x, w4, y)
    y2 = torch.zeros_like(y)
    m.mtp_head_linear_fp4(x, *w4, y2, ws)
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


def test_linear_magnitudes_and_bad_rows():
    x = bf16(rng_matrix(20, 300, 3, "wide"))
    x[4] = 0.0
    x[7, 299] = float("nan")
    x[9, 0] = float("inf")
    w = bf16(rng_matrix(50, 300, 4, "outliers") * 1e10)
    w[3] = 0.0
    w4, _ = make_copy(w)
    y = torch.full((20, 50), 5.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mtp_head_linear_fp4(x, *w4, y, m.linear_fp4_workspace(20, 50, 300, DEV), st)
    assert int(st.item()) == m.ERR_NONFINITE
    assert not y[[4, 7, 9]].any() and not y[:, 3].any()
    keep = [i for i in range(20) if i not in (7, 9)]
    check_linear(x[keep].contiguous(), w4, y[keep])


def test_linear_graph_replay_on_new_rows():
    r = np.random.default_rng(5)
    x = bf16(r.standard_normal((24, 512)))
    w4, _ = make_copy(bf16(rng_matrix(640, 512, 6)))
    ws = m.linear_fp4_workspace(24, 640, 512, DEV)
    y = torch.zeros(24, 640, dtype=torch.bfloat16, device=DEV)
    g = m.MtpDraftHead.capture(lambda s: m.mtp_head_linear_fp4(x, *w4, y, ws, stream=s))
    for seed in (1, 2):
        x.copy_(bf16(np.random.default_rng(seed).standard_normal((24, 512))))
        g.replay()
        torch.cuda.synchronize()
        check_linear(x, w4, y)


def test_linear_long_weights():
    """Weights that do not stay in L2 (69 MB) and 18 activation tiles: the schedule that passes over them once for
    each group of 16, the last group short and the last weight tile ragged; sampled rows and columns."""
    R, N, K = 4000, 120003, 1000
    g = torch.Generator(DEV).manual_seed(8)
    x = torch.randn(R, K, device=DEV, generator=g).bfloat16()
    w4, _ = make_copy((torch.randn(N, K, device=DEV, generator=g) * 0.02).bfloat16())
    y = torch.full((R, N), 1e30, dtype=torch.bfloat16, device=DEV)
    m.mtp_head_linear_fp4(x, *w4, y, m.linear_fp4_workspace(R, N, K, DEV))
    rows = torch.arange(0, R, 31, device=DEV)
    cols = torch.cat([torch.arange(0, N, 523, device=DEV), torch.arange(N - 140, N, device=DEV)])
    check_linear(x[rows].contiguous(), tuple(t[cols].contiguous() for t in w4), y[rows][:, cols])
    assert not bool((y == 1e30).any())


def test_linear_calls_in_flight_together():
    """Calls of every schedule (k split, whole tiles, pairs) on streams of their own at once, with workspaces of
    their own, and graphs of them replayed beside: the bits of the plain calls."""
    shapes = [(4, 300, 1024), (40, 10240, 100), (700, 6144, 256), (1, 6144, 2048)]
    ins, want = [], []
    for R, N, K in shapes:
        x = bf16(np.random.default_rng(R).standard_normal((R, K)))
        w4, _ = make_copy(bf16(rng_matrix(N, K, R + 1)))
        ins.append((x, w4))
        y = torch.zeros(R, N, dtype=torch.bfloat16, device=DEV)
        m.mtp_head_linear_fp4(x, *w4, y, m.linear_fp4_workspace(R, N, K, DEV))
        want.append(y)
    new = lambda: [(torch.zeros_like(y), m.linear_fp4_workspace(*s, DEV)) for y, s in zip(want, shapes)]  # noqa: E731
    eager, rec = new(), new()
    graphs = [m.MtpDraftHead.capture(lambda s, i=i: m.mtp_head_linear_fp4(ins[i][0], *ins[i][1], *rec[i], stream=s))
              for i in range(len(shapes))]
    streams = [torch.cuda.Stream() for _ in range(2 * len(shapes))]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (x, w4) in enumerate(ins):
            m.mtp_head_linear_fp4(x, *w4, *eager[i], stream=streams[i])
            with torch.cuda.stream(streams[len(shapes) + i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for y, (e, _), (r, _) in zip(want, eager, rec):
        assert torch.equal(y, e) and torch.equal(y, r)


def test_linear_output_as_the_next_stages_weights():
    """Each kernel of a chain launches early only past its own wait: a matrix made by the linear, copied to FP4
    and multiplied again in the same breath gives what the calls give one by one."""
    a = bf16(np.random.default_rng(1).standard_normal((512, 768)))
    w4, _ = make_copy(bf16(rng_matrix(256, 768, 2)))
    x = bf16(np.random.default_rng(3).standard_normal((9, 256)))
    y, out = torch.zeros(512, 256, dtype=torch.bfloat16, device=DEV), torch.zeros(9, 512, dtype=torch.bfloat16, device=DEV)
    y4 = m.fp4_empty(512, 256, DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws, ws2 = m.linear_fp4_workspace(512, 256, 768, DEV), m.linear_fp4_workspace(9, 512, 256, DEV)

    def chain(wait):
        m.mtp_head_linear_fp4(a, *w4, y, ws)
        wait()
        m.mtp_head_quantize_fp4(y, *y4, st)
        wait()
        m.mtp_head_linear_fp4(x, *y4, out, ws2)
        wait()
    chain(torch.cuda.synchronize)
    want = out.clone()
    for _ in range(20):
        out.zero_()
        y.zero_()
        for t in y4:
            t.zero_()
        chain(lambda: None)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


# ---------------------------------------------------------------------------- input stage
@pytest.mark.parametrize("R,H", [(1, 64), (3, 264), (16, 512), (40, 256), (300, 1024)])
def test_context_rows(R, H):
    V = 500
    w = synth.make_weights(H, V, 3, "cpu")
    tokens, hidden = synth.make_step_inputs(H, V, R, 4, "cpu", distinct=False)
    tokens[R // 2] = V if R > 1 else tokens[0]
    wb = {k: synth.bits(v) for k, v in w.as_dict().items()}
    ok = (tokens.numpy() >= 0) & (tokens.numpy() < V)
    concat = np.concatenate([ref.norm(wb["embed"][np.where(ok, tokens.numpy(), 0)], wb["enorm_w"], EPS),
                             ref.norm(synth.bits(hidden), wb["hnorm_w"], EPS)], 1)
    g = {k: v.to(DEV) for k, v in w.as_dict().items()}
    eh, st0 = make_copy(g["eh_proj"])
    assert st0 == 0
    x = torch.full((R, H), 9.0, dtype=torch.bfloat16, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.mtp_head_context_rows_fp4(g["embed"], g["enorm_w"], g["hnorm_w"], *eh, tokens.to(DEV), hidden.to(DEV), x,
                                m.context_fp4_workspace(R, H, DEV), st, eps=EPS)
    assert int(st.item()) == (0 if ok.all() else m.ERR_TOKEN_RANGE)
    assert not x[torch.from_numpy(~ok).to(DEV)].any()
    check_linear(bf16(concat[ok]), eh, x[torch.from_numpy(ok).to(DEV)])


# ---------------------------------------------------------------------------- the head
def test_head_over_fp4_copies():
    """A draft step of the head over its FP4 copies is its input stage followed by its output stage,
    and its logits stay near the BF16 head's (four-bit weights: a loose bound on the whole)."""
    H, V, B = 512, 3000, 6
    w = synth.make_weights(H, V, 1, "cpu")
    g = {k: v.to(DEV) for k, v in w.as_dict().items()}
    head = m.MtpDraftHead(g["embed"], g["lm_head"], g["eh_proj"], g["enorm_w"], g["hnorm_w"], g["final_norm_w"],
                          max_batch=B)
    tokens, hidden = (t.to(DEV) for t in synth.make_step_inputs(H, V, B, 2, "cpu"))
    with pytest.raises(RuntimeError, match="quantize_fp4"):
        head.forward(tokens, hidden, fp4=True)
    assert head.quantize_fp4() == 0
    with pytest.raises(ValueError):
        head.logits_argmax(hidden, fp8=True, fp4=True)
    x, lg, d = head.forward(tokens, hidden, fp4=True, logits=True)
    x2 = head.input(tokens, hidden, fp4=True)
    lg2, d2 = head.logits_argmax(x2, fp4=True)
    assert torch.equal(x, x2) and torch.equal(lg, lg2) and torch.equal(d, d2)
    check_sweep(x, g["final_norm_w"], head.lm_head_fp4, lg, d)
    _, full, _ = head.forward(tokens, hidden, logits=True)
    cos = torch.nn.functional.cosine_similarity(lg.double(), full.double(), dim=1)
    assert float(cos.min()) > 0.9


def test_refusals_on_device():
    w = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w4 = m.fp4_empty(4, 64, DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="bfloat16"):
        m.mtp_head_quantize_fp4(w.float(), *w4, st)
    with pytest.raises(ValueError, match="contiguous"):
        m.mtp_head_quantize_fp4(torch.zeros(64, 4, dtype=torch.bfloat16, device=DEV).t(), *w4, st)
    with pytest.raises(ValueError, match="shape"):
        m.mtp_head_quantize_fp4(w, w4[0][:, :64].contiguous(), w4[1], w4[2], st)
    with pytest.raises(ValueError, match="required|tensor"):
        m.mtp_head_quantize_fp4(w, *w4, None)
    x = torch.zeros(17, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(m.MTPError) as e:
        m.mtp_head_logits_argmax_fp4(x, x[0], *w4, None, torch.zeros(17, dtype=torch.int32, device=DEV),
                                     torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))
    assert e.value.code == m.ERR_SHAPE
    with pytest.raises(m.MTPError) as e:
        m.mtp_head_linear_fp4(x, *w4, torch.zeros(17, 4, dtype=torch.bfloat16, device=DEV),
                              torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.code == m.ERR_WORKSPACE
