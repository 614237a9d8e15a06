"""The attention half's operators where values, scales, streams and waits are out of the ordinary."""
import numpy as np
import pytest
import torch

import mtp_speculative_draft_head_gb300 as m
from mtp_speculative_draft_head_gb300 import _lib
import oracle
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, I32, F32, F64 = torch.bfloat16, torch.int32, torch.float32, torch.float64
INF, NAN = float("inf"), float("nan")


def i32(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def status():
    return torch.zeros(1, dtype=I32, device=DEV)


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


# ------------------------------------------------------------------------------------- prompts
def prompt(q, k, v, starts, st=None):
    out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    m.mtp_head_attention_prompt(q, k, v, i32(starts), out, lse, status=st)
    return out, lse


def with_values_planted(starts, good, v, plant):
    """What the outputs `good` become when the elements {(row, key head, column): value} of v are infinite or NaN: a row that
    sees infinities of one sign has them, one that sees a NaN or both signs has a NaN, and every other element stays."""
    G = good.shape[1] // v.shape[1]
    want = good.clone()
    for (row, h, c), x in plant.items():
        end = next(b for a, b in zip(starts[:-1], starts[1:]) if a <= row < b)
        part = want[row:end, h * G:(h + 1) * G, c]
        part.copy_(torch.where(torch.isfinite(part), torch.tensor(x, dtype=BF, device=DEV), part + x))
    return want


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [{0: INF, 5: NAN, 127: -INF}, {300: INF, 310: NAN}, {5: INF, 130: -INF, 255: NAN, 256: INF, 599: INF}])
def test_prompt_carries_infinities_and_nan_of_every_place(D, rows):
    """Non-finite values in the first and in the second 128 rows of each 256: every later row of the sequence has them, those
    of the second 128 as well, whose products read the rows of the first after these were cleared."""
    starts = [3, 303, 903, 1159]
    g = gen(D)
    q, k, v = (torch.randn((1164, n, D), generator=g, device=DEV).bfloat16() for n in (4, 2, 2))
    good, good_lse = prompt(q, k, v, starts)
    plant = {}
    for s, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        for i, (r, x) in enumerate(rows.items()):
            if a + r < b:
                plant[a + r, (s + i) % 2, (7 * i + 13 * s) % D] = x
                plant[a + r, (s + i) % 2, D - 1] = x  # (a column where several meet)
    for (r, h, c), x in plant.items():
        v[r, h, c] = x
    out, lse = prompt(q, k, v, starts)
    assert same(out, with_values_planted(starts, good, v, plant))
    assert torch.equal(lse, good_lse)


def test_prompt_marks_of_one_piece_do_not_reach_the_next():
    """Thousands of short pieces, one after another in the same CTAs, every third with an infinity among its values: one
    and two tiles long by turns."""
    lens = [(1, 100, 128, 129, 200, 256)[(i * i + i // 7) % 6] for i in range(600)]
    starts = np.concatenate(([0], np.cumsum(lens))).tolist()
    g = gen(3)
    q, k, v = (torch.randn((starts[-1], n, 64), generator=g, device=DEV).bfloat16() for n in (4, 4, 4))
    good, _ = prompt(q, k, v, starts)
    plant = {}
    for i, a in enumerate(starts[:-1]):
        if i % 3 == 0:
            plant[a + (37 * i) % lens[i], i % 4, i % 64] = INF if i % 2 else NAN
    for (r, h, c), x in plant.items():
        v[r, h, c] = x
    want = with_values_planted(starts, good, v, plant)
    for _ in range(5):
        assert same(prompt(q, k, v, starts)[0], want)


def test_prompt_waits_that_give_up_return_and_leave_nothing_behind():
    """A limit of 0: every wait gives up at once, the call says so and returns; with the old limit the same call is what it
    was, and a recorded one keeps the limit of its recording."""
    starts = [0, 300, 301, 1500]
    g = gen(4)
    q, k, v = (torch.randn((1500, n, 128), generator=g, device=DEV).bfloat16() for n in (4, 2, 2))
    good, good_lse = prompt(q, k, v, starts)
    at, out, st = i32(starts), torch.empty_like(good), status()
    graph = m.MtpDraftHead.capture(lambda s: m.mtp_head_attention_prompt(q, k, v, at, out, status=st, stream=s))
    old = m.mtp_head_set_wait_limit_ns(0)
    try:
        for _ in range(3):
            none = status()
            prompt(q, k, v, starts, none)
            torch.cuda.synchronize()
            assert int(none.item()) == m.ERR_TIMEOUT
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.equal(out, good)
    finally:
        m.mtp_head_set_wait_limit_ns(old)
    again, lse = prompt(q, k, v, starts, st)
    assert int(st.item()) == 0 and torch.equal(again, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("starts,certain", [([0, 300, 301, 1500, 4000], False), ([0, 20000], True)])
def test_prompt_waits_that_run_out_under_way(starts, certain):
    """A limit of 1 ns: waits run out wherever their data is not there within the hardware's own polling time, in the
    middle of pieces too. A call says so, or has the usual results; what was under way lands, and the next call is right.
    In the second case a CTA has eight pieces one after another, the next but one of which waits for a whole piece (tens
    of us): some wait runs out."""
    g = gen(5)
    q, k, v = (torch.randn((starts[-1], n, 64), generator=g, device=DEV).bfloat16() for n in (16, 2, 2))
    good, good_lse = prompt(q, k, v, starts)
    codes = []
    old = m.mtp_head_set_wait_limit_ns(1)
    try:
        for _ in range(20):
            st = status()
            out, lse = prompt(q, k, v, starts, st)
            codes.append(int(st.item()))
            assert codes[-1] in (0, m.ERR_TIMEOUT)
            if codes[-1] == 0:
                assert torch.equal(out, good) and torch.equal(lse, good_lse)
    finally:
        m.mtp_head_set_wait_limit_ns(old)
    assert not certain or m.ERR_TIMEOUT in codes
    st = status()
    out, lse = prompt(q, k, v, starts, st)
    assert int(st.item()) == 0 and torch.equal(out, good) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("scale", [2.0 ** 60, 2.0 ** -100])
def test_scores_of_zero_stay_zero_at_any_scale(scale):
    """Queries of 2^120 in a column where every key is zero: the weights are equal, so the outputs are the values' mean."""
    n, D = 48, 64
    g = gen(6)
    q = torch.zeros((n, 2, D), dtype=BF, device=DEV)
    q[..., 0] = 2.0 ** 120
    k = torch.randn((n, 1, D), generator=g, device=DEV).bfloat16()
    k[..., 0] = 0.0
    v = torch.randint(-8, 9, (n, 1, D), generator=g, device=DEV).bfloat16()
    v[:, :, ::16] = 8.0  # (blocks and rows whose FP4 copies hold these integers' multiples)
    out, lse = torch.empty_like(q), torch.empty((n, 2), device=DEV)
    m.mtp_head_attention_prompt(q, k, v, i32([0, n]), out, lse, scale)
    mean = v[:, 0].double().cumsum(0) / torch.arange(1, n + 1, device=DEV).view(-1, 1)
    # equal weights of 1: the sums are exact, their quotient rounds twice in fp32 and once to BF16
    tol = mean.abs() * (2.0 ** -8 + 2.0 ** -21)
    assert bool(((out.double() - mean.view(n, 1, D)).abs() <= tol.view(n, 1, D)).all())
    cache, table = m.cache_empty(3, 16, 1, D, DEV), i32([[0, 1, 2]])
    m.mtp_head_cache_write_fp4(k, v, i32([0, n]), i32([0]), table, *cache)
    held = [torch.zeros((n, 1, D), dtype=BF, device=DEV) for _ in range(2)]
    m.mtp_head_cache_read_fp4(*cache, i32([0, n]), i32([0]), table, *held)
    assert not bool(held[0][..., 0].any())
    one, ws = torch.empty((1, 1, 2, D), dtype=BF, device=DEV), m.attention_fp4_workspace(1, 1, 2, 1, D, 48, DEV)
    m.mtp_head_attention_fp4(q[-1:].view(1, 1, 2, D), *cache, table, i32([n]), one, ws, scale=scale)
    mean = held[1][:, 0].double().mean(0)
    # the values read back are BF16 (2^-8 of each), the weights carry log2 of row scales near 8 / 2688 (8.4: an error of
    # 3 * 8.4 * 2^-24 in the exponent) and round to f16 (2^-11); the result rounds to BF16
    size = held[1][:, 0].double().abs().mean(0)
    assert bool(((one.double() - mean).abs() <= size * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) + mean.abs() * 2.0 ** -8).all())
    assert bool(((lse.double() - torch.arange(1, n + 1, device=DEV).double().log().view(-1, 1)).abs() <= 2.0 ** -20).all())


# ------------------------------------------------------------------------------------- residual norm
def bf16(a):
    return torch.from_numpy(oracle.f64_to_bf16(a).view(np.int16).copy()).view(BF).to(DEV)


def vals(t):
    return oracle.bf16_to_f64(synth.bits(t))


def norm_is_rounded_once(x, w, eps, delta=None):
    """y, bit for bit, against the formula in 64 bits, whatever its factors' sizes; zeros of either sign are alike."""
    t = vals(x) if delta is None else oracle.bf16_to_f64(oracle.f64_to_bf16(vals(x) + vals(delta)))
    with np.errstate(over="ignore"):
        want = oracle.bf16_to_f64(oracle.f64_to_bf16(t * (vals(w)[None] / np.sqrt((t * t).mean(1, keepdims=True) + eps))))
    y = torch.empty_like(x)
    m.mtp_head_norm_residual(x, w, delta, y=y, eps=eps)
    assert np.array_equal(vals(y), want)


@pytest.mark.parametrize("H", [200, 1003, 2048, 6144, 9000])
@pytest.mark.parametrize("xs,ws", [(2.0 ** 60, 2.0 ** 70), (2.0 ** 30, 2.0 ** 110), (2.0 ** -20, 2.0 ** -115), (2.0 ** -49, 2.0 ** -80),
                                   (2.0 ** 100, 2.0 ** 90), (2.0 ** -100, 2.0 ** 90), (2.0 ** -100, 2.0 ** -60)])
def test_norm_weights_of_any_size(xs, ws, H):
    """x w beyond the fp32 range on either side, where x w / rms is within it."""
    r = np.random.default_rng(H)
    x, w = bf16(r.standard_normal((5, H)) * xs), bf16(r.standard_normal(H) * ws)
    for eps in (0.0, 1e-6):
        norm_is_rounded_once(x, w, eps)


@pytest.mark.parametrize("H", [200, 1003, 4096, 6144, 9000])
@pytest.mark.parametrize("top", [2.0 ** 90, 2.0 ** 40, 1.0, 2.0 ** -45, 2.0 ** -70])
def test_norm_rows_of_elements_far_apart(top, H):
    """Elements down to 2^-133 beside the row's largest, zeros among them, with weights that bring them back."""
    r = np.random.default_rng(H + 1)
    x = r.standard_normal((6, H)) * top * 2.0 ** -r.uniform(0, 160, (6, H))
    x[:, ::5] = 0.0
    x[:, 3] = top
    w = r.standard_normal(H) * 2.0 ** r.uniform(-60, 120, H)
    w[2::7] = 0.0
    norm_is_rounded_once(bf16(x), bf16(w), 0.0)
    norm_is_rounded_once(bf16(x), bf16(w), 1e-6, bf16(r.standard_normal((6, H)) * top * 2.0 ** -r.uniform(0, 160, (6, H))))


# ------------------------------------------------------------------------------------- the layer and its cache
H, HQ, KV, D = 128, 4, 2, 64


def layer_weights(seed=50):
    g = gen(seed)
    r = lambda *s: (torch.randn(s, generator=g, device=DEV) * 0.06).bfloat16()  # noqa: E731
    return 1 + r(H), r((HQ + 2 * KV) * D, H), r(H, HQ * D), HQ, KV


def rows(n, seed):
    return torch.randn((n, H), generator=gen(seed), device=DEV).bfloat16()


def test_layer_buffers_are_filled_before_another_stream_may_use_them(monkeypatch):
    """Zero fills run on the stream of the construction, or of a step's first number of rows. They are over when the call
    returns: nothing orders them before a call on another stream."""
    late = torch.cuda.Stream()
    with torch.cuda.stream(late):
        torch.cuda._sleep(100_000_000)
        cache = m.LayerCache(2, 64, KV, D, page=16, device=DEV)
        assert late.query()
        real = _lib.attention_fp4_workspace

        def slow(*args):
            torch.cuda._sleep(100_000_000)
            return real(*args)

        monkeypatch.setattr(_lib, "attention_fp4_workspace", slow)
        layer = m.DraftLayer(*layer_weights(), cache, max_rows=6)
        assert late.query()
        calls = []
        monkeypatch.setattr(_lib, "mtp_head_norm_residual", lambda *a, **k: calls.append(late.query()))
        layer.step(rows(6, 1), i32([3, 3]))
        assert calls[0]
    torch.cuda.synchronize()


def test_cache_read_fills_its_rows_on_the_stream_that_reads():
    cache = m.LayerCache(1, 64, KV, D, page=16, device=DEV)
    k, v = (torch.randn((20, KV, D), generator=gen(i), device=DEV).bfloat16() for i in (51, 52))
    starts, at = i32([0, 20]), i32([0])
    cache.write(k, v, starts, at)
    good = cache.read(starts, at, 22)
    assert bool(good[0][:20].any()) and not bool(good[0][20:].any())
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # the current stream is busy
    got = cache.read(starts, at, 22, stream=other)
    raw = cache.read(starts, at, 22, stream=other.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *raw), (*good, *good)))


def test_layer_takes_the_streams_that_the_binding_takes():
    """A torch.cuda.Stream, its raw handle, the default stream's handle (0), or none; also through the head's forward."""
    x0, x1 = rows(5, 53), rows(2, 54)
    starts, length = i32([0, 3, 5]), i32([4, 3])
    head_w = synth.make_weights(H, 512, 0, "cpu")
    gw = {k: t.to(DEV) for k, t in head_w.as_dict().items()}
    head = m.MtpDraftHead(gw["embed"], gw["lm_head"], gw["eh_proj"], gw["enorm_w"], gw["hnorm_w"], gw["final_norm_w"], max_batch=2)
    tokens, hidden = (t.to(DEV) for t in synth.make_step_inputs(H, 512, 2, 0, "cpu"))
    layer = m.DraftLayer(*layer_weights(), m.LayerCache(2, 64, KV, D, page=16, device=DEV), max_rows=5)
    other = torch.cuda.Stream()
    seen = []
    for stream in (None, other, other.cuda_stream, 0):
        a, b = x0.clone(), x1.clone()
        torch.cuda.synchronize()
        layer.prompt(a, starts, stream=stream)
        torch.cuda.synchronize()
        layer.step(b, length, stream=stream)
        torch.cuda.synchronize()
        x, _, draft = head.forward(tokens, hidden, stream=stream, layer=lambda x, **kw: layer.step(x, length, **kw))
        torch.cuda.synchronize()
        seen.append((a, b, x, draft))
    for s in seen[1:]:
        assert all(torch.equal(t, u) for t, u in zip(s, seen[0]))


@pytest.mark.parametrize("mlp", [False, True])
def test_layer_keeps_the_errors_of_calls_without_a_status(mlp):
    cache = m.LayerCache(2, 32, KV, D, page=16, device=DEV)
    half = dict(mlp=lambda y, q, s: y, mlp_norm_w=layer_weights()[0]) if mlp else {}
    layer = m.DraftLayer(*layer_weights(), cache, max_rows=80, **half)

    def code():
        c = int(layer.status.item())
        layer.status.zero_()
        return c

    layer.prompt(rows(30, 55), i32([0, 20, 30]))
    layer.step(rows(2, 56), i32([21, 11]))
    assert code() == 0
    layer.step(rows(2, 57), i32([33, 12]))  # a place behind the cache
    assert code() == m.ERR_ARG
    layer.prompt(rows(50, 58), i32([0, 40, 50]))  # more rows than the cache holds
    assert code() == m.ERR_ARG
    bad = rows(2, 59)
    bad[1, 3] = NAN
    layer.step(bad, i32([21, 11]))
    assert code() == m.ERR_NONFINITE
    own = status()
    layer.step(rows(2, 60), i32([33, 12]), own)
    assert int(own.item()) == m.ERR_ARG and code() == 0
    table = cache.table.clone()
    cache.table[1, 0] = 99
    layer.step(rows(2, 61), i32([21, 11]))
    assert code() == m.ERR_ARG
    cache.table.copy_(table)
    layer.step(rows(2, 62), i32([21, 11]))
    assert code() == 0


def test_layer_rotates_at_places_of_the_cache_only():
    """Rows of no sequence, lengths below the step's rows or past the cache: the positions that a rotation may look up in a
    table of max_len rows stay within it, and those of rows that have a place are theirs."""
    cache = m.LayerCache(3, 48, KV, D, page=16, device=DEV)
    seen = []
    layer = m.DraftLayer(*layer_weights(), cache, max_rows=200, rotate=lambda q, k, p: seen.append(p.clone()))
    layer.prompt(rows(200, 63), i32([4, 24, 24, 60]))
    p = seen.pop()
    assert p.dtype == I32 and int(p.min()) >= 0 and int(p.max()) < cache.max_len
    assert torch.equal(p[4:24], torch.arange(20, dtype=I32, device=DEV))
    assert torch.equal(p[24:60], torch.arange(36, dtype=I32, device=DEV))
    layer.prompt(rows(100, 64), i32([0, 100]))
    p = seen.pop()
    assert torch.equal(p, torch.arange(100, dtype=I32, device=DEV).clamp_(max=cache.max_len - 1))
    layer.step(rows(6, 65), i32([0, 21, 60]))
    assert seen.pop().tolist() == [0, 0, 19, 20, 47, 47]
    layer.step(rows(3, 66), i32([1, 48, 22]))
    assert seen.pop().tolist() == [0, 47, 21]
