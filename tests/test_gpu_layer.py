"""The attention half's operators against 64-bit forms of their definitions (layer_helpers)."""
import numpy as np
import pytest
import torch

import fp4_helpers as ref
import layer_helpers as lh
import mtp_speculative_draft_head_gb300 as m
import oracle
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6
BF, I32, F32, F64, U8 = torch.bfloat16, torch.int32, torch.float32, torch.float64, torch.uint8


def bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(oracle.f64_to_bf16(a).view(np.int16).copy()).view(BF).to(DEV)


def vals(t: torch.Tensor) -> np.ndarray:
    return oracle.bf16_to_f64(synth.bits(t))


def status():
    return torch.zeros(1, dtype=I32, device=DEV)


def i32(v):
    return torch.tensor(v, dtype=I32, device=DEV)


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


# ------------------------------------------------------------------------------------- residual norm
def plain_norm(x, delta, w, eps=EPS):
    t = x if delta is None else oracle.bf16_to_f64(oracle.f64_to_bf16(x + delta))
    y = t * w / np.sqrt((t * t).mean(1, keepdims=True) + eps)
    return t, oracle.bf16_to_f64(oracle.f64_to_bf16(y))


def plain_codes(y, group):
    """(E4M3 codes, scales) of BF16 values y, by torch on the host: fp32 quotients, one conversion."""
    R, H = y.shape
    n = group or H
    p = torch.zeros((R, -(-H // n) * n))
    p[:, :H] = torch.from_numpy(y.astype(np.float32))
    p = p.view(R, -1, n)
    s = torch.from_numpy(p.abs().amax(2).numpy() / np.float32(448.0))
    q = torch.where(s.unsqueeze(2) > 0, p / torch.where(s > 0, s, 1.0).unsqueeze(2), torch.tensor(0.0))
    q = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(U8).view(R, -1)[:, :H]
    return q, (s if group else s.view(-1))


def run_norm(x, w, delta, group, eps=EPS, want=("total", "y", "q")):
    R, H = x.shape
    st = status()
    total = torch.full((R, H), 7.0, dtype=BF, device=DEV) if "total" in want else None
    y = torch.full((R, H), 7.0, dtype=BF, device=DEV) if "y" in want else None
    q = torch.full((R, H), 77, dtype=U8, device=DEV) if "q" in want else None
    sc = torch.full((R,) if group == 0 else (R, -(-H // group)), -1.0, device=DEV) if "q" in want else None
    m.mtp_head_norm_residual(x, w, delta, total, y, q, sc, st, group=group, eps=eps)
    return total, y, q, sc, int(st.item())


@pytest.mark.parametrize("with_delta", [False, True])
@pytest.mark.parametrize("R,H", [(1, 1), (3, 7), (2, 8), (5, 127), (9, 129), (4, 136), (16, 6144), (700, 1016), (300, 1024),
                                 (301, 1032), (7, 4093), (200, 2050), (2, 8184), (200, 8184), (3, 8192), (160, 8185), (2, 8200),
                                 (1, 65536), (2, 65535), (1300, 250)])
def test_norm_bits(R, H, with_delta):
    r = np.random.default_rng(R * 131 + H)
    x = bf16(r.standard_normal((R, H)) * 3.0)
    d = bf16(r.standard_normal((R, H)) * 2.0 ** r.integers(-12, 2, (R, H))) if with_delta else None
    w = bf16(1.0 + 0.1 * r.standard_normal(H))
    t_ref, y_ref = plain_norm(vals(x), None if d is None else vals(d), vals(w)[None])
    for group in (0, 128):
        total, y, q, sc, st = run_norm(x, w, d, group)
        assert st == 0
        assert np.array_equal(vals(total), t_ref)
        assert np.array_equal(vals(y), y_ref)
        q_ref, s_ref = plain_codes(y_ref, group)
        assert torch.equal(sc.cpu(), s_ref)
        assert torch.equal(q.cpu() & 127, q_ref & 127)
        assert torch.equal((q.cpu() > 127) & (q_ref != 0), (q_ref > 127) & (q_ref != 0))
    # the row's copy is the library's 8-bit copy of y
    q8, s8, st8 = torch.empty_like(q), torch.empty(R, device=DEV), status()
    m.mtp_head_quantize_fp8(y, q8, s8, st8)
    _, _, q, sc, _ = run_norm(x, w, d, 0)
    assert torch.equal(q, q8) and torch.equal(sc, s8)


@pytest.mark.parametrize("want", [("total",), ("y",), ("q",), ("total", "q"), ("y", "q"), ("total", "y")])
def test_norm_each_output_alone(want):
    g = gen(1)
    x, d = (torch.randn((70, 1000), generator=g, device=DEV).bfloat16() for _ in range(2))
    w = torch.randn(1000, generator=g, device=DEV).bfloat16()
    whole = run_norm(x, w, d, 128)
    some = run_norm(x, w, d, 128, want=want)
    for a, b in zip(some, whole):
        assert a is None or (a == b if isinstance(a, int) else torch.equal(a, b))


@pytest.mark.parametrize("H", [6144, 999])
@pytest.mark.parametrize("place", ["total_x", "total_delta", "y_x", "y_delta", "both"])
def test_norm_in_place(place, H):
    g = gen(2)
    x, d = (torch.randn((33, H), generator=g, device=DEV).bfloat16() for _ in range(2))
    w = torch.randn(H, generator=g, device=DEV).bfloat16()
    t_ref, y_ref, _, _, _ = run_norm(x, w, d, 0)
    x, d = x.clone(), d.clone()
    total, y = torch.empty_like(x), torch.empty_like(x)
    total = {"total_x": x, "total_delta": d, "both": x}.get(place, total)
    y = {"y_x": x, "y_delta": d, "both": d}.get(place, y)
    m.mtp_head_norm_residual(x, w, d, total, y, eps=EPS)
    assert torch.equal(total, t_ref) and torch.equal(y, y_ref)


@pytest.mark.parametrize("H", [256, 1003, 9000])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-22, 1e-12, 1e12, 1e22, 1e35])
def test_norm_rows_of_any_size(size, H):
    """Squares beyond the fp32 range on either side; without eps, so that the small rows are normalised too."""
    r = np.random.default_rng(H)
    x = bf16(r.standard_normal((5, H)) * size)
    w = bf16(1.0 + 0.1 * r.standard_normal(H))
    _, y_ref = plain_norm(vals(x), None, vals(w)[None], eps=0.0)
    _, y, _, _, st = run_norm(x, w, None, 0, eps=0.0)
    assert st == 0 and np.array_equal(vals(y), y_ref)


def test_norm_sums_on_rounding_borders():
    """x + delta half-way between BF16 values, and just beside it by what fp32 cannot hold."""
    x = torch.tensor([1.0, 1.0, 1.0, 1.0, -1.0, 256.0, 256.0, 3.0e38], device=DEV).bfloat16().view(1, -1)
    d = torch.tensor([2.0 ** -8, 2.0 ** -8, -2.0 ** -9, 2.0 ** -30, -2.0 ** -8, 1.0, 2.0 ** -40, 3.0e38], device=DEV).bfloat16().view(1, -1)
    x = torch.cat((x, torch.tensor([[1.0 + 2.0 ** -7, 2.0 ** 60, -(2.0 ** 60)]], device=DEV).bfloat16()), 1)
    d = torch.cat((d, torch.tensor([[2.0 ** -8, 2.0 ** 52, -(2.0 ** 52)]], device=DEV).bfloat16()), 1)
    x, d = x.repeat(3, 1), d.repeat(3, 1)
    with np.errstate(over="ignore"):
        t_ref = oracle.bf16_to_f64(oracle.f64_to_bf16(vals(x) + vals(d)))
    total, *_ = run_norm(x, torch.ones(x.shape[1], dtype=BF, device=DEV), d, 0, want=("total",))
    assert np.array_equal(vals(total), t_ref)


@pytest.mark.parametrize("H", [640, 1003])
def test_norm_nonfinite_rows(H):
    g = gen(3)
    x = torch.randn((6, H), generator=g, device=DEV).bfloat16()
    w = torch.ones(H, dtype=BF, device=DEV)
    clean = run_norm(x, w, None, 128)
    x[1, 200] = float("nan")
    x[3, 300] = float("inf")
    _, y, q, sc, st = run_norm(x, w, None, 128)
    assert st == m.ERR_NONFINITE
    assert bool(y[1].isnan().all()) and int(q[1].max()) == 0 and float(sc[1].abs().max()) == 0.0
    assert bool(y[3, 300].isnan()) and int((y[3] != 0).sum()) == 1  # the mean is infinite: the others are zeros
    assert int(q[3].max()) == 0 and float(sc[3].max()) == 0.0
    for row in (0, 2, 4, 5):
        assert torch.equal(q[row], clean[2][row]) and torch.equal(sc[row], clean[3][row])
    zero = torch.zeros((2, H), dtype=BF, device=DEV)
    _, y, q, sc, st = run_norm(zero, w, None, 0)
    assert st == 0 and not bool(y.any()) and not bool(q.any()) and not bool(sc.any())


# ------------------------------------------------------------------------------------- the cache
def rows_of(T, heads, D, seed, kind="normal", strided=True):
    r = np.random.default_rng(seed)
    a = r.standard_normal((T, 2, heads, D))
    if kind == "wide":
        a *= 10.0 ** r.uniform(-9, 3, a.shape)
    elif kind == "tiny":
        a *= 1e-38
    elif kind == "huge":
        a *= 5e37
    elif kind == "ties":
        a = r.integers(-24, 25, a.shape) * 0.25
        a[..., 0] = 6.0
    t = bf16(a.reshape(T, -1)).view(a.shape)
    if not strided:
        return t[:, 0].contiguous(), t[:, 1].contiguous()
    return t[:, 0], t[:, 1]


def paged(lens, page, seed, extra=3):
    """A table that hands out pages in no order, and the number of pages (some belong to nobody)."""
    need = [-(-n // page) for n in lens]
    perm = torch.randperm(sum(need) + extra, generator=torch.Generator().manual_seed(seed)).to(I32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=I32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table.to(DEV), sum(need) + extra


def garbage_cache(pages, page, heads, D):
    """What a pool may hold behind its sequences: NaN and infinite scales, any codes."""
    q, bs, rs = m.cache_empty(pages, page, heads, D, DEV)
    q.random_(0, 256, generator=gen(9))
    bs.fill_(0x7F)
    rs.fill_(float("nan"))
    rs[..., ::2] = float("inf")
    return q, bs, rs


@pytest.mark.parametrize("D,heads,page", [(64, 1, 16), (64, 3, 64), (128, 8, 64), (128, 5, 16), (128, 2, 256)])
@pytest.mark.parametrize("kind", ["normal", "wide", "tiny", "huge", "ties"])
def test_cache_bits_and_back(kind, D, heads, page):
    counts, before = [5, 0, 1, 37, 16, 100], [0, 9, 15, 250, 16, 3]
    T = sum(counts) + 4  # two rows in front of the sequences and two behind belong to nobody
    starts = np.concatenate(([2], 2 + np.cumsum(counts)))
    k, v = rows_of(T, heads, D, D + heads, kind)
    table, pages = paged([a + b for a, b in zip(counts, before)], page, 1)
    cache = garbage_cache(pages, page, heads, D)
    was = [t.clone() for t in cache]
    st = status()
    m.mtp_head_cache_write_fp4(k, v, i32(starts.tolist()), i32(before), table, *cache, st)
    assert int(st.item()) == 0
    touched = torch.zeros((pages, page), dtype=torch.bool)
    tab = table.cpu()
    for b, n in enumerate(counts):
        for i in range(n):
            pos = before[b] + i
            pg, off, row = int(tab[b, pos // page]), pos % page, int(starts[b]) + i
            touched[pg, off] = True
            for kind_i, src in enumerate((k, v)):
                if (row + kind_i) % 7:  # (sampled rows: the reference is slow)
                    continue
                q_ref, s_ref, r_ref = lh.quantize(vals(src[row].contiguous()))
                assert np.array_equal(cache[0][pg, kind_i, :, off].cpu().numpy(), q_ref)
                assert np.array_equal(cache[1][pg, kind_i, :, off].cpu().numpy(), s_ref)
                assert np.array_equal(cache[2][pg, kind_i, :, off].cpu().numpy().view(np.uint32), r_ref.view(np.uint32))
    for t, w in zip(cache, was):  # what no row goes to stays as it was, bit for bit
        a, b = (x.movedim(3, 1)[~touched.to(DEV)].contiguous().view(U8) for x in (t, w))
        assert torch.equal(a, b)
    out = torch.full((T, 2, heads, D), 7.0, dtype=BF, device=DEV)
    m.mtp_head_cache_read_fp4(*cache, i32(starts.tolist()), i32(before), table, out[:, 0], out[:, 1], st)
    assert int(st.item()) == 0
    for row in (*range(int(starts[0])), *range(int(starts[-1]), T)):
        assert bool((out[row] == 7.0).all())
    b = np.repeat(np.arange(len(counts)), counts)
    rows = torch.arange(int(starts[0]), int(starts[-1]))
    pos = torch.tensor(before)[b] + rows - torch.from_numpy(starts)[b]
    pg, off = tab[b, pos // page].long(), pos % page
    for kind_i in range(2):
        c, s, r = (t.cpu()[pg, kind_i, :, off] for t in cache)
        codes = torch.stack((c & 15, c >> 4), -1).flatten(-2).long()
        f = torch.cat((lh.E2M1, -lh.E2M1)).float()[codes] * torch.from_numpy(ref.E4M3).float()[s.long()].repeat_interleave(16, -1)
        assert torch.equal(out[rows.to(DEV), kind_i].cpu(), (f * r.unsqueeze(-1)).bfloat16())


def test_cache_rows_that_have_no_place():
    k, v = rows_of(8, 2, 64, 1)
    cache = garbage_cache(4, 16, 2, 64)
    was = [t.clone() for t in cache]
    good = i32([[0, 1]])
    # past the table, in front of it, on pages that do not exist; an empty batch of rows writes nothing
    for starts, at, table in (([0, 8], [30], good), ([0, 8], [-3], good), ([0, 8], [12], i32([[4, 5]])), ([0, 8], [12], i32([[0, -1]]))):
        for t, w in zip(cache, was):
            t.copy_(w)
        st = status()
        m.mtp_head_cache_write_fp4(k, v, i32(starts), i32(at), table, *cache, st)
        assert int(st.item()) == m.ERR_ARG
        ko, vo = (torch.full((8, 2, 64), 7.0, dtype=BF, device=DEV) for _ in range(2))
        m.mtp_head_cache_read_fp4(*cache, i32(starts), i32(at), table, ko, vo, st)
        n = sum(0 <= at[0] + i < 32 and 0 <= int(table[0, (at[0] + i) // 16]) < 4 for i in range(8))
        zero = [not bool(ko[i].any()) and not bool(vo[i].any()) for i in range(8)]
        assert sum(zero) == 8 - n
    for t, w in zip(cache, was):
        t.copy_(w)
    for starts in ([0, 0], [8, 8], [9, 20], [5, 2], [-4, -1]):
        st = status()
        m.mtp_head_cache_write_fp4(k, v, i32(starts), i32([0]), good, *cache, st)
        torch.cuda.synchronize()
    assert all(torch.equal(t.view(U8), w.view(U8)) for t, w in zip(cache, was))


def test_cache_nonfinite_rows_become_zeros():
    k, v = rows_of(6, 3, 128, 2, strided=False)
    table, at = i32([[0]]), i32([4])
    clean = m.cache_empty(1, 16, 3, 128, DEV)
    m.mtp_head_cache_write_fp4(k, v, i32([0, 6]), at, table, *clean)
    k[2, 1, 77] = float("nan")
    v[5, 2, 0] = float("-inf")
    cache = garbage_cache(1, 16, 3, 128)
    st = status()
    m.mtp_head_cache_write_fp4(k, v, i32([0, 6]), at, table, *cache, st)
    assert int(st.item()) == m.ERR_NONFINITE
    for kind, row, h in ((0, 2, 1), (1, 5, 2)):
        assert not any(bool(t[0, kind, h, 4 + row].any()) for t in cache)
        for t in clean:
            t[0, kind, h, 4 + row] = 0
    assert all(torch.equal(t[:, :, :, 4:10], w[:, :, :, 4:10]) for t, w in zip(cache, clean))


def test_cache_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes, rows on its first and on its last pages."""
    heads, page, D = 8, 256, 128
    pages = (1 << 32) // (2 * heads * page * D // 2) + 40
    q = torch.empty((pages, 2, heads, page, D // 2), dtype=U8, device=DEV)
    bs = torch.empty((pages, 2, heads, page, D // 16), dtype=U8, device=DEV)
    rs = torch.empty((pages, 2, heads, page), device=DEV)
    assert q.numel() > 1 << 32
    table = i32([[pages - 1, 0], [pages - 20, pages - 30]])
    k, v = rows_of(200, heads, D, 4)
    starts, at = i32([0, 120, 200]), i32([200, 250])
    m.mtp_head_cache_write_fp4(k, v, starts, at, table, q, bs, rs)
    small = (m.cache_empty(4, page, heads, D, DEV))
    t2 = i32([[0, 1], [2, 3]])
    m.mtp_head_cache_write_fp4(k, v, starts, at, t2, *small)
    out = [torch.zeros((200, heads, D), dtype=BF, device=DEV) for _ in range(4)]
    m.mtp_head_cache_read_fp4(q, bs, rs, starts, at, table, *out[:2])
    m.mtp_head_cache_read_fp4(*small, starts, at, t2, *out[2:])
    assert torch.equal(out[0], out[2]) and torch.equal(out[1], out[3]) and bool(out[0].any())
    # and the attention over them
    qr = torch.randn((2, 1, heads, D), generator=gen(1), device=DEV).bfloat16()
    whole = [torch.empty_like(qr) for _ in range(2)]
    for (c, tb, o) in (((q, bs, rs), table, whole[0]), (small, t2, whole[1])):
        for t, pg in ((c, tb),):
            m.mtp_head_cache_write_fp4(*rows_of(512, heads, D, 5), i32([0, 256, 512]), i32([0, 256]), pg, *t)
            m.mtp_head_cache_write_fp4(*rows_of(512, heads, D, 6), i32([0, 256, 512]), i32([256, 0]), pg, *t)
        ws = m.attention_fp4_workspace(2, 1, heads, heads, D, 512, DEV)
        m.mtp_head_attention_fp4(qr, *c, tb, i32([512, 511]), o, ws)
    assert torch.equal(whole[0], whole[1]) and bool(whole[0].any())


# ------------------------------------------------------------------------------------- attention over the cache
def filled(lens, page, heads, D, seed, kind="normal"):
    table, pages = paged(lens, page, seed)
    cache = garbage_cache(pages, page, heads, D)
    T = sum(lens)
    if T:
        k, v = rows_of(T, heads, D, seed, kind)
        starts = np.concatenate(([0], np.cumsum(lens)))
        st = status()
        m.mtp_head_cache_write_fp4(k, v, i32(starts.tolist()), i32([0] * len(lens)), table, *cache, st)
        assert int(st.item()) == 0
    return cache, table


def check_attention(cache, table, lens, q, rows, out, lse, scale, untouched=7.0):
    B, Q, hq, D = q.shape
    page, kv = cache[0].shape[3], cache[0].shape[2]
    G = hq // kv
    for b in range(B):
        n = Q if rows is None else rows[b]
        held = [t[table[b, :-(-lens[b] // page)].long()] for t in cache]
        kvals = lh.values(*held).permute(1, 2, 0, 3, 4).reshape(2, kv, -1, D)[:, :, :lens[b]]
        r = held[2][:, 1].permute(1, 0, 2).reshape(kv, -1)[:, :lens[b]]  # the values' row scales
        log_scale = float(torch.log2(r[r > 0].double()).abs().max()) if bool((r > 0).any()) else 0.0
        for h in range(kv):
            x = q[b, :n, h * G:(h + 1) * G].double().reshape(-1, D)
            limits = (lens[b] - n + 1 + torch.arange(n, device=DEV)).repeat_interleave(G)
            o, z, A, E, P = lh.attention(x, kvals[0, h], kvals[1, h], limits, scale)
            got = out[b, :n, h * G:(h + 1) * G].double().reshape(-1, D)
            err = (got - o).abs()
            tol = lh.bound_out(o, A, E, P, D, max(lens[b], 1), 2.0 ** -11, log_scale)
            assert bool((err <= tol).all()), (b, h, float((err / tol).max()))
            gz = lse[b, :n, h * G:(h + 1) * G].double().reshape(-1)
            none = limits <= 0
            assert bool((gz[none] == float("-inf")).all()) and not bool(got[none].any())
            ez = (gz - z)[~none].abs()
            tz = lh.bound_lse(z, E, D, lens[b])[~none]
            assert bool((ez <= tz).all()), (b, h, float((ez / tz).max()))
        assert bool((out[b, n:] == untouched).all()) and bool((lse[b, n:] == untouched).all())


def attend(cache, table, lens, q, rows=None, scale=None, ws=None):
    B, Q, hq, D = q.shape
    out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
    lse = torch.full((B, Q, hq), 7.0, device=DEV)
    st = status()
    if ws is None:
        ws = m.attention_fp4_workspace(B, Q, hq, cache[0].shape[2], D, table.shape[1] * cache[0].shape[3], DEV)
    m.mtp_head_attention_fp4(q, *cache, table, i32(lens), out, ws, rows=None if rows is None else i32(rows), lse=lse,
                             scale=scale, status=st)
    return out, lse, int(st.item())


def queries(B, Q, hq, D, seed, size=1.0):
    return (torch.randn((B, Q, hq, D), generator=gen(seed), device=DEV) * size).bfloat16()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,G,Q,page", [(1, 1, 1, 16), (2, 6, 1, 64), (3, 1, 2, 32), (1, 16, 1, 256), (2, 5, 5, 64), (2, 17, 1, 16),
                                         (1, 8, 9, 128)])
def test_attention_over_lengths(D, kv, G, Q, page):
    """Lengths on both sides of a step, a round, a page and a range, shorter than the rows, and nothing at all."""
    lens = [0, 1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1100]
    cache, table = filled(lens, page, kv, D, D + kv + G)
    q = queries(len(lens), Q, kv * G, D, 3, 2.0)
    out, lse, st = attend(cache, table, lens, q)
    assert st == 0
    check_attention(cache, table, lens, q, None, out, lse, D ** -0.5)


def test_attention_rows_of_each_sequence():
    lens, rows = [40, 40, 40, 3, 3, 0, 900, 7], [0, 1, 4, 4, 2, 3, 3, 4]
    cache, table = filled(lens, 32, 2, 128, 5)
    q = queries(len(lens), 4, 12, 128, 6)
    out, lse, st = attend(cache, table, lens, q, rows, scale=0.3)
    assert st == 0
    check_attention(cache, table, lens, q, rows, out, lse, 0.3)


@pytest.mark.parametrize("B,Q,kv,G,D,lens", [(1, 1, 8, 6, 128, [20011]), (2, 5, 2, 8, 128, [9001, 130]), (1, 2, 1, 1, 64, [33000]),
                                             (40, 1, 8, 4, 64, None)])
def test_attention_long_and_many(B, Q, kv, G, D, lens):
    lens = lens or [(977 * i) % 700 for i in range(B)]
    cache, table = filled(lens, 64, kv, D, 8)
    q = queries(B, Q, kv * G, D, 9, 1.5)
    out, lse, st = attend(cache, table, lens, q)
    assert st == 0
    check_attention(cache, table, lens, q, None, out, lse, D ** -0.5)
    again = attend(cache, table, lens, q)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("B,Q,kv,G,D,top", [(100, 1, 8, 2, 64, 700), (70, 3, 4, 4, 128, 900), (3, 1, 1, 1, 128, 100000),
                                            (33, 1, 2, 1, 64, 300), (1500, 1, 1, 1, 64, 260), (200, 1, 8, 1, 64, 4200)])
@pytest.mark.parametrize("some", [False, True])
def test_attention_work_shared_out(B, Q, kv, G, D, top, some):
    """Work that the CTAs share out in pieces that end inside sequences, over several of them, or (few long ones) in as many
    pieces as are joined at once, and work of so many sequences that each has its own; sequences without rows in front, behind
    and in runs longer than a warp."""
    lens = [(top * (i % 7 + 1)) // 7 - i % 5 for i in range(B)]
    rows = [0 if i < B // 2 or i % 4 == 1 else i % (Q + 1) for i in range(B)] if some else None
    cache, table = filled(lens, 64, kv, D, 31)
    q = queries(B, Q, kv * G, D, 32, 1.5)
    ws = m.attention_fp4_workspace(B, Q, kv * G, kv, D, table.shape[1] * 64, DEV)
    first = attend(cache, table, lens, q, rows, ws=ws)
    assert first[2] == 0
    check_attention(cache, table, lens, q, rows, first[0], first[1], D ** -0.5)
    again = attend(cache, table, lens, q, rows, ws=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_nothing_to_do():
    cache, table = filled([20] * 40, 16, 2, 64, 33)
    q = queries(40, 2, 4, 64, 34)
    out, lse, st = attend(cache, table, [20] * 40, q, [0] * 40)
    assert st == 0 and bool((out == 7.0).all()) and bool((lse == 7.0).all())
    out, lse, st = attend(cache, table, [0] * 40, q)
    assert st == 0 and not bool(out.any()) and bool((lse == float("-inf")).all())


@pytest.mark.parametrize("kind", ["wide", "tiny", "huge", "ties"])
def test_attention_values_of_any_size(kind):
    """Rows whose sizes differ by many orders of magnitude from token to token, queries to match (scores of order one)."""
    lens = [300, 77, 1]
    cache, table = filled(lens, 16, 2, 128, 11, kind)
    size = {"wide": 1e-2, "tiny": 1e36, "huge": 1e-37, "ties": 0.1}[kind]
    q = queries(3, 2, 8, 128, 12, size)
    q[0, 0, 1] = 0.0
    out, lse, st = attend(cache, table, lens, q)
    assert st == 0
    check_attention(cache, table, lens, q, None, out, lse, 128 ** -0.5)


def test_attention_values_far_apart_in_size():
    """Tokens with large weights and small values next to tokens with small weights and large values: neither may be
    lost. Keys: one column decides the score; values: a constant per token."""
    n, D = 160, 64
    k = torch.zeros((n, 1, D), dtype=BF, device=DEV)
    v = torch.zeros((n, 1, D), dtype=BF, device=DEV)
    i = torch.arange(n, device=DEV)
    k[:, 0, 0] = (24.0 - 48.0 * (i % 2)).bfloat16()               # scores +24 and -24
    v[:, 0] = torch.where(i % 2 == 0, 1e-18, 1e3).view(-1, 1).expand(n, D).bfloat16() * (1 + (i % 3)).view(-1, 1)
    cache = m.cache_empty(10, 16, 1, D, DEV)
    table = torch.arange(10, dtype=I32, device=DEV).view(1, -1)
    m.mtp_head_cache_write_fp4(k, v, i32([0, n]), i32([0]), table, *cache)
    q = torch.zeros((1, 1, 1, D), dtype=BF, device=DEV)
    q[..., 0] = 1.0
    out, lse, st = attend(cache, table, [n], q, scale=1.0)
    assert st == 0
    check_attention(cache, table, [n], q, None, out, lse, 1.0)


def test_attention_errors_in_device_data():
    lens = [50, 60, 70]
    cache, table = filled(lens, 16, 1, 64, 13)
    q = queries(3, 2, 2, 64, 14)
    good, good_lse, _ = attend(cache, table, lens, q)
    cap = table.shape[1] * 16
    for bad_len, rows in ((cap + 1, None), (-1, None), (60, [2, 3, 2]), (60, [2, -1, 2])):
        out, lse, st = attend(cache, table, [50, bad_len, 70], q, rows)
        assert st == m.ERR_ARG
        assert not bool(out[1].any()) and bool((lse[1] == float("-inf")).all())
        assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.equal(lse[[0, 2]], good_lse[[0, 2]])
    for page in (-1, cache[0].shape[0]):
        t = table.clone()
        t[1, 1] = page
        out, lse, st = attend(cache, t, lens, q)
        assert st == m.ERR_ARG and torch.equal(out[[0, 2]], good[[0, 2]]) and bool(torch.isfinite(out[1]).all())


def test_attention_nonfinite_queries_stay_in_their_rows():
    lens = [200]
    cache, table = filled(lens, 16, 1, 128, 15)
    q = queries(1, 3, 4, 128, 16)
    good, good_lse, _ = attend(cache, table, lens, q)
    q[0, 1, 2, 5] = float("nan")
    q[0, 2, 0, 0] = float("inf")
    out, lse, _ = attend(cache, table, lens, q)
    bad = torch.zeros((1, 3, 4), dtype=torch.bool, device=DEV)
    bad[0, 1, 2] = bad[0, 2, 0] = True
    assert torch.equal(out[~bad], good[~bad]) and torch.equal(lse[~bad], good_lse[~bad])
    assert bool(out[bad].isnan().all())


def test_attention_strided_rows_one_workspace_and_a_graph():
    """Queries and outputs inside wider rows; one workspace for calls of several sizes, one after another; a recorded
    call replayed on new lengths and rows."""
    lens, kv, G, D = [700, 90], 2, 3, 64
    cache, table = filled([800, 800], 32, kv, D, 17)
    wide = torch.randn((2, 4, 10, D), generator=gen(18), device=DEV).bfloat16()
    q = wide[:, :, 2:8]
    res = torch.full((2, 4, 9, D), 7.0, dtype=BF, device=DEV)
    ws = m.attention_fp4_workspace(2, 4, kv * G, kv, D, 800, DEV)
    length = i32(lens)
    m.mtp_head_attention_fp4(q, *cache, table, length, res[:, :, 1:7], ws)
    plain, _, _ = attend(cache, table, lens, q.contiguous())
    assert torch.equal(res[:, :, 1:7], plain)
    assert bool((res[:, :, 0] == 7.0).all()) and bool((res[:, :, 7:] == 7.0).all())
    for Q in (1, 4, 2):
        for b in (1, 2):
            x = q[:b, :Q].contiguous()
            a, _, _ = attend(cache, table[:b].contiguous(), lens[:b], x, ws=ws)
            c, _, _ = attend(cache, table[:b].contiguous(), lens[:b], x)
            assert torch.equal(a, c)
    rows = i32([4, 4])
    out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
    g = m.MtpDraftHead.capture(lambda s: m.mtp_head_attention_fp4(q, *cache, table, length, out, ws, rows=rows, stream=s))
    for new, r in (([700, 90], [4, 4]), ([5, 800], [4, 1]), ([0, 333], [2, 4])):
        length.copy_(i32(new))
        rows.copy_(i32(r))
        out.fill_(7.0)
        g.replay()
        c, _, _ = attend(cache, table, new, q.contiguous(), r)
        assert torch.equal(out, c)
    assert not bool(ws[:256].any())  # the counters are back at zero


def test_attention_calls_side_by_side():
    """Calls on two streams at once, each with its own workspace, and two recorded ones beside them."""
    sets = []
    for i, lens in enumerate(([3000, 1500], [800, 4000])):
        cache, table = filled(lens, 64, 2, 128, 20 + i)
        q = queries(2, 2, 8, 128, 30 + i)
        sets.append((cache, table, lens, q, attend(cache, table, lens, q)[0]))
    outs = [torch.empty_like(s[3]) for s in sets]
    wss = [m.attention_fp4_workspace(2, 2, 8, 2, 128, s[1].shape[1] * 64, DEV) for s in sets]
    lens = [i32(s[2]) for s in sets]
    recorded = [m.MtpDraftHead.capture(lambda st, i=i: m.mtp_head_attention_fp4(sets[i][3], *sets[i][0], sets[i][1], lens[i],
                                                                                outs[i], wss[i], stream=st)) for i in (0, 1)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for use_graph in (False, True):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    if use_graph:
                        recorded[i].replay()
                    else:
                        m.mtp_head_attention_fp4(sets[i][3], *sets[i][0], sets[i][1], lens[i], outs[i], wss[i])
        torch.cuda.synchronize()
        assert all(torch.equal(o, s[4]) for o, s in zip(outs, sets))


# ------------------------------------------------------------------------------------- prompts
def prompt_inputs(T, hq, kv, D, seed, size=1.0, strided=True):
    qkv = torch.randn((T, hq + 2 * kv, D), generator=gen(seed), device=DEV)
    qkv[:, :hq] *= size
    parts = qkv.bfloat16().split([hq, kv, kv], 1)
    return parts if strided else tuple(p.contiguous() for p in parts)


def prompt(q, k, v, starts, scale=None):
    T, hq, D = q.shape
    out = torch.full((T, hq, D), 7.0, dtype=BF, device=DEV)
    lse = torch.full((T, hq), 7.0, device=DEV)
    st = status()
    m.mtp_head_attention_prompt(q, k, v, i32(starts), out, lse, scale, st)
    return out, lse, int(st.item())


def check_prompt(q, k, v, starts, out, lse, scale, heads=None):
    hq, kv, D = q.shape[1], k.shape[1], q.shape[2]
    for a, b in zip(starts[:-1], starts[1:]):
        if b <= a:
            continue
        for h in heads or range(hq):
            kk, vv = k[a:b, h * kv // hq].double(), v[a:b, h * kv // hq].double()
            for i in range(a, b, 2048):
                j = min(b, i + 2048)
                limits = torch.arange(i - a + 1, j - a + 1, device=DEV)
                o, z, A, E, P = lh.attention(q[i:j, h].double(), kk[:j - a], vv[:j - a], limits, scale)
                tol = lh.bound_out(o, A, E, P, D, j - a, 2.0 ** -8)
                err = (out[i:j, h].double() - o).abs()
                assert bool((err <= tol).all()), (a, b, h, float((err / tol).max()))
                tz = lh.bound_lse(z, E, D, j - a)
                ez = (lse[i:j, h].double() - z).abs()
                assert bool((ez <= tz).all()), (a, b, h, float((ez / tz).max()))
    inside = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    for a, b in zip(starts[:-1], starts[1:]):
        inside[a:b] = True
    assert bool((out[~inside] == 7.0).all()) and bool((lse[~inside] == 7.0).all())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,kv", [(1, 1), (6, 2), (5, 5), (8, 1)])
def test_prompt_lengths(D, hq, kv):
    lens = [1, 2, 0, 15, 64, 127, 128, 129, 200, 255, 256, 257, 1, 384, 600, 0]
    starts = np.concatenate(([3], 3 + np.cumsum(lens))).tolist()
    T = starts[-1] + 5
    q, k, v = prompt_inputs(T, hq, kv, D, D + hq, 2.0)
    out, lse, st = prompt(q, k, v, starts)
    assert st == 0
    check_prompt(q, k, v, starts, out, lse, D ** -0.5)


@pytest.mark.parametrize("D,hq,kv,starts", [(128, 2, 1, [0, 5003]), (64, 4, 2, [0, 1, 4100]), (128, 12, 2, [0, 700, 701, 2000, 2300])])
def test_prompt_long(D, hq, kv, starts):
    q, k, v = prompt_inputs(starts[-1], hq, kv, D, 5, strided=False)
    out, lse, st = prompt(q, k, v, starts, 0.2)
    assert st == 0
    check_prompt(q, k, v, starts, out, lse, 0.2)
    again = prompt(q, k, v, starts, 0.2)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_prompt_many_sequences():
    """More sequences than a warp looks at once, most of them short."""
    lens = [(13 * i) % 40 for i in range(150)] + [500]
    starts = np.concatenate(([0], np.cumsum(lens))).tolist()
    q, k, v = prompt_inputs(starts[-1], 2, 1, 64, 6)
    out, lse, st = prompt(q, k, v, starts)
    assert st == 0
    check_prompt(q, k, v, starts, out, lse, 0.125)


@pytest.mark.parametrize("size", [1e-3, 30.0, 300.0])
def test_prompt_scores_of_any_size(size):
    """Flat rows, peaked rows, and rows whose maximum keeps rising (keys that grow along the sequence)."""
    q, k, v = (t.clone() for t in prompt_inputs(700, 2, 1, 128, 7, size))
    k[:, 0, 3] = torch.linspace(-8.0, 8.0, 700, device=DEV).bfloat16()
    q[:, :, 3] = (q[:, :, 3].abs() + 1.0).bfloat16()
    out, lse, st = prompt(q, k, v, [0, 700])
    assert st == 0
    check_prompt(q, k, v, [0, 700], out, lse, 128 ** -0.5)


def test_prompt_values_that_are_not_seen_do_not_matter():
    """Infinities and NaN in keys and values of other sequences, of rows outside every sequence, and behind a row in its
    own sequence: rows that do not see them are what they were, rows that do carry them."""
    starts = [2, 130, 133, 420]
    q, k, v = (t.clone() for t in prompt_inputs(430, 4, 2, 64, 8))
    good, good_lse, _ = prompt(q, k, v, starts)
    bad = torch.tensor([0, 1, 421, 429], device=DEV)
    for t in (q, k, v):
        t[bad] = float("nan")
    out, lse, st = prompt(q, k, v, starts)
    assert st == 0 and torch.equal(out, good) and torch.equal(lse, good_lse)
    # within a sequence: value row 300 (head 0) has an infinity in column 5 and a NaN in column 9, key row 350 a NaN
    v[300, 0, 5], v[300, 0, 9], k[350, 1, 0] = float("inf"), float("nan"), float("nan")
    v[132, 1, 1] = float("-inf")
    out, lse, _ = prompt(q, k, v, starts)
    seen = torch.zeros((430, 4, 64), dtype=torch.bool, device=DEV)
    seen[300:420, 0:2, 5] = seen[300:420, 0:2, 9] = seen[350:420, 2:4] = seen[132, 2:4, 1] = True
    assert torch.equal(out[~seen], good[~seen])
    assert bool((out[300:389, 0:2, 5] == float("inf")).all()) and bool(out[300:420, 0:2, 9].isnan().all())
    assert bool((out[132, 2:4, 1] == float("-inf")).all())
    assert not bool(torch.isfinite(out[350:420, 2:4]).any())


def test_prompt_sequences_that_do_not_fit():
    q, k, v = prompt_inputs(300, 2, 1, 64, 9)
    good, _, _ = prompt(q, k, v, [0, 100, 300])
    for starts in ([0, 100, 301], [0, 100, 50], [-1, 100, 100]):
        out, _, st = prompt(q, k, v, starts)
        assert st == m.ERR_ARG
        if starts[0] == 0:
            assert torch.equal(out[:100], good[:100])


def test_prompt_graph_streams_and_strides():
    starts = i32([0, 50, 333, 333])
    wide = torch.randn((333, 9, 128), generator=gen(10), device=DEV).bfloat16()
    q, k, v = wide[:, 0:4], wide[:, 5:7], wide[:, 7:9]
    plain, _, _ = prompt(q.contiguous(), k.contiguous(), v.contiguous(), [0, 50, 333, 333])
    res = torch.full((333, 6, 128), 7.0, dtype=BF, device=DEV)
    m.mtp_head_attention_prompt(q, k, v, starts, res[:, 1:5])
    assert torch.equal(res[:, 1:5], plain) and bool((res[:, 0] == 7.0).all()) and bool((res[:, 5] == 7.0).all())
    outs = [torch.zeros((333, 4, 128), dtype=BF, device=DEV) for _ in range(2)]
    graphs = [m.MtpDraftHead.capture(lambda s, o=o: m.mtp_head_attention_prompt(q, k, v, starts, o, stream=s)) for o in outs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, plain) for o in outs)
    starts.copy_(i32([0, 10, 20, 333]))  # a recorded call on other sequences
    graphs[0].replay()
    other, _, _ = prompt(q, k, v, [0, 10, 20, 333])
    assert torch.equal(outs[0], other)


# ------------------------------------------------------------------------------------- the layer
def plain_linear(x, w):
    """x times FP4 copies of both operands, 64 bits, rounded to BF16 once (layouts: fp4_helpers)."""
    def copy(a):
        codes, sc, rs = ref.quantize(vals(a))
        return ref.values(ref.pack(codes), sc, rs, a.shape[1])
    return oracle.bf16_to_f64(oracle.f64_to_bf16(copy(x) @ copy(w).T))


@pytest.mark.parametrize("mlp", [False, True])
def test_layer_prompt_then_steps(mlp):
    """Prompts through the layer, then steps of one and of three rows: each step's rows against the same arithmetic done
    call by call (norm, projections, rotation, cache, attention), and the cache's contents read back."""
    H, hq, kv, D, B = 256, 4, 2, 64, 3
    g = gen(40)
    r = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    norm_w, mlp_w = (1 + 0.1 * r(H)).bfloat16(), (1 + 0.1 * r(H)).bfloat16()
    qkv_w, o_w = (r((hq + 2 * kv) * D, H) * 0.06).bfloat16(), (r(H, hq * D) * 0.06).bfloat16()

    def rotate(q, k, positions):  # pairs of columns turned by the position
        a = positions.double().view(-1, 1, 1) / 10.0 ** (4.0 * torch.arange(D // 2, device=DEV) / (D // 2))
        for t in (q, k):
            x, y = t[..., :D // 2].double(), t[..., D // 2:].double()
            t.copy_(torch.cat((x * a.cos() - y * a.sin(), x * a.sin() + y * a.cos()), 2))

    seen = []

    def second_half(y, q8, scale):
        seen.append((y.clone(), q8.clone(), scale.clone()))
        return (y.float() * 0.5).bfloat16()

    cache = m.LayerCache(B, 300, kv, D, page=16, device=DEV)
    layer = m.DraftLayer(norm_w, qkv_w, o_w, hq, kv, cache, eps=EPS, max_rows=300, rotate=rotate,
                         mlp=second_half if mlp else None, mlp_norm_w=mlp_w if mlp else None)

    def project(x):
        y = torch.empty_like(x)
        m.mtp_head_norm_residual(x, norm_w, y=y, eps=EPS)
        _, y_ref = plain_norm(vals(x), None, vals(norm_w)[None])
        assert np.array_equal(vals(y), y_ref)
        out = torch.empty((x.shape[0], hq + 2 * kv, D), dtype=BF, device=DEV)
        m.mtp_head_linear_fp4(y, *layer.qkv_fp4, out.view(x.shape[0], -1), layer.ws_qkv)
        want = plain_linear(y, qkv_w)
        assert np.abs(vals(out.view(x.shape[0], -1)) - want).max() <= 2.0 ** -7 * np.abs(want).max()
        return out.split([hq, kv, kv], 1)

    def finish(x, heads):
        delta = torch.empty_like(x)
        m.mtp_head_linear_fp4(heads.reshape(x.shape[0], -1), *layer.o_fp4, delta, layer.ws_o)
        total = bf16(vals(x) + vals(delta))
        if mlp:
            _, y = plain_norm(vals(total), None, vals(mlp_w)[None])
            q8, sc = plain_codes(y, 128)
            got = seen.pop()
            assert np.array_equal(vals(got[0]), y) and torch.equal(got[2].cpu(), sc)
            assert torch.equal(got[1].cpu() & 127, q8 & 127)
            total = bf16(vals(total) + vals((got[0].float() * 0.5).bfloat16()))
        return total

    lens = [40, 1, 129]
    starts = [0, 40, 41, 170]
    x = r(170, H).bfloat16()
    st = status()
    after = layer.prompt(x.clone(), i32(starts), status=st)
    q, k, v = project(x)
    rotate(q, k, torch.cat([torch.arange(n, dtype=I32, device=DEV) for n in lens]))
    heads, lse, _ = prompt(q, k, v, starts)
    check_prompt(q, k, v, starts, heads, lse, D ** -0.5)
    assert torch.equal(after, finish(x, heads)) and int(st.item()) == 0
    kk, vv = cache.read(i32(starts), i32([0] * B), 170)
    for t, src in ((kk, k), (vv, v)):
        c = lh.quantize(vals(src.reshape(-1, D)))
        assert np.array_equal(vals(t.view(-1, D)), vals(lh.values(*(torch.from_numpy(a.copy()) for a in c)).float().bfloat16()))
    for Q in (1, 3):
        lens = [n + Q for n in lens]
        x = r(B * Q, H).bfloat16()
        length = i32(lens)
        after = layer.step(x.clone(), length, status=st)
        q, k, v = project(x)
        pos = torch.cat([torch.arange(n - Q, n, dtype=I32, device=DEV) for n in lens])
        rotate(q, k, pos)
        kk, _ = cache.read(i32(list(range(0, B * Q + 1, Q))), i32([n - Q for n in lens]), B * Q)
        c = lh.quantize(vals(k.reshape(-1, D)))
        assert np.array_equal(vals(kk.view(-1, D)), vals(lh.values(*(torch.from_numpy(a.copy()) for a in c)).float().bfloat16()))
        qq = q.unflatten(0, (B, Q)).contiguous()
        heads, lse, _ = attend(cache.arrays, cache.table, lens, qq)
        check_attention(cache.arrays, cache.table, lens, qq, None, heads, lse, D ** -0.5)
        assert torch.equal(after, finish(x, heads)) and int(st.item()) == 0


def test_head_with_a_layer():
    """A draft step with the layer between the stages: the stages' own results around it, greedy and FP4; and the layer's
    step inside a recorded graph."""
    H, V, hq, kv, D, B = 256, 4096, 4, 2, 64, 2
    w = synth.make_weights(H, V, 0, "cpu")
    gw = {k: t.to(DEV) for k, t in w.as_dict().items()}
    head = m.MtpDraftHead(gw["embed"], gw["lm_head"], gw["eh_proj"], gw["enorm_w"], gw["hnorm_w"], gw["final_norm_w"], max_batch=B)
    head.quantize_fp4()
    tokens, hidden = synth.make_step_inputs(H, V, B, 0, "cpu")
    tokens, hidden = tokens.to(DEV), hidden.to(DEV)
    g = gen(41)
    r = lambda *s: (torch.randn(s, generator=g, device=DEV) * 0.06).bfloat16()  # noqa: E731
    cache = m.LayerCache(B, 64, kv, D, page=16, device=DEV)
    layer = m.DraftLayer(1 + r(H), r((hq + 2 * kv) * D, H), r(H, hq * D), hq, kv, cache, max_rows=B)
    for fp4 in (False, True):
        length = i32([1, 1])
        call = lambda x, status=None, stream=None: layer.step(x, length, status, stream)  # noqa: E731
        x, logits, draft = head.forward(tokens, hidden, logits=True, fp4=fp4, layer=call)
        x0 = head.input(tokens, hidden, fp4=fp4)
        x1 = layer.step(x0.clone(), length)
        lg, d = head.logits_argmax(x1, fp4=fp4)
        assert torch.equal(x, x1) and torch.equal(logits, lg) and torch.equal(draft, d)
        assert not torch.equal(x, x0)
        y = torch.empty_like(x0)
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            y.copy_(x0)
            layer.step(y, length)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, x1)


def test_layer_made_for_prompts_steps_too(monkeypatch):
    """A layer made for the rows of long prompts takes steps of one and of three rows as one made for just those does; a
    step whose workspace is not there yet is not recorded into a graph."""
    H, hq, kv, D, B = 128, 4, 2, 64, 2
    g = gen(42)
    r = lambda *s: (torch.randn(s, generator=g, device=DEV) * 0.06).bfloat16()  # noqa: E731
    w = (1 + r(H), r((hq + 2 * kv) * D, H), r(H, hq * D), hq, kv)
    layers = [m.DraftLayer(*w, m.LayerCache(B, 64, kv, D, page=16, device=DEV), max_rows=n) for n in (2000, B * 3)]
    n = 0
    for Q in (1, 3, 1):
        n += Q
        x = r(B * Q, H)
        a, b = (layer.step(x.clone(), i32([n, n])) for layer in layers)
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        layers[1].step(r(8, H), i32([n, n]))
    with pytest.raises(ValueError):
        layers[0].step(r(4, H), i32([]))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError):
        layers[0].step(r(B * 2, H), i32([n + 2, n + 2]))
    layers[0].step(r(B * 3, H), i32([n + 3, n + 3]))
