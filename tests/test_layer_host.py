"""The attention half's entry points without a GPU: sizes, the documented status codes (every call below fails
validation before anything is launched; the addresses are never dereferenced) and the binding's refusals."""
import ctypes

import pytest
import torch

import mtp_speculative_draft_head_gb300 as m

A = 0x10000  # an aligned fake device address
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def lib():
    return m.load()


def spread(names, step=0x100000000):
    return {k: A + step * (i + 1) for i, k in enumerate(names)}


NORM = ("x", "delta", "w", "total", "y", "q", "scale", "status")


def norm(lib, a):
    return lib.mtp_head_norm_residual(*(a[k] for k in NORM), a["R"], a["H"], a["group"], ctypes.c_float(a["eps"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), m.ERR_ARG), (dict(w=None), m.ERR_ARG), (dict(total=None, y=None, q=None), m.ERR_ARG),
    (dict(scale=None), m.ERR_ARG), (dict(status=None), m.ERR_ARG), (dict(eps=-1.0), m.ERR_ARG),
    (dict(eps=float("nan")), m.ERR_ARG), (dict(group=64), m.ERR_ARG), (dict(group=-1), m.ERR_ARG), (dict(R=0), m.ERR_SHAPE),
    (dict(R=65537), m.ERR_SHAPE), (dict(H=0), m.ERR_SHAPE), (dict(H=65537), m.ERR_SHAPE), (dict(x=A + 2), m.ERR_ALIGN),
    (dict(delta=A + 8), m.ERR_ALIGN), (dict(w=A + 4), m.ERR_ALIGN), (dict(total=A + 2), m.ERR_ALIGN),
    (dict(y=A + 8), m.ERR_ALIGN), (dict(q=A + 8), m.ERR_ALIGN), (dict(scale=A + 2), m.ERR_ALIGN),
    (dict(status=A + 1), m.ERR_ALIGN)])
def test_norm_validation(lib, kw, code):
    a = dict(spread(NORM), R=3, H=200, group=128, eps=1e-6)
    a.update(kw)
    assert norm(lib, a) == code


def test_norm_outputs_on_what_is_still_read_are_refused(lib):
    R, H = 3, 200
    size = dict(x=R * H * 2, delta=R * H * 2, w=H * 2, total=R * H * 2, y=R * H * 2, q=R * H, scale=R * 2 * 4, status=4)
    base = dict(spread(NORM), R=R, H=H, group=128, eps=1e-6)
    outs = ("total", "y", "q", "scale", "status")
    for o in outs:
        for other in (*outs, "w", "x", "delta"):
            if other == o:
                continue
            in_place = o in ("total", "y") and other in ("x", "delta")
            for at in (base[other], base[other] + (size[other] - 1) // 16 * 16, base[other] - (size[o] - 1) // 16 * 16):
                if not (in_place and at == base[other]):
                    assert norm(lib, dict(base, **{o: at})) == m.ERR_ARG, (o, other)


CACHE = ("k", "v", "starts", "at", "table", "q", "bs", "rs", "status")


def cache_call(lib, a, read):
    ints = (a["T"], a["B"], a["heads"], a["D"], a["pages"], a["page"], a["mp"], None)
    if read:
        return lib.mtp_head_cache_read_fp4(a["q"], a["bs"], a["rs"], a["starts"], a["at"], a["table"], a["k"], a["ldk"], a["v"],
                                           a["ldv"], a["status"], *ints)
    return lib.mtp_head_cache_write_fp4(a["k"], a["ldk"], a["v"], a["ldv"], a["starts"], a["at"], a["table"], a["q"], a["bs"],
                                        a["rs"], a["status"], *ints)


CACHE_SIZES = dict(T=5, B=2, heads=3, D=64, pages=7, page=16, mp=4, ldk=192, ldv=200)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("kw,code", [
    *[({k: None}, m.ERR_ARG) for k in CACHE if k != "status"],
    (dict(T=0), m.ERR_SHAPE), (dict(T=(1 << 22) + 1), m.ERR_SHAPE), (dict(B=0), m.ERR_SHAPE), (dict(B=65537), m.ERR_SHAPE),
    (dict(heads=0), m.ERR_SHAPE), (dict(heads=1025), m.ERR_SHAPE), (dict(pages=0), m.ERR_SHAPE), (dict(page=24), m.ERR_SHAPE),
    (dict(page=8), m.ERR_SHAPE), (dict(page=512), m.ERR_SHAPE), (dict(mp=0), m.ERR_SHAPE), (dict(mp=1 << 27), m.ERR_SHAPE),
    (dict(D=0), m.ERR_SHAPE), (dict(D=96), m.ERR_NOT_IMPLEMENTED), (dict(D=256), m.ERR_NOT_IMPLEMENTED),
    (dict(ldk=191), m.ERR_SHAPE), (dict(ldv=100), m.ERR_SHAPE), (dict(ldk=196), m.ERR_ALIGN), (dict(ldv=202), m.ERR_ALIGN),
    *[({k: A + 8}, m.ERR_ALIGN) for k in ("k", "v", "q", "bs", "rs")],
    *[({k: A + 2}, m.ERR_ALIGN) for k in ("starts", "at", "table", "status")]])
def test_cache_validation(lib, read, kw, code):
    a = dict(spread(CACHE), **CACHE_SIZES)
    a.update(kw)
    assert cache_call(lib, a, read) == code


def test_cache_outputs_on_what_is_still_read_are_refused(lib):
    z = CACHE_SIZES
    rows = z["pages"] * 2 * z["heads"] * z["page"]
    size = dict(k=((z["T"] - 1) * z["ldk"] + 192) * 2, v=((z["T"] - 1) * z["ldv"] + 192) * 2, starts=12, at=8, table=32,
                q=rows * 32, bs=rows * 4, rs=rows * 4, status=4)
    base = dict(spread(CACHE), **z)
    for read, outs, ins in ((False, ("q", "bs", "rs", "status"), ("k", "v", "starts", "at", "table")),
                            (True, ("k", "v", "status"), ("q", "bs", "rs", "starts", "at", "table"))):
        for o in outs:
            for other in (*outs, *ins):
                if o == other:
                    continue
                for at in (base[other], base[other] + (size[other] - 1) // 16 * 16, base[other] - (size[o] - 1) // 16 * 16):
                    assert cache_call(lib, dict(base, **{o: at}), read) == m.ERR_ARG, (read, o, other)


ATT = ("query", "q", "bs", "rs", "table", "length", "rows", "out", "lse", "status", "ws")
ATT_SIZES = dict(B=2, Q=3, hq=6, kv=3, D=64, pages=7, page=16, mp=4, ldq=384, ldo=392, scale=0.125, ws_bytes=1 << 31)


def attend(lib, a):
    return lib.mtp_head_attention_fp4(a["query"], a["ldq"], a["q"], a["bs"], a["rs"], a["table"], a["length"], a["rows"],
                                      a["out"], a["ldo"], a["lse"], a["status"], a["ws"], a["ws_bytes"], a["B"], a["Q"],
                                      a["hq"], a["kv"], a["D"], a["pages"], a["page"], a["mp"], ctypes.c_float(a["scale"]), None)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, m.ERR_ARG) for k in ("query", "q", "bs", "rs", "table", "length", "out")],
    (dict(scale=0.0), m.ERR_ARG), (dict(scale=-1.0), m.ERR_ARG), (dict(scale=float("inf")), m.ERR_ARG),
    (dict(scale=float("nan")), m.ERR_ARG), (dict(B=0), m.ERR_SHAPE), (dict(B=65537), m.ERR_SHAPE), (dict(Q=0), m.ERR_SHAPE),
    (dict(Q=1025), m.ERR_SHAPE), (dict(hq=7), m.ERR_SHAPE), (dict(hq=0), m.ERR_SHAPE), (dict(kv=0), m.ERR_SHAPE),
    (dict(hq=1026, ldq=1 << 20, ldo=1 << 20), m.ERR_SHAPE), (dict(B=65536, Q=1024), m.ERR_SHAPE),
    (dict(page=48), m.ERR_SHAPE), (dict(D=80, ldq=1024, ldo=1024), m.ERR_NOT_IMPLEMENTED), (dict(ldq=380), m.ERR_SHAPE),
    (dict(ldo=376), m.ERR_SHAPE), (dict(ldq=388), m.ERR_ALIGN), (dict(ldo=386), m.ERR_ALIGN),
    *[({k: A + 8}, m.ERR_ALIGN) for k in ("query", "q", "bs", "rs", "out", "ws")],
    *[({k: A + 2}, m.ERR_ALIGN) for k in ("table", "length", "rows", "lse", "status")],
    (dict(ws=None), m.ERR_WORKSPACE), (dict(ws_bytes=256), m.ERR_WORKSPACE)])
def test_attention_fp4_validation(lib, kw, code):
    a = dict(spread(ATT), **ATT_SIZES)
    a.update(kw)
    assert attend(lib, a) == code


def test_attention_fp4_outputs_on_what_is_still_read_are_refused(lib):
    z = dict(ATT_SIZES)
    z["ws_bytes"] = m.mtp_head_attention_fp4_workspace_bytes(2, 3, 6, 3, 64, 64)
    rows = z["pages"] * 2 * z["kv"] * z["page"]
    size = dict(query=(5 * 384 + 384) * 2, q=rows * 32, bs=rows * 4, rs=rows * 4, table=32, length=8, rows=8,
                out=(5 * 392 + 384) * 2, lse=36 * 4, status=4, ws=z["ws_bytes"])
    base = dict(spread(ATT), **z)
    for o in ("out", "lse", "status", "ws"):
        for other in ATT:
            if o == other:
                continue
            for at in (base[other], base[other] + (size[other] - 1) // 16 * 16, base[other] - (size[o] - 1) // 16 * 16):
                assert attend(lib, dict(base, **{o: at})) == m.ERR_ARG, (o, other)


def test_attention_fp4_workspace_serves_smaller_calls(lib):
    f = m.mtp_head_attention_fp4_workspace_bytes
    assert f(0, 1, 8, 8, 64, 100) == 0 and f(1, 0, 8, 8, 64, 100) == 0 and f(1, 1, 9, 8, 64, 100) == 0
    assert f(1, 1, 8, 8, 96, 100) == 0 and f(1, 1, 8, 8, 64, 0) == 0 and f(1, 1, 8, 8, 64, (1 << 30) + 1) == 0
    for B, Q, hq, kv, D, n in ((16, 5, 48, 8, 128, 32768), (3, 1, 8, 8, 64, 100), (200, 2, 16, 2, 128, 131072)):
        top = f(B, Q, hq, kv, D, n)
        assert top > 0
        for b in (1, B // 2 or 1, B):
            for q in (1, Q):
                for length in (16, n // 3 or 1, n):
                    assert 0 < f(b, q, hq, kv, D, length) <= top
                    assert 0 < f(b, q, kv, kv, 64, length) <= top


def test_attention_fp4_refuses_more_rounds_than_it_counts(lib):
    """2^31 rounds of 128 tokens over all sequences, key heads and groups of 16 rows."""
    sizes = dict(spread(ATT), **dict(ATT_SIZES, B=65536, Q=1, hq=8, kv=8, ldq=512, ldo=512, pages=1 << 20, page=128, ws_bytes=0))
    assert attend(lib, dict(sizes, mp=4096)) == m.ERR_WORKSPACE
    assert attend(lib, dict(sizes, mp=4097)) == m.ERR_SHAPE
    f = m.mtp_head_attention_fp4_workspace_bytes
    assert f(65536, 1, 8, 8, 64, 4096 * 128) > 0 and f(65536, 1, 8, 8, 64, 4097 * 128) == 0


PROMPT = ("q", "k", "v", "starts", "out", "lse", "status")
PROMPT_SIZES = dict(T=9, B=2, hq=6, kv=3, D=64, ldq=384, ldk=192, ldv=200, ldo=392, scale=0.125)


def prompt(lib, a):
    return lib.mtp_head_attention_prompt(a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["starts"], a["out"], a["ldo"],
                                         a["lse"], a["status"], a["T"], a["B"], a["hq"], a["kv"], a["D"],
                                         ctypes.c_float(a["scale"]), None)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, m.ERR_ARG) for k in ("q", "k", "v", "starts", "out")], (dict(scale=0.0), m.ERR_ARG),
    (dict(scale=float("nan")), m.ERR_ARG), (dict(T=0), m.ERR_SHAPE), (dict(T=(1 << 22) + 1), m.ERR_SHAPE), (dict(B=0), m.ERR_SHAPE),
    (dict(B=65537), m.ERR_SHAPE), (dict(hq=7), m.ERR_SHAPE), (dict(kv=0), m.ERR_SHAPE), (dict(D=0), m.ERR_SHAPE),
    (dict(D=32), m.ERR_NOT_IMPLEMENTED), (dict(ldq=376), m.ERR_SHAPE), (dict(ldk=184), m.ERR_SHAPE), (dict(ldv=10), m.ERR_SHAPE),
    (dict(ldo=383), m.ERR_SHAPE), (dict(ldq=388), m.ERR_ALIGN), (dict(ldk=194), m.ERR_ALIGN), (dict(ldv=204), m.ERR_ALIGN),
    (dict(ldo=390), m.ERR_ALIGN), *[({k: A + 8}, m.ERR_ALIGN) for k in ("q", "k", "v", "out")],
    *[({k: A + 2}, m.ERR_ALIGN) for k in ("starts", "lse", "status")]])
def test_prompt_validation(lib, kw, code):
    a = dict(spread(PROMPT), **PROMPT_SIZES)
    a.update(kw)
    assert prompt(lib, a) == code


def test_prompt_outputs_on_what_is_still_read_are_refused(lib):
    base = dict(spread(PROMPT), **PROMPT_SIZES)
    size = dict(q=9 * 384 * 2, k=9 * 192 * 2, v=(8 * 200 + 192) * 2, starts=12, out=(8 * 392 + 384) * 2, lse=9 * 6 * 4, status=4)
    for o in ("out", "lse", "status"):
        for other in PROMPT:
            if o == other:
                continue
            for at in (base[other], base[other] + (size[other] - 1) // 16 * 16, base[other] - (size[o] - 1) // 16 * 16):
                assert prompt(lib, dict(base, **{o: at})) == m.ERR_ARG, (o, other)


def test_binding_refuses_host_tensors_and_wrong_ranks():
    cache = m.cache_empty(4, 16, 2, 64, "cpu")
    assert [tuple(t.shape) for t in cache] == [(4, 2, 2, 16, 32), (4, 2, 2, 16, 4), (4, 2, 2, 16)]
    for bad in ((0, 16, 2, 64), (4, 8, 2, 64), (4, 16, 0, 64), (4, 16, 2, 60)):
        with pytest.raises(m.MTPError):
            m.cache_empty(*bad, "cpu")
    z = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        m.mtp_head_norm_residual(z(2, 64), z(64), y=z(2, 64))
    with pytest.raises(ValueError, match="dimensions"):
        m.mtp_head_norm_residual(z(64), z(64), y=z(64))
    with pytest.raises(ValueError, match="CUDA"):
        m.mtp_head_cache_write_fp4(z(3, 2, 64), z(3, 2, 64), z(2, dtype=I32), z(1, dtype=I32), z(1, 4, dtype=I32), *cache)
    with pytest.raises(ValueError, match="CUDA"):
        m.mtp_head_attention_fp4(z(1, 1, 2, 64), *cache, z(1, 4, dtype=I32), z(1, dtype=I32), z(1, 1, 2, 64), None)
    with pytest.raises(ValueError, match="CUDA"):
        m.mtp_head_attention_prompt(z(3, 2, 64), z(3, 2, 64), z(3, 2, 64), z(2, dtype=I32), z(3, 2, 64))
    with pytest.raises(m.MTPError):
        m.attention_fp4_workspace(1, 1, 3, 2, 64, 100, "cpu")


def test_layer_refuses_shapes_that_do_not_fit():
    cache = m.LayerCache(2, 100, 2, 64, page=16, device="cpu")
    assert cache.max_pages == 7 and cache.max_len == 112 and cache.table.shape == (2, 7)
    w = torch.zeros(64, dtype=BF)
    with pytest.raises(ValueError, match="shapes"):
        m.DraftLayer(w, torch.zeros(100, 64, dtype=BF), torch.zeros(64, 256, dtype=BF), 4, 2, cache)
    with pytest.raises(ValueError, match="key heads"):
        m.DraftLayer(w, torch.zeros(6 * 64, 64, dtype=BF), torch.zeros(64, 256, dtype=BF), 4, 1, cache)
    with pytest.raises(ValueError, match="together"):
        m.DraftLayer(w, torch.zeros(8 * 64, 64, dtype=BF), torch.zeros(64, 256, dtype=BF), 4, 2, cache, mlp=lambda *a: None)
