"""The FP4, sampling and acceptance entry points without a GPU: sizes, the documented status codes
(every call below fails validation before anything is launched; the addresses are never
dereferenced) and the binding's refusals."""
import ctypes

import pytest
import torch

import mtp_speculative_draft_head_gb300 as m

A = 0x10000  # an aligned fake device address


@pytest.fixture(scope="module")
def lib():
    return m.load()


@pytest.mark.parametrize("h,hp", [(1, 256), (255, 256), (256, 256), (257, 512), (6144, 6144), (12288, 12288),
                                  (131072, 131072), (0, 0), (-5, 0), (131073, 0)])
def test_padded_row(lib, h, hp):
    assert m.mtp_head_fp4_padded(h) == hp


def test_workspace_sizes(lib):
    assert m.mtp_head_fp4_workspace_bytes(0, 64, 10) == 0 and m.mtp_head_fp4_workspace_bytes(17, 64, 10) == 0
    assert m.mtp_head_fp4_workspace_bytes(1, 65537, 10) == 0 and m.mtp_head_fp4_workspace_bytes(1, 64, 0) == 0
    sizes = [m.mtp_head_fp4_workspace_bytes(b, 6144, 154880) for b in range(1, 17)]
    assert sizes[0] > 2304 and sizes == sorted(sizes)
    assert m.mtp_head_linear_fp4_workspace_bytes(0, 1, 1) == 0 and m.mtp_head_linear_fp4_workspace_bytes(65537, 1, 1) == 0
    assert m.mtp_head_linear_fp4_workspace_bytes(1, 0, 1) == 0 and m.mtp_head_linear_fp4_workspace_bytes(1, 1, 131073) == 0
    assert m.mtp_head_linear_fp4_workspace_bytes(3, 5, 7) > 0
    assert m.mtp_head_context_fp4_workspace_bytes(4, 60) == 0  # H % 8 != 0
    assert m.mtp_head_context_fp4_workspace_bytes(4, 64) > m.mtp_head_linear_fp4_workspace_bytes(4, 64, 128)
    with pytest.raises(m.MTPError):
        m.fp4_empty(4, 0, "cpu")


@pytest.mark.parametrize("kw,code", [
    (dict(w=None), m.ERR_ARG), (dict(q=None), m.ERR_ARG), (dict(bs=None), m.ERR_ARG), (dict(rs=None), m.ERR_ARG),
    (dict(status=None), m.ERR_ARG), (dict(V=0), m.ERR_SHAPE), (dict(H=0), m.ERR_SHAPE), (dict(H=131073), m.ERR_SHAPE),
    (dict(w=A + 8), m.ERR_ALIGN), (dict(q=A + 8), m.ERR_ALIGN), (dict(bs=A + 2), m.ERR_ALIGN),
    (dict(rs=A + 2), m.ERR_ALIGN), (dict(status=A + 1), m.ERR_ALIGN)])
def test_quantize_validation(lib, kw, code):
    a = dict(w=A, q=A, bs=A, rs=A, status=A, V=4, H=64)
    a.update(kw)
    assert lib.mtp_head_quantize_fp4(a["w"], a["q"], a["bs"], a["rs"], a["status"], a["V"], a["H"], None) == code
    if "status" not in kw:
        assert lib.mtp_head_dequantize_fp4(a["q"], a["bs"], a["rs"], a["w"], a["V"], a["H"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), m.ERR_ARG), (dict(fw=None), m.ERR_ARG), (dict(q=None), m.ERR_ARG), (dict(draft=None), m.ERR_ARG),
    (dict(eps=float("nan")), m.ERR_ARG), (dict(eps=-1.0), m.ERR_ARG), (dict(B=0), m.ERR_SHAPE),
    (dict(B=17), m.ERR_SHAPE), (dict(H=65537), m.ERR_SHAPE), (dict(V=0), m.ERR_SHAPE), (dict(x=A + 2), m.ERR_ALIGN),
    (dict(q=A + 8), m.ERR_ALIGN), (dict(logits=A + 2), m.ERR_ALIGN), (dict(ws=A + 8), m.ERR_ALIGN),
    (dict(ws=None), m.ERR_WORKSPACE), (dict(ws_bytes=2304), m.ERR_WORKSPACE)])
def test_sweep_validation(lib, kw, code):
    a = dict(x=A, fw=A, q=A, bs=A, rs=A, logits=None, draft=A, status=None, ws=A, ws_bytes=1 << 20, B=1, H=64, V=100,
             eps=1e-6)
    a.update(kw)
    assert lib.mtp_head_logits_argmax_fp4(a["x"], a["fw"], a["q"], a["bs"], a["rs"], a["logits"], a["draft"],
                                          a["status"], a["ws"], a["ws_bytes"], a["B"], a["H"], a["V"],
                                          ctypes.c_float(a["eps"]), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), m.ERR_ARG), (dict(y=None), m.ERR_ARG), (dict(rs=None), m.ERR_ARG), (dict(R=0), m.ERR_SHAPE),
    (dict(R=65537), m.ERR_SHAPE), (dict(N=0), m.ERR_SHAPE), (dict(K=0), m.ERR_SHAPE), (dict(K=131073), m.ERR_SHAPE),
    (dict(x=A + 8), m.ERR_ALIGN), (dict(y=A + 2), m.ERR_ALIGN), (dict(bs=A + 8), m.ERR_ALIGN),
    (dict(ws=None), m.ERR_WORKSPACE), (dict(ws_bytes=16), m.ERR_WORKSPACE)])
def test_linear_validation(lib, kw, code):
    a = dict(x=A, q=A, bs=A, rs=A, y=A, status=None, ws=A, ws_bytes=1 << 30, R=4, N=8, K=64)
    a.update(kw)
    assert lib.mtp_head_linear_fp4(a["x"], a["q"], a["bs"], a["rs"], a["y"], a["status"], a["ws"], a["ws_bytes"],
                                   a["R"], a["N"], a["K"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(embed=None), m.ERR_ARG), (dict(q=None), m.ERR_ARG), (dict(tokens=None), m.ERR_ARG),
    (dict(eps=float("inf")), m.ERR_ARG), (dict(R=0), m.ERR_SHAPE), (dict(H=65544), m.ERR_SHAPE), (dict(V=0), m.ERR_SHAPE),
    (dict(tokens=A + 2), m.ERR_ALIGN), (dict(x=A + 8), m.ERR_ALIGN), (dict(H=60), m.ERR_NOT_IMPLEMENTED),
    (dict(ws=None), m.ERR_WORKSPACE), (dict(ws_bytes=64), m.ERR_WORKSPACE)])
def test_context_rows_validation(lib, kw, code):
    a = dict(embed=A, en=A, hn=A, q=A, bs=A, rs=A, tokens=A, hidden=A, x=A, status=None, ws=A, ws_bytes=1 << 30, R=4,
             H=64, V=100, eps=1e-6)
    a.update(kw)
    assert lib.mtp_head_context_rows_fp4(a["embed"], a["en"], a["hn"], a["q"], a["bs"], a["rs"], a["tokens"],
                                         a["hidden"], a["x"], a["status"], a["ws"], a["ws_bytes"], a["R"], a["H"],
                                         a["V"], ctypes.c_float(a["eps"]), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), m.ERR_ARG), (dict(token=None, prob=None, probs=None), m.ERR_ARG), (dict(u=None), m.ERR_ARG),
    (dict(u=None, token=None), m.ERR_ARG), (dict(dtype=2), m.ERR_ARG), (dict(R=0), m.ERR_SHAPE),
    (dict(R=65537), m.ERR_SHAPE), (dict(V=0), m.ERR_SHAPE), (dict(ld=99), m.ERR_SHAPE), (dict(logits=A + 2), m.ERR_ALIGN),
    (dict(dtype=1, logits=A + 1), m.ERR_ALIGN), (dict(token=A + 2), m.ERR_ALIGN), (dict(top_k=A + 1), m.ERR_ALIGN),
    (dict(probs=A + 2), m.ERR_ALIGN)])
def test_sample_validation(lib, kw, code):
    a = dict(logits=A, dtype=m.LOGITS_FP32, ld=100, t=A, top_k=A, top_p=A, min_p=A, u=A, token=A, prob=A, probs=A,
             status=A, R=2, V=100)
    a.update(kw)
    assert lib.mtp_head_sample(a["logits"], a["dtype"], a["ld"], a["t"], a["top_k"], a["top_p"], a["min_p"], a["u"],
                               a["token"], a["prob"], a["probs"], a["status"], a["R"], a["V"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(p=None), m.ERR_ARG), (dict(x=None), m.ERR_ARG), (dict(u=None), m.ERR_ARG), (dict(tokens=None), m.ERR_ARG),
    (dict(accepted=None), m.ERR_ARG), (dict(B=0), m.ERR_SHAPE), (dict(B=65537), m.ERR_SHAPE), (dict(D=0), m.ERR_SHAPE),
    (dict(D=1025), m.ERR_SHAPE), (dict(V=0), m.ERR_SHAPE), (dict(p=A + 2), m.ERR_ALIGN), (dict(q=A + 2), m.ERR_ALIGN),
    (dict(n=A + 1), m.ERR_ALIGN), (dict(prob=A + 3), m.ERR_ALIGN)])
def test_verify_validation(lib, kw, code):
    a = dict(p=A, q=A, x=A, n=A, u=A, tokens=A, accepted=A, prob=A, status=A, B=2, D=3, V=100)
    a.update(kw)
    assert lib.mtp_head_verify(a["p"], a["q"], a["x"], a["n"], a["u"], a["tokens"], a["accepted"], a["prob"],
                               a["status"], a["B"], a["D"], a["V"], None) == code


def test_outputs_on_their_inputs_are_refused(lib):
    """probs on any byte of the (strided) logits, tokens on any byte of the drafts: refused before a launch."""
    R, V, ld = 3, 100, 128
    span = ((R - 1) * ld + V) * 4
    for probs in (A, A + span - 4, A - R * V * 4 + 4):
        assert lib.mtp_head_sample(A, m.LOGITS_FP32, ld, None, None, None, None, A, A, A, probs, None, R, V,
                                   None) == m.ERR_ARG
    B, D = 2, 3
    for tokens in (A, A + B * D * 4 - 4, A - B * (D + 1) * 4 + 4):
        assert lib.mtp_head_verify(A, A, A, None, A, tokens, A, None, None, B, D, V, None) == m.ERR_ARG


@pytest.mark.parametrize("out", ["tokens", "accepted", "prob", "status"])
@pytest.mark.parametrize("other", ["p", "q", "x", "n", "u", "tokens", "accepted", "prob", "status"])
def test_verify_outputs_on_any_other_array_are_refused(lib, out, other):
    """Every output of the acceptance against every other array, on its first byte and on its last."""
    B, D, V = 2, 3, 100
    size = dict(p=B * (D + 1) * V, q=B * D * V, x=B * D, n=B, u=B * (D + 1), tokens=B * (D + 1), accepted=B, prob=B, status=1)
    base = {k: A + 0x100000 * i for i, k in enumerate(size)}
    if out == other:
        return
    for at in (base[other], base[other] + 4 * (size[other] - 1), base[other] - 4 * (size[out] - 1)):
        a = dict(base)
        a[out] = at
        assert lib.mtp_head_verify(a["p"], a["q"], a["x"], a["n"], a["u"], a["tokens"], a["accepted"], a["prob"],
                                   a["status"], B, D, V, None) == m.ERR_ARG


def _refused(call, size, pairs):
    """call(addresses) is refused with MTP_ERR_ARG whenever the first array of a pair shares the first or the last
    bytes of the second (arrays are 16-byte aligned, so are the shifts)."""
    base = {k: A + 0x10000000 * i for i, k in enumerate(size)}
    for out, other in pairs:
        last = (size[other] - 1) // 16 * 16
        for at in (base[other], base[other] + last, base[other] - (size[out] - 1) // 16 * 16):
            assert call(dict(base, **{out: at})) == m.ERR_ARG, (out, other)


COPY = ("q", "bs", "rs")


def test_fp4_outputs_on_what_is_still_read_are_refused(lib):
    V, H = 40, 500
    copy = dict(q=V * 256, bs=V * 32, rs=V * 4)
    _refused(lambda a: lib.mtp_head_quantize_fp4(a["w"], a["q"], a["bs"], a["rs"], a["st"], V, H, None),
             dict(copy, w=V * H * 2, st=4),
             [(o, i) for o in (*COPY, "st") for i in ("w", *COPY, "st") if o != i])
    _refused(lambda a: lib.mtp_head_dequantize_fp4(a["q"], a["bs"], a["rs"], a["w"], V, H, None),
             dict(copy, w=V * H * 2), [("w", i) for i in COPY])
    B = 3
    ws = m.mtp_head_fp4_workspace_bytes(B, H, V)
    _refused(lambda a: lib.mtp_head_logits_argmax_fp4(a["x"], a["fw"], a["q"], a["bs"], a["rs"], a["lg"], a["d"], a["st"],
                                                      a["ws"], ws, B, H, V, ctypes.c_float(1e-6), None),
             dict(copy, x=B * H * 2, fw=H * 2, lg=B * V * 4, d=B * 4, st=4, ws=ws),
             [(o, i) for o in ("lg", "d", "st", "ws") for i in (*COPY, "lg", "d", "st", "ws") if o != i] +
             [("ws", "x"), ("ws", "fw")])
    R = 5
    wl = m.mtp_head_linear_fp4_workspace_bytes(R, V, H)
    _refused(lambda a: lib.mtp_head_linear_fp4(a["x"], a["q"], a["bs"], a["rs"], a["y"], a["st"], a["ws"], wl, R, V, H,
                                               None),
             dict(copy, x=R * H * 2, y=R * V * 2, st=4, ws=wl),
             [(o, i) for o in ("y", "st", "ws") for i in (*COPY, "y", "st", "ws") if o != i] + [("ws", "x"), ("st", "x")])
    h, v = 64, 40
    wc = m.mtp_head_context_fp4_workspace_bytes(R, h)
    _refused(lambda a: lib.mtp_head_context_rows_fp4(a["e"], a["en"], a["hn"], a["q"], a["bs"], a["rs"], a["t"], a["h"],
                                                     a["x"], a["st"], a["ws"], wc, R, h, v, ctypes.c_float(1e-6), None),
             dict(q=h * 128, bs=h * 16, rs=h * 4, e=v * h * 2, en=h * 2, hn=h * 2, t=R * 4, h=R * h * 2, x=R * h * 2, st=4,
                  ws=wc),
             [(o, i) for o in ("x", "st", "ws") for i in (*COPY, "x", "st", "ws") if o != i] +
             [("ws", i) for i in ("e", "en", "hn", "t", "h")])


def test_sampler_outputs_on_what_is_still_read_are_refused(lib):
    R, V, ld = 7, 100, 128
    par = ("t", "k", "tp", "mp", "u")
    size = dict(l=((R - 1) * ld + V) * 2, token=R * 4, prob=R * 4, probs=R * V * 4, st=4, **{p: R * 4 for p in par})
    call = lambda a: lib.mtp_head_sample(a["l"], m.LOGITS_BF16, ld, *(a[p] for p in par), a["token"], a["prob"],  # noqa: E731
                                         a["probs"], a["st"], R, V, None)
    outs = ("token", "prob", "probs", "st")
    _refused(call, size, [(o, i) for o in outs for i in ("l", *outs) if o != i] +
             [(o, p) for o in ("probs", "st") for p in par])
    base = {k: A + 0x10000000 * i for i, k in enumerate(size)}
    for o in ("token", "prob"):  # one row off: another row's parameter
        for p in par:
            for shift in (4, -4, 4 * (R - 1)):
                assert call(dict(base, **{o: base[p] + shift})) == m.ERR_ARG


def test_binding_refuses_host_tensors_and_wrong_ranks():
    bf, i32 = torch.bfloat16, torch.int32
    w4 = m.fp4_empty(4, 64, "cpu")
    assert [tuple(t.shape) for t in w4] == [(4, 128), (4, 16), (4,)]
    st = torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError, match="CUDA"):
        m.mtp_head_quantize_fp4(torch.zeros(4, 64, dtype=bf), *w4, st)
    with pytest.raises(ValueError, match="dimensions"):
        m.mtp_head_quantize_fp4(torch.zeros(64, dtype=bf), *w4, st)
    with pytest.raises(ValueError, match="CUDA"):
        m.mtp_head_linear_fp4(torch.zeros(2, 64, dtype=bf), *w4, torch.zeros(2, 4, dtype=bf), None)
    with pytest.raises(ValueError, match="CUDA"):
        m.mtp_head_sample(torch.zeros(2, 10), torch.zeros(2), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="dimensions"):
        m.mtp_head_verify(torch.zeros(2, 10), None, torch.zeros(2, 1, dtype=i32), torch.zeros(2, 2),
                          torch.zeros(2, 2, dtype=i32), torch.zeros(2, dtype=i32))


def test_head_refuses_two_weight_formats_before_any_launch(monkeypatch):
    """forward(fp8=True, fp4=True): nothing of the step has run when it is refused."""
    head = object.__new__(m.MtpDraftHead)
    monkeypatch.setattr(m.MtpDraftHead, "input", lambda *a, **k: pytest.fail("the input stage was launched"))
    with pytest.raises(ValueError, match="exclude"):
        head.forward(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 64, dtype=torch.bfloat16), fp8=True, fp4=True)
