"""The FP4 and sampling operators of the draft head: what is measured, and their plain forms.

Five operators, in the order in which a speculative decoder uses them:

* ``copy``    the two-level FP4 copy of a BF16 matrix and the BF16 matrix that the copy stands for
* ``sweep``   final norm, lm_head sweep over the FP4 copy, argmax (1 to 16 sequences)
* ``linear``  rows of activations quantised to FP4, times an FP4 weight matrix
* ``sample``  one token per row of logits: temperature, top-k, top-p, min-p, one given uniform number
* ``verify``  drafts accepted or rejected against the target's distributions, and the token after them

``run`` computes them with elementary torch operations, or with the library's own calls when
``own`` is set.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
BLOCK = 16     # codes that share a block scale
ROW = 256      # rows of codes are padded to a multiple of this
DEV = "cuda"


def listed():
    return [
        # the concat rows of 16 sequences of a draft step, before an FP4 eh_proj: latency counts
        {"name": "copy_rows16", "op": "copy", "V": 16, "H": 12288},
        # the whole lm_head, copied once when the weights are loaded
        {"name": "copy_lm_head", "op": "copy", "V": 154880, "H": 6144},
        # the smallest head of the tests: a step that is all latency
        {"name": "sweep_tiny", "op": "sweep", "B": 1, "H": 256, "V": 4096},
        # one sequence of the full-size head: an ordinary draft step
        {"name": "sweep_b1", "op": "sweep", "B": 1, "H": 6144, "V": 154880},
        # a full batch of the full-size head
        {"name": "sweep_b16", "op": "sweep", "B": 16, "H": 6144, "V": 154880},
        # eh_proj for 16 sequences of a draft step
        {"name": "linear_16", "op": "linear", "R": 16, "N": 6144, "K": 12288},
        # eh_proj over a prompt (context rows)
        {"name": "linear_4096", "op": "linear", "R": 4096, "N": 6144, "K": 12288},
        # one sequence, all filters on
        {"name": "sample_1", "op": "sample", "R": 1, "V": 154880, "bf16": False, "top_k": True, "top_p": True,
         "min_p": True, "probs": False},
        # a draft step of 16 sequences from BF16 logits, with the distribution kept for the acceptance
        {"name": "sample_16_bf16", "op": "sample", "R": 16, "V": 154880, "bf16": True, "top_k": False, "top_p": True,
         "min_p": False, "probs": True},
        # the target's rows of 16 sequences with 4 drafts each: 80 distributions
        {"name": "sample_80", "op": "sample", "R": 80, "V": 154880, "bf16": False, "top_k": True, "top_p": True,
         "min_p": False, "probs": True},
        # one sequence, one draft, on the smallest head of the tests
        {"name": "verify_1", "op": "verify", "B": 1, "D": 1, "V": 4096, "onehot": False},
        # 16 sequences with 4 drafts each
        {"name": "verify_16", "op": "verify", "B": 16, "D": 4, "V": 154880, "onehot": False},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["copy", "sweep", "linear", "sample", "verify"])
    if op == "copy":
        return {"op": op, "V": _between(rng, 1, 154880), "H": _between(rng, 16, 6144)}
    if op == "sweep":
        return {"op": op, "B": rng.randint(1, 16), "H": _between(rng, 64, 6144), "V": _between(rng, 1000, 154880)}
    if op == "linear":
        return {"op": op, "R": _between(rng, 1, 4096), "N": _between(rng, 64, 6144), "K": _between(rng, 64, 12288)}
    if op == "sample":
        return {"op": op, "R": _between(rng, 1, 80), "V": _between(rng, 1000, 154880), "bf16": rng.random() < 0.5,
                "top_k": rng.random() < 0.5, "top_p": rng.random() < 0.7, "min_p": rng.random() < 0.5,
                "probs": rng.random() < 0.5}
    return {"op": op, "B": _between(rng, 1, 16), "D": rng.randint(1, 4), "V": _between(rng, 1000, 154880),
            "onehot": rng.random() < 0.3}


def _padded(n):
    return (n + ROW - 1) // ROW * ROW


def work(c):
    if c["op"] == "copy":
        V, H = c["V"], c["H"]
        # the copy is written and read once, the matrix read once and written once
        return {"bytes": V * H * 2 * 2 + 2 * (V * H * 9 // 16 + 4 * V), "flops": 4 * V * H}
    if c["op"] == "sweep":
        B, H, V = c["B"], c["H"], c["V"]
        return {"bytes": V * H * 9 // 16 + 4 * V + 2 * B * H + 4 * B * V + 4 * B, "flops": 2 * B * V * H}
    if c["op"] == "linear":
        R, N, K = c["R"], c["N"], c["K"]
        return {"bytes": N * K * 9 // 16 + 4 * N + 2 * R * K + 2 * R * N, "flops": 2 * R * N * K}
    if c["op"] == "sample":
        n = c["R"] * c["V"]
        return {"bytes": n * (2 if c["bf16"] else 4) + (4 * n if c["probs"] else 0), "flops": 10 * n}
    # per sequence: one row of the target's distributions and, unless the drafts are greedy, one of the drafter's
    return {"bytes": c["B"] * c["V"] * 4 * (1 if c["onehot"] else 2), "flops": 3 * c["B"] * c["V"]}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _fp4_weights(n, k, g):
    """An FP4 copy as a loader hands it over: Gaussian weights, quantised in 32 bits."""
    q = torch.empty((n, _padded(k) // 2), dtype=torch.uint8, device=DEV)
    bs = torch.empty((n, _padded(k) // BLOCK), dtype=torch.uint8, device=DEV)
    rs = torch.empty((n,), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // _padded(k))
    for i in range(0, n, step):  # slices keep the 32-bit copies small
        m = min(step, n - i)
        w = torch.zeros((m, _padded(k)), device=DEV)
        w[:, :k] = (torch.randn((m, k), generator=g, device=DEV) * 0.02).bfloat16().float()
        r = w.abs().amax(1) / 2688.0
        b = w.view(m, -1, BLOCK)
        s = (b.abs().amax(2) / (6.0 * r).view(-1, 1)).clamp(max=448.0).to(torch.float8_e4m3fn)
        y = (b.abs() / (s.float() * r.view(-1, 1)).view(m, -1, 1).clamp(min=1e-30)).clamp(max=6.0)
        c = torch.bucketize(y, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV))
        c = (c + 8 * (b < 0)).to(torch.uint8).view(m, -1)
        q[i:i + m] = c[:, 0::2] | (c[:, 1::2] << 4)
        bs[i:i + m] = s.view(torch.uint8)
        rs[i:i + m] = r
    return q, bs, rs


def _logits(rows, V, g):
    """Logits like a language model's: a broad bulk and a few tokens well above it."""
    l = torch.randn((rows, V), generator=g, device=DEV) * 2.0
    top = torch.randint(0, V, (rows, 24), generator=g, device=DEV)
    return l.scatter_add_(1, top, torch.rand((rows, 24), generator=g, device=DEV) * 12.0)


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": c, "kept": {}}
    if c["op"] == "copy":
        s["w"] = (torch.randn((c["V"], c["H"]), generator=g, device=DEV) * 0.02).bfloat16()
    elif c["op"] == "sweep":
        s["x"] = (torch.randn((c["B"], c["H"]), generator=g, device=DEV)).bfloat16()
        s["norm"] = (1.0 + 0.1 * torch.randn((c["H"],), generator=g, device=DEV)).bfloat16()
        s["q"], s["bs"], s["rs"] = _fp4_weights(c["V"], c["H"], g)
    elif c["op"] == "linear":
        s["x"] = (torch.randn((c["R"], c["K"]), generator=g, device=DEV)).bfloat16()
        s["q"], s["bs"], s["rs"] = _fp4_weights(c["N"], c["K"], g)
    elif c["op"] == "sample":
        R, V = c["R"], c["V"]
        l = _logits(R, V, g)
        s["logits"] = l.bfloat16() if c["bf16"] else l
        s["temperature"] = 0.6 + 0.6 * torch.rand((R,), generator=g, device=DEV)
        s["top_k"] = torch.randint(1, 200, (R,), generator=g, device=DEV, dtype=torch.int32) if c["top_k"] else None
        s["top_p"] = 0.8 + 0.19 * torch.rand((R,), generator=g, device=DEV) if c["top_p"] else None
        s["min_p"] = 0.1 * torch.rand((R,), generator=g, device=DEV) if c["min_p"] else None
        s["u"] = torch.rand((R,), generator=g, device=DEV)
    else:
        B, D, V = c["B"], c["D"], c["V"]
        l = _logits(B * (D + 1), V, g).view(B, D + 1, V)
        s["p"] = torch.softmax(l, 2)
        ql = l[:, :D] + 0.5 * torch.randn((B, D, V), generator=g, device=DEV)
        q = torch.softmax(ql, 2)
        pick = torch.rand((B, D, 1), generator=g, device=DEV)
        s["draft"] = (ql.argmax(2) if c["onehot"] else (q.cumsum(2) < pick).sum(2).clamp(max=V - 1)).to(torch.int32)
        s["draft_probs"] = None if c["onehot"] else q
        s["u"] = torch.rand((B, D + 1), generator=g, device=DEV)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _round(x, bits, low):
    """x (64 bits) to `bits` significant bits, no finer than 2^(low - bits + 1), ties to even."""
    e = torch.frexp(x)[1] - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=low) - (bits - 1))
    return torch.round(x / step) * step


def _fp4(w):
    """The copy of a BF16 matrix as values in 64 bits: codes [V, H'], block scales [V, H'/16], and
    the row scales [V] in 32 bits; H' is H rounded up to whole blocks."""
    w = torch.nn.functional.pad(w, (0, -w.shape[1] % BLOCK)).double().view(w.shape[0], -1, BLOCK)
    rs = (w.abs().amax((1, 2)) / 2688.0).float()
    r = rs.double().view(-1, 1)
    s = w.abs().amax(2) / torch.where(r > 0, 6.0 * r, torch.ones_like(r))
    s = torch.where(r > 0, _round(s, 4, -6).clamp(max=448.0), torch.zeros_like(s))
    d = (s * r).unsqueeze(2)
    c = w / torch.where(d > 0, d, torch.ones_like(d))
    c = torch.where(d > 0, _round(c, 2, 0).clamp(-6.0, 6.0), torch.zeros_like(c))
    return c.view(w.shape[0], -1), s, rs


def _unpack(q, bs, k):
    """code * block scale of a packed copy, in 32 bits (exact), [n, k]."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=q.device)
    c = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), 2).view(q.shape[0], -1, BLOCK)
    return (c * bs.view(torch.float8_e4m3fn).float().unsqueeze(2)).view(q.shape[0], -1)[:, :k]


def _plain_copy(s):
    c, bs, rs = _fp4(s["w"])
    n, h = s["w"].shape
    w = (c.float().view(n, -1, BLOCK) * bs.float().unsqueeze(2) * rs.view(-1, 1, 1)).view(n, -1)[:, :h]
    return {"w": w.bfloat16(), "row_scale": rs, "block_scale": bs.float().to(torch.float8_e4m3fn)}


def _plain_sweep(s):
    x = s["x"].double()
    xhat = _round(x * s["norm"].double() / torch.sqrt((x * x).mean(1, keepdim=True) + EPS), 8, -126).float()
    logits = (xhat @ _unpack(s["q"], s["bs"], x.shape[1]).t()) * s["rs"]
    return {"logits": logits, "draft": torch.argmax(logits, 1).to(torch.int32)}


def _plain_linear(s):
    c, bs, rs = _fp4(s["x"])
    k = s["x"].shape[1]
    a = (c.view(c.shape[0], -1, BLOCK) * bs.unsqueeze(2)).view(c.shape[0], -1)[:, :k].float()
    return (a @ _unpack(s["q"], s["bs"], k).t() * rs.view(-1, 1) * s["rs"]).bfloat16()


def _plain_sample(s):
    l = s["logits"].double()
    R, V = l.shape
    t = s["temperature"].double().view(-1, 1)
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    w = torch.exp((v - v[:, :1]) / t)
    if s["top_k"] is not None:
        w = torch.where(torch.arange(V, device=l.device) < s["top_k"].view(-1, 1), w, 0.0)
    if s["top_p"] is not None:
        cum = w.cumsum(1)
        w = torch.where(cum - w < s["top_p"].double().view(-1, 1) * cum[:, -1:], w, 0.0)
    if s["min_p"] is not None:
        w = torch.where(v >= v[:, :1] + t * torch.log(s["min_p"].double().view(-1, 1)), w, 0.0)
    w = torch.zeros_like(w).scatter_(1, i, w)
    cum = w.cumsum(1)
    z = cum[:, -1:]
    token = (cum <= s["u"].double().view(-1, 1) * z).sum(1, keepdim=True).clamp(max=V - 1)
    p = (w / z).float()
    out = {"token": token.view(-1).to(torch.int32), "prob": p.gather(1, token).view(-1)}
    if s["case"]["probs"]:
        out["probs"] = p
    return out


def _plain_verify(s):
    p, q, x, u = s["p"], s["draft_probs"], s["draft"].long(), s["u"].double()
    B, D = x.shape
    V = p.shape[2]
    px = p[:, :D].gather(2, x.unsqueeze(2)).squeeze(2).double()
    qx = torch.ones_like(px) if q is None else q.gather(2, x.unsqueeze(2)).squeeze(2).double()
    n = (u[:, :D] * qx < px).long().cumprod(1).sum(1)
    row = p[torch.arange(B, device=p.device), n].double()
    at = n.clamp(max=D - 1)
    if q is None:
        other = torch.zeros_like(row).scatter_(1, x.gather(1, at.view(-1, 1)), 2.0)
    else:
        other = q[torch.arange(B, device=p.device), at].double()
    left = (row - torch.where((n < D).view(-1, 1), other, torch.zeros_like(other))).clamp(min=0.0)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, row)
    cum = left.cumsum(1)
    token = (cum <= u[:, D:] * cum[:, -1:]).sum(1, keepdim=True).clamp(max=V - 1)
    i = torch.arange(D + 1, device=p.device).view(1, -1)
    out = torch.where(i < n.view(-1, 1), torch.nn.functional.pad(x, (0, 1)), torch.where(i == n.view(-1, 1), token, -1))
    prob = (left.gather(1, token) / cum[:, -1:]).float().view(-1)
    return {"tokens": out.to(torch.int32), "accepted": n.to(torch.int32), "prob": prob}


# ------------------------------------------------------------------------------------- the library's calls
def _kept(s, name, make):
    """A buffer that a user's program makes once and uses for every call."""
    if name not in s["kept"]:
        s["kept"][name] = make()
    return s["kept"][name]


def _own(s):
    import mtp_speculative_draft_head_gb300 as m
    c = s["case"]
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)  # noqa: E731
    if c["op"] == "copy":
        V, H = c["V"], c["H"]
        w4 = _kept(s, "w4", lambda: m.fp4_empty(V, H, DEV))
        status = _kept(s, "status", lambda: torch.zeros(1, dtype=torch.int32, device=DEV))
        back = _kept(s, "back", lambda: new(V, H, dtype=torch.bfloat16))
        m.mtp_head_quantize_fp4(s["w"], *w4, status)
        m.mtp_head_dequantize_fp4(*w4, back)
        q, bs, rs = w4
        blocks = -(-H // BLOCK)
        return {"w": back, "row_scale": rs, "block_scale": bs[:, :blocks].view(torch.float8_e4m3fn)}
    if c["op"] == "sweep":
        B, H, V = c["B"], c["H"], c["V"]
        ws = _kept(s, "ws", lambda: m.fp4_workspace(B, H, V, DEV))
        logits = _kept(s, "logits", lambda: new(B, V, dtype=torch.float32))
        draft = _kept(s, "draft", lambda: new(B, dtype=torch.int32))
        m.mtp_head_logits_argmax_fp4(s["x"], s["norm"], s["q"], s["bs"], s["rs"], logits, draft, ws, eps=EPS)
        return {"logits": logits, "draft": draft}
    if c["op"] == "linear":
        ws = _kept(s, "ws", lambda: m.linear_fp4_workspace(c["R"], c["N"], c["K"], DEV))
        y = _kept(s, "y", lambda: new(c["R"], c["N"], dtype=torch.bfloat16))
        m.mtp_head_linear_fp4(s["x"], s["q"], s["bs"], s["rs"], y, ws)
        return y
    if c["op"] == "sample":
        R, V = c["R"], c["V"]
        token = _kept(s, "token", lambda: new(R, dtype=torch.int32))
        prob = _kept(s, "prob", lambda: new(R, dtype=torch.float32))
        probs = _kept(s, "probs", lambda: new(R, V, dtype=torch.float32)) if c["probs"] else None
        m.mtp_head_sample(s["logits"], s["u"], token, prob, probs, temperature=s["temperature"], top_k=s["top_k"],
                          top_p=s["top_p"], min_p=s["min_p"])
        out = {"token": token, "prob": prob}
        if c["probs"]:
            out["probs"] = probs
        return out
    tokens = _kept(s, "tokens", lambda: new(c["B"], c["D"] + 1, dtype=torch.int32))
    accepted = _kept(s, "accepted", lambda: new(c["B"], dtype=torch.int32))
    prob = _kept(s, "prob", lambda: new(c["B"], dtype=torch.float32))
    m.mtp_head_verify(s["p"], s["draft_probs"], s["draft"], s["u"], tokens, accepted, prob)
    return {"tokens": tokens, "accepted": accepted, "prob": prob}


def run(s):
    if own:
        return _own(s)
    return {"copy": _plain_copy, "sweep": _plain_sweep, "linear": _plain_linear, "sample": _plain_sample,
            "verify": _plain_verify}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------- 64 bits
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest(y, values):
    """Index of the nearest of the ascending `values` for each y >= 0 (64 bits); a tie goes to the even index."""
    v = torch.tensor(values, dtype=torch.float64, device=y.device)
    mid = (v[1:] + v[:-1]) / 2
    below = torch.bucketize(y, mid, right=False)   # values whose upper midpoint is < y
    upto = torch.bucketize(y, mid, right=True)     # ... <= y: one more on a tie
    return torch.where(below % 2 == 0, below, upto)


def _exact_fp4(w):
    n, h = w.shape
    blocks = -(-h // BLOCK)
    a = torch.zeros((n, blocks * BLOCK), dtype=torch.float64, device=w.device)
    a[:, :h] = w.to(torch.float64)
    rs = (a.abs().max(1).values / 2688.0).to(torch.float32)
    r = rs.to(torch.float64)
    table = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    top = a.view(n, blocks, BLOCK).abs().max(2).values
    s = torch.tensor(table, dtype=torch.float64, device=w.device)[_nearest(top / (6.0 * r)[:, None].clamp(min=1e-300), table)]
    d = (s * r[:, None]).repeat_interleave(BLOCK, 1)
    d = torch.where(d > 0, d, torch.full_like(d, math.inf))
    code = _nearest(a.abs() / d, _E2M1)
    return torch.sign(a) * torch.tensor(_E2M1, dtype=torch.float64, device=w.device)[code], s, rs


def _exact_weights(q, bs, k):
    code = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.uint8, device=q.device)
    code[:, 0::2] = q & 15
    code[:, 1::2] = q >> 4
    e = (bs >> 3).to(torch.float64)
    m = (bs & 7).to(torch.float64)
    s = torch.where(e > 0, (8 + m) * torch.exp2(e - 10), m * 2.0 ** -9)
    v = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)[(code & 7).long()]
    return (torch.where(code > 7, -v, v) * s.repeat_interleave(BLOCK, 1))[:, :k]


def _exact_verify(s):
    """The probability of each sequence's last token in the distribution that it was drawn from."""
    get = lambda k: s[k].double().cpu().numpy()  # noqa: E731
    u, x = get("u"), s["draft"].cpu().numpy()
    B, D = x.shape
    prob = np.zeros(B)
    for b in range(B):
        d = s["p"][b].double().cpu().numpy()
        n = 0
        while n < D:
            q = np.zeros(d.shape[1]) if s["draft_probs"] is None else s["draft_probs"][b, n].double().cpu().numpy()
            if s["draft_probs"] is None:
                q[x[b, n]] = 1.0
            if u[b, n] * q[x[b, n]] >= d[n, x[b, n]]:
                break
            n += 1
        w = d[n] if n == D else np.maximum(d[n] - q, 0.0)
        w = w / (np.sum(w) if np.sum(w) > 0 else 1.0)
        cum = np.cumsum(w)
        prob[b] = w[min(int(np.searchsorted(cum, u[b, D] * cum[-1], side="right")), w.size - 1)]
    return prob


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "copy":
        h = c["H"]
        v, bs, rs = _exact_fp4(s["w"])
        v *= bs.repeat_interleave(BLOCK, 1)
        return {"w": v[:, :h] * rs.double()[:, None], "row_scale": rs.double(), "block_scale": bs}
    if c["op"] == "sweep":
        x = s["x"].cpu().double().numpy()
        y = x * s["norm"].cpu().double().numpy() / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + EPS)
        m, e = np.frexp(y)  # the norm's output is a BF16 value
        xhat = torch.from_numpy(np.ldexp(np.rint(m * 256.0), e - 8)).to(DEV)
        logits = torch.matmul(xhat, _exact_weights(s["q"], s["bs"], c["H"]).T) * s["rs"].double()
        return {"logits": logits, "draft": None}
    if c["op"] == "linear":
        v, bs, rs = _exact_fp4(s["x"])
        a = (v * bs.repeat_interleave(BLOCK, 1) * rs.double()[:, None])[:, :c["K"]]
        return torch.matmul(a, _exact_weights(s["q"], s["bs"], c["K"]).T) * s["rs"].double()
    if c["op"] == "verify":
        return {"tokens": None, "accepted": None, "prob": _exact_verify(s)}
    l = s["logits"].double().cpu().numpy()
    get = lambda k: None if s[k] is None else s[k].double().cpu().numpy()  # noqa: E731
    t, tk, tp, mp, u = (get(k) for k in ("temperature", "top_k", "top_p", "min_p", "u"))
    probs = np.zeros_like(l)
    prob = np.zeros(c["R"])
    for r in range(c["R"]):
        order = np.argsort(-l[r], kind="stable")
        v = l[r][order]
        w = np.exp((v - v[0]) / t[r])
        keep = c["V"] if tk is None else min(c["V"], int(tk[r]))
        if tp is not None:
            before = np.concatenate(([0.0], np.cumsum(w[:keep])[:-1]))
            keep = int(np.sum(before < tp[r] * np.sum(w[:keep])))
        if mp is not None:
            keep = min(keep, int(np.sum((v - v[0]) / t[r] >= np.log(mp[r]))))
        probs[r, order[:keep]] = w[:keep] / np.sum(w[:keep])
        cum = np.cumsum(probs[r])
        prob[r] = probs[r, min(int(np.sum(cum <= u[r] * cum[-1])), c["V"] - 1)]
    out = {"token": None, "prob": prob}
    if c["probs"]:
        out["probs"] = probs
    return out
