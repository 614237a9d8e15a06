"""The operators of a draft layer's attention half: what is measured, and their plain forms.

Four operators, in the order in which a layer between the head's two stages uses them:

* ``norm``    the residual's addition, the norm of the sum, and an E4M3 copy of it with scales
* ``cache``   rows of keys and values written into a paged FP4 cache, and the same rows read back
* ``attend``  a few query rows of each sequence over its FP4 pages (a draft step, a verification)
* ``prompt``  causal attention over packed prompts of different lengths

``run`` computes them with elementary torch operations, or with the library's own calls when
``own`` is set.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 16     # codes that share a block scale
DEV = "cuda"


def listed():
    return [
        # 16 sequences of a draft step, the sum normalised for an 8-bit projection: latency counts
        {"name": "norm_step", "op": "norm", "R": 16, "H": 6144, "delta": True, "group": 0},
        # a prompt's rows with a scale per 128 columns
        {"name": "norm_prompt", "op": "norm", "R": 4096, "H": 6144, "delta": True, "group": 128},
        # rows that are not made of 16-byte pieces, without a sum and without the copy
        {"name": "norm_odd", "op": "norm", "R": 1021, "H": 5003, "delta": False, "group": -1},
        # the rows of one draft step and its verification, 16 sequences
        {"name": "cache_step", "op": "cache", "B": 16, "T": 61, "heads": 8, "D": 128, "page": 64},
        # four prompts
        {"name": "cache_prompt", "op": "cache", "B": 4, "T": 16384, "heads": 8, "D": 128, "page": 64},
        # one sequence, one row, a short context: a step that is all latency
        {"name": "attend_1", "op": "attend", "B": 1, "Q": 1, "kv": 8, "G": 6, "D": 128, "page": 64, "L": 2048},
        # a draft step of 16 sequences with long contexts of different lengths
        {"name": "attend_16", "op": "attend", "B": 16, "Q": 1, "kv": 8, "G": 6, "D": 128, "page": 64, "L": 32768},
        # the verification of 4 drafts of 16 sequences
        {"name": "attend_verify", "op": "attend", "B": 16, "Q": 5, "kv": 8, "G": 6, "D": 128, "page": 64, "L": 16384},
        # small heads, one key head for each query head, small pages
        {"name": "attend_mha", "op": "attend", "B": 7, "Q": 2, "kv": 16, "G": 1, "D": 64, "page": 16, "L": 5000},
        # short prompts of odd lengths, small heads
        {"name": "prompt_short", "op": "prompt", "B": 9, "T": 1003, "kv": 4, "G": 4, "D": 64},
        # prompts packed into one batch
        {"name": "prompt_packed", "op": "prompt", "B": 8, "T": 16384, "kv": 8, "G": 6, "D": 128},
        # one long prompt
        {"name": "prompt_long", "op": "prompt", "B": 1, "T": 16384, "kv": 8, "G": 6, "D": 128},
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "cache", "attend", "prompt"])
    if op == "norm":
        return {"op": op, "R": _between(rng, 1, 4096), "H": _between(rng, 64, 6144), "delta": rng.random() < 0.7,
                "group": rng.choice([-1, 0, 0, 128])}
    D = rng.choice([64, 128, 128])
    if op == "cache":
        B = _between(rng, 1, 32)
        return {"op": op, "B": B, "T": _between(rng, max(B, 8), 16384), "heads": rng.choice([1, 2, 4, 8]), "D": D,
                "page": rng.choice([16, 32, 64, 128])}
    kv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    if op == "attend":
        B, Q = _between(rng, 1, 16), rng.choice([1, 1, 1, 2, 3, 5, 8])
        top = max(2048, min(32768, 16 * 32768 * 48 // (B * Q * kv * G)))
        return {"op": op, "B": B, "Q": Q, "kv": kv, "G": G, "D": D, "page": rng.choice([16, 32, 64, 128]),
                "L": _between(rng, 16, top)}
    B = _between(rng, 1, 16)
    return {"op": op, "B": B, "T": _between(rng, max(B, 16), 16384), "kv": kv, "G": min(G, 6), "D": D}


def _lengths(c):
    """Lengths of the case's sequences: they differ, and are the same for every seed."""
    B = c["B"]
    share = [1.0 + 0.75 * math.cos(2.4 * i) for i in range(B)]
    if c["op"] == "attend":  # L is the longest
        return [max(c["Q"], int(c["L"] * s / max(share))) for s in share]
    n = [max(1, int(c["T"] * s / sum(share))) for s in share]  # T is the total
    n[0] += c["T"] - sum(n)
    while n[0] < 1:  # (many short sequences: the longest gives)
        i = n.index(max(n))
        n[i] -= 1
        n[0] += 1
    return n


def work(c):
    if c["op"] == "norm":
        n = c["R"] * c["H"]
        each = 2 + 2 + (4 if c["delta"] else 0) + (1 if c["group"] >= 0 else 0)
        scales = 0 if c["group"] < 0 else 4 * c["R"] * (1 if c["group"] == 0 else -(-c["H"] // c["group"]))
        return {"bytes": n * each + 2 * c["H"] + scales, "flops": 6 * n}
    D = c["D"]
    row = D // 2 + D // BLOCK + 4  # bytes of a token's key (or value) in the cache, one head
    if c["op"] == "cache":
        n = 2 * c["T"] * c["heads"]
        return {"bytes": 2 * n * (2 * D + row), "flops": 4 * n * D}
    hq = c["kv"] * c["G"]
    if c["op"] == "attend":
        tokens = sum(_lengths(c))
        return {"bytes": 2 * tokens * c["kv"] * row + c["B"] * c["Q"] * hq * (4 * D + 4),
                "flops": 4 * D * hq * sum(c["Q"] * n - c["Q"] * (c["Q"] - 1) // 2 for n in _lengths(c))}
    return {"bytes": c["T"] * (2 * hq + 2 * c["kv"]) * D * 2 + 4 * c["T"] * hq,
            "flops": 4 * D * hq * sum(n * (n + 1) // 2 for n in _lengths(c))}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(c, lens, g):
    """Pages of each sequence in a pool that serves them all, handed out in no order."""
    need = [-(-n // c["page"]) for n in lens]
    perm = torch.randperm(sum(need), generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need)


def _filled_cache(pages, heads, page, D, g):
    """A cache as earlier steps left it: Gaussian keys and values with a few large channels, quantised."""
    q = torch.empty((pages, 2, heads, page, D // 2), dtype=torch.uint8, device=DEV)
    bs = torch.empty((pages, 2, heads, page, D // BLOCK), dtype=torch.uint8, device=DEV)
    rs = torch.empty((pages, 2, heads, page), dtype=torch.float32, device=DEV)
    channel = 1.0 + 2.0 * (torch.rand((2, heads, 1, D), generator=g, device=DEV) < 0.03)
    channel[1] = 1.0
    step = max(1, (1 << 26) // (2 * heads * page * D))
    for i in range(0, pages, step):  # slices keep the 32-bit copies small
        n = min(step, pages - i)
        w = (torch.randn((n, 2, heads, page, D), generator=g, device=DEV) * channel).bfloat16().float()
        r = w.abs().amax(4) / 2688.0
        b = w.view(n, 2, heads, page, -1, BLOCK)
        s = (b.abs().amax(5) / (6.0 * r).unsqueeze(4)).clamp(max=448.0).to(torch.float8_e4m3fn)
        y = (b.abs() / (s.float() * r.unsqueeze(4)).clamp(min=1e-30).unsqueeze(5)).clamp(max=6.0)
        code = torch.bucketize(y, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV))
        code = (code + 8 * (b < 0)).to(torch.uint8).view(n, 2, heads, page, D)
        q[i:i + n] = code[..., 0::2] | (code[..., 1::2] << 4)
        bs[i:i + n] = s.view(torch.uint8)
        rs[i:i + n] = r
    return q, bs, rs


def prepare(c, seed):
    g = _gen(seed)
    s = {"case": c, "kept": {}}
    rand = lambda *shape: torch.randn(shape, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "norm":
        s["x"] = (rand(c["R"], c["H"]) * 3.0).bfloat16()
        s["delta"] = rand(c["R"], c["H"]).bfloat16() if c["delta"] else None
        s["w"] = (1.0 + 0.1 * rand(c["H"])).bfloat16()
        return s
    lens = s["lens"] = _lengths(c)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    D = c["D"]
    if c["op"] == "cache":
        # (the rows of one projection: keys and values side by side, as it leaves them)
        kv = (rand(c["T"], 2, c["heads"], D) * (1.0 + 2.0 * (torch.rand((D,), generator=g, device=DEV) < 0.03))).bfloat16()
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        before = [(37 * b) % 200 for b in range(c["B"])]  # tokens that each sequence holds already
        s["table"], pages = _table(c, [n + p for n, p in zip(lens, before)], g)
        s["starts"], s["at"] = _i32(starts), _i32(before)
        s["cache"] = (torch.zeros((pages, 2, c["heads"], c["page"], D // 2), dtype=torch.uint8, device=DEV),
                      torch.zeros((pages, 2, c["heads"], c["page"], D // BLOCK), dtype=torch.uint8, device=DEV),
                      torch.zeros((pages, 2, c["heads"], c["page"]), dtype=torch.float32, device=DEV))
        return s
    hq = c["kv"] * c["G"]
    if c["op"] == "attend":
        s["q"] = (rand(c["B"], c["Q"], hq, D) * 1.5).bfloat16()
        s["table"], pages = _table(c, lens, g)
        s["length"] = _i32(lens)
        s["cache"] = _filled_cache(pages, c["kv"], c["page"], D, g)
        return s
    # queries, keys and values side by side, as one projection leaves them
    qkv = rand(c["T"], hq + 2 * c["kv"], D).bfloat16()
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + c["kv"]], qkv[:, hq + c["kv"]:]
    s["starts"] = _i32(starts)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _round(x, bits, low):
    """x (64 bits) to `bits` significant bits, no finer than 2^(low - bits + 1), ties to even."""
    e = (torch.frexp(x)[1] - 1).clamp(min=low) - (bits - 1)
    step = ((e.long() + 1023) << 52).view(torch.float64)  # 2^e, exactly
    return torch.round(x / step) * step


def _plain_norm(s):
    c = s["case"]
    x = s["x"].double()  # 64 bits: the results are rounded to few bits, next to whose borders 32 decide otherwise
    if s["delta"] is not None:
        x = _round(x + s["delta"].double(), 8, -126)
    y = _round(x * s["w"].double() / torch.sqrt((x * x).mean(1, keepdim=True) + EPS), 8, -126).float()
    out = {"y": y.bfloat16()}
    if s["delta"] is not None:
        out["total"] = x.bfloat16()
    if c["group"] >= 0:
        n = c["group"] or c["H"]
        p = torch.nn.functional.pad(y, (0, -c["H"] % n)).view(c["R"], -1, n)
        scale = p.abs().amax(2) / 448.0
        q = p / torch.where(scale > 0, scale, 1.0).unsqueeze(2)
        out["q"] = q.reshape(c["R"], -1)[:, :c["H"]].clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out["scale"] = scale if c["group"] else scale.view(-1)
    return out


def _fp4(w):
    """The FP4 copy of rows [..., D] as values in 64 bits: code * block scale * row scale."""
    b = w.double().unflatten(-1, (-1, BLOCK))
    r = (b.abs().amax((-2, -1)) / 2688.0).float().double().unsqueeze(-1)
    s = b.abs().amax(-1) / torch.where(r > 0, 6.0 * r, 1.0)
    s = torch.where(r > 0, _round(s, 4, -6).clamp(max=448.0), 0.0)
    d = (s * r).unsqueeze(-1)
    code = _round(b / torch.where(d > 0, d, 1.0), 2, 0).clamp(-6.0, 6.0)
    return (torch.where(d > 0, code, 0.0) * d).flatten(-2)


def _plain_cache(s):
    c = s["case"]
    # where each row goes: its sequence's page, and its place in it
    row = torch.arange(c["T"], device=DEV)
    b = torch.bucketize(row, s["starts"][1:].long(), right=True)
    at = s["at"].long()[b] + row - s["starts"].long()[b]
    page, off = s["table"].long()[b, at // c["page"]], at % c["page"]
    held = torch.zeros((s["cache"][0].shape[0], c["page"], 2, c["heads"], c["D"]), device=DEV)
    held[page, off, 0] = _fp4(s["k"]).float()
    held[page, off, 1] = _fp4(s["v"]).float()
    return {"k": held[page, off, 0].bfloat16(), "v": held[page, off, 1].bfloat16()}


def _unpack(q, bs, rs):
    """Cached rows as 32-bit values [..., D]."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=DEV)
    v = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), -1).flatten(-2).unflatten(-1, (-1, BLOCK))
    return (v * bs.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2) * rs.unsqueeze(-1)


def _softmax(a):
    """Weights and the logarithm of their sum for scores [..., keys], -inf where masked."""
    m = a.amax(-1, keepdim=True)
    w = torch.exp(a - m)
    z = w.sum(-1, keepdim=True)
    return w / z, (m + torch.log(z)).squeeze(-1)


def _plain_attend(s):
    c = s["case"]
    Q, kv, G, D, page = c["Q"], c["kv"], c["G"], c["D"], c["page"]
    q, bs, rs = s["cache"]
    out, lse = [], []
    for b, n in enumerate(s["lens"]):
        at = s["table"][b, :-(-n // page)].long()
        held = _unpack(q[at], bs[at], rs[at]).permute(1, 2, 0, 3, 4).reshape(2, kv, -1, D)[:, :, :n]
        x = s["q"][b].float().view(Q, kv, G, D).permute(1, 0, 2, 3).reshape(kv, Q * G, D)
        a = (x @ held[0].transpose(1, 2) / math.sqrt(D)).view(kv, Q, G, n)
        last = n - Q + torch.arange(Q, device=DEV).view(1, Q, 1, 1)
        a = a.masked_fill(torch.arange(n, device=DEV) > last, float("-inf"))
        w, z = _softmax(a)
        o = (w.view(kv, Q * G, n) @ held[1]).view(kv, Q, G, D)
        out.append(o.permute(1, 0, 2, 3).reshape(Q, kv * G, D))
        lse.append(z.permute(1, 0, 2).reshape(Q, kv * G))
    return {"out": torch.stack(out).bfloat16(), "lse": torch.stack(lse)}


def _plain_prompt(s):
    c = s["case"]
    out = torch.empty((c["T"], c["kv"] * c["G"], c["D"]), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((c["T"], c["kv"] * c["G"]), device=DEV)
    at = 0
    for n in s["lens"]:
        for h in range(c["kv"] * c["G"]):  # head by head: a long prompt's scores are large
            k, v = s["k"][at:at + n, h // c["G"]].float(), s["v"][at:at + n, h // c["G"]].float()
            for i in range(0, n, 4096):
                j = min(n, i + 4096)
                a = s["q"][at + i:at + j, h].float() @ k[:j].t() / math.sqrt(c["D"])
                a.masked_fill_(torch.arange(j, device=DEV) > torch.arange(i, j, device=DEV).view(-1, 1), float("-inf"))
                w, z = _softmax(a)
                out[at + i:at + j, h] = (w @ v[:j]).bfloat16()
                lse[at + i:at + j, h] = z
        at += n
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------------------------- the library's calls
def _kept(s, name, make):
    """A buffer that a user's program makes once and uses for every call."""
    if name not in s["kept"]:
        s["kept"][name] = make()
    return s["kept"][name]


def _own(s):
    import mtp_speculative_draft_head_gb300 as m
    c = s["case"]
    buf = lambda name, shape, dtype: _kept(s, name, lambda: torch.empty(shape, dtype=dtype, device=DEV))  # noqa: E731
    if c["op"] == "norm":
        R, H = c["R"], c["H"]
        y = buf("y", (R, H), torch.bfloat16)
        total = buf("total", (R, H), torch.bfloat16) if c["delta"] else None
        q = scale = status = None
        if c["group"] >= 0:
            q = buf("q", (R, H), torch.uint8)
            scale = buf("scale", (R, -(-H // c["group"])) if c["group"] else (R,), torch.float32)
            status = _kept(s, "status", lambda: torch.zeros(1, dtype=torch.int32, device=DEV))
        m.mtp_head_norm_residual(s["x"], s["w"], s["delta"], total, y, q, scale, status, group=max(c["group"], 0), eps=EPS)
        out = {"y": y}
        if c["delta"]:
            out["total"] = total
        if c["group"] >= 0:
            out["q"], out["scale"] = q.view(torch.float8_e4m3fn), scale
        return out
    if c["op"] == "cache":
        shape = (c["T"], c["heads"], c["D"])
        k, v = buf("k", shape, torch.bfloat16), buf("v", shape, torch.bfloat16)
        m.mtp_head_cache_write_fp4(s["k"], s["v"], s["starts"], s["at"], s["table"], *s["cache"])
        m.mtp_head_cache_read_fp4(*s["cache"], s["starts"], s["at"], s["table"], k, v)
        return {"k": k, "v": v}
    hq = c["kv"] * c["G"]
    if c["op"] == "attend":
        B, Q, D = c["B"], c["Q"], c["D"]
        out, lse = buf("out", (B, Q, hq, D), torch.bfloat16), buf("lse", (B, Q, hq), torch.float32)
        ws = _kept(s, "ws", lambda: m.attention_fp4_workspace(B, Q, hq, c["kv"], D, s["table"].shape[1] * c["page"], DEV))
        m.mtp_head_attention_fp4(s["q"], *s["cache"], s["table"], s["length"], out, ws, lse=lse)
        return {"out": out, "lse": lse}
    out, lse = buf("out", (c["T"], hq, c["D"]), torch.bfloat16), buf("lse", (c["T"], hq), torch.float32)
    m.mtp_head_attention_prompt(s["q"], s["k"], s["v"], s["starts"], out, lse=lse)
    return {"out": out, "lse": lse}


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "cache": _plain_cache, "attend": _plain_attend, "prompt": _plain_prompt}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------- 64 bits
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest(y, values):
    """Index of the nearest of the ascending `values` for each y >= 0 (64 bits); a tie goes to the even index."""
    v = torch.tensor(values, dtype=torch.float64, device=y.device)
    mid = (v[1:] + v[:-1]) / 2
    below = torch.bucketize(y, mid, right=False)   # values whose upper midpoint is < y
    upto = torch.bucketize(y, mid, right=True)     # ... <= y: one more on a tie
    return torch.where(below % 2 == 0, below, upto)


def _exact_fp4(x):
    """x [rows, D] -> what its FP4 copy stands for, by tables of the codes' values."""
    a = x.to(torch.float64).reshape(x.shape[0], -1, BLOCK)
    r = (a.abs().reshape(x.shape[0], -1).max(1).values / 2688.0).to(torch.float32).to(torch.float64)[:, None]
    table = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]
    top = a.abs().max(2).values
    s = torch.tensor(table, dtype=torch.float64, device=x.device)[_nearest(top / (6.0 * r).clamp(min=1e-300), table)]
    d = (s * r)[:, :, None]
    code = _nearest(a.abs() / torch.where(d > 0, d, torch.full_like(d, math.inf)), _E2M1)
    return (torch.sign(a) * torch.tensor(_E2M1, dtype=torch.float64, device=x.device)[code] * d).reshape(x.shape)


def _exact_values(q, bs, rs):
    code = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.uint8, device=q.device)
    code[..., 0::2] = q & 15
    code[..., 1::2] = q >> 4
    e = (bs >> 3).to(torch.float64)
    m = (bs & 7).to(torch.float64)
    s = torch.where(e > 0, (8 + m) * torch.exp2(e - 10), m * 2.0 ** -9)
    v = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)[(code & 7).long()]
    return torch.where(code > 7, -v, v) * s.repeat_interleave(BLOCK, -1) * rs.double()[..., None]


def _exact_rows(x, k, v, scale):
    """Rows x [n, D] over the first i + 1 + (keys - n) of the keys, row by row of i."""
    n, j = x.shape[0], k.shape[0]
    a = torch.einsum("nd,jd->nj", x.double(), k.double()) * scale
    a = torch.where(torch.ones((n, j), dtype=torch.bool, device=x.device).tril(j - n), a, torch.full_like(a, -math.inf))
    z = torch.logsumexp(a, 1)
    return torch.einsum("nj,jd->nd", torch.exp(a - z[:, None]), v.double()), z


def _to_bf16(x):
    """64-bit values rounded to 8 significant bits, ties to even, on their bit patterns."""
    b = x.contiguous().view(torch.int64)
    b = b + ((1 << 44) - 1) + ((b >> 45) & 1)
    return ((b >> 45) << 45).view(torch.float64)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "norm":
        x = s["x"].double()
        out = {}
        if s["delta"] is not None:
            x = x + s["delta"].double()
            out["total"] = x
            x = _to_bf16(x)  # the norm is of the BF16 sum
        y = x * s["w"].double() * torch.rsqrt(x.pow(2).sum(1, keepdim=True) / c["H"] + EPS)
        out["y"] = y
        if c["group"] >= 0:
            y = _to_bf16(y)  # the 8-bit copy is of the BF16 rows
            scales, copies = [], []
            for part in torch.split(y, c["group"] or c["H"], 1):
                scales.append(part.abs().max(1).values / 448.0)
                copies.append(part / scales[-1].float().double()[:, None].clamp(min=1e-300))
            out["q"] = torch.cat(copies, 1)
            out["scale"] = torch.stack(scales, 1) if c["group"] else scales[0]
        return {k: out[k] for k in ("y", "total", "q", "scale") if k in out}
    D = c["D"]
    if c["op"] == "cache":
        return {"k": _exact_fp4(s["k"].reshape(-1, D)).view(s["k"].shape),
                "v": _exact_fp4(s["v"].reshape(-1, D)).view(s["v"].shape)}
    hq, scale = c["kv"] * c["G"], 1.0 / math.sqrt(D)
    if c["op"] == "attend":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(s["q"].shape[:3], dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"]):
            at = s["table"][b, :-(-n // c["page"])].long()
            for h in range(c["kv"]):
                k, v = (_exact_values(*(t[at, i, h] for t in s["cache"])).reshape(-1, D)[:n] for i in (0, 1))
                for j in range(h * c["G"], (h + 1) * c["G"]):
                    out[b, :, j], lse[b, :, j] = _exact_rows(s["q"][b, :, j], k, v, scale)
        return {"out": out, "lse": lse}
    out = torch.empty((c["T"], hq, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((c["T"], hq), dtype=torch.float64, device=DEV)
    at = 0
    for n in s["lens"]:
        for h in range(hq):
            k, v = (s[name][at:at + n, h // c["G"]] for name in ("k", "v"))
            for i in range(0, n, 2048):
                j = min(n, i + 2048)
                out[at + i:at + j, h], lse[at + i:at + j, h] = _exact_rows(s["q"][at + i:at + j, h], k[:j], v[:j], scale)
        at += n
    return {"out": out, "lse": lse}
