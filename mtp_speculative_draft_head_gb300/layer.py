"""``DraftLayer``: the attention half of the layer between the head's two stages, as a thin owner of
buffers around the C ABI (include/mtp_head.h).

In the source the drafter runs one decoder layer between the input and the output stage
("glm5next_mtp_head.rs", `forward_one`: the block call over the drafter's own one-layer KV pool). The
head here leaves it out unless it is given one: ``MtpDraftHead.forward(layer=...)`` calls it on the block input. Its
projections run over FP4 copies, its keys and values live in a paged FP4 cache, and what is a model's
own (the rotation of queries and keys, the second half of the layer) is passed in as functions.
"""
from __future__ import annotations

import torch

from . import _lib


def _filled(device) -> None:
    """Waits for the fills of new buffers: calls on any stream may use them from here on."""
    if device.type == "cuda":
        torch.cuda.current_stream(device).synchronize()


def _on(stream, device):
    """The context of a stream as the binding takes it: a torch.cuda.Stream, a raw handle or None (the current one)."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


class LayerCache:
    """A paged FP4 cache of keys and values for ``batch`` sequences of up to ``max_len`` tokens: the three
    arrays, and a table that gives every sequence pages of its own (``table`` may be replaced by one that
    shares or reorders them)."""

    def __init__(self, batch: int, max_len: int, kv_heads: int, head_dim: int, page: int = 64, device=None):
        self.max_pages = -(-max_len // page)
        self.page, self.max_len = page, self.max_pages * page
        self.kv_heads, self.head_dim, self.batch = kv_heads, head_dim, batch
        self.arrays = _lib.cache_empty(batch * self.max_pages, page, kv_heads, head_dim, device)
        self.device = self.arrays[0].device
        self.table = torch.arange(batch * self.max_pages, dtype=torch.int32, device=self.device).view(batch, -1)
        _filled(self.device)

    def write(self, k, v, row_start, position, status=None, stream=None) -> None:
        """Packed rows k, v [T, kv_heads, head_dim] to the sequences' places, as mtp_head_cache_write_fp4."""
        _lib.mtp_head_cache_write_fp4(k, v, row_start, position, self.table, *self.arrays, status, stream)

    def read(self, row_start, position, rows: int, status=None, stream=None):
        """``rows`` packed rows (k, v) back as BF16, as mtp_head_cache_read_fp4 (rows of no sequence: zeros)."""
        with _on(stream, self.device):  # (the fills too)
            k, v = (torch.zeros((rows, self.kv_heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
                    for _ in range(2))
        _lib.mtp_head_cache_read_fp4(*self.arrays, row_start, position, self.table, k, v, status, stream)
        return k, v


class DraftLayer:
    """x <- x + o_proj . attention(qkv_proj . norm(x)), then, with ``mlp``, x <- x + mlp(norm(x)).

    ``norm_w`` [H], ``qkv_proj`` [(q_heads + 2 kv_heads) head_dim, H], ``o_proj`` [H, q_heads head_dim] BF16: the
    projections are copied to FP4 here. ``rotate(q, k, positions)``, if given, rotates the views q
    [R, q_heads, head_dim] and k [R, kv_heads, head_dim] in place (positions [R] int32, never negative and always
    below cache.max_len: rows that have no place there, which the status tells, and rows of no sequence are given the nearest). ``mlp(y, q, q_scale)``, with
    ``mlp_norm_w`` [H], takes the normalised rows in BF16 and in E4M3 (a scale per 128 columns) and returns what is
    added to x. ``max_rows``: rows of a call at most.

    ``status`` [1] int32 takes the errors of calls that are given none (a length or a prompt that the cache does not hold, a
    page that is not there, a NaN or Inf in what is copied): it keeps the first until the caller sets it to 0.

    Its workspaces serve one call at a time: calls of one layer (and replays of graphs that recorded some) follow one
    another, on one stream or ordered by events."""

    def __init__(self, norm_w, qkv_proj, o_proj, q_heads: int, kv_heads: int, cache: LayerCache, eps: float = 1e-6,
                 max_rows: int = 16, rotate=None, mlp=None, mlp_norm_w=None):
        self.H, self.D = norm_w.numel(), cache.head_dim
        self.q_heads, self.kv_heads = q_heads, kv_heads
        width = (q_heads + 2 * kv_heads) * self.D
        if qkv_proj.shape != (width, self.H) or o_proj.shape != (self.H, q_heads * self.D):
            raise ValueError("shapes: qkv_proj [(q_heads + 2 kv_heads) head_dim, H], o_proj [H, q_heads head_dim]")
        if kv_heads != cache.kv_heads:
            raise ValueError("the cache is for another number of key heads")
        if (mlp is None) != (mlp_norm_w is None):
            raise ValueError("mlp and mlp_norm_w go together")
        self.norm_w, self.mlp_norm_w, self.eps = norm_w, mlp_norm_w, float(eps)
        self.cache, self.rotate, self.mlp, self.max_rows = cache, rotate, mlp, max_rows
        dev = self.device = cache.device
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        self.qkv_fp4 = _lib.fp4_empty(width, self.H, dev)
        _lib.mtp_head_quantize_fp4(qkv_proj, *self.qkv_fp4, st)
        self.o_fp4 = _lib.fp4_empty(self.H, q_heads * self.D, dev)
        _lib.mtp_head_quantize_fp4(o_proj, *self.o_fp4, st)
        if int(st.item()) != 0:
            raise _lib.MTPError(int(st.item()), "DraftLayer")
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.ws_qkv = _lib.linear_fp4_workspace(max_rows, width, self.H, dev)
        self.ws_o = _lib.linear_fp4_workspace(max_rows, self.H, q_heads * self.D, dev)
        self.ws_step = {1: self._step_workspace(1)}  # by the rows of a sequence (waits for all fills up to here)

    def _step_workspace(self, Q: int):
        """For steps of Q rows of as many sequences as max_rows and the cache allow."""
        ws = _lib.attention_fp4_workspace(min(self.cache.batch, self.max_rows // Q), Q, self.q_heads, self.kv_heads, self.D,
                                          self.cache.max_len, self.device)
        _filled(self.device)
        return ws

    def _project(self, x, status, stream):
        R = x.shape[0]
        if R > self.max_rows:
            raise ValueError(f"{R} rows, made for {self.max_rows}")
        y = torch.empty_like(x)
        _lib.mtp_head_norm_residual(x, self.norm_w, y=y, eps=self.eps, stream=stream)
        qkv = torch.empty((R, self.q_heads + 2 * self.kv_heads, self.D), dtype=torch.bfloat16, device=self.device)
        _lib.mtp_head_linear_fp4(y, *self.qkv_fp4, qkv.view(R, -1), self.ws_qkv, status, stream)
        return qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)

    def _finish(self, x, heads, status, stream):
        delta = torch.empty_like(x)
        _lib.mtp_head_linear_fp4(heads.view(x.shape[0], -1), *self.o_fp4, delta, self.ws_o, status, stream)
        if self.mlp is None:
            _lib.mtp_head_norm_residual(x, self.norm_w, delta, total=x, eps=self.eps, stream=stream)
            return x
        y = torch.empty_like(x)
        q = torch.empty(x.shape, dtype=torch.uint8, device=self.device)
        scale = torch.empty((x.shape[0], -(-self.H // 128)), dtype=torch.float32, device=self.device)
        _lib.mtp_head_norm_residual(x, self.mlp_norm_w, delta, x, y, q, scale, status, 128, self.eps, stream)
        _lib.mtp_head_norm_residual(x, self.mlp_norm_w, self.mlp(y, q, scale), total=x, eps=self.eps, stream=stream)
        return x

    def step(self, x, length, status=None, stream=None):
        """The layer over the next rows of each sequence, in place: x [B Q, H] (Q rows of each of B sequences, the
        first B of the cache), length [B] int32 (Q at least) the tokens that the cache holds with them. Their keys and values are
        written to the cache first. Every sequence has Q rows (mtp_head_attention_fp4 itself takes fewer of some). The first step of another Q than 1 makes that Q's workspace, waits for its zero fill and is
        not recorded into a graph: the fill would only run with the graph."""
        B = length.numel()
        if B < 1 or x.shape[0] < B or x.shape[0] % B != 0 or B > self.cache.batch:
            raise ValueError("x: an equal number of rows for each sequence of the cache")
        Q = x.shape[0] // B
        if x.shape[0] > self.max_rows:
            raise ValueError(f"{x.shape[0]} rows, made for {self.max_rows}")
        status = self.status if status is None else status
        with _on(stream, self.device):
            if Q not in self.ws_step:
                if torch.cuda.is_current_stream_capturing():
                    raise RuntimeError(f"DraftLayer: make one step of {Q} rows before recording one")
                self.ws_step[Q] = self._step_workspace(Q)
            q, k, v = self._project(x, status, stream)
            starts = torch.arange(0, (B + 1) * Q, Q, dtype=torch.int32, device=self.device)
            first = length - Q
            if self.rotate is not None:
                at = (first.view(-1, 1) + torch.arange(Q, dtype=torch.int32, device=self.device)).view(-1)
                self.rotate(q, k, at.clamp_(0, self.cache.max_len - 1))
            table = self.cache.table[:B]
            _lib.mtp_head_cache_write_fp4(k, v, starts, first, table, *self.cache.arrays, status, stream)
            heads = torch.empty((B, Q, self.q_heads, self.D), dtype=torch.bfloat16, device=self.device)
            _lib.mtp_head_attention_fp4(q.unflatten(0, (B, Q)), *self.cache.arrays, table, length, heads, self.ws_step[Q],
                                        status=status, stream=stream)
            return self._finish(x, heads, status, stream)

    def prompt(self, x, row_start, status=None, stream=None):
        """The layer over whole prompts, in place: x [T, H], sequence b's rows row_start[b] .. row_start[b + 1]
        (row_start [B + 1] int32), from its first position on. Their keys and values fill the cache. The rows attend to them in
        BF16, as they are; steps attend to the cache's FP4 copies, so a row is not quite the same through either. Rows of
        no sequence attend to nothing, but are projected all the same (the status tells a NaN in one)."""
        B = row_start.numel() - 1
        if B < 1 or B > self.cache.batch:
            raise ValueError("row_start: one sequence at least, and no more than the cache has")
        status = self.status if status is None else status
        with _on(stream, self.device):
            q, k, v = self._project(x, status, stream)
            if self.rotate is not None:
                row = torch.arange(x.shape[0], dtype=torch.int32, device=self.device)
                which = torch.bucketize(row, row_start[1:], out_int32=True, right=True).clamp_(max=B - 1)
                self.rotate(q, k, (row - row_start[which.long()]).clamp_(0, self.cache.max_len - 1))
            first = torch.zeros(B, dtype=torch.int32, device=self.device)
            _lib.mtp_head_cache_write_fp4(k, v, row_start, first, self.cache.table[:B], *self.cache.arrays, status, stream)
            heads = torch.zeros((x.shape[0], self.q_heads, self.D), dtype=torch.bfloat16, device=self.device)
            _lib.mtp_head_attention_prompt(q, k, v, row_start, heads, status=status, stream=stream)
            return self._finish(x, heads, status, stream)
