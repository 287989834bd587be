"""Norm and rotation as a layer, and a block cache with its device buffers.

    rope = NormRope(d, pairs=(22, 21, 21), rows=64, device="cuda")     # (frame, row, column)
    q, k = rope(q, k, grid_positions(T, H, W))            # normed, rotated, [B, heads, N, d]

    cache = BlockCache(B, heads, d, max_tokens, code="e4m3")
    cache.append(k, v)                                    # new tokens of every sequence
    o = cache.attend(q)                                   # q: the newest Tq tokens, causal
    idx, cnt = cache.select(q, cap=64)                    # or: choose blocks for each query ...
    o = cache.attend(q, idx, cnt)                         # ... and attend to those

Each call is the entry point of the same purpose in include/svsa.h on the
current stream, or on `stream`; nothing is copied to the host, so a step
captured into a CUDA graph stays valid while the cache grows.  A call on
`stream` does all its work there, workspaces and allocations included, as under
torch.cuda.stream(stream): it does not wait for the current stream, nor the
current stream for it.
"""
from __future__ import annotations

import contextlib

import torch

from . import (BLOCK, block_cache, cache_query, cache_tokens, norm_rope_params, svsa_cache_append, svsa_cache_attn,
               svsa_cache_attn_workspace_bytes, svsa_cache_select, svsa_qk_norm_rope, svsa_qk_norm_rope_bwd,
               svsa_qk_norm_rope_bwd_workspace_bytes)

_CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def rope_tables(rows: int, pairs, theta: float = 10000.0, device="cuda"):
    """cos and sin, fp32 [rows, d / 2]: pair i of an axis with m pairs turns by position * theta^(-i / m), computed in
    double and rounded once."""
    f = torch.cat([theta ** (-torch.arange(m, dtype=torch.float64) / m) for m in pairs]).to(device)
    angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return angle.cos().float(), angle.sin().float()


def grid_positions(T: int, H: int, W: int, frame: int = 0, device="cuda"):
    """int32 [1, T*H*W, 3]: (frame, row, column) of the tokens of T frames from `frame` on, in raster order."""
    axes = (torch.arange(frame, frame + T), torch.arange(H), torch.arange(W))
    return torch.stack([v.reshape(-1) for v in torch.meshgrid(*axes, indexing="ij")], -1).to(torch.int32).unsqueeze(0).to(device)


@contextlib.contextmanager
def _on(stream, device):
    """Makes `stream` the current one: what is allocated inside belongs to it, so a workspace that a call drops goes to
    no other stream while the call still runs.  The call's outputs are also marked (`keep`) as used by the stream that
    was current, where the caller will use them."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    if stream.device != device:                            # (the tensors' allocations and launches would not be on it)
        raise ValueError(f"the stream is one of {stream.device}, the tensors are on {device}")
    caller = torch.cuda.current_stream(device)

    def keep(*tensors):
        for t in tensors:
            if t is not None:
                t.record_stream(caller)

    with torch.cuda.stream(stream):
        yield keep


class _NormRopeGrad(torch.autograd.Function):
    """NormRope.__call__ with its gradients (svsa_qk_norm_rope_bwd)."""

    @staticmethod
    def forward(ctx, layer, q, k, wq, wk, pos, perm, iperm):
        ctx.layer, ctx.rows = layer, None if perm is None else perm.shape[0]
        ctx.save_for_backward(q, k, wq, wk, pos, iperm)
        return layer._forward(q, k, wq, wk, pos, perm, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gq, gk):
        q, k, wq, wk, pos, iperm = ctx.saved_tensors
        gq, gk = gq.contiguous(), None if k is None else gk.contiguous()
        dq, dk, dwq, dwk = ctx.layer._backward(gq, gk, q, k, wq, wk, pos, iperm, ctx.rows, None)
        return None, dq, dk, None if wq is None else dwq, None if wk is None else dwk, None, None, None


class NormRope:
    """Per-head RMS norm and position rotation of queries and keys (svsa_qk_norm_rope), with its weights and tables.
    Differentiable in q, k and the weights."""

    def __init__(self, d: int, *, pairs=(), rows: int = 0, theta: float = 10000.0, halves: bool = False, eps: float = 1e-6,
                 wq=None, wk=None, device="cuda"):
        """pairs: pairs of each position axis (their sum is d / 2; empty: norm only); rows: positions of the tables
        (0 .. rows - 1).  wq, wk: fp32 [d] weights, ones by default."""
        if pairs and sum(pairs) != d // 2:
            raise ValueError(f"the axes' pairs sum to {sum(pairs)}, not d / 2 = {d // 2}")
        if pairs and rows < 1:
            raise ValueError("rows: the tables need at least one position")
        self.d, self.pairs, self.halves, self.eps = d, tuple(pairs), bool(halves), float(eps)
        self.wq, self.wk = wq, wk
        self.cos, self.sin = rope_tables(rows, self.pairs, theta, device) if pairs else (None, None)

    def params(self, q, k, pos, rows=None):
        return norm_rope_params(q, k, self.cos, pos, rows=rows, pairs=self.pairs, halves=self.halves, eps=self.eps)

    def __call__(self, q, k, pos=None, *, perm=None, iperm=None, out=None, stream=None):
        """q [B, heads_q, N, d], k [B, heads_k, N, d] or None: views with a contiguous last dimension.  perm int32 [rows]:
        token of each output row (-1: zeros).  Returns (yq, yk) [B, heads, rows, d], into `out` if given.

        Where q, k or a weight requires gradients the outputs carry them; with a perm that takes its inverse too (iperm
        int32 [N], the output row of each token, -1 for none; no token may have two), and `out` is not possible.  As with any
        function of torch, drop the eager graphs of the same leaves before a backward is captured into a CUDA graph."""
        if stream is not None:
            with _on(stream, q.device) as keep:
                y = self(q, k, pos, perm=perm, iperm=iperm, out=out)
                if out is None:
                    keep(*y)
                return y
        wq, wk = self.wq, self.wk if k is not None else None
        if torch.is_grad_enabled() and (q.requires_grad or k is not None and k.requires_grad or
                                        wq is not None and wq.requires_grad or wk is not None and wk.requires_grad):
            if out is not None:
                raise RuntimeError("an input requires gradients, which outputs given by the caller cannot carry: leave `out` "
                                   "away, or call under torch.no_grad()")
            if perm is not None and iperm is None:
                raise ValueError("an input requires gradients: with a perm, its inverse iperm is needed")
            return _NormRopeGrad.apply(self, q, k, wq, wk, pos, perm, iperm)
        return self._forward(q, k, wq, wk, pos, perm, out)

    def _forward(self, q, k, wq, wk, pos, perm, out):
        rows = q.shape[2] if perm is None else perm.shape[0]
        if out is None:
            out = tuple(None if x is None else torch.empty((x.shape[0], x.shape[1], rows, x.shape[3]), dtype=x.dtype, device=x.device)
                        for x in (q, k))
        svsa_qk_norm_rope(q, k, wq, wk, self.cos, self.sin, pos, perm, *out, self.params(q, k, pos, rows))
        return out

    def backward(self, gq, gk, q, k, pos=None, *, iperm=None, rows=None, out=None, stream=None):
        """Gradients of a call with these inputs: (dq, dk, dwq, dwk).  iperm int32 [N]: the output row of each token and
        `rows` their number, where the call had a perm.  dq, dk go into `out` if given (views of any strides); dwq, dwk
        are fp32 [d]."""
        if stream is not None:
            with _on(stream, q.device) as keep:
                dx = self.backward(gq, gk, q, k, pos, iperm=iperm, rows=rows, out=out)
                keep(*(dx if out is None else dx[2:]))
                return dx
        return self._backward(gq, gk, q, k, self.wq, self.wk if k is not None else None, pos, iperm, rows, out)

    def _backward(self, gq, gk, q, k, wq, wk, pos, iperm, rows, out):
        p = self.params(q, k, pos, rows)
        if out is None:
            out = tuple(None if x is None else torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in (q, k))
        dw = torch.empty((2, self.d), dtype=torch.float32, device=q.device)
        ws = torch.empty(svsa_qk_norm_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device=q.device)
        dwk = dw[1] if k is not None else None
        svsa_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, self.cos, self.sin, pos, iperm, *out, dw[0], dwk, p, ws, ws.numel())
        return (*out, dw[0], dwk)


class BlockCache:
    """Keys and values of B sequences in 8-bit pages of 64 tokens (struct svsa_cache), with its buffers.  For answering, not
    for training: what it returns carries no gradients."""

    def __init__(self, B: int, heads: int, d: int, max_tokens: int, *, code: str = "e4m3", n_pages: int | None = None,
                 table=None, means: bool = True, device="cuda"):
        """max_tokens: of one sequence.  By default every sequence has pages of its own; for a shared pool give n_pages
        and a table int32 [B, max_blocks] (kept, so its entries may be filled in as pages are handed out: each must be
        set before tokens reach it).  means: keep the key means that `select` needs."""
        blocks = -(-max_tokens // BLOCK)
        if table is None:
            if n_pages is not None and n_pages < B * blocks:
                raise ValueError(f"n_pages={n_pages}: {B * blocks} are needed without a table")
            table = torch.arange(B * blocks, dtype=torch.int32, device=device).view(B, blocks)
        elif n_pages is None:
            raise ValueError("a table needs the number of pages it points into")
        n = B * blocks if n_pages is None else n_pages
        self.code = code
        self.k = torch.zeros((n, heads, BLOCK, d), dtype=torch.uint8, device=device).view(_CODES[code])
        self.v = torch.zeros((n, heads, BLOCK, d), dtype=torch.uint8, device=device).view(_CODES[code])
        self.k_scale = torch.zeros((n, heads), device=device)
        self.v_scale = torch.zeros((n, heads), device=device)
        self.mean = torch.zeros((n, heads, d), dtype=torch.int8, device=device) if means else None
        self.mean_scale = torch.zeros((n, heads), device=device) if means else None
        self.table = table
        self.length = torch.zeros(B, dtype=torch.int32, device=device)
        self._next = torch.zeros_like(self.length)
        self.cache = block_cache(self.k, self.v, self.k_scale, self.v_scale, self.table, self.length, self.mean, self.mean_scale)

    def append(self, k, v, n_new=None, *, stream=None):
        """k, v [B, heads, N, d] (views with a contiguous last dimension); n_new int32 [B]: how many of the N are real.
        The lengths are updated on the same stream."""
        if stream is not None:
            with _on(stream, k.device):
                return self.append(k, v, n_new)
        svsa_cache_append(self.cache, k, v, n_new, self._next, cache_tokens(k, v))
        self.length.copy_(self._next)

    def select(self, q, cap: int, *, first: int = 1, last: int = 1, causal: bool = True, stream=None):
        """Blocks for each query and key head: (idx [B, Tq, heads, cap] ascending, cnt [B, Tq, heads])."""
        if stream is not None:
            with _on(stream, q.device) as keep:
                lists = self.select(q, cap, first=first, last=last, causal=causal)
                keep(*lists)
                return lists
        c = self.cache
        idx = torch.empty((c.B, q.shape[2], c.heads, cap), dtype=torch.int32, device=q.device)
        cnt = torch.empty((c.B, q.shape[2], c.heads), dtype=torch.int32, device=q.device)
        svsa_cache_select(c, q, idx, cnt, cache_query(q, causal=causal, cap=cap, first=first, last=last))
        return idx, cnt

    def attend(self, q, idx=None, cnt=None, *, causal: bool = True, out=None, lse=None, stream=None):
        """Attention of q [B, heads_q, Tq, d] over the cache, or over each query's listed blocks."""
        if stream is not None:
            with _on(stream, q.device) as keep:
                o = self.attend(q, idx, cnt, causal=causal, out=out, lse=lse)
                if out is None:
                    keep(o)
                return o
        p = cache_query(q, causal=causal, cap=0 if idx is None else idx.shape[-1])
        if out is None:
            out = torch.empty_like(q)
        ws = torch.empty(svsa_cache_attn_workspace_bytes(self.cache, p), dtype=torch.uint8, device=q.device)
        svsa_cache_attn(self.cache, q, idx, cnt, out, lse, p, ws, ws.numel())
        return out

    def reset(self, *, stream=None):
        """Empty every sequence; the pages keep what they hold until written again."""
        if stream is not None:
            with _on(stream, self.length.device):
                return self.reset()
        self.length.zero_()
