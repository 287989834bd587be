"""Streaming entry points on the GPU against the fp64 oracle: per-head norm and rotation with gradients, the 8-bit block
cache, block selection and attention over the cache.

Tolerances, counted before the first run (u = the output type's half step, finfo.eps / 2):
  * norm and rotation: fp32 throughout.  The sum of d <= 128 squares is a chain of at most 8 + 4 additions, then the
    scale, rsqrtf (2 ulp), two products and a rotation (3 roundings): under 32 roundings of 2^-24, so 2^-19 of the
    pair's length, plus the one rounding of the result, u |y| (2^-25 where an fp16 result is subnormal).
  * its gradients: the same count for each of the two terms, 2^-18 of their sizes, plus u |dx|; dw: fp32 sums of R
    rows, at most (R + 64) 2^-24 of the sum of the terms' sizes.
  * appended codes, scales and means, and selected lists: equal.
  * attention: weights rounded to fp16 (2^-11 each), logits off by less than 2^-13 (fp32 products and sums with
    sum |q k| / sqrt(d) under 2^10 / 16, and the exponent's argument), so (2^-11 + 2^-12) W with W = sum p |v|, plus
    u |o|; the log-sum-exp 2^-13.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_hilbert_b200 as svsa
import oracle
from oracle import stream

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    svsa.lib()


@pytest.fixture(autouse=True)
def _clean():
    yield
    svsa.svsa_sync_status()                                # no test leaves a recorded failure behind unread


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _np(t):
    return t.detach().double().cpu().numpy()


def _half(dtype):
    return torch.finfo(dtype).eps / 2


# ---- norm and rotation --------------------------------------------------------------

def _rope_case(B, hq, hk, N, d, dtype, axes, layout, order, seed=0):
    g = _gen(seed)
    heads = hq + 2 * hk
    if layout == "tokens":                                 # views of a fused projection's output
        qkv = torch.randn(B, N, heads, d, generator=g).mul(1.7).to(dtype).cuda()
        q, k = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hk].transpose(1, 2)
    else:
        q = torch.randn(B, hq, N, d, generator=g).mul(1.7).to(dtype).cuda()
        k = torch.randn(B, hk, N, d, generator=g).to(dtype).cuda()
    pairs = {0: (), 1: (d // 2,), 2: (5, d // 2 - 5), 3: (d // 2 - 2 * (d // 6), d // 6, d // 6)}[axes]
    table = 50
    pos = torch.randint(0, table, (B if axes == 1 else 1, N, axes), generator=g, dtype=torch.int32).cuda() if axes else None
    ang = torch.rand(table, d // 2, generator=g, dtype=torch.float64) * 6 - 3
    cos, sin = (ang.cos().float().cuda(), ang.sin().float().cuda()) if axes else (None, None)
    wq, wk = (1 + 0.3 * torch.randn(d, generator=g)).cuda(), (1 + 0.3 * torch.randn(d, generator=g)).cuda()
    perm = iperm = None
    rows = N
    if order:
        rows = -(-N // 64) * 64
        p = torch.full((rows,), -1, dtype=torch.int32)
        p[:N] = torch.randperm(N, generator=g, dtype=torch.int32)
        ip = torch.empty(N, dtype=torch.int32)
        ip[p[:N].long()] = torch.arange(N, dtype=torch.int32)
        perm, iperm = p.cuda(), ip.cuda()
    return dict(q=q, k=k, wq=wq, wk=wk, cos=cos, sin=sin, pos=pos, perm=perm, iperm=iperm, pairs=pairs, rows=rows)


def _turns(s, B, N, d):
    """cos and sin [B, 1, N, d/2] of every token's pairs, in fp64 from the fp32 tables."""
    if s["cos"] is None:
        return None, None
    axis = np.repeat(np.arange(len(s["pairs"])), s["pairs"])
    pos = s["pos"].cpu().numpy()[:, :, axis]
    pos = np.broadcast_to(pos, (B,) + pos.shape[1:])
    i = np.arange(d // 2)
    return _np(s["cos"])[pos, i][:, None], _np(s["sin"])[pos, i][:, None]


def _rows_out(y, perm):
    if perm is None:
        return y
    p = perm.cpu().numpy()
    out = np.zeros(y.shape[:2] + (len(p), y.shape[3]))
    out[:, :, p >= 0] = y[:, :, p[p >= 0]]
    return out


def _pair_length(y, halves):
    a, b = (y[..., :y.shape[-1] // 2], y[..., y.shape[-1] // 2:]) if halves else (y[..., 0::2], y[..., 1::2])
    n = np.hypot(a, b)
    return np.concatenate([n, n], -1) if halves else np.repeat(n, 2, -1)


ROPE = [
    # B, hq, hk, N, d, dtype, axes, halves, layout, order
    (1, 1, 1, 1, 64, BF, 1, True, "heads", False),
    (3, 8, 2, 1, 128, HF, 1, True, "tokens", False),
    (1, 5, 3, 67, 128, BF, 3, False, "tokens", True),
    (2, 12, 12, 130, 64, HF, 2, False, "heads", True),
    (2, 9, 1, 33, 128, HF, 0, False, "tokens", False),
    (1, 3, 0, 200, 64, BF, 3, True, "heads", True),
    (2, 40, 40, 300, 128, BF, 3, True, "tokens", True),
    (1, 17, 4, 1001, 128, BF, 1, False, "tokens", False),
]


def _rope_run(c, weights=True):
    B, hq, hk, N, d, dtype, axes, halves, layout, order = c
    s = _rope_case(B, hq, hk, N, d, dtype, axes, layout, order, seed=hash((B, hq, N)) % 1000)
    k = s["k"] if hk else None
    w = (s["wq"], s["wk"] if hk else None) if weights else (None, None)
    p = svsa.norm_rope_params(s["q"], k, s["cos"], s["pos"], rows=s["rows"], pairs=s["pairs"], halves=halves, eps=1e-5)
    return s, k, w, p


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("c", ROPE)
def test_norm_rope_matches_the_oracle(c, weights):
    B, hq, hk, N, d, dtype, axes, halves, layout, order = c
    s, k, w, p = _rope_run(c, weights)
    yq = torch.full((B, hq, s["rows"], d), float("nan"), dtype=dtype, device="cuda")
    yk = torch.full((B, hk, s["rows"], d), float("nan"), dtype=dtype, device="cuda") if hk else None
    svsa.svsa_qk_norm_rope(s["q"], k, w[0], w[1], s["cos"], s["sin"], s["pos"], s["perm"], yq, yk, p)
    svsa.svsa_sync_status()
    cos, sin = _turns(s, B, N, d)
    for y, x, wt in ((yq, s["q"], w[0]), (yk, k, w[1])):
        if x is None:
            continue
        ref = _rows_out(stream.norm_rope(_np(x), 1.0 if wt is None else _np(wt), cos, sin, halves, np.float32(1e-5)), s["perm"])
        tol = _half(dtype) * np.abs(ref) * (1 + 2**-7) + 2.0**-19 * _pair_length(ref, halves) + 2.0**-25
        err = np.abs(_np(y) - ref)
        assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("c", ROPE)
def test_norm_rope_gradients_match_the_oracle(c):
    B, hq, hk, N, d, dtype, axes, halves, layout, order = c
    s, k, w, p = _rope_run(c)
    g = _gen(5)
    gq = torch.randn(B, hq, s["rows"], d, generator=g).to(dtype).cuda()
    gk = torch.randn(B, hk, s["rows"], d, generator=g).to(dtype).cuda() if hk else None
    # gradients into views of one buffer with a gap between tokens: the gap stays as it was
    buf = torch.full((B, N, hq + hk + 1, d), 7.0, dtype=dtype, device="cuda")
    dq = buf[:, :, :hq].transpose(1, 2)
    dk = buf[:, :, hq:hq + hk].transpose(1, 2) if hk else None
    dw = torch.full((2, d), float("nan"), device="cuda")
    ws = torch.empty(svsa.svsa_qk_norm_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    args = (gq, gk, s["q"], k, w[0], w[1], s["cos"], s["sin"], s["pos"], s["iperm"])
    svsa.svsa_qk_norm_rope_bwd(*args, dq, dk, dw[0], dw[1] if hk else None, p, ws, ws.numel())
    svsa.svsa_sync_status()
    assert torch.all(buf[:, :, hq + hk] == 7.0)
    cos, sin = _turns(s, B, N, d)
    ip = np.arange(N) if s["iperm"] is None else s["iperm"].cpu().numpy()
    for x, wt, go, dx, dwt in ((s["q"], w[0], gq, dq, dw[0]), (k, w[1], gk, dk, dw[1])):
        if x is None:
            continue
        xs, gs, wn = _np(x), _np(go)[:, :, ip], _np(wt)
        ref, dwr = stream.norm_rope_bwd(gs, xs, wn, cos, sin, halves, np.float32(1e-5))
        r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-5)
        size = _pair_length(gs, halves) * np.abs(wn)
        size = r * (size + np.abs(xs * r) * (size * np.abs(xs * r)).mean(-1, keepdims=True))
        tol = _half(dtype) * np.abs(ref) * (1 + 2**-7) + 2.0**-18 * size + 2.0**-25
        err = np.abs(_np(dx) - ref)
        assert np.all(err <= tol), float((err / tol).max())
        R = dwr[..., 0].size
        terms = (_pair_length(gs, halves) * np.abs(xs * r)).sum((0, 1, 2))
        assert np.all(np.abs(_np(dwt) - dwr.sum((0, 1, 2))) <= (R + 64) * 2.0**-24 * terms)
    # the same call gives the same bits
    again = torch.empty_like(dw)
    dq1 = dq.clone()
    svsa.svsa_qk_norm_rope_bwd(*args, dq, dk, again[0], again[1] if hk else None, p, ws, ws.numel())
    assert torch.equal(dq1, dq) and torch.equal(again[0], dw[0]) and (not hk or torch.equal(again[1], dw[1]))


def test_norm_rope_bwd_without_weight_gradients_and_with_unused_tokens():
    B, h, N, d = 1, 2, 70, 64
    g = _gen(9)
    q = torch.randn(B, h, N, d, generator=g).to(BF).cuda()
    perm = torch.arange(3, 60, dtype=torch.int32).cuda()   # rows of tokens 3 .. 59 only
    iperm = torch.full((N,), -1, dtype=torch.int32)
    iperm[3:60] = torch.arange(57, dtype=torch.int32)
    p = svsa.norm_rope_params(q, None, rows=57)
    y = torch.empty(B, h, 57, d, dtype=BF, device="cuda")
    svsa.svsa_qk_norm_rope(q, None, None, None, None, None, None, perm, y, None, p)
    full = torch.empty(B, h, N, d, dtype=BF, device="cuda")
    svsa.svsa_qk_norm_rope(q, None, None, None, None, None, None, None, full, None, svsa.norm_rope_params(q, None))
    assert torch.equal(y, full[:, :, 3:60])
    gy = torch.randn(B, h, 57, d, generator=g).to(BF).cuda()
    dq = torch.full_like(q, float("nan"))
    ws = torch.empty(svsa.svsa_qk_norm_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    svsa.svsa_qk_norm_rope_bwd(gy, None, q, None, None, None, None, None, None, iperm.cuda(), dq, None, None, None, p, ws,
                               ws.numel())
    svsa.svsa_sync_status()
    assert torch.all(dq[:, :, :3] == 0) and torch.all(dq[:, :, 60:] == 0) and torch.isfinite(dq.float()).all()
    assert torch.count_nonzero(dq[:, :, 3:60]) > 0


def test_norm_rope_takes_the_place_of_the_reorder():
    """With the library's own token order, norm only and no weights, the rows are the reordered rows, normed."""
    T, H, W, h, d = 4, 9, 7, 2, 128
    N = T * H * W
    sh = svsa.shape(1, h, T, H, W, d)
    rows = -(-N // 64) * 64
    q = torch.randn(1, h, N, d, generator=_gen(3)).to(BF).cuda()
    perm, iperm = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(N, dtype=torch.int32, device="cuda")
    ws = torch.empty(svsa.svsa_perm_workspace_bytes(sh, svsa.ORDER_HILBERT), dtype=torch.uint8, device="cuda")
    svsa.svsa_build_perm(sh, svsa.ORDER_HILBERT, perm, iperm, ws, ws.numel())
    y, full, want = (torch.empty(1, h, n, d, dtype=BF, device="cuda") for n in (rows, N, rows))
    svsa.svsa_qk_norm_rope(q, None, None, None, None, None, None, perm, y, None, svsa.norm_rope_params(q, None, rows=rows))
    svsa.svsa_qk_norm_rope(q, None, None, None, None, None, None, None, full, None, svsa.norm_rope_params(q, None))
    svsa.svsa_reorder(full, want, perm, sh)
    assert torch.equal(y, want)


# ---- the cache -----------------------------------------------------------------------

class GpuCache:
    """Cache tensors whose pages hold noise at first, so that a read of a row that is not there shows."""

    def __init__(self, B, heads, d, code, max_blocks, seed=0, spare=3, lens=None):
        g = _gen(seed)
        n = B * max_blocks + spare
        dt = torch.float8_e4m3fn if code == "e4m3" else torch.int8
        self.code, self.B, self.heads, self.d = code, B, heads, d
        noise = lambda: torch.randint(0, 256, (n, heads, 64, d), generator=g, dtype=torch.uint8).cuda()
        self.k, self.v = noise().view(dt), noise().view(dt)
        self.k.view(torch.uint8)[:, :, 1::2] = 0x7F        # NaN in e4m3
        self.v.view(torch.uint8)[:, :, 1::2] = 0x7F
        self.k_scale, self.v_scale, self.mean_scale = (torch.full((n, heads), float("nan"), device="cuda") for _ in range(3))
        self.mean = torch.randint(-128, 128, (n, heads, d), generator=g, dtype=torch.int8).cuda()
        self.table = torch.randperm(n, generator=g, dtype=torch.int32)[:B * max_blocks].view(B, max_blocks).cuda()
        self.len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.c = svsa.block_cache(self.k, self.v, self.k_scale, self.v_scale, self.table, self.len, self.mean, self.mean_scale)

    def append(self, k, v, n_new=None):
        out = torch.empty_like(self.len)
        svsa.svsa_cache_append(self.c, k, v, n_new, out, svsa.cache_tokens(k, v))
        self.len.copy_(out)

    def oracle(self):
        cpu = [t.cpu().numpy() for t in (self.k.view(torch.uint8), self.v.view(torch.uint8), self.k_scale, self.v_scale,
                                         self.mean, self.mean_scale, self.table, self.len)]
        return stream.BlockCache(*cpu, self.code)

    def attend(self, q, causal=True, idx=None, cnt=None, lse=True):
        p = svsa.cache_query(q, causal=causal, cap=0 if idx is None else idx.shape[-1])
        o = torch.full_like(q, 99.0)
        l = torch.full(q.shape[:3], 99.0, device="cuda") if lse else None
        ws = torch.full((svsa.svsa_cache_attn_workspace_bytes(self.c, p),), 0xFF, dtype=torch.uint8, device="cuda")
        svsa.svsa_cache_attn(self.c, q, idx, cnt, o, l, p, ws, ws.numel())
        return o, l

    def select(self, q, cap, first=0, last=0, causal=True):
        idx = torch.full((self.B, q.shape[2], self.heads, cap), -5, dtype=torch.int32, device="cuda")
        cnt = torch.full(idx.shape[:3], -5, dtype=torch.int32, device="cuda")
        svsa.svsa_cache_select(self.c, q, idx, cnt, svsa.cache_query(q, causal=causal, cap=cap, first=first, last=last))
        return idx, cnt


def _tokens(g, B, heads, N, d, dtype, layout="heads", scale=1.0):
    x = torch.randn(B, N, 2 * heads + 1, d, generator=g).mul(scale).to(dtype).cuda()
    k, v = x[:, :, :heads].transpose(1, 2), x[:, :, heads:2 * heads].transpose(1, 2)
    return (k, v) if layout == "tokens" else (k.contiguous(), v.contiguous())


def _same_cache(gpu, ref, what):
    assert np.array_equal(gpu.len.cpu().numpy(), ref.len), what
    for name in ("k", "v"):
        assert np.count_nonzero(getattr(gpu, name).view(torch.uint8).cpu().numpy() != getattr(ref, name)) == 0, (what, name)
    assert np.count_nonzero(gpu.mean.cpu().numpy() != ref.mean) == 0, what
    for name in ("k_scale", "v_scale", "mean_scale"):
        assert np.array_equal(_np(getattr(gpu, name)), getattr(ref, name), equal_nan=True), (what, name)


@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF), (128, BF)])
def test_appending_in_pieces_matches_the_oracle(code, d, dtype):
    B, heads = 3, 2
    gpu = GpuCache(B, heads, d, code, 8)
    ref = gpu.oracle()
    g = _gen(1)
    # (tokens, how many of each sequence's are real, size of the values)
    steps = [(1, None, 1.0), (1, None, 8.0), (62, [62, 0, 1], 0.5), (65, [65, 64, 63], 20.0), (130, [130, 5, 129], 1.0),
             (1, [0, 0, 0], 1.0), (3, None, 1e-3), (3, None, 0.0), (64, [64, 64, 0], 3e-7), (17, None, 100.0)]
    for i, (N, real, scale) in enumerate(steps):
        k, v = _tokens(g, B, heads, N, d, dtype, "tokens" if i % 2 else "heads", scale)
        n_new = None if real is None else torch.tensor(real, dtype=torch.int32)
        gpu.append(k, v, None if real is None else n_new.cuda())
        ref.append(_np(k), _np(v), [N] * B if real is None else real)
        svsa.svsa_sync_status()
        _same_cache(gpu, ref, i)


def test_append_fills_the_table_to_its_end_and_without_means():
    B, heads, d = 1, 1, 64
    gpu = GpuCache(B, heads, d, "i8", 2)
    ref = gpu.oracle()
    gpu.c = svsa.block_cache(gpu.k, gpu.v, gpu.k_scale, gpu.v_scale, gpu.table, gpu.len)
    k, v = _tokens(_gen(2), B, heads, 128, d, BF)
    gpu.append(k, v)
    svsa.svsa_sync_status()
    before, scale = ref.mean.copy(), ref.mean_scale.copy()
    ref.append(_np(k), _np(v), [128])
    ref.mean, ref.mean_scale = before, scale               # not kept, so not touched
    _same_cache(gpu, ref, "full")


def test_append_saturates_values_that_are_not_finite():
    gpu = GpuCache(1, 1, 64, "e4m3", 1)
    k, v = _tokens(_gen(4), 1, 1, 5, 64, BF)
    k[0, 0, 1, 3], k[0, 0, 2, 4], v[0, 0, 0, 0] = float("inf"), float("-inf"), float("nan")
    ref = gpu.oracle()
    clean = _np(k), _np(v)
    fin = np.where(np.isfinite(clean[0]), clean[0], 0), np.where(np.isfinite(clean[1]), clean[1], 0)
    ref.append(*fin, [5])
    gpu.append(k, v)
    with pytest.raises(svsa.SvsaError) as e:
        svsa.svsa_sync_status()
    assert e.value.status == 6
    svsa.svsa_sync_status()                                # reported once
    got = gpu.oracle()
    page = int(gpu.table[0, 0])
    assert np.array_equal(got.k_scale, ref.k_scale, equal_nan=True) and np.array_equal(got.v_scale, ref.v_scale, equal_nan=True)
    kk, vv = got.tokens(0, 0)
    s = got.k_scale[page, 0]
    assert kk[1, 3] == 448 * s and kk[2, 4] == -448 * s and vv[0, 0] == 0
    kr, vr = ref.tokens(0, 0)
    kk[1, 3] = kk[2, 4] = 0
    assert np.array_equal(kk, kr) and np.array_equal(vv, vr)


# ---- attention over the cache ------------------------------------------------------------

def _check_attention(gpu, q, o, lse, causal, lists=None):
    ref, rl = stream.cache_attention(gpu.oracle(), _np(q), causal, lists)
    # W = sum p |v|: the same attention over |v|
    a = gpu.oracle()
    if a.code == "i8":
        a.v = np.abs(a.v.view(np.int8).astype(np.int16)).astype(np.uint8)
    else:
        a.v = a.v & 0x7F
    w, _ = stream.cache_attention(a, _np(q), causal, lists)
    tol = (2.0**-11 + 2.0**-12) * np.abs(w) + _half(q.dtype) * np.abs(ref) * (1 + 2**-7) + 2.0**-25
    err = np.abs(_np(o) - ref)
    assert np.all(err <= tol), float((err / tol).max())
    if lse is not None:
        got = _np(lse)
        assert np.array_equal(np.isinf(got), np.isinf(rl)) and np.all(got[np.isinf(rl)] == -np.inf)
        fin = np.isfinite(rl)
        assert np.all(np.abs(got[fin] - rl[fin]) <= 2.0**-13 + 2.0**-20 * np.abs(rl[fin]))
    return ref, rl


def _filled(B, heads, d, code, lens, dtype=BF, seed=0, blocks=None):
    gpu = GpuCache(B, heads, d, code, blocks or max(1, -(-max(lens) // 64)), seed=seed)
    if max(lens):
        k, v = _tokens(_gen(seed + 100), B, heads, max(lens), d, dtype)
        gpu.append(k, v, torch.tensor(lens, dtype=torch.int32).cuda())
    return gpu


ATTN = [
    # lens, heads, group, Tq, d, dtype, code
    ([1], 1, 1, 1, 128, BF, "e4m3"),
    ([0, 5], 2, 4, 1, 64, HF, "i8"),
    ([64, 63, 65, 0], 2, 8, 1, 128, HF, "i8"),
    ([777, 1, 130], 1, 5, 3, 128, BF, "i8"),
    ([2000], 2, 16, 1, 128, BF, "e4m3"),
    ([300, 640], 1, 20, 1, 64, BF, "e4m3"),
    ([1500, 20], 3, 2, 17, 128, HF, "e4m3"),
    ([513, 700, 3, 64, 65], 2, 1, 8, 64, HF, "i8"),
    ([100, 40], 1, 3, 33, 128, BF, "i8"),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads,group,Tq,d,dtype,code", ATTN)
def test_attention_matches_the_oracle(lens, heads, group, Tq, d, dtype, code, causal):
    B = len(lens)
    gpu = _filled(B, heads, d, code, lens, blocks=-(-max(lens) // 64) + 2)
    q = torch.randn(B, heads * group, Tq, d, generator=_gen(7)).to(dtype).cuda()
    o, lse = gpu.attend(q, causal)
    svsa.svsa_sync_status()
    _check_attention(gpu, q, o, lse, causal)
    again, _ = gpu.attend(q, causal, lse=False)
    assert torch.equal(o, again)


def test_attention_with_scales_of_any_size():
    """Blocks whose scales differ by many powers of two, and are no powers of two."""
    gpu = _filled(1, 1, 128, "i8", [640])
    pages = gpu.table[0, :10].long()
    gpu.v_scale[pages, 0] = torch.tensor([3e-20, 1e10, 0.3, 1.7e-5, 0.0, 2.0, 1e-30, 5e9, 1.0, 0.01], device="cuda")
    gpu.k_scale[pages, 0] *= torch.tensor([1.1, 0.0, 0.9, 1.3, 1.0, 0.7, 1.0, 0.33, 1.0, 1.9], device="cuda")
    q = torch.randn(1, 3, 1, 128, generator=_gen(8)).to(BF).cuda()
    o, lse = gpu.attend(q)
    _check_attention(gpu, q, o, lse, True)


def test_attention_over_one_dominant_key():
    """Logits far apart: the weights of all but one key vanish, whatever block it is in."""
    gpu = _filled(1, 1, 64, "e4m3", [300])
    q = torch.randn(1, 2, 1, 64, generator=_gen(9)).mul(40).to(HF).cuda()
    o, lse = gpu.attend(q)
    ref, rl = stream.cache_attention(gpu.oracle(), _np(q), True)
    assert np.abs(rl).max() > 40
    # logits of size L are off by less than 2^-18 L here, and so are the weights' exponents
    w = np.abs(gpu.oracle().tokens(0, 0)[1]).max()
    assert np.abs(_np(o) - ref).max() <= (2.0**-11 + 2.0**-17 * np.abs(rl).max()) * w
    assert np.abs(_np(lse) - rl).max() <= 2.0**-17 * np.abs(rl).max()


def test_query_rows_of_any_size_and_rows_that_are_not_finite():
    gpu = _filled(1, 2, 128, "e4m3", [200])
    q = torch.randn(1, 8, 1, 128, generator=_gen(10)).to(BF)
    for h, f in enumerate((1e-30, 1e-5, 0.0, 1.0)):
        q[0, h] *= f
    q[0, 5, 0, 7], q[0, 6, 0, 100] = float("inf"), float("nan")
    q = q.cuda()
    o, lse = gpu.attend(q)
    good = [0, 1, 2, 3, 4, 7]
    ref, rl = stream.cache_attention(gpu.oracle(), np.where(np.isfinite(_np(q)), _np(q), 0), True)
    w = np.abs(np.stack([gpu.oracle().tokens(0, h)[1] for h in range(2)])).max()
    assert np.abs(_np(o) - ref)[0, good].max() <= (2.0**-11 + 2.0**-12 + 2.0**-8) * w
    assert np.abs(_np(lse) - rl)[0, good].max() <= 2.0**-13
    assert torch.isnan(o[0, [5, 6]]).all() and torch.isnan(lse[0, [5, 6]]).all()


def test_long_cache_beyond_32_bit_offsets():
    """Pages whose byte offsets pass 2^31 and 2^32."""
    heads, d, n = 8, 128, 70000                            # 4.6 GB of codes for keys, and for values
    k = torch.empty(n, heads, 64, d, dtype=torch.int8, device="cuda")
    v = torch.empty_like(k)
    ks, vs, ms = (torch.zeros(n, heads, device="cuda") for _ in range(3))
    mean = torch.zeros(n, heads, d, dtype=torch.int8, device="cuda")
    table = torch.tensor([[n - 1, 1, 33000, 66000], [32768, 65536, 2, n - 2]], dtype=torch.int32, device="cuda")
    length = torch.zeros(2, dtype=torch.int32, device="cuda")
    small = _filled(2, heads, d, "i8", [250, 130], blocks=4)
    c = svsa.block_cache(k, v, ks, vs, table, length, mean, ms)
    kn, vn = _tokens(_gen(100), 2, heads, 250, d, BF)
    new = torch.tensor([250, 130], dtype=torch.int32, device="cuda")
    out = torch.empty_like(length)
    svsa.svsa_cache_append(c, kn, vn, new, out, svsa.cache_tokens(kn, vn))
    length.copy_(out)
    q = torch.randn(2, 16, 2, d, generator=_gen(11)).to(BF).cuda()
    o, lse = small.attend(q)
    p = svsa.cache_query(q, cap=2, last=1)
    ws = torch.empty(svsa.svsa_cache_attn_workspace_bytes(c, p), dtype=torch.uint8, device="cuda")
    o2, l2 = torch.empty_like(o), torch.empty_like(lse)
    svsa.svsa_cache_attn(c, q, None, None, o2, l2, p, ws, ws.numel())
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    idx, cnt = small.select(q, 2, last=1)
    i2, c2 = torch.empty_like(idx), torch.empty_like(cnt)
    svsa.svsa_cache_select(c, q, i2, c2, p)
    assert torch.equal(idx, i2) and torch.equal(cnt, c2)
    svsa.svsa_sync_status()


# ---- lists ----------------------------------------------------------------------------------

def _lists(idx, cnt):
    i, n = idx.cpu().numpy(), cnt.cpu().numpy()
    out = np.empty(n.shape, dtype=object)
    for at in np.ndindex(n.shape):
        out[at] = list(i[at][:n[at]])
    return out


@pytest.mark.parametrize("lens,heads,group,Tq,d,dtype,code", ATTN)
def test_attention_over_lists_matches_the_oracle(lens, heads, group, Tq, d, dtype, code):
    B, cap = len(lens), 6
    gpu = _filled(B, heads, d, code, lens, blocks=-(-max(lens) // 64) + 1)
    rng = np.random.default_rng(3)
    idx = np.full((B, Tq, heads, cap), 12345, dtype=np.int32)          # past cnt: not read
    cnt = np.zeros((B, Tq, heads), dtype=np.int32)
    for b in range(B):
        nb = -(-lens[b] // 64)
        for t in range(Tq):
            for h in range(heads):
                n = int(rng.integers(0, min(cap, nb) + 1))             # empty lists among them
                cnt[b, t, h] = n
                idx[b, t, h, :n] = np.sort(rng.permutation(nb)[:n])
    idx, cnt = torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()
    q = torch.randn(B, heads * group, Tq, d, generator=_gen(12)).to(dtype).cuda()
    for causal in (False, True):
        o, lse = gpu.attend(q, causal, idx, cnt)
        svsa.svsa_sync_status()
        _check_attention(gpu, q, o, lse, causal, _lists(idx, cnt))


def test_lists_of_all_blocks_are_the_whole_cache():
    gpu = _filled(2, 2, 128, "e4m3", [1000, 333])
    q = torch.randn(2, 8, 3, 128, generator=_gen(13)).to(BF).cuda()
    idx = torch.arange(16, dtype=torch.int32, device="cuda").repeat(2, 3, 2, 1)
    cnt = torch.tensor([16, 6], dtype=torch.int32, device="cuda").view(2, 1, 1).repeat(1, 3, 2).contiguous()
    o, lse = gpu.attend(q, True, idx, cnt)
    _check_attention(gpu, q, o, lse, True)


@pytest.mark.parametrize("nb,cap,first,last,group,Tq,d,code", [
    (5, 8, 0, 0, 1, 1, 64, "i8"),           # fewer blocks than entries
    (9, 9, 1, 1, 2, 1, 64, "e4m3"),         # as many
    (40, 1, 0, 0, 3, 2, 128, "i8"),
    (40, 3, 2, 1, 4, 1, 128, "e4m3"),       # every entry forced
    (300, 17, 1, 2, 5, 3, 64, "i8"),        # several CTAs per query
    (1100, 64, 1, 1, 2, 1, 128, "e4m3"),
    (2100, 100, 0, 3, 1, 1, 64, "i8"),
])
def test_selection_matches_the_oracle(nb, cap, first, last, group, Tq, d, code):
    B, heads = 2, 1
    lens = [64 * nb - 13, max(1, 64 * (nb // 2) - 63)]
    gpu = _filled(B, heads, d, code, lens, blocks=nb + 3)
    q = torch.randn(B, heads * group, Tq, d, generator=_gen(14)).to(BF).cuda()
    for causal in (True, False):
        idx, cnt = gpu.select(q, cap, first, last, causal)
        svsa.svsa_sync_status()
        want = stream.select_blocks(gpu.oracle(), _np(q), cap, first, last, causal)
        got = _lists(idx, cnt)
        for at in np.ndindex(got.shape):
            assert got[at] == want[at], at
        tail = torch.arange(cap, device="cuda") >= cnt[..., None]
        assert torch.all(idx[tail] == 0)


@pytest.mark.parametrize("nb", [70, 600, 2500])
def test_selection_breaks_ties_by_the_lower_block(nb):
    gpu = _filled(1, 1, 64, "i8", [64 * nb])
    pages = gpu.table[0, :nb].long()
    gpu.mean[pages, 0] = torch.arange(64, dtype=torch.int8, device="cuda") - 32
    gpu.mean_scale[pages, 0] = 1.0
    gpu.mean[pages[nb // 2], 0] = -gpu.mean[pages[nb // 2], 0]        # one block apart: best for q, worst for -q
    q = torch.arange(64).sub(32).neg().to(BF).view(1, 1, 1, 64).cuda().contiguous()
    idx, cnt = gpu.select(q, 7)
    assert idx[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, nb // 2]
    idx, cnt = gpu.select(-q, 7)
    assert idx[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6]
    # a zero query: every score is equal
    idx, cnt = gpu.select(q * 0, 7, first=0, last=2)
    assert idx[0, 0, 0].tolist() == [0, 1, 2, 3, 4, nb - 2, nb - 1]


# ---- streams, graphs, a run of them together --------------------------------------------------

def test_a_stream_of_frames_eager_and_captured():
    """Norm and rotation, append, selection and attention step by step, as a streaming layer runs them, against the
    oracle's cache; then the same steps replayed from one captured graph: the same bits."""
    B, hq, hk, d, N, steps = 2, 8, 2, 128, 48, 9
    ang = torch.rand(600, d // 2, generator=_gen(20), dtype=torch.float64) * 6
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    qkv_all = torch.randn(steps, B, N, hq + 2 * hk, d, generator=_gen(21)).to(BF).cuda()
    w = (1 + 0.2 * torch.randn(2, d, generator=_gen(22))).cuda()

    qkv = torch.empty_like(qkv_all[0])
    pos = torch.empty(1, N, 1, dtype=torch.int32, device="cuda")
    yq = torch.empty(B, hq, N, d, dtype=BF, device="cuda")
    yk = torch.empty(B, hk, N, d, dtype=BF, device="cuda")
    o, lse = torch.empty_like(yq), torch.empty(B, hq, N, device="cuda")
    q, k, v = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hk].transpose(1, 2), qkv[:, :, hq + hk:].transpose(1, 2)
    rp = svsa.norm_rope_params(q, k, cos, pos, pairs=(d // 2,), halves=True)
    qp = svsa.cache_query(yq, cap=4, first=1, last=1)
    idx = torch.empty(B, N, hk, 4, dtype=torch.int32, device="cuda")
    cnt = torch.empty(B, N, hk, dtype=torch.int32, device="cuda")

    def layer(cache, ws, out_len):
        svsa.svsa_qk_norm_rope(q, k, w[0], w[1], cos, sin, pos, None, yq, yk, rp)
        svsa.svsa_cache_append(cache.c, yk, v, None, out_len, svsa.cache_tokens(yk, v))
        cache.len.copy_(out_len)
        svsa.svsa_cache_select(cache.c, yq, idx, cnt, qp)
        svsa.svsa_cache_attn(cache.c, yq, idx, cnt, o, lse, qp, ws, ws.numel())

    eager, ref = GpuCache(B, hk, d, "e4m3", 8, seed=5), None
    ref = eager.oracle()
    ws = torch.empty(svsa.svsa_cache_attn_workspace_bytes(eager.c, qp), dtype=torch.uint8, device="cuda")
    out_len = torch.empty_like(eager.len)
    kept = []
    for i in range(steps):
        qkv.copy_(qkv_all[i])
        pos.copy_(torch.arange(i * N, i * N + N, dtype=torch.int32).view(1, N, 1))
        layer(eager, ws, out_len)
        svsa.svsa_sync_status()
        ref.append(_np(yk), _np(v), [N] * B)
        _same_cache(eager, ref, i)
        lists = stream.select_blocks(ref, _np(yq), 4, 1, 1, True)
        got = _lists(idx, cnt)
        assert all(got[at] == lists[at] for at in np.ndindex(got.shape))
        _check_attention(eager, yq, o, lse, True, lists)
        kept.append((o.clone(), lse.clone()))

    cap = GpuCache(B, hk, d, "e4m3", 8, seed=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer(cap, ws, out_len)
    for i in range(steps):
        qkv.copy_(qkv_all[i])
        pos.copy_(torch.arange(i * N, i * N + N, dtype=torch.int32).view(1, N, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, kept[i][0]) and torch.equal(lse, kept[i][1]), i
    _same_cache(cap, ref, "captured")


def test_two_streams_at_once():
    gpu = _filled(3, 2, 128, "i8", [5000, 300, 2222])
    q = [torch.randn(3, 8, 1, 128, generator=_gen(s)).to(BF).cuda() for s in (1, 2)]
    want = [gpu.attend(x) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    p = svsa.cache_query(q[0])
    ws = [torch.empty(svsa.svsa_cache_attn_workspace_bytes(gpu.c, p), dtype=torch.uint8, device="cuda") for _ in q]
    out = [torch.empty_like(x) for x in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st, w, o in zip(q, streams, ws, out):
            svsa.svsa_cache_attn(gpu.c, x, None, None, o, None, p, w, w.numel(), stream=st)
    torch.cuda.synchronize()
    for o, (w, _) in zip(out, want):
        assert torch.equal(o, w)


def test_a_page_shared_by_two_sequences():
    gpu = _filled(2, 1, 64, "i8", [128, 128])
    gpu.table[1, 0] = gpu.table[0, 0]                      # the second reads the first's opening block
    q = torch.randn(2, 2, 1, 64, generator=_gen(15)).to(BF).cuda()
    o, lse = gpu.attend(q)
    svsa.svsa_sync_status()
    _check_attention(gpu, q, o, lse, True)


# ---- values read from device memory that lie outside their range ---------------------------------

def _index_error():
    with pytest.raises(svsa.SvsaError) as e:
        svsa.svsa_sync_status()
    assert e.value.status == 8
    svsa.svsa_sync_status()                                # reported once, then cleared


def test_positions_and_map_entries_out_of_range_are_clamped_and_reported():
    N, d = 20, 64
    q = torch.randn(1, 2, N, d, generator=_gen(16)).to(BF).cuda()
    cos = torch.rand(8, 32, generator=_gen(17)).cuda()
    pos = torch.arange(N, dtype=torch.int32).remainder(8).view(1, N, 1)
    p = svsa.norm_rope_params(q, None, cos, pos.cuda(), pairs=(32,))
    run = lambda pos, perm=None: (svsa.svsa_qk_norm_rope(q, None, None, None, cos, cos, pos.cuda(), perm, y, None, p), y.clone())[1]
    y = torch.empty(1, 2, N, d, dtype=BF, device="cuda")
    bad, clamped = pos.clone(), pos.clone()
    bad[0, 3], bad[0, 5], clamped[0, 3], clamped[0, 5] = 8, -1, 7, 0
    got = run(bad)
    _index_error()
    assert torch.equal(got, run(clamped))
    svsa.svsa_sync_status()
    perm = torch.arange(N, dtype=torch.int32).cuda()
    perm[4], perm[6], perm[7] = N, -2, -1                  # (-1 alone is a pad row, not an error)
    got = run(pos, perm)
    _index_error()
    assert torch.all(got[:, :, [4, 6, 7]] == 0) and torch.equal(got[:, :, 8:], run(pos)[:, :, 8:])


def test_pages_and_lengths_out_of_range_are_left_out_and_reported():
    gpu = _filled(2, 1, 64, "i8", [200, 100], blocks=4)
    q = torch.randn(2, 2, 1, 64, generator=_gen(18)).to(BF).cuda()
    good = gpu.table.clone()
    k, v = _tokens(_gen(19), 2, 1, 3, 64, BF)
    for page in (-1, gpu.k.shape[0]):
        gpu.table.copy_(good)
        gpu.table[0, 1] = page                             # block 1 of sequence 0 is not there
        o, lse = gpu.attend(q)
        _index_error()
        gpu.table.copy_(good)
        lists = np.empty((2, 1, 1), dtype=object)
        lists[0, 0, 0], lists[1, 0, 0] = [0, 2, 3], [0, 1]
        _check_attention(gpu, q, o, lse, True, lists)
        # the block that receives tokens: nothing is written
        gpu.table[0, 3] = page
        before = gpu.oracle()
        n = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
        svsa.svsa_cache_append(gpu.c, k, v, n, None, svsa.cache_tokens(k, v))
        _index_error()
        _same_cache(gpu, before, "bad page")
    gpu.table.copy_(good)
    idx, cnt = gpu.select(q, 2)
    svsa.svsa_sync_status()
    # lengths: clamped to [0, 64 max_blocks]
    gpu.len.copy_(torch.tensor([-7, 1 << 20], dtype=torch.int32))
    out = torch.empty_like(gpu.len)
    svsa.svsa_cache_append(gpu.c, k, v, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), out, svsa.cache_tokens(k, v))
    _index_error()
    assert out.tolist() == [0, 256]                        # no room: nothing appended
    svsa.svsa_sync_status()
    gpu.len.copy_(torch.tensor([-7, 100], dtype=torch.int32))
    o, lse = gpu.attend(q)
    _index_error()
    gpu.len.copy_(torch.tensor([0, 100], dtype=torch.int32))
    _check_attention(gpu, q, o, lse, True)
    svsa.svsa_sync_status()


def test_list_entries_that_are_not_ascending_or_past_the_end_are_left_out_and_reported():
    gpu = _filled(1, 1, 64, "e4m3", [300])                 # 5 blocks
    q = torch.randn(1, 2, 1, 64, generator=_gen(23)).to(BF).cuda()
    for entries, n, kept in (([1, 1, 3, 0], 3, [1, 3]), ([0, 2, 5, 7], 4, [0, 2]), ([-1, 2, 3, 4], 4, [2, 3, 4]),
                             ([0, 1, 2, 3], 9, [0, 1, 2, 3]), ([0, 1, 2, 3], -2, []), ([2**31 - 1, 0, 1, 2], 1, [])):
        idx = torch.tensor(entries, dtype=torch.int32, device="cuda").view(1, 1, 1, 4)
        cnt = torch.tensor([[[n]]], dtype=torch.int32, device="cuda")
        o, lse = gpu.attend(q, True, idx, cnt)
        _index_error()
        lists = np.empty((1, 1, 1), dtype=object)
        lists[0, 0, 0] = kept
        _check_attention(gpu, q, o, lse, True, lists)


# ---- the layer classes ------------------------------------------------------------------------------

def test_layer_classes_run_a_stream_and_its_gradients():
    """NormRope and BlockCache against the oracle over a few pieces, and NormRope.backward against autograd of the same
    formula in 64 bits."""
    B, h, d, T, H, W = 1, 2, 64, 1, 6, 9
    N = T * H * W
    rope = svsa.NormRope(d, pairs=(12, 10, 10), rows=20, halves=True, wq=torch.linspace(0.5, 1.5, d).cuda(), wk=None)
    cache = svsa.BlockCache(B, h, d, 4 * N, code="i8")
    ref = stream.BlockCache(*(t.cpu().numpy() for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale,
                                                        cache.v_scale, cache.mean, cache.mean_scale, cache.table,
                                                        cache.length)), "i8")
    for f in range(4):
        x = torch.randn(B, N, 3 * h, d, generator=_gen(30 + f)).to(BF).cuda()
        q, k, v = (x[:, :, i * h:(i + 1) * h].transpose(1, 2) for i in range(3))
        pos = svsa.grid_positions(T, H, W, frame=f)
        yq, yk = rope(q, k, pos)
        cache.append(yk, v)
        ref.append(_np(yk), _np(v), [N])
        assert np.count_nonzero(cache.k.view(torch.uint8).cpu().numpy() != ref.k) == 0
        idx, cnt = cache.select(yq, 2, causal=False)
        o = cache.attend(yq, idx, cnt, causal=False)
        want, _ = stream.cache_attention(ref, _np(yq), False, _lists(idx, cnt))
        assert np.abs(_np(o) - want).max() <= (2.0**-11 + 2.0**-12 + 2.0**-8) * np.abs(ref.tokens(0, 0)[1]).max() * 2
    svsa.svsa_sync_status()
    # gradients
    gq, gk = (torch.randn(B, h, N, d, generator=_gen(i)).to(BF).cuda() for i in (1, 2))
    dq, dk, dwq, dwk = rope.backward(gq, gk, q, k, pos)
    axis = torch.repeat_interleave(torch.arange(3), torch.tensor(rope.pairs)).cuda()
    ang = [t.double()[pos[0].long()[:, axis], torch.arange(d // 2, device="cuda")] for t in (rope.cos, rope.sin)]
    for x, w, g, got, gw in ((q, rope.wq, gq, dq, dwq), (k, torch.ones(d).cuda(), gk, dk, dwk)):
        a, b = x.double().requires_grad_(), w.double().requires_grad_()
        y = a / (a.square().mean(-1, keepdim=True) + rope.eps).sqrt() * b
        lo, hi = y[..., :d // 2], y[..., d // 2:]
        y = torch.cat([lo * ang[0] - hi * ang[1], lo * ang[1] + hi * ang[0]], -1)
        ga, gb = torch.autograd.grad(y, (a, b), g.double())
        assert float((got.double() - ga).abs().max()) <= 2.0**-8 * float(ga.abs().max())
        # (B h N = 108 rows, fp32 sums of terms of unit size: (108 + 64) 2^-24 of their total)
        terms = (g.double().abs().amax(-1, keepdim=True) * (a / a.square().mean(-1, keepdim=True).sqrt()).abs()).sum((0, 1, 2))
        assert torch.all((gw.double() - gb).abs() <= 172 * 2.0**-24 * 2 * terms)
    cache.reset()
    assert torch.all(cache.attend(yq) == 0)


@pytest.mark.parametrize("order", ["raster", "hilbert"])
def test_sparse_layer_with_norm_and_rotation(order):
    """SparseVideoAttention with norm_rope gives, bit for bit, the layer on queries and keys normed and rotated
    beforehand."""
    B, h, T, H, W, d = 1, 2, 3, 8, 10, 128
    N = T * H * W
    x = torch.randn(B, N, 3 * h, d, generator=_gen(40)).to(BF).cuda()
    q, k, v = (x[:, :, i * h:(i + 1) * h].transpose(1, 2) for i in range(3))
    v = v.contiguous()
    rope = svsa.NormRope(d, pairs=(24, 20, 20), rows=16, wq=torch.linspace(0.8, 1.2, d).cuda())
    pos = svsa.grid_positions(T, H, W)
    kw = dict(order=order, select="topk", keep_frac=0.5)
    got = svsa.SparseVideoAttention(B, h, T, H, W, d, norm_rope=(rope, pos), **kw)
    o = got(q, k, v)
    assert o.is_contiguous()
    yq, yk = rope(q, k, pos)
    want = svsa.SparseVideoAttention(B, h, T, H, W, d, **kw)(yq, yk, v)
    svsa.svsa_sync_status()
    assert torch.equal(o, want)
    with pytest.raises(ValueError):
        got.forward_host(q, k, v, o)
    with pytest.raises(ValueError):
        got(q, k, x[:, :, 2 * h:].transpose(1, 2))         # a view as v


# ---- many query rows per key head -----------------------------------------------------------------------

@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads,group,Tq,d,dtype,code", [
    ([64], 1, 1, 33, 128, BF, "i8"),             # one page, rows that see little
    ([20, 0, 130], 1, 1, 40, 64, HF, "e4m3"),    # more queries than keys, an empty sequence
    ([300], 2, 1, 128, 128, HF, "e4m3"),         # one full tile
    ([700, 64, 65], 1, 1, 129, 64, BF, "i8"),    # one row past a tile
    ([2100], 1, 3, 111, 128, BF, "e4m3"),        # several tiles, shared over CTAs
    ([1300, 5], 2, 40, 2, 64, HF, "i8"),         # a wide group
])
def test_attention_of_many_rows_matches_the_oracle(lens, heads, group, Tq, d, dtype, code, causal):
    gpu = _filled(len(lens), heads, d, code, lens, blocks=max(1, -(-max(lens) // 64)) + 1)
    q = torch.randn(len(lens), heads * group, Tq, d, generator=_gen(24)).to(dtype).cuda()
    o, lse = gpu.attend(q, causal)
    svsa.svsa_sync_status()
    _check_attention(gpu, q, o, lse, causal)
    again, _ = gpu.attend(q, causal, lse=False)
    assert torch.equal(o, again)


@pytest.mark.parametrize("heads,group,Tq,d,blocks", [(4, 4, 5, 128, 1400), (4, 8, 4, 128, 1400), (4, 4, 12, 64, 2700), (2, 2, 12, 64, 40)])
def test_rows_of_few_tiles_in_caches_of_any_room(heads, group, Tq, d, blocks):
    gpu = _filled(2, heads, d, "e4m3", [1500, 70], blocks=blocks)
    q = torch.randn(2, heads * group, Tq, d, generator=_gen(26)).to(BF).cuda()
    o, lse = gpu.attend(q, True)
    svsa.svsa_sync_status()
    _check_attention(gpu, q, o, lse, True)


def test_many_rows_with_scales_of_any_size_and_rows_that_are_not_finite():
    gpu = _filled(1, 1, 128, "i8", [1280])
    pages = gpu.table[0, :20].long()
    scale = torch.tensor([3e-20, 1e10, 0.3, 1.7e-5, 0.0, 2.0, 1e-30, 5e9, 1.0, 0.01], device="cuda")
    gpu.v_scale[pages, 0] = torch.cat([scale, scale.flip(0) * 7])
    gpu.k_scale[pages, 0] *= torch.linspace(0.0, 2.0, 20, device="cuda")
    q = torch.randn(1, 3, 50, 128, generator=_gen(25)).to(BF)
    q[0, 0, 7] *= 1e-20
    q[0, 1, 3] = 0
    q = q.cuda()
    o, lse = gpu.attend(q)
    _check_attention(gpu, q, o, lse, True)
    # a few large contributions only: blocks of tiny values carry the rest
    gpu.v_scale[pages, 0] = 1e-12
    gpu.v_scale[pages[3], 0] = 1e12
    gpu.k[pages[3], 0] = torch.full_like(gpu.k[pages[3], 0], -127)
    gpu.k_scale[pages[3], 0] = 30.0
    qp = q.abs()                                           # the page of huge values is 2^-1000 away for every row
    o, lse = gpu.attend(qp)
    _check_attention(gpu, qp, o, lse, True)
    q[0, 2, 11, 5], q[0, 2, 12, 6] = float("inf"), float("nan")
    gpu2 = _filled(1, 1, 128, "e4m3", [200])
    o, lse = gpu2.attend(q)
    bad = torch.zeros(1, 3, 50, dtype=torch.bool, device="cuda")
    bad[0, 2, 11:13] = True
    assert torch.isnan(o[bad]).all() and torch.isnan(lse[bad]).all() and torch.isfinite(o[~bad].float()).all()


def test_many_rows_leave_out_pages_out_of_range():
    gpu = _filled(2, 1, 64, "e4m3", [500, 100], blocks=8)
    q = torch.randn(2, 4, 30, 64, generator=_gen(26)).to(BF).cuda()
    good = gpu.table.clone()
    gpu.table[0, 3], gpu.table[0, 5] = -1, gpu.k.shape[0]
    o, lse = gpu.attend(q, causal=False)
    _index_error()
    gpu.table.copy_(good)
    lists = np.empty((2, 30, 1), dtype=object)
    for t in range(30):
        lists[0, t, 0], lists[1, t, 0] = [0, 1, 2, 4, 6, 7], [0, 1]
    _check_attention(gpu, q, o, lse, False, lists)
    gpu.len.copy_(torch.tensor([-3, 10000], dtype=torch.int32))
    o, lse = gpu.attend(q)
    _index_error()
    assert torch.all(o[0] == 0)


def test_many_rows_keep_the_weights_of_pages_with_tiny_values():
    """Pages whose value scales lie 170 and more binary orders below others': they add nothing to the sums but all of
    their weight to the row sum."""
    gpu = _filled(1, 1, 64, "e4m3", [640])
    pages = gpu.table[0, :10].long()
    gpu.v_scale[pages, 0] = torch.tensor([1e25, 1e-25, 1e-25, 1e25, 1.0, 1e-30, 1e-27, 1.0, 1e25, 1e20], device="cuda")
    q = torch.randn(1, 1, 70, 64, generator=_gen(27)).to(BF).cuda()
    o, lse = gpu.attend(q, causal=False)
    _check_attention(gpu, q, o, lse, False)


GATHERED = [
    # lens, heads, group, Tq, d, dtype, code, cap, the lists' blocks: shared ones and drawn ones
    ([3840], 2, 1, 200, 128, BF, "e4m3", 40, "drawn"),
    ([3800], 3, 3, 150, 64, HF, "i8", 40, "drawn"),
    ([3840], 2, 5, 230, 128, HF, "i8", 40, "near"),
    ([6000, 100, 0], 1, 1, 200, 64, BF, "e4m3", 60, "near"),
]


@pytest.mark.parametrize("lens,heads,group,Tq,d,dtype,code,cap,kind", GATHERED)
def test_lists_of_many_queries_match_the_oracle(lens, heads, group, Tq, d, dtype, code, cap, kind):
    """Enough queries that their lists are gathered per tile: drawn lists, and lists of neighbours that share most of
    their blocks; empty ones among them."""
    B = len(lens)
    gpu = _filled(B, heads, d, code, lens)
    launches = svsa.svsa_launch_count()
    rng = np.random.default_rng(4)
    idx = np.zeros((B, Tq, heads, cap), dtype=np.int32)
    cnt = np.zeros((B, Tq, heads), dtype=np.int32)
    for b in range(B):
        nb = -(-lens[b] // 64)
        for t in range(Tq):
            for h in range(heads):
                if kind == "near":
                    pool = np.unique(np.clip(t * nb // Tq + np.arange(-8, 9), 0, nb - 1)) if nb else np.zeros(0, int)
                else:
                    pool = np.arange(nb)
                n = int(rng.integers(0, min(cap, len(pool)) + 1))
                cnt[b, t, h] = n
                idx[b, t, h, :n] = np.sort(rng.permutation(pool)[:n])
    idx, cnt = torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()
    q = torch.randn(B, heads * group, Tq, d, generator=_gen(28)).to(dtype).cuda()
    launches = svsa.svsa_launch_count()
    o, lse = gpu.attend(q, False, idx, cnt)
    assert svsa.svsa_launch_count() - launches == 3        # gathered: lists, tiles, joining
    svsa.svsa_sync_status()
    _check_attention(gpu, q, o, lse, False, _lists(idx, cnt))
    o, lse = gpu.attend(q, True, idx, cnt)
    _check_attention(gpu, q, o, lse, True, _lists(idx, cnt))
    again, _ = gpu.attend(q, True, idx, cnt, lse=False)
    assert torch.equal(o, again)


def test_gathered_lists_leave_out_bad_entries_and_pages():
    gpu = _filled(1, 2, 128, "i8", [3840])
    Tq, cap = 200, 40
    idx = torch.arange(20, 60, dtype=torch.int32, device="cuda").repeat(1, Tq, 2, 1)
    cnt = torch.full((1, Tq, 2), cap, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, Tq, 128, generator=_gen(29)).to(BF).cuda()
    gpu.attend(q, True, idx, cnt)
    svsa.svsa_sync_status()
    idx[0, 7, 0, 5] = 3                                    # not ascending
    idx[0, 9, 1, 39] = 60                                  # past the sequence
    cnt[0, 11, 0], cnt[0, 12, 0] = -4, 41
    o, lse = gpu.attend(q, True, idx, cnt)
    _index_error()
    lists = np.empty((1, Tq, 2), dtype=object)
    for t in range(Tq):
        for h in range(2):
            lists[0, t, h] = list(range(20, 60))
    lists[0, 7, 0].remove(25)                              # (the entry after it ascends again)
    lists[0, 9, 1].remove(59)
    lists[0, 11, 0] = []
    _check_attention(gpu, q, o, lse, True, lists)
    gpu.table[0, 30] = -1
    idx[0, 7, 0, 5], idx[0, 9, 1, 39] = 25, 59
    cnt.fill_(cap)
    o, lse = gpu.attend(q, True, idx, cnt)
    _index_error()
    for t in range(Tq):
        for h in range(2):
            lists[0, t, h] = [j for j in range(20, 60) if j != 30]
    gpu.table[0, 30] = 5
    _check_attention(gpu, q, o, lse, True, lists)
