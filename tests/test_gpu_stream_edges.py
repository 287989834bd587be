"""Streaming entry points at the edges of their definitions, on the GPU against 64 bits.

Tolerances of the attention, counted before the first run (u = the output type's half step, finfo.eps / 2), with p_t the
softmax weights under their largest and S their sum:
  * (2^-11 + 2^-12) W, W = sum p |v| / S, and u |o|, as in test_gpu_stream.py, but no absolute term: bf16 outputs have
    none, so outputs of any size are held to the same relative error.
  * weights below fp16's normal range are off by at most half its smallest step, 2^-25, of what a weight of 1 stands for.
    The few-row tiles hold p times 2^14: sum 2^-39 |v| / S.  The 128-row tiles hold p times the page's value scale times
    2^11 or more against the largest such product Y: sum 2^-36 Y |code| / S.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_attention_hilbert_b200 as svsa
from oracle import stream
from test_gpu_stream import BF, HF, GpuCache, _filled, _gen, _half, _index_error, _np, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    svsa.lib()


@pytest.fixture(autouse=True)
def _clean():
    yield
    svsa.svsa_sync_status()


def _check(gpu, q, o, lse, causal, lists=None, many=True):
    """o and lse against 64 bits, element by element."""
    ref, qn, got, got_l = gpu.oracle(), _np(q), _np(o), _np(lse)
    B, hq, Tq, d = qn.shape
    g = hq // gpu.heads
    for b in range(B):
        n = int(ref.len[b])
        see = np.arange(n)[None] < np.array([stream.visible(n, Tq, t, causal) for t in range(Tq)])[:, None]
        pages = ref.table[b, :-(-n // 64)]
        for h in range(gpu.heads):
            k, v = ref.tokens(b, h)
            vs = np.repeat(ref.v_scale[pages, h], 64)[:n, None]
            code = np.abs(v) / np.where(vs > 0, vs, 1.0)
            mask = see.copy()
            if lists is not None:
                for t in range(Tq):
                    mine = np.zeros(len(pages), dtype=bool)
                    mine[lists[b, t, h]] = True
                    mask[t] &= np.repeat(mine, 64)[:n]
            for e in range(h * g, h * g + g):
                s = np.where(mask, qn[b, e] @ k.T / math.sqrt(d), -np.inf)
                empty = ~mask.any(-1)
                top = np.where(empty, 0.0, s.max(-1, initial=-np.inf))[:, None]
                p = np.exp(s - top)
                total = np.where(empty, 1.0, p.sum(-1))[:, None]
                want, W = p @ v / total, p @ np.abs(v) / total
                if many:
                    low = 2.0**-36 * (p * vs[:, 0]).max(-1, initial=0.0)[:, None] * (mask @ code) / total
                else:
                    low = 2.0**-39 * (mask @ np.abs(v)) / total
                tol = (2.0**-11 + 2.0**-12) * W + _half(q.dtype) * np.abs(want) * (1 + 2**-7) + low
                if q.dtype == HF:
                    tol = tol + 2.0**-25                     # half of fp16's smallest step
                err = np.abs(got[b, e] - want)
                assert np.all(err <= tol), (b, e, float((err / np.maximum(tol, 1e-300)).max()))
                rl = np.where(empty, -np.inf, top[:, 0] + np.log(np.where(empty, 1.0, p.sum(-1))))
                assert np.array_equal(np.isinf(got_l[b, e]), empty) and np.all(got_l[b, e][empty] == -np.inf)
                fin = ~empty
                assert np.all(np.abs(got_l[b, e][fin] - rl[fin]) <= 2.0**-13 + 2.0**-20 * np.abs(rl[fin]))


# ---- blocks of zero values ----------------------------------------------------------------

@pytest.mark.parametrize("code", ["e4m3", "i8"])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-5, 1e-9])
@pytest.mark.parametrize("gathered", [False, True])
def test_blocks_of_zero_values_beside_small_ones(size, code, gathered):
    """A block whose values are all zero has the value scale 0: it adds to the row sums alone, however small the other
    blocks' values are."""
    n, d, heads, Tq = (3840, 128, 2, 200) if gathered else (1270, 128, 1, 60)
    gpu = GpuCache(1, heads, d, code, -(-n // 64), seed=1)
    k, v = _tokens(_gen(101), 1, heads, n, d, BF)
    v = v * size
    for j in (0, 1, 7, 12):
        v[:, :, 64 * j:64 * j + 64] = 0
    gpu.append(k, v)
    assert torch.count_nonzero(gpu.v_scale[gpu.table[0].long()] == 0) == 4 * heads
    q = torch.randn(1, heads, Tq, d, generator=_gen(41)).to(BF).cuda()
    if not gathered:
        for causal in (True, False):
            o, lse = gpu.attend(q, causal)
            svsa.svsa_sync_status()
            _check(gpu, q, o, lse, causal)
        return
    rng = np.random.default_rng(5)
    lists = np.empty((1, Tq, heads), dtype=object)
    idx, cnt = np.zeros((1, Tq, heads, 40), dtype=np.int32), np.zeros((1, Tq, heads), dtype=np.int32)
    for t in range(Tq):
        for h in range(heads):
            m = int(rng.integers(0, 41))
            pick = {0, 1, 7} if t == 3 else set(rng.permutation(60)[:m].tolist()) | ({0, 12} if m < 38 else set())
            lists[0, t, h] = sorted(pick)
            cnt[0, t, h] = len(pick)
            idx[0, t, h, :len(pick)] = lists[0, t, h]
    launches = svsa.svsa_launch_count()
    o, lse = gpu.attend(q, False, torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda())
    assert svsa.svsa_launch_count() - launches == 3        # gathered
    svsa.svsa_sync_status()
    _check(gpu, q, o, lse, False, lists)


# ---- a dominant key without a value ---------------------------------------------------------

@pytest.mark.parametrize("code,dtype", [("e4m3", BF), ("i8", HF)])
@pytest.mark.parametrize("logit", [10.0, 15.0, 17.5, 20.0])
@pytest.mark.parametrize("Tq", [1, 4, 50])
def test_the_tail_below_a_dominant_key_without_a_value(logit, Tq, code, dtype):
    """One key takes nearly all of the weight and its value is zero, so the output is what the others add."""
    n, d, heads = 2600, 128, 2
    gpu = GpuCache(1, heads, d, code, -(-n // 64) + 1, seed=2)
    k, v = _tokens(_gen(102), 1, heads, n, d, BF, scale=0.25)
    u = torch.randn(d, generator=_gen(42)).sign().to(BF).cuda()
    for at in (0, 64 * 6 + 3):                              # in a page of either parity
        k[0, at // 64 % 2, at], v[0, at // 64 % 2, at] = u, 0
    k[0, 1, 5], v[0, 1, 5] = u, 0
    gpu.append(k, v * 4)
    q = (u * (logit / math.sqrt(d)) + 0.1 * torch.randn(1, 3 * heads, Tq, d, generator=_gen(43)).cuda()).to(dtype)
    o, lse = gpu.attend(q, False)
    svsa.svsa_sync_status()
    assert logit - 1 < float(lse.min()) and float(lse.max()) < logit + 9
    _check(gpu, q, o, lse, False, many=3 * Tq > 48)


# ---- rows that see nothing --------------------------------------------------------------------

@pytest.mark.parametrize("Tq", [4, 60])
@pytest.mark.parametrize("d,dtype,code", [(128, BF, "e4m3"), (64, HF, "i8")])
def test_rows_that_see_nothing_give_zeros_whatever_their_values(Tq, d, dtype, code):
    """Queries before the first key, and lists without a visible key: zeros and -inf, for rows that are not finite too."""
    gpu = _filled(2, 1, d, code, [2, 0], dtype=dtype, blocks=3)
    q = torch.randn(2, 2, Tq, d, generator=_gen(44)).to(dtype).cuda()
    q[:, 0, 0, 3], q[:, 1, 1, 9], q[:, :, -1, 0] = float("nan"), float("inf"), float("-inf")
    o, lse = gpu.attend(q, True)
    svsa.svsa_sync_status()
    assert torch.all(o[:, :, :-2] == 0) and torch.all(lse[:, :, :-2] == -math.inf)
    assert torch.all(o[1] == 0) and torch.all(lse[1] == -math.inf)
    assert torch.isfinite(o[0, :, -2].float()).all() and torch.isnan(o[0, :, -1]).all() and torch.isnan(lse[0, :, -1]).all()
    # lists: empty, or of blocks that the query does not see yet
    gpu = _filled(1, 1, d, code, [66], dtype=dtype, blocks=2)
    q = q[:1, :, -4:].contiguous()
    q[0, :, 0, 1] = q[0, :, 1, 1] = float("nan")
    idx = torch.tensor([[0], [1], [1], [0]], dtype=torch.int32, device="cuda").view(1, 4, 1, 1)
    cnt = torch.tensor([0, 1, 1, 1], dtype=torch.int32, device="cuda").view(1, 4, 1)
    o, lse = gpu.attend(q, True, idx, cnt)
    svsa.svsa_sync_status()
    assert torch.all(o[:, :, :2] == 0) and torch.all(lse[:, :, :2] == -math.inf)
    assert torch.isfinite(o[:, :, 2].float()).all() and torch.isnan(o[:, :, 3]).all()


def test_gathered_rows_that_are_not_finite():
    """Many queries' lists, gathered: a row without a listed key gives zeros, a row that is not finite NaN, and neither
    touches its neighbours."""
    gpu = _filled(1, 2, 128, "e4m3", [3840])
    Tq, cap = 200, 40
    idx = torch.arange(20, 60, dtype=torch.int32, device="cuda").repeat(1, Tq, 2, 1)
    cnt = torch.full((1, Tq, 2), cap, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, Tq, 128, generator=_gen(48)).to(BF).cuda()
    cnt[0, 11, 0] = 0
    want, want_l = gpu.attend(q, True, idx, cnt)
    q[0, 0, 11, 5], q[0, 1, 12, 6] = float("inf"), float("nan")
    o, lse = gpu.attend(q, True, idx, cnt)
    svsa.svsa_sync_status()
    assert torch.all(o[0, 0, 11] == 0) and lse[0, 0, 11] == -math.inf
    assert torch.isnan(o[0, 1, 12]).all() and torch.isnan(lse[0, 1, 12])
    o[0, 1, 12], lse[0, 1, 12] = want[0, 1, 12], want_l[0, 1, 12]
    assert torch.equal(o, want) and torch.equal(lse, want_l)


# ---- lists that name a block twice ------------------------------------------------------------

@pytest.mark.parametrize("Tq", [2, 200])
def test_a_list_that_comes_back_to_a_block_is_reported_and_touches_no_other(Tq):
    """[5, 3, 5]: the call is reported, whichever tiles it takes, and the other queries' results are what they were."""
    gpu = _filled(1, 2, 64, "i8", [3840])
    cap = 40
    idx = torch.arange(20, 60, dtype=torch.int32, device="cuda").repeat(1, Tq, 2, 1)
    cnt = torch.full((1, Tq, 2), cap, dtype=torch.int32, device="cuda")
    q = torch.randn(1, 2, Tq, 64, generator=_gen(45)).to(BF).cuda()
    want, want_l = gpu.attend(q, True, idx, cnt)
    svsa.svsa_sync_status()
    idx[0, 1, 0, :3] = torch.tensor([25, 23, 25], dtype=torch.int32)
    o, lse = gpu.attend(q, True, idx, cnt)
    _index_error()
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse).all()
    o[0, 0, 1], lse[0, 0, 1] = want[0, 0, 1], want_l[0, 0, 1]
    assert torch.equal(o, want) and torch.equal(lse, want_l)


# ---- the layers on streams -------------------------------------------------------------------------

def test_layer_calls_in_flight_on_two_streams():
    """attend, with and without lists, select and gradients queued on two side streams behind some work, while the current
    stream asks for memory of the same sizes and writes it: each gives what it gives alone."""
    B, heads, d, n = 2, 4, 128, 9000
    cache = svsa.BlockCache(B, heads, d, n)
    k, v = _tokens(_gen(60), B, heads, n, d, BF)
    cache.append(k, v, torch.tensor([n, 1234], dtype=torch.int32, device="cuda"))
    rope = svsa.NormRope(d, pairs=(64,), rows=64, wq=torch.linspace(0.5, 1.5, d).cuda())
    pos = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40, 1)
    q = [torch.randn(B, 4 * heads, t, d, generator=_gen(61 + t)).to(BF).cuda() for t in (1, 1, 40, 40)]

    def both(i, s):
        x = q[i]
        idx, cnt = cache.select(x, 9, stream=s)
        out = [idx, cnt, cache.attend(x, stream=s), cache.attend(x, idx, cnt, stream=s)]
        if x.shape[2] == 40:
            out += rope(x, x, pos, stream=s)
            out += rope.backward(x, x, x, x, pos, stream=s)
        return out

    want = [both(i, None) for i in range(4)]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:
        with torch.cuda.stream(s):
            torch.cuda._sleep(3_000_000)
    for _ in range(5):
        for i in range(4):
            got.append((i, both(i, side[i % 2])))
            for w in want[i]:
                torch.full_like(w, 7)                      # on the current stream, dropped at once
            torch.full((4 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for i, out in got:
        for a, b in zip(out, want[i]):
            assert torch.equal(a, b)
    svsa.svsa_sync_status()


def test_a_chain_on_one_side_stream():
    """append, select, attend and reset through `stream=` alone, against the current stream's."""
    B, heads, d = 2, 2, 64
    plain, chained = (svsa.BlockCache(B, heads, d, 500, code="i8") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(1_000_000)
    outs = [[], []]
    xs = [torch.randn(B, heads, 100, d, generator=_gen(70 + i)).to(BF).cuda() for i in range(4)]
    s.wait_stream(torch.cuda.current_stream())
    for c, st, out in ((plain, None, outs[0]), (chained, s, outs[1])):
        for x in xs:
            c.append(x, x, stream=st)
            idx, cnt = c.select(x, 3, stream=st)
            out += [idx, cnt, c.attend(x, idx, cnt, stream=st), c.attend(x, stream=st)]
    torch.cuda.synchronize()
    assert plain.length.tolist() == chained.length.tolist() == [400, 400]
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    chained.reset(stream=s)
    o = chained.attend(xs[0], stream=s)
    torch.cuda.synchronize()
    assert torch.all(o == 0) and chained.length.tolist() == [0, 0]
    svsa.svsa_sync_status()


# ---- gradients through autograd ---------------------------------------------------------------------

@pytest.mark.parametrize("order", [False, True])
@pytest.mark.parametrize("dtype,halves", [(BF, True), (HF, False)])
def test_autograd_of_norm_and_rotation(dtype, halves, order):
    """Gradients of a fused projection's output and of the weights, through autograd: those of the call itself, on the
    current stream and on another."""
    B, hq, hk, N, d = 2, 6, 2, 70, 64
    pos = torch.arange(N, dtype=torch.int32, device="cuda").view(1, N, 1)
    perm = iperm = None
    if order:
        perm = torch.cat([torch.randperm(N, generator=_gen(80)), torch.full((58,), -1)]).to(torch.int32).cuda()
        iperm = torch.argsort(perm[:N]).to(torch.int32)
    wq, wk = (torch.nn.Parameter(1 + 0.3 * torch.randn(d, generator=_gen(i)).cuda()) for i in (81, 82))
    rope = svsa.NormRope(d, pairs=(32,), rows=N, halves=halves, wq=wq, wk=wk)
    x = torch.randn(B, N, hq + hk, d, generator=_gen(83)).to(dtype).cuda().requires_grad_()
    rows = N if perm is None else 128
    gq, gk = (torch.randn(B, h, rows, d, generator=_gen(84)).to(dtype).cuda() for h in (hq, hk))
    with torch.no_grad():
        q, k = x[:, :, :hq].transpose(1, 2), x[:, :, hq:].transpose(1, 2)
        want = rope(q, k, pos, perm=perm)
        dq, dk, dwq, dwk = rope.backward(gq, gk, q, k, pos, iperm=iperm, rows=rows)
    side = torch.cuda.Stream()
    for s in (None, side):
        side.wait_stream(torch.cuda.current_stream())
        y = x.grad = wq.grad = wk.grad = None              # (no graph of an earlier stream stays)
        y = rope(x[:, :, :hq].transpose(1, 2), x[:, :, hq:].transpose(1, 2), pos, perm=perm, iperm=iperm, stream=s)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
        torch.autograd.backward(y, (gq, gk))
        torch.cuda.synchronize()
        assert torch.equal(x.grad, torch.cat([dq, dk], 1).transpose(1, 2))
        assert torch.equal(wq.grad, dwq) and torch.equal(wk.grad, dwk)
    # only one output used, its gradient broadcast
    y = x.grad = wq.grad = wk.grad = None
    y = rope(x[:, :, :hq].transpose(1, 2), x[:, :, hq:].transpose(1, 2), pos, perm=perm, iperm=iperm)
    y[1].sum().backward()
    with torch.no_grad():
        dq, dk, dwq, dwk = rope.backward(torch.zeros_like(gq), torch.ones_like(gk), q, k, pos, iperm=iperm, rows=rows)
    assert torch.equal(x.grad, torch.cat([dq, dk], 1).transpose(1, 2)) and torch.equal(wk.grad, dwk)
    assert torch.all(wq.grad == 0) and torch.all(x.grad[:, :, :hq] == 0)
    svsa.svsa_sync_status()


def test_sparse_layer_with_weights_that_require_gradients():
    """A layer used for inference, its norm weights parameters: it runs, as it does on inputs that require gradients."""
    B, h, T, H, W, d = 1, 2, 3, 8, 10, 128
    q, k, v = (torch.randn(B, h, T * H * W, d, generator=_gen(90 + i)).to(BF).cuda() for i in range(3))
    rope = svsa.NormRope(d, wq=torch.nn.Parameter(torch.linspace(0.8, 1.2, d).cuda()))
    kw = dict(order="raster", select="topk", keep_frac=0.5)
    o = svsa.SparseVideoAttention(B, h, T, H, W, d, norm_rope=(rope, None), **kw)(q, k, v)
    with torch.no_grad():
        want = svsa.SparseVideoAttention(B, h, T, H, W, d, **kw)(*rope(q, k), v)
    svsa.svsa_sync_status()
    assert torch.equal(o, want)


# ---- strides of dimensions of size 1 ------------------------------------------------------------

def test_strides_of_dimensions_of_size_one_do_not_matter():
    """A batch, head or token dimension of size 1 may have any stride: nothing is ever a step away along it."""
    d = 64
    x = torch.randn(3, 1, 5, d, generator=_gen(46)).to(BF).cuda()
    q = x[1:2].as_strided((1, 1, 5, d), (3, 5, d, 1), x.stride(0))
    t = x[0, 0, :1].as_strided((1, 1, 1, d), (1, 2, 3, 1))
    for a in (q, t):
        rope = svsa.NormRope(d)
        want = rope(a.contiguous().clone(), a.contiguous().clone())
        got = rope(a, a)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        g = torch.randn(a.shape, generator=_gen(47)).to(BF).cuda()
        for u, w in zip(rope.backward(g, g, a, a), rope.backward(g, g, a.contiguous().clone(), a.contiguous().clone())):
            assert torch.equal(u, w)
        caches = [svsa.BlockCache(1, 1, d, 64) for _ in range(2)]
        caches[0].append(a, a)
        caches[1].append(a.contiguous().clone(), a.contiguous().clone())
        for u, w in ((caches[0].k, caches[1].k), (caches[0].v, caches[1].v)):
            assert torch.equal(u.view(torch.uint8), w.view(torch.uint8))
    svsa.svsa_sync_status()


# ---- the largest selection ------------------------------------------------------------------------------

@pytest.mark.parametrize("d,group,cap", [(128, 128, 4097), (64, 1, 32767)])
def test_selection_over_the_most_blocks(d, group, cap):
    """32,768 blocks and 128 query heads per key head: scores are whole numbers under powers of two, exact in 64 bits."""
    nb = 32768
    rng = np.random.default_rng(7)
    mean = rng.integers(-127, 128, (nb, 1, d)).astype(np.int8)
    scale = np.exp2(rng.integers(-9, 3, (nb, 1))).astype(np.float32)
    codes = torch.zeros(nb, 1, 64, d, dtype=torch.int8, device="cuda")
    one = torch.ones(nb, 1, device="cuda")
    order = rng.permutation(nb).astype(np.int32)
    dev = lambda a: torch.from_numpy(a).cuda()
    n = torch.tensor([64 * nb - 3], dtype=torch.int32, device="cuda")
    mean_t, scale_t, table = dev(mean), dev(scale), dev(order[None])
    c = svsa.block_cache(codes, codes.clone(), one, one.clone(), table, n, mean_t, scale_t)
    q = torch.randn(1, group, 2, d, generator=_gen(50)).to(BF).cuda()
    idx = torch.full((1, 2, 1, cap), -5, dtype=torch.int32, device="cuda")
    cnt = torch.full((1, 2, 1), -5, dtype=torch.int32, device="cuda")
    svsa.svsa_cache_select(c, q, idx, cnt, svsa.cache_query(q, causal=True, cap=cap, first=2, last=3))
    svsa.svsa_sync_status()
    for t in range(2):
        score = np.full(nb, -np.inf)
        for e in range(group):
            row = _np(q[0, e, t])
            s = stream.pow2_scale(np.abs(row).max(), "i8")
            qi = stream.encode(row, s, "i8").view(np.int8).astype(np.float64)
            score = np.maximum(score, (mean[order, 0].astype(np.float64) @ qi) * (s * scale[order, 0].astype(np.float64)))
        score[:2] = score[-3:] = np.inf
        want = np.sort(np.lexsort((np.arange(nb), -score))[:cap])
        assert cnt[0, t, 0] == cap and np.array_equal(idx[0, t, 0].cpu().numpy(), want)


def test_autograd_of_norm_and_rotation_captured():
    """Forward and backward in one CUDA graph, replayed on other values: the eager gradients."""
    B, hq, hk, N, d = 1, 4, 2, 50, 128
    pos = torch.arange(N, dtype=torch.int32, device="cuda").view(1, N, 1)
    wq, wk = (torch.nn.Parameter(1 + 0.3 * torch.randn(d, generator=_gen(i)).cuda()) for i in (91, 92))
    rope = svsa.NormRope(d, pairs=(64,), rows=N, wq=wq, wk=wk)
    x = torch.randn(B, N, hq + hk, d, generator=_gen(93)).to(BF).cuda().requires_grad_()
    gq, gk = (torch.randn(B, h, N, d, generator=_gen(94)).to(BF).cuda() for h in (hq, hk))

    def step():
        y = rope(x[:, :, :hq].transpose(1, 2), x[:, :, hq:].transpose(1, 2), pos)
        return torch.autograd.grad(y, (x, wq, wk), (gq, gk))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (95, 96):
        with torch.no_grad():
            x.copy_(torch.randn(x.shape, generator=_gen(seed)).to(BF))
            wq.mul_(1.1)
        graph.replay()
        torch.cuda.synchronize()
        kept = [g.clone() for g in got]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b)
    svsa.svsa_sync_status()
