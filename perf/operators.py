"""Cases, plain forms and 64-bit values of the operators around the block cache.

Six operators, in the order in which a model that streams its tokens uses them:

    norm_rope       per-head RMS norm of the queries and keys and their position
                    rotation, in the library's token order where one is given
    norm_rope_bwd   its gradients (inputs and norm weights)
    append          new keys and values into the 8-bit cache of 64-token blocks,
                    with one power-of-two scale and (for keys) one 8-bit mean
                    per block and head
    select          the key blocks of the cache that each query attends to
    attend          attention over the whole cache
    attend_blocks   attention over each query's own list of cache blocks

`run` computes them with elementary torch operations in 32 bits, or, with `own`
set, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False
device = "cuda"

BLOCK = 64
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
CODES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
TOP = {"e4m3": (0.875, 9), "i8": (127.0 / 128.0, 7)}       # the largest code, as frexp gives it


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of 32 running sequences of a decoder: latency
        {"name": "norm_rope_token", "op": "norm_rope", "B": 32, "T": 1, "H": 1, "W": 1, "hq": 32, "hk": 8, "d": 128,
         "dtype": "bf16", "axes": 1, "halves": True, "order": False},
        # a 40-head video layer, rotated by (frame, row, column) and put in block order
        {"name": "norm_rope_video", "op": "norm_rope", "B": 1, "T": 21, "H": 30, "W": 52, "hq": 40, "hk": 40, "d": 128,
         "dtype": "bf16", "axes": 3, "halves": False, "order": True},
        # training a 12-head video layer
        {"name": "norm_rope_bwd_video", "op": "norm_rope_bwd", "B": 1, "T": 21, "H": 30, "W": 52, "hq": 12, "hk": 12,
         "d": 128, "dtype": "bf16", "axes": 3, "halves": False, "order": True},
        # a small odd batch with shared key heads
        {"name": "norm_rope_bwd_odd", "op": "norm_rope_bwd", "B": 2, "T": 5, "H": 9, "W": 7, "hq": 6, "hk": 2, "d": 64,
         "dtype": "fp16", "axes": 1, "halves": True, "order": False},
        # one new token of 32 sequences
        {"name": "append_token", "op": "append", "B": 32, "N": 1, "len": 2000, "len_min": 0, "hk": 8, "d": 128,
         "dtype": "bf16", "code": "i8"},
        # five latent frames of 30 x 52 tokens appended to two streams
        {"name": "append_frames", "op": "append", "B": 2, "N": 7800, "len": 1000, "len_min": 77, "hk": 12, "d": 128,
         "dtype": "bf16", "code": "e4m3"},
        # single-token decoding over long caches
        {"name": "select_token", "op": "select", "B": 8, "Tq": 1, "len": 131072, "len_min": 30001, "hq": 32, "hk": 8,
         "d": 128, "dtype": "bf16", "code": "e4m3", "cap": 64, "first": 1, "last": 2, "causal": True},
        # a chunk of tokens of a 12-head video stream, a quarter of the blocks each
        {"name": "select_chunk", "op": "select", "B": 1, "Tq": 60, "len": 32760, "len_min": 32760, "hq": 12, "hk": 12,
         "d": 128, "dtype": "bf16", "code": "i8", "cap": 128, "first": 0, "last": 1, "causal": False},
        # five drafted tokens over a short cache: latency, causal among themselves
        {"name": "attend_draft", "op": "attend", "B": 2, "Tq": 5, "len": 777, "len_min": 130, "hq": 8, "hk": 2, "d": 64,
         "dtype": "fp16", "code": "i8", "causal": True},
        # single-token decoding over long caches: bandwidth
        {"name": "attend_long", "op": "attend", "B": 8, "Tq": 1, "len": 131072, "len_min": 30001, "hq": 32, "hk": 8,
         "d": 128, "dtype": "bf16", "code": "e4m3", "causal": True},
        # the same caches, 64 blocks of each
        {"name": "attend_blocks_token", "op": "attend_blocks", "B": 8, "Tq": 1, "len": 131072, "len_min": 30001, "hq": 32,
         "hk": 8, "d": 128, "dtype": "bf16", "code": "e4m3", "cap": 64, "causal": True},
        # a chunk of tokens of a 12-head video stream, 64 blocks for each token and head
        {"name": "attend_blocks_chunk", "op": "attend_blocks", "B": 1, "Tq": 60, "len": 32760, "len_min": 32760, "hq": 12,
         "hk": 12, "d": 128, "dtype": "bf16", "code": "i8", "cap": 64, "causal": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "select", "attend", "attend_blocks"])
    c = {"op": op, "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "fp16"])}
    hk = rng.choice([1, 2, 3, 4, 8, 12])
    group = rng.choice([1, 1, 2, 4, 5, 8, 16])
    if op in ("norm_rope", "norm_rope_bwd"):
        most = (1 * 21 * 30 * 52 * 40 * 128) if op == "norm_rope" else (21 * 30 * 52 * 12 * 128)
        c.update(B=_log(rng, 1, 48), T=rng.choice([1, 1, 3, 8, 21]), H=_log(rng, 1, 30), W=_log(rng, 1, 52), hk=hk,
                 hq=hk * group, axes=rng.choice([0, 1, 3]), halves=rng.random() < 0.5, order=rng.random() < 0.5)
        while c["B"] * c["T"] * c["H"] * c["W"] * c["hq"] * c["d"] > most:
            c["B"], c["H"] = max(1, c["B"] // 2), max(1, c["H"] - 3)
            if c["B"] == 1 and c["H"] == 1:
                c["T"] = 1
        return c
    c.update(B=_log(rng, 1, 40), hk=hk, code=rng.choice(["e4m3", "i8"]))
    if op == "append":
        c.update(N=_log(rng, 1, 8000), len=_log(rng, 1, 4000))
        c["len_min"] = rng.randint(0, c["len"])
        while c["B"] * (c["N"] + c["len"]) * hk * c["d"] > 2 * 8800 * 12 * 128:
            c["B"], c["N"] = max(1, c["B"] // 2), max(1, c["N"] * 3 // 4)
            c["len"] = max(1, c["len"] * 3 // 4)
            c["len_min"] = min(c["len_min"], c["len"])
        return c
    c.update(hq=hk * group, Tq=rng.choice([1, 1, 1, 2, 3, 4, 7, 8, 17, 33]), len=_log(rng, 1, 131072),
             causal=rng.random() < 0.6)
    c["len_min"] = max(1, int(c["len"] * rng.uniform(0.05, 1.0)))
    cap = _log(rng, 1, 128)
    if op == "select":
        c.update(cap=cap, first=rng.randint(0, min(cap, 2)), last=0)
        c["last"] = rng.randint(0, min(cap - c["first"], 3))
    if op == "attend_blocks":
        c["cap"] = cap
    while (c["B"] * (c["len"] + c["len_min"]) / 2 * hk * c["d"] > 8 * 80000 * 8 * 128
           or c["B"] * c["Tq"] * c["hq"] * c["len"] > 8 * 32 * 131072
           or (op == "select" and c["B"] * c["Tq"] * c["hq"] * c["len"] * c["d"] > 60 * 12 * 32760 * 128)
           or (op == "attend_blocks" and c["B"] * c["Tq"] * hk * cap * c["d"] > 60 * 12 * 64 * 128)):
        c["B"], c["Tq"] = max(1, c["B"] // 2), max(1, c["Tq"] // 2)
        if c["B"] == 1 and c["Tq"] == 1:
            c["len"] = max(1, c["len"] // 2)
            c["len_min"] = min(c["len_min"], c["len"])
    return c


def _lens(case):
    """The cache lengths of a case's sequences: from len_min to len, the longest first."""
    lo, hi = case["len_min"], case["len"]
    return [hi if b == 0 else lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(case["B"])]


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- inputs

def _randn(seed, k, shape):
    g = torch.Generator(device=device)
    g.manual_seed(1_000_003 * int(seed) + k)
    return torch.randn(shape, generator=g, device=device, dtype=torch.float32)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=device)


def _pow2_scale(amax, code):
    """The smallest power of two with amax / scale within the codes (0 for amax = 0)."""
    most, bits = TOP[code]
    f, e = torch.frexp(amax)
    e = torch.where(f <= most, e - bits, e - bits + 1).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _encode(x, scale, code):
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    return (y.clamp(-127, 127).round() if code == "i8" else y.clamp(-448, 448)).to(CODES[code])


def _pick(x, *index):
    """x[index] for codes (indexed as bytes)."""
    return x.view(torch.uint8)[index].view(x.dtype)


def _summary(k_codes, k_scale, count, code):
    """8-bit means of a cache's key blocks [..., 64, d] over their first `count` tokens, with their scales."""
    unit = 1.0 if code == "i8" else 2.0 ** -9
    rows = torch.arange(BLOCK, device=k_codes.device).view(-1, 1) < count[..., None, None]
    total = torch.where(rows, k_codes.float() / unit, 0.0).sum(-2)       # whole numbers below 2^24: exact
    mean = total / count.clamp(min=1)[..., None].float()
    s = _pow2_scale(mean.abs().amax(-1), "i8")
    return _encode(mean, s[..., None], "i8"), s * unit * k_scale


def _make_cache(case, seed, room):
    """A cache with its sequences' lengths, and pages for `room` more tokens each, in shuffled pages."""
    B, h, d, code = case["B"], case["hk"], case["d"], case["code"]
    lens = _lens(case)
    blocks = [_blocks(n + room) for n in lens]
    n_pages, width = sum(blocks) + 3, max(1, max(blocks))
    order = np.random.RandomState(int(seed) % (1 << 31)).permutation(n_pages)
    table, at = np.full((B, width), -1, dtype=np.int32), 0
    count = np.zeros(n_pages, dtype=np.int64)
    for b in range(B):
        pages = order[at:at + blocks[b]]
        table[b, :blocks[b]] = pages
        count[pages] = np.clip(lens[b] - BLOCK * np.arange(blocks[b]), 0, BLOCK)
        at += blocks[b]
    # channels of unlike size and a slow drift over the tokens, as keys have; values plain
    size = torch.exp(0.5 * _randn(seed, 1, (h, 1, d)))
    state = {"table": torch.from_numpy(table).to(device), "len": _ints(lens)}
    count = torch.from_numpy(count).to(device)
    for name, k in (("k", 2), ("v", 4)):
        codes = torch.empty((n_pages, h, BLOCK, d), dtype=CODES[code], device=device)
        scales = torch.empty((n_pages, h), device=device)
        for i in range(0, n_pages, 4096):
            j = min(n_pages, i + 4096)
            x = _randn(seed, 100 * k + i, (j - i, h, BLOCK, d))
            if name == "k":
                x = (x + 0.7 * _randn(seed, 100 * k + 50 + i, (j - i, h, 1, d))) * size
            x = torch.where(torch.arange(BLOCK, device=device).view(-1, 1) < count[i:j, None, None, None], x, 0.0)
            s = _pow2_scale(x.abs().amax((-1, -2)), code)
            codes[i:j], scales[i:j] = _encode(x, s[..., None, None], code), s
        state[name], state[name + "_scale"] = codes, scales
    state["mean"], state["mean_scale"] = torch.empty((n_pages, h, d), dtype=torch.int8, device=device), torch.empty((n_pages, h), device=device)
    for i in range(0, n_pages, 4096):
        j = min(n_pages, i + 4096)
        state["mean"][i:j], state["mean_scale"][i:j] = _summary(state["k"][i:j], state["k_scale"][i:j], count[i:j, None].expand(-1, h), code)
    return state


def _make_norm_rope(case, seed):
    B, T, H, W, hq, hk, d = (case[x] for x in ("B", "T", "H", "W", "hq", "hk", "d"))
    dt, n = TYPES[case["dtype"]], T * H * W
    # the projection's output, tokens first: q and k are views of it
    qkv = (_randn(seed, 1, (B, n, hq + 2 * hk, d)) * torch.exp(0.3 * _randn(seed, 2, (hq + 2 * hk, d)))).to(dt)
    q, k = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hk].transpose(1, 2)
    state = {"q": q, "k": k, "wq": 1 + 0.2 * _randn(seed, 3, (d,)), "wk": 1 + 0.2 * _randn(seed, 4, (d,)),
             "eps": EPS, "axes": case["axes"], "halves": case["halves"], "op": case["op"]}
    if case["axes"] == 3:
        t, y, x = (v.reshape(-1) for v in torch.meshgrid(torch.arange(T), torch.arange(H), torch.arange(W), indexing="ij"))
        pos = torch.stack([t, y, x], -1).to(torch.int32).to(device).unsqueeze(0)
        each = [d // 2 - 2 * (d // 6), d // 6, d // 6]
        rows = max(T, H, W)
    elif case["axes"] == 1:
        # sequences at positions of their own
        start = torch.from_numpy(np.random.RandomState(int(seed) % (1 << 31)).randint(0, 4000, (B, 1, 1)))
        pos = (start + torch.arange(n).view(1, n, 1)).to(torch.int32).to(device)
        each, rows = [d // 2], 4000 + n
    else:
        pos, each, rows = None, [], 0
    state["pairs"] = tuple(each)
    state["axis"] = torch.tensor([a for a, m in enumerate(each) for _ in range(m)], dtype=torch.long, device=device)
    if rows:
        f = torch.cat([10000.0 ** (-torch.arange(m, dtype=torch.float64) / m) for m in each]).to(device)
        angle = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
    else:
        state["cos"] = state["sin"] = None
    state["pos"] = pos
    state["perm"] = state["iperm"] = None
    if case["order"]:
        # a space-filling order of the grid (bits of the three coordinates in turn), padded to whole blocks
        t, y, x = np.meshgrid(np.arange(T), np.arange(H), np.arange(W), indexing="ij")
        key = sum(((c.reshape(-1).astype(np.int64) >> b) & 1) << (3 * b + 2 - a) for a, c in enumerate((t, y, x)) for b in range(8))
        perm = np.full(_blocks(n) * BLOCK, -1, dtype=np.int32)
        perm[:n] = np.argsort(key, kind="stable")
        iperm = np.empty(n, dtype=np.int32)
        iperm[perm[:n]] = np.arange(n)
        state["perm"], state["iperm"] = torch.from_numpy(perm).to(device), torch.from_numpy(iperm).to(device)
    if case["op"] == "norm_rope_bwd":
        rows = n if state["perm"] is None else state["perm"].numel()
        state["gq"] = (0.1 * _randn(seed, 5, (B, hq, rows, d))).to(dt)
        state["gk"] = (0.1 * _randn(seed, 6, (B, hk, rows, d))).to(dt)
    return state


def prepare(case, seed):
    if case["op"].startswith("norm_rope"):
        return _make_norm_rope(case, seed)
    dt, B, h, d = TYPES[case["dtype"]], case["B"], case["hk"], case["d"]
    if case["op"] == "append":
        state = _make_cache(case, seed, case["N"])
        size = torch.exp(0.5 * _randn(seed, 1, (h, d)))
        kv = torch.stack([_randn(seed, 7, (B, case["N"], h, d)) * size, _randn(seed, 8, (B, case["N"], h, d))], 2).to(dt)
        # a padded batch: the last tokens of some sequences are no tokens
        new = [case["N"] - (b % 3) * (case["N"] // 5) for b in range(B)]
        state.update(op="append", new_k=kv[:, :, 0].transpose(1, 2), new_v=kv[:, :, 1].transpose(1, 2), n_new=_ints(new), code=case["code"])
        return state
    state = _make_cache(case, seed, 0)
    q = 1.2 * _randn(seed, 9, (B, h, case["hq"] // h, case["Tq"], d)) / torch.exp(0.5 * _randn(seed, 1, (h, 1, d))).view(1, h, 1, 1, d)
    state.update(op=case["op"], code=case["code"], causal=case["causal"], q=q.reshape(B, case["hq"], case["Tq"], d).to(dt), cap=case.get("cap", 0),
                 first=case.get("first", 0), last=case.get("last", 0))
    if case["op"] == "attend_blocks":
        # each query's list: distinct blocks of its sequence, ascending, the newest among them
        nb = torch.tensor([_blocks(n) for n in _lens(case)], device=device)
        u = torch.rand((B, case["Tq"], h, state["table"].shape[1]), generator=torch.Generator(device=device).manual_seed(int(seed) + 77), device=device)
        j = torch.arange(u.shape[-1], device=device)
        u = torch.where(j < nb.view(-1, 1, 1, 1), u, 2.0)
        u = torch.where(j == nb.view(-1, 1, 1, 1) - 1, -1.0, u)
        take = min(case["cap"], u.shape[-1])
        idx = u.topk(take, dim=-1, largest=False).indices
        idx = torch.where(idx < nb.view(-1, 1, 1, 1), idx, 1 << 30).sort(-1).values
        cnt = (idx < (1 << 30)).sum(-1)
        full = torch.zeros((B, case["Tq"], h, case["cap"]), dtype=torch.int32, device=device)
        full[..., :take] = torch.where(idx < (1 << 30), idx, 0).to(torch.int32)
        state.update(idx=full, cnt=cnt.to(torch.int32))
    return state


# ---------------------------------------------------------------- plain forms (32 bits)

def _take(x, index):
    """Rows `index` of x [B, h, n, d] (zeros where it is -1); all of them without one."""
    if index is None:
        return x
    return torch.where((index >= 0).view(1, 1, -1, 1), x[:, :, index.clamp(min=0).long()], torch.zeros((), dtype=x.dtype, device=x.device))


def _angles(s, n):
    """cos and sin [B or 1, 1, n, d / 2] of the tokens' pairs."""
    rows = s["pos"].long()[:, :, s["axis"]]
    pair = torch.arange(s["axis"].numel(), device=rows.device)
    return s["cos"][rows, pair].unsqueeze(1), s["sin"][rows, pair].unsqueeze(1)


def _split(x, halves):
    return (x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:]) if halves else (x[..., 0::2], x[..., 1::2])


def _join(a, b, halves):
    return torch.cat([a, b], -1) if halves else torch.stack([a, b], -1).flatten(-2)


def _norm_rope(s, x, w):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w
    if s["pos"] is not None:
        c, n = _angles(s, x.shape[2])
        a, b = _split(y, s["halves"])
        y = _join(a * c - b * n, a * n + b * c, s["halves"])
    return y


def _norm_rope_bwd(s, g, x, w):
    g, x = _take(g, s["iperm"]).float(), x.float()
    if s["pos"] is not None:
        c, n = _angles(s, x.shape[2])
        a, b = _split(g, s["halves"])
        g = _join(a * c + b * n, b * c - a * n, s["halves"])
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    y = x * r
    gw = g * w
    return r * (gw - y * (gw * y).mean(-1, keepdim=True)), (g * y).sum((0, 1, 2))


def _append(s):
    """The cache with the new tokens in it: a block whose scale grows is held in the new scale from then on."""
    k, v, n_new, length, table = s["new_k"], s["new_v"], s["n_new"].long(), s["len"].long(), s["table"].long()
    B, h, n, d = k.shape
    wide = _blocks(n) + 1                                    # blocks that n tokens can touch
    blk = (length // BLOCK)[:, None] + torch.arange(wide, device=k.device)
    pos = blk[..., None] * BLOCK + torch.arange(BLOCK, device=k.device)          # [B, wide, 64]
    src = pos - length[:, None, None]
    new = (src >= 0) & (src < n_new[:, None, None])
    old = src < 0
    touched = new.any(-1)
    page = torch.gather(table, 1, blk.clamp(max=table.shape[1] - 1)).clamp(min=0)
    count = (old | new).sum(-1)
    out = {}
    for name, x in (("k", k), ("v", v)):
        b = torch.arange(B, device=k.device).view(B, 1, 1)
        rows = x.permute(0, 2, 1, 3)[b, src.clamp(0, n - 1)].permute(0, 1, 3, 2, 4).float()      # [B, wide, h, 64, d]
        codes, scale = _pick(s[name], page), s[name + "_scale"][page]
        had = old.any(-1)[..., None]
        start = torch.where(had, scale, 0.0)
        need = torch.where(new[:, :, None, :, None], rows, 0.0).abs().amax((-1, -2))
        grown = torch.maximum(start, _pow2_scale(need, s["code"]))
        held = codes.float() * start[..., None, None]
        value = torch.where(new[:, :, None, :, None], rows, held)
        made = _encode(value, grown[..., None, None], s["code"])
        keep = (old | new)[:, :, None, :, None]
        made = torch.where(keep, made.view(torch.uint8), codes.view(torch.uint8)).view(CODES[s["code"]])
        s[name].view(torch.uint8)[page[touched]] = made.view(torch.uint8)[touched]
        s[name + "_scale"][page[touched]] = grown[touched]
        out[name], out[name + "_scale"] = s[name], s[name + "_scale"]
        if name == "k":
            m, ms = _summary(made, grown, count[..., None].expand(-1, -1, h), s["code"])
            s["mean"][page[touched]], s["mean_scale"][page[touched]] = m[touched], ms[touched]
            out["mean"], out["mean_scale"] = s["mean"], s["mean_scale"]
    out["len"] = (length + n_new).to(torch.int32)
    return out


def _visible(s, Tq):
    """Keys that each query sees, [B, Tq]."""
    length = s["len"].long()[:, None]
    back = torch.arange(Tq, device=length.device) - (Tq - 1) if s["causal"] else torch.zeros(Tq, dtype=torch.long, device=length.device)
    return (length + back).clamp(min=0)


def _select(s):
    q, cap = s["q"], s["cap"]
    B, hq, Tq, d = q.shape
    h = s["k"].shape[1]
    x = q.float().view(B, h, hq // h, Tq, d)
    scale = _pow2_scale(x.abs().amax(-1), "i8")
    qi = _encode(x, scale[..., None], "i8").float()
    page = s["table"].long().clamp(min=0)
    mean = s["mean"][page].float().permute(0, 2, 3, 1)                              # [B, h, d, blocks]
    dot = torch.matmul(qi.view(B, h, -1, d), mean).view(B, h, hq // h, Tq, -1)      # whole numbers below 2^24: exact
    score = dot * (scale[..., None] * s["mean_scale"][page].permute(0, 2, 1)[:, :, None, None])
    score = score.amax(2).permute(0, 2, 1, 3)                                       # [B, Tq, h, blocks]
    nb = ((_visible(s, Tq) + BLOCK - 1) // BLOCK)[:, :, None, None]
    j = torch.arange(score.shape[-1], device=q.device)
    score = torch.where((j < s["first"]) | (j >= nb - s["last"]), math.inf, score)
    score = torch.where(j < nb, score, -math.inf)
    take = min(cap, score.shape[-1])
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :take]
    far = 1 << 30
    order = torch.where(order < nb, order, far).sort(-1).values
    cnt = (order < far).sum(-1)
    idx = torch.zeros((B, Tq, h, cap), dtype=torch.int32, device=q.device)
    idx[..., :take] = torch.where(order < far, order, 0).to(torch.int32)
    return {"idx": idx, "cnt": cnt.to(torch.int32)}


def _softmax_av(logit, seen, v):
    """exp(logit) v / sum over the last axis where `seen`; zeros and -inf where nothing is."""
    logit = torch.where(seen, logit, -math.inf)
    m = logit.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(logit - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    return o, (m + torch.log(total)).squeeze(-1)


def _attend(s):
    q = s["q"]
    B, hq, Tq, d = q.shape
    h = s["k"].shape[1]
    page = s["table"].long().clamp(min=0)
    k = (_pick(s["k"], page).float() * s["k_scale"][page][..., None, None]).transpose(1, 2).reshape(B, h, -1, d)
    at = torch.arange(k.shape[2], device=q.device)
    qf = q.float().view(B, h, -1, d) / math.sqrt(d)
    logit = torch.matmul(qf, k.transpose(-1, -2)).view(B, hq, Tq, -1)
    del k
    v = (_pick(s["v"], page).float() * s["v_scale"][page][..., None, None]).transpose(1, 2).reshape(B, h, -1, d)
    v = torch.where((at < s["len"].view(B, 1)).view(B, 1, -1, 1), v, 0.0)
    seen = (at < _visible(s, Tq)[..., None]).view(B, 1, Tq, -1)
    logit = torch.where(seen, logit, -math.inf).view(B, h, -1, at.numel())
    o, lse = _softmax_av(logit, logit > -math.inf, v)
    return {"o": o.view(B, hq, Tq, d).to(q.dtype), "lse": lse.view(B, hq, Tq)}


def _attend_blocks(s):
    q, idx, cnt = s["q"], s["idx"].long(), s["cnt"]
    B, hq, Tq, d = q.shape
    h, cap = s["k"].shape[1], idx.shape[-1]
    page = torch.gather(s["table"].long().clamp(min=0), 1, idx.view(B, -1)).view(idx.shape)        # [B, Tq, h, cap]
    head = torch.arange(h, device=q.device).view(1, 1, h, 1)
    k = (_pick(s["k"], page, head).float() * s["k_scale"][page, head][..., None, None]).view(B, Tq, h, cap * BLOCK, d)
    qf = q.float().view(B, h, hq // h, Tq, d).permute(0, 3, 1, 2, 4) / math.sqrt(d)                # [B, Tq, h, group, d]
    logit = torch.matmul(qf, k.transpose(-1, -2))
    del k
    v = (_pick(s["v"], page, head).float() * s["v_scale"][page, head][..., None, None]).view(B, Tq, h, cap * BLOCK, d)
    at = (idx[..., None] * BLOCK + torch.arange(BLOCK, device=q.device)).view(B, Tq, h, -1)
    live = (torch.arange(cap, device=q.device) < cnt[..., None]).repeat_interleave(BLOCK, -1)
    seen = live & (at < _visible(s, Tq)[:, :, None, None])
    v = torch.where(seen[..., None], v, 0.0)
    o, lse = _softmax_av(logit, seen[:, :, :, None], v)
    return {"o": o.permute(0, 2, 3, 1, 4).reshape(B, hq, Tq, d).to(q.dtype), "lse": lse.permute(0, 2, 3, 1).reshape(B, hq, Tq)}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "norm_rope":
        return {"q": _take(_norm_rope(s, s["q"], s["wq"]).to(s["q"].dtype), s["perm"]),
                "k": _take(_norm_rope(s, s["k"], s["wk"]).to(s["k"].dtype), s["perm"])}
    if op == "norm_rope_bwd":
        dq, dwq = _norm_rope_bwd(s, s["gq"], s["q"], s["wq"])
        dk, dwk = _norm_rope_bwd(s, s["gk"], s["k"], s["wk"])
        return {"dq": dq.to(s["q"].dtype), "dk": dk.to(s["k"].dtype), "dwq": dwq, "dwk": dwk}
    return {"append": _append, "select": _select, "attend": _attend, "attend_blocks": _attend_blocks}[op](s)


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    import block_sparse_attention_hilbert_b200 as svsa
    op = s["op"]
    if op.startswith("norm_rope"):
        q, k = s["q"], s["k"]
        B, hq, n, d = q.shape
        rows = n if s["perm"] is None else s["perm"].numel()
        p = svsa.norm_rope_params(q, k, s["cos"], s["pos"], rows=rows, pairs=s["pairs"], halves=s["halves"], eps=s["eps"])
        if op == "norm_rope":
            yq = torch.empty((B, hq, rows, d), dtype=q.dtype, device=q.device)
            yk = torch.empty((B, k.shape[1], rows, d), dtype=q.dtype, device=q.device)
            svsa.svsa_qk_norm_rope(q, k, s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["perm"], yq, yk, p)
            return {"q": yq, "k": yk}
        # gradients in a token-first buffer, as the projection's backward takes them
        grad = torch.empty((B, n, hq + k.shape[1], d), dtype=q.dtype, device=q.device)
        dq, dk = grad[:, :, :hq].transpose(1, 2), grad[:, :, hq:].transpose(1, 2)
        dw = torch.empty((2, d), dtype=torch.float32, device=q.device)
        ws = torch.empty(svsa.svsa_qk_norm_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device=q.device)
        svsa.svsa_qk_norm_rope_bwd(s["gq"], s["gk"], q, k, s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["iperm"], dq, dk, dw[0], dw[1], p, ws, ws.numel())
        return {"dq": dq, "dk": dk, "dwq": dw[0], "dwk": dw[1]}
    c = svsa.block_cache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["len"], s["mean"], s["mean_scale"])
    if op == "append":
        length = torch.empty_like(s["len"])
        svsa.svsa_cache_append(c, s["new_k"], s["new_v"], s["n_new"], length, svsa.cache_tokens(s["new_k"], s["new_v"]))
        return {"k": s["k"], "k_scale": s["k_scale"], "v": s["v"], "v_scale": s["v_scale"], "mean": s["mean"], "mean_scale": s["mean_scale"], "len": length}
    q = s["q"]
    B, hq, Tq, d = q.shape
    if op == "select":
        idx = torch.empty((B, Tq, s["k"].shape[1], s["cap"]), dtype=torch.int32, device=q.device)
        cnt = torch.empty(idx.shape[:3], dtype=torch.int32, device=q.device)
        svsa.svsa_cache_select(c, q, idx, cnt, svsa.cache_query(q, causal=s["causal"], cap=s["cap"], first=s["first"], last=s["last"]))
        return {"idx": idx, "cnt": cnt}
    p = svsa.cache_query(q, causal=s["causal"], cap=s["cap"])
    o = torch.empty_like(q)
    lse = torch.empty((B, hq, Tq), dtype=torch.float32, device=q.device)
    ws = torch.empty(svsa.svsa_cache_attn_workspace_bytes(c, p), dtype=torch.uint8, device=q.device)
    svsa.svsa_cache_attn(c, q, s.get("idx"), s.get("cnt"), o, lse, p, ws, ws.numel())
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- work

def work(case):
    op, B, hk, d = case["op"], case["B"], case["hk"], case["d"]
    if op.startswith("norm_rope"):
        n = case["T"] * case["H"] * case["W"]
        rows = _blocks(n) * BLOCK if case["order"] else n
        heads = case["hq"] + hk
        tables = 4 * d * (n + 4000 if case["axes"] == 1 else max(case["T"], case["H"], case["W"])) if case["axes"] else 0
        tables += 4 * case["axes"] * n * (B if case["axes"] == 1 else 1) + (4 * rows if case["order"] else 0)
        if case["axes"] == 1 and n < 4000:
            tables = 4 * d * min(B * n, n + 4000) + 4 * n * B
        if op == "norm_rope":
            return {"bytes": 2 * B * heads * d * (n + rows) + tables, "flops": 10 * B * heads * n * d}
        return {"bytes": 2 * B * heads * d * 3 * n + tables, "flops": 20 * B * heads * n * d}
    lens = _lens(case)
    nb = [_blocks(x) for x in lens]
    if op == "append":
        new = [case["N"] - (b % 3) * (case["N"] // 5) for b in range(B)]
        tail = [x % BLOCK for x in lens]
        blocks = sum(_blocks(t + m) for t, m in zip(tail, new))
        # new tokens read, their codes written, the open block's key codes read for its mean
        return {"bytes": sum(new) * hk * d * (4 + 2) + sum(t for t, m in zip(tail, new) if m) * hk * d + blocks * hk * (d + 12 + 8) + 12 * B,
                "flops": 6 * sum(new) * hk * d}
    q = 2 * B * case["hq"] * case["Tq"] * d
    if op == "select":
        return {"bytes": sum(nb) * (hk * (d + 4) + 4) + q + 4 * B * case["Tq"] * hk * (case["cap"] + 1),
                "flops": 2 * case["hq"] * case["Tq"] * d * sum(nb)}
    out = 2 * q + 4 * B * case["hq"] * case["Tq"]
    if op == "attend":
        return {"bytes": sum(lens) * hk * d * 2 + sum(nb) * (8 * hk + 4) + out, "flops": 4 * case["hq"] * case["Tq"] * d * sum(lens)}
    took = [min(case["cap"], n) for n in nb]
    # a block that several queries list is read once
    read = sum(n * (1 - (1 - t / max(n, 1)) ** case["Tq"]) for t, n in zip(took, nb))
    return {"bytes": int(read * hk * (BLOCK * d * 2 + 8) + 4 * B * case["Tq"] * hk * (case["cap"] + 1) + out),
            "flops": 4 * case["hq"] * case["Tq"] * d * BLOCK * sum(took)}


# ---------------------------------------------------------------- 64 bits

def _exact_rotate(s, y):
    """y [B, h, n, d] in 64 bits, its pairs turned as complex numbers."""
    if s["pos"] is None:
        return y
    cols, at = [], 0
    for a, m in enumerate(s["pairs"]):
        p = s["pos"][:, :, a].long()
        cols.append(torch.complex(s["cos"][:, at:at + m].double(), s["sin"][:, at:at + m].double())[p])
        at += m
    turn = torch.cat(cols, -1)[:, None]
    half = y.shape[-1] // 2
    if s["halves"]:
        z = torch.complex(y[..., :half].contiguous(), y[..., half:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)
    return torch.view_as_real(torch.view_as_complex(y.reshape(*y.shape[:-1], half, 2).contiguous()) * turn).reshape(y.shape)


def _exact_norm_rope(s, x, w):
    return _exact_rotate(s, x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w)


def _exact_out(s, y):
    if s["perm"] is None:
        return y
    pad = torch.cat([y, y.new_zeros(y.shape[0], y.shape[1], 1, y.shape[3])], 2)
    where = torch.where(s["perm"] < 0, y.shape[2], s["perm"].long())
    return pad.index_select(2, where)


def _exact_append(s):
    """The blocks' tokens one sequence and block at a time."""
    code, (h, d) = s["code"], (s["k"].shape[1], s["k"].shape[3])
    unit, most = (1.0, 127.0) if code == "i8" else (2.0 ** -9, 448.0)
    for b in range(s["len"].numel()):
        n0, m = int(s["len"][b]), int(s["n_new"][b])
        for j in range(n0 // BLOCK, -(-(n0 + m) // BLOCK) if m else 0):
            page, lo, hi = int(s["table"][b, j]), max(n0, j * BLOCK), min(n0 + m, (j + 1) * BLOCK)
            had, end = lo - j * BLOCK, hi - j * BLOCK
            for name in ("k", "v"):
                new = s["new_" + name][b, :, lo - n0:hi - n0].double()
                codes, scale = s[name][page].double(), s[name + "_scale"][page].double()
                start = scale if had > 0 else torch.zeros_like(scale)
                top = new.abs().amax((1, 2))
                need = torch.where(top > 0, 2.0 ** torch.ceil(torch.log2(top.clamp(min=1e-300) / most)).clamp(min=-126), 0.0)
                need = torch.where(need * most < top, need * 2, need)
                need = torch.where((need > 2.0 ** -126) & (need / 2 * most >= top), need / 2, need)
                grown = torch.maximum(start, need)
                div = torch.where(grown > 0, grown, 1.0)[:, None, None]
                value = torch.cat([codes[:, :had] * start[:, None, None], new], 1) / div
                value = value.round() if code == "i8" else value.float()      # exact in 32 bits: a power of two apart from its input
                s[name][page][:, :end] = value.to(CODES[code])
                s[name + "_scale"][page] = grown.float()
                if name == "k":
                    mean = s["k"][page][:, :end].double().sum(1) / unit / end
                    ms = mean.abs().amax(-1)
                    e = torch.where(ms > 0, 2.0 ** torch.ceil(torch.log2(ms.clamp(min=1e-300) / 127)), 0.0)
                    e = torch.where(e * 127 < ms, e * 2, e)
                    e = torch.where((e > 0) & (e / 2 * 127 >= ms), e / 2, e)
                    s["mean"][page] = (mean / torch.where(e > 0, e, 1.0)[:, None]).round().to(torch.int8)
                    s["mean_scale"][page] = (e * unit * grown).float()
    return {"k": s["k"], "k_scale": s["k_scale"], "v": s["v"], "v_scale": s["v_scale"], "mean": s["mean"], "mean_scale": s["mean_scale"], "len": None}


def _exact_attend(s, case):
    q, lens = s["q"].double(), _lens(case)
    B, hq, Tq, d = q.shape
    h, g = s["k"].shape[1], q.shape[1] // s["k"].shape[1]
    o, lse = torch.zeros_like(q), torch.full((B, hq, Tq), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        page = s["table"][b, :_blocks(lens[b])].long()
        for e in range(h):
            k = (_pick(s["k"], page, e).double() * s["k_scale"][page, e].double()[:, None, None]).reshape(-1, d)[:lens[b]]
            v = (_pick(s["v"], page, e).double() * s["v_scale"][page, e].double()[:, None, None]).reshape(-1, d)[:lens[b]]
            logit = q[b, e * g:(e + 1) * g] @ k.T / math.sqrt(d)                 # [g, Tq, len]
            at = torch.arange(lens[b], device=q.device)
            for t in range(Tq):
                see = at <= lens[b] - Tq + t if s["causal"] else at >= 0
                if "idx" in s:
                    mine = torch.zeros(page.numel(), dtype=torch.bool, device=q.device)
                    mine[s["idx"][b, t, e, :int(s["cnt"][b, t, e])].long()] = True
                    see = see & mine[at // BLOCK]
                if bool(see.any()):
                    z = logit[:, t][:, see]
                    o[b, e * g:(e + 1) * g, t] = torch.softmax(z, -1) @ v[see]
                    lse[b, e * g:(e + 1) * g, t] = torch.logsumexp(z, -1)
    return {"o": o, "lse": lse}


def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None                                          # whole numbers
    s = prepare(case, seed)
    if op == "norm_rope":
        return {"q": _exact_out(s, _exact_norm_rope(s, s["q"].double(), s["wq"].double())),
                "k": _exact_out(s, _exact_norm_rope(s, s["k"].double(), s["wk"].double()))}
    if op == "norm_rope_bwd":
        out = {}
        for x, w, g in (("q", "wq", "gq"), ("k", "wk", "gk")):
            a, b = s[x].double().requires_grad_(), s[w].double().requires_grad_()
            out["d" + x], out["d" + w] = torch.autograd.grad(_exact_out(s, _exact_norm_rope(s, a, b)), (a, b), s[g].double())
        return out
    if op == "append":
        return _exact_append(s)
    return _exact_attend(s, case)
