"""Argument checks of the streaming entry points (no GPU: everything is refused before a launch)."""
import ctypes
import os

import pytest
import torch

import block_sparse_attention_hilbert_b200 as svsa
from block_sparse_attention_hilbert_b200 import Cache, CacheQuery, CacheTokens, NormRopeParams

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _err():
    return svsa.lib().svsa_last_error().decode()


def test_struct_layouts_match_the_c_compiler(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    structs = {"svsa_norm_rope": NormRopeParams, "svsa_cache": Cache, "svsa_cache_tokens": CacheTokens,
               "svsa_cache_query": CacheQuery}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "svsa.h"', "int main(void) {"]
    for cname, cls in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f[0]} %zu\\n", offsetof({cname}, {f[0]}));' for f in cls._fields_]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    seen = 0
    for line in filter(None, out):
        cname, field, val = line.split()
        cls = structs[cname]
        assert int(val) == (ctypes.sizeof(cls) if field == "size" else getattr(cls, field).offset), line
        seen += 1
    assert seen == sum(len(c._fields_) + 1 for c in structs.values())


def test_status_code():
    text = open(os.path.join(ROOT, "include", "svsa.h")).read()
    assert "SVSA_ERR_INDEX = 8" in text and svsa.STATUS[8] == "INDEX"


# ---- C entry points -----------------------------------------------------------

def _rope(**kw):
    f = dict(B=1, heads_q=4, heads_k=2, N=10, rows=10, d=64, dtype=0, pairing=0, axes=1, pairs=(32, 0, 0),
             table_rows=16, eps=1e-6, pos_stride=0, q_stride=(4 * 640, 640, 64), k_stride=(2 * 640, 640, 64),
             dq_stride=(4 * 640, 640, 64), dk_stride=(2 * 640, 640, 64))
    f.update(kw)
    return NormRopeParams(*(f[n] for n, _ in NormRopeParams._fields_))


def _fwd(p, q=16, k=32, wq=48, wk=64, cos=80, sin=96, pos=112, mp=None, yq=144, yk=160):
    return svsa.lib().svsa_qk_norm_rope(q, k, wq, wk, cos, sin, pos, mp, yq, yk, p, None)


def _bwd(p, dyq=16, dyk=32, q=48, k=64, wq=80, wk=96, cos=112, sin=128, pos=144, imap=None, dq=176, dk=192, dwq=208,
         dwk=224, ws=240, ws_bytes=1 << 30):
    return svsa.lib().svsa_qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, cos, sin, pos, imap, dq, dk, dwq, dwk, p, ws, ws_bytes,
                                            None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(rows=0), 1), (dict(heads_q=0), 1), (dict(heads_k=-1), 1), (dict(d=96), 2),
    (dict(dtype=2), 2), (dict(pairing=2), 1), (dict(axes=4), 1), (dict(axes=-1), 1), (dict(pairs=(31, 0, 0)), 1),
    (dict(axes=2, pairs=(40, -8, 0)), 1), (dict(table_rows=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(pos_stride=-1), 1), (dict(q_stride=(2560, 640, 60)), 1), (dict(k_stride=(1280, -640, 64)), 1),
    (dict(rows=12), 1), (dict(B=1 << 16, N=1 << 15, rows=1 << 15), 2)])
def test_norm_rope_rejects(kw, status):
    p = _rope(**kw)
    assert _fwd(p) == status and _err()
    assert _bwd(p) == status and _err()


def test_norm_rope_rejects_pointers():
    p = _rope()
    for bad in (dict(q=None), dict(k=None), dict(q=17), dict(wq=50), dict(cos=None), dict(sin=None), dict(pos=None),
                dict(mp=20), dict(yq=None), dict(yk=None), dict(yq=16), dict(yk=32), dict(yk=144)):
        assert _fwd(p, **bad) == 1, bad
    assert svsa.lib().svsa_qk_norm_rope(16, 32, 48, 64, 80, 96, 112, None, 144, 160, None, None) == 1
    for bad in (dict(dyq=None), dict(dq=None), dict(dk=None), dict(dq=16), dict(dq=48), dict(dk=176), dict(dwq=210),
                dict(ws=None)):
        assert _bwd(p, **bad) == 1, bad
    need = svsa.svsa_qk_norm_rope_bwd_workspace_bytes(p)
    assert need > 0 and _bwd(p, ws_bytes=need - 1) == 3
    # rows of the gradients that overlap: a head broadcast by a stride of 0, tokens closer than a row
    assert _bwd(_rope(dq_stride=(2560, 0, 64))) == 1 and "overlap" in _err()
    assert _bwd(_rope(dk_stride=(1280, 640, 32))) == 1 and "overlap" in _err()


CACHE = dict(k=16, v=32, k_scale=48, v_scale=64, mean=80, mean_scale=96, table=112, len=128, B=2, heads=2, d=128, code=0,
             n_pages=9, max_blocks=5)
QUERY = dict(heads_q=4, Tq=1, dtype=0, causal=1, cap=3, first=1, last=1)


def _cache(**kw):
    f = {**CACHE, **kw}
    return Cache(*(f[n] for n, _ in Cache._fields_))


def _query(**kw):
    f = {**QUERY, **kw}
    return CacheQuery(*(f[n] for n, _ in CacheQuery._fields_))


def _append(c, N=3, dtype=0, ks=(768, 384, 128), vs=(768, 384, 128), k=144, v=160, n_new=None, len_out=None):
    return svsa.lib().svsa_cache_append(c, k, v, n_new, len_out, CacheTokens(N, dtype, ks, vs), None)


def _select(c, p, q=144, idx=160, cnt=176):
    return svsa.lib().svsa_cache_select(c, q, idx, cnt, p, None)


def _attn(c, p, q=144, idx=None, cnt=None, o=160, lse=None, ws=192, ws_bytes=1 << 30):
    return svsa.lib().svsa_cache_attn(c, q, idx, cnt, o, lse, p, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(heads=0), 1), (dict(n_pages=0), 1), (dict(max_blocks=0), 1), (dict(d=96), 2), (dict(code=2), 2),
    (dict(n_pages=1 << 24), 2), (dict(max_blocks=(1 << 24) + 1), 2), (dict(k=None), 1), (dict(v=33), 1),
    (dict(k_scale=None), 1), (dict(v_scale=None), 1), (dict(table=None), 1), (dict(len=None), 1), (dict(mean=None), 1),
    (dict(mean_scale=None), 1)])
def test_cache_rejects(kw, status):
    c = _cache(**kw)
    for got in (_append(c), _select(c, _query()), _attn(c, _query(heads_q=4))):
        assert got == status and _err()


def test_cache_without_means_appends_and_attends_but_does_not_select():
    c = _cache(mean=None, mean_scale=None)
    assert _select(c, _query()) == 1 and "mean" in _err()
    # (the others get as far as the argument that is wrong here)
    assert _append(c, k=None) == 1 and "k is NULL" in _err()
    assert _attn(c, _query(), q=None) == 1 and "q is NULL" in _err()


def test_append_of_more_tokens_than_fit_32_bits_of_blocks():
    assert _append(_cache(B=1 << 20, heads=1 << 10), N=1 << 30) == 2
    # (the most tokens that a call can name pass the size check, and fail at the pointer)
    assert _append(_cache(B=1, heads=1), N=2**31 - 1, k=None) == 1 and "k is NULL" in _err()


def test_append_rejects():
    c = _cache()
    for bad in (dict(N=0), dict(ks=(768, 384, 4)), dict(vs=(768, -384, 128)), dict(k=None), dict(v=161), dict(n_new=3),
                dict(len_out=5), dict(len_out=128), dict(n_new=208, len_out=208)):
        assert _append(c, **bad) == 1, bad
    assert _append(c, dtype=7) == 2
    assert _append(_cache(v=16)) == 1 and _append(_cache(v_scale=48)) == 1
    assert svsa.lib().svsa_cache_append(c, 144, 160, None, None, None, None) == 1
    assert svsa.lib().svsa_cache_append(None, 144, 160, None, None, CacheTokens(1, 0, (8, 8, 8), (8, 8, 8)), None) == 1


def test_select_and_attention_reject():
    c = _cache()
    for bad in (dict(heads_q=0), dict(heads_q=3), dict(Tq=0), dict(causal=2)):
        assert _select(c, _query(**bad)) == 1 and _attn(c, _query(**bad)) == 1, bad
    assert _select(c, _query(dtype=2)) == 2 and _attn(c, _query(dtype=2)) == 2
    assert _attn(c, _query(Tq=1 << 25)) == 2
    for bad in (dict(cap=0), dict(first=-1), dict(last=-1), dict(first=2, last=2)):
        assert _select(c, _query(**bad)) == 1, bad
    assert _select(_cache(max_blocks=32769), _query()) == 2
    assert _select(c, _query(heads_q=2 * 129)) == 2
    for bad in (dict(q=None), dict(idx=None), dict(cnt=None), dict(q=145)):
        assert _select(c, _query(), **bad) == 1, bad
    assert _select(c, None) == 1 and _attn(c, None) == 1 and _attn(None, _query()) == 1
    for bad in (dict(q=None), dict(o=None), dict(o=144), dict(lse=3), dict(idx=208), dict(cnt=208), dict(ws=None)):
        assert _attn(c, _query(), **bad) == 1, bad
    assert _attn(c, _query(cap=0), idx=208, cnt=224) == 1
    need = svsa.svsa_cache_attn_workspace_bytes(c, _query())
    assert need > 0 and _attn(c, _query(), ws_bytes=need - 1) == 3
    assert svsa.lib().svsa_cache_attn_workspace_bytes(None, None) == 0


# ---- the binding's checks of tensors -------------------------------------------

def test_binding_checks_tensors():
    q = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16)
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    cos, pos = torch.zeros(8, 32), torch.zeros(1, 3, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        svsa.norm_rope_params(q.float(), k)
    with pytest.raises(ValueError):
        svsa.norm_rope_params(q.transpose(2, 3), k)
    with pytest.raises(ValueError):
        svsa.norm_rope_params(q, k.half())
    with pytest.raises(ValueError):
        svsa.norm_rope_params(q, k, pairs=(32,))
    p = svsa.norm_rope_params(q, k, cos, pos, pairs=(32,))
    good = dict(q=q, k=k, wq=None, wk=None, cos=cos, sin=cos, pos=pos, perm=None, yq=torch.empty_like(q), yk=torch.empty_like(k))
    for name, t in (("q", q.half()), ("q", q[:, :, :2]), ("k", None), ("k", k.half()), ("wq", torch.zeros(32)),
                    ("cos", cos.double()), ("sin", None), ("sin", cos[:4]), ("pos", pos.long()),
                    ("perm", torch.zeros(4, dtype=torch.int32)), ("yq", q.transpose(1, 2).contiguous().transpose(1, 2)),
                    ("yk", q)):
        with pytest.raises(ValueError):
            svsa.svsa_qk_norm_rope(**{**good, name: t}, p=p)
    codes, sc = torch.zeros(3, 2, 64, 64, dtype=torch.int8), torch.zeros(3, 2)
    tab, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in ((codes.float(), codes, sc, sc, tab, n), (codes[:, :, :32], codes, sc, sc, tab, n),
                (codes, codes[:2], sc, sc, tab, n), (codes, codes, sc.double(), sc, tab, n),
                (codes, codes, sc, sc, tab.long(), n), (codes, codes, sc, sc, tab, n[:1]),
                (codes, codes, sc, sc, tab.t().contiguous().t(), n)):
        with pytest.raises(ValueError):
            svsa.block_cache(*bad)
    c = svsa.block_cache(codes, codes.clone(), sc, sc.clone(), tab, n)
    with pytest.raises(ValueError):
        svsa.cache_tokens(k, k.half())
    t = svsa.cache_tokens(k, k)
    with pytest.raises(ValueError):
        svsa.svsa_cache_append(c, k[:1], k, None, None, t)
    with pytest.raises(ValueError):
        svsa.svsa_cache_append(c, k, k, n.long(), None, t)
    qp = svsa.cache_query(q, cap=2)
    with pytest.raises(ValueError):
        svsa.svsa_cache_attn(c, q.half(), None, None, q, None, qp, None, 0)
    with pytest.raises(ValueError):
        svsa.svsa_cache_attn(c, q, None, None, torch.empty_like(q).half(), None, qp, None, 0)
    ws = torch.zeros(svsa.svsa_cache_attn_workspace_bytes(c, qp) - 1, dtype=torch.uint8)
    with pytest.raises(ValueError):                        # fewer bytes than the call says
        svsa.svsa_cache_attn(c, q, None, None, torch.empty_like(q), None, qp, ws, ws.numel() + 1)
    with pytest.raises(ValueError):
        svsa.svsa_cache_select(c, q, torch.zeros(2, 3, 2, 3, dtype=torch.int32), torch.zeros(2, 3, 2, dtype=torch.int32), qp)


def test_layer_classes_check_their_arguments():
    with pytest.raises(ValueError):
        svsa.NormRope(64, pairs=(16, 8), rows=4, device="cpu")
    with pytest.raises(ValueError):
        svsa.NormRope(64, pairs=(32,), device="cpu")
    with pytest.raises(ValueError):
        svsa.BlockCache(2, 1, 64, 200, n_pages=7, device="cpu")
    with pytest.raises(ValueError):
        svsa.BlockCache(2, 1, 64, 200, table=torch.zeros(2, 4, dtype=torch.int32), device="cpu")
    c = svsa.BlockCache(2, 1, 64, 200, code="i8", means=False, device="cpu")
    assert c.table.tolist() == [[0, 1, 2, 3], [4, 5, 6, 7]] and c.cache.mean is None and c.cache.code == svsa.CODE_I8
    with pytest.raises(ValueError):
        svsa.SparseVideoAttention(1, 1, 2, 8, 8, 64, order="cocluster", norm_rope=(None, None), device="cpu")


def test_rope_tables_and_grid_positions():
    cos, sin = svsa.rope_tables(9, (3, 1), theta=100.0, device="cpu")
    assert cos.shape == (9, 4)
    f = torch.tensor([1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3), 1.0], dtype=torch.float64)
    want = torch.arange(9, dtype=torch.float64)[:, None] * f
    # one rounding to fp32: at most half a step
    assert (cos.double() - want.cos()).abs().max() <= 2.0**-24 and (sin.double() - want.sin()).abs().max() <= 2.0**-24
    pos = svsa.grid_positions(2, 3, 4, frame=5, device="cpu")
    assert pos.shape == (1, 24, 3) and pos[0, 0].tolist() == [5, 0, 0] and pos[0, 23].tolist() == [6, 2, 3]
    assert pos[0, 1 * 12 + 2 * 4 + 1].tolist() == [6, 2, 1]


def test_strides_of_dimensions_of_size_one_are_not_looked_at():
    """A dimension of size 1 is never stepped along (each call gets as far as the missing pointer)."""
    odd = (3, 640, 64)
    for p in (_rope(q_stride=odd), _rope(k_stride=(-7, 640, 64)), _rope(heads_q=1, q_stride=(1, 1 << 50, 64)),
              _rope(N=1, rows=1, q_stride=(2560, 64, 1), k_stride=(0, 64, 3))):
        assert _fwd(p, yq=None) == 1 and "yq is NULL" in _err()
    for p in (_rope(dq_stride=odd), _rope(dk_stride=(-1, 640, 64))):
        assert _bwd(p, ws=None) == 1 and "ws is NULL" in _err()
    c = _cache(B=1, heads=1)
    assert _append(c, N=1, ks=(1, 2, 3), vs=(-1, 5, 7), k=None) == 1 and "k is NULL" in _err()
    # those of the others still are
    assert _fwd(_rope(q_stride=(3, 641, 64))) == 1 and _append(c, N=2, ks=(1, 2, 3)) == 1
    # and a view may differ from the parameters' tensor there
    q = torch.zeros(1, 4, 3, 64, dtype=torch.bfloat16)
    other = torch.zeros(7, 4, 3, 64, dtype=torch.bfloat16)[::7].as_strided((1, 4, 3, 64), (5, 192, 64, 1))
    p = svsa.norm_rope_params(q, None)
    for x in (q, other):                                   # (as far as the device)
        with pytest.raises(ValueError, match="CUDA"):
            svsa.svsa_qk_norm_rope(x, None, None, None, None, None, None, None, torch.empty_like(q), None, p)
