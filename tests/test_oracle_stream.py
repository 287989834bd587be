"""Pins for the oracle's norm, rotation, 8-bit cache and cache attention (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import stream


def _angles(rng, shape, d):
    t = rng.uniform(-3, 3, shape + (d // 2,))
    return np.cos(t), np.sin(t)


@pytest.mark.parametrize("halves", [False, True])
def test_rotation_is_complex_multiplication_and_keeps_norms(halves):
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((5, 16)), rng.uniform(0.5, 1.5, 16)
    c, s = _angles(rng, (5,), 16)
    plain = stream.norm_rope(x, w, None, None, halves, 1e-6)
    got = stream.norm_rope(x, w, c, s, halves, 1e-6)
    z = plain[:, :8] + 1j * plain[:, 8:] if halves else plain[:, 0::2] + 1j * plain[:, 1::2]
    z = z * (c + 1j * s)
    want = np.concatenate([z.real, z.imag], -1) if halves else np.stack([z.real, z.imag], -1).reshape(5, 16)
    assert np.allclose(got, want, atol=1e-14)
    assert np.allclose(np.linalg.norm(got, axis=-1), np.linalg.norm(plain, axis=-1))


def test_norm_is_the_library_rms_norm():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((7, 64)), rng.uniform(0.5, 1.5, 64)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), eps=1e-5).numpy()
    assert np.allclose(stream.norm_rope(x, w, None, None, False, 1e-5), want, atol=1e-14)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("turn", [False, True])
def test_gradients_match_central_differences(halves, turn):
    rng = np.random.default_rng(2)
    x, w, g = rng.standard_normal((3, 8)), rng.uniform(0.5, 1.5, 8), rng.standard_normal((3, 8))
    c, s = _angles(rng, (3,), 8) if turn else (None, None)
    f = lambda x, w: float((g * stream.norm_rope(x, w, c, s, halves, 1e-3)).sum())
    dx, dw = stream.norm_rope_bwd(g, x, w, c, s, halves, 1e-3)
    h = 1e-5                                               # error of the difference ~ h^2 + 1e-16 / h
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-8
    for i in range(8):
        e = np.zeros(8)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw.sum(0)[i]) < 1e-8


def test_e4m3_values_and_rounding_are_the_library_type():
    bytes_ = np.arange(256, dtype=np.uint8)
    lib = torch.from_numpy(bytes_).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(lib, stream.E4M3, equal_nan=True)
    # every value, every midpoint of neighbours, and points around them
    v = stream.E4M3[:127]
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, mid * (1 + 2**-20), mid * (1 - 2**-20)])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(stream.encode(x, 1.0, "e4m3"), want)
    # brute force: no other code is nearer
    y = np.random.default_rng(3).uniform(-448, 448, 200)
    got = stream.E4M3[stream.encode(y, 1.0, "e4m3")]
    assert np.all(np.abs(got - y) <= np.nanmin(np.abs(stream.E4M3[None] - y[:, None]), axis=1))


def test_int8_rounding_and_saturation():
    x = np.array([0.5, 1.5, -0.5, -2.5, 126.5, 200.0, -200.0])
    assert list(stream.encode(x, 1.0, "i8").view(np.int8)) == [0, 2, 0, -2, 126, 127, -127]


@pytest.mark.parametrize("code", ["e4m3", "i8"])
def test_scale_is_the_smallest_power_of_two_that_holds_the_largest(code):
    top = stream.TOP[code]
    for a in (top, top * (1 + 2**-20), 1.0, 3e-5, 1e30, top / 2, 1e-30):
        s = stream.pow2_scale(a, code)
        assert math.frexp(s)[0] == 0.5 and a / s <= top and a / (s / 2) > top
    assert stream.pow2_scale(0.0, code) == 0.0


def _empty(rng, n_pages, heads, d, table, length, code):
    z = np.zeros((n_pages, heads, 64, d), np.uint8)
    s = np.zeros((n_pages, heads))
    return stream.BlockCache(z, z, s, s, np.zeros((n_pages, heads, d), np.int8), s, table, length, code)


@pytest.mark.parametrize("code", ["e4m3", "i8"])
def test_appending_holds_every_value_within_half_a_step(code):
    rng = np.random.default_rng(4)
    k, v = rng.standard_normal((2, 1, 2, 100, 8))
    c = _empty(rng, 3, 2, 8, np.array([[2, 0]]), [0], code)
    c.append(k, v, [100])
    for h in range(2):
        kk, vv = c.tokens(0, h)
        for got, x, sc in ((kk, k[0, h], c.k_scale), (vv, v[0, h], c.v_scale)):
            step = np.repeat(sc[[2, 0], h], 64)[:100, None]
            bound = step / 2 if code == "i8" else np.maximum(np.abs(x) * 2**-4, step * 2.0**-10)
            assert np.all(np.abs(got - x) <= bound)
    # the mean is the mean of what is held, to half a step of its own scale
    for j, n in ((0, 64), (1, 36)):
        page = c.table[0, j]
        held = c.tokens(0, 1)[0][64 * j:64 * j + n].mean(0)
        assert np.all(np.abs(c.mean[page, 1] * c.mean_scale[page, 1] - held) <= c.mean_scale[page, 1] * (0.5 + 1e-12))


def test_a_block_whose_scale_grows_is_held_in_the_new_scale():
    rng = np.random.default_rng(5)
    c = _empty(rng, 1, 1, 4, np.array([[0]]), [0], "i8")
    k = np.full((1, 1, 2, 4), 127.0)
    k[0, 0, 1] = 254.0
    c.append(k[:, :, :1], k[:, :, :1], [1])
    assert c.k_scale[0, 0] == 1.0 and list(c.k[0, 0, 0].view(np.int8)) == [127] * 4
    c.append(k[:, :, 1:], k[:, :, 1:], [1])
    assert c.k_scale[0, 0] == 2.0
    assert list(c.k[0, 0, 0].view(np.int8)) == [64] * 4 and list(c.k[0, 0, 1].view(np.int8)) == [127] * 4


def test_selection_keeps_the_forced_blocks_and_the_largest_scores():
    rng = np.random.default_rng(6)
    c = _empty(rng, 7, 1, 8, np.arange(7)[None], [0], "i8")
    k = rng.integers(-5, 6, (1, 1, 400, 8)).astype(float)
    c.append(k, k, [400])
    q = rng.integers(-127, 128, (1, 2, 1, 8)).astype(float)
    q[..., 0] = 127                                        # scale 1: the codes are the values
    got = stream.select_blocks(c, q, 4, 1, 1, True)[0, 0, 0]
    score = np.array([max(float(q[0, e, 0] @ (c.mean[j, 0] * c.mean_scale[j, 0])) for e in range(2)) for j in range(7)])
    rest = sorted(range(1, 6), key=lambda j: (-score[j], j))[:2]
    assert got == sorted([0, 6] + rest)
    # equal scores: the lower index
    c.mean[:], c.mean_scale[:] = 1, 1.0
    assert stream.select_blocks(c, q, 3, 0, 0, True)[0, 0, 0] == [0, 1, 2]


@pytest.mark.parametrize("causal", [False, True])
def test_cache_attention_is_the_library_attention(causal):
    rng = np.random.default_rng(7)
    c = _empty(rng, 3, 2, 8, np.array([[1, 2, 0]]), [0], "i8")
    kv = rng.standard_normal((2, 1, 2, 150, 8))
    c.append(kv[0], kv[1], [150])
    q = rng.standard_normal((1, 4, 3, 8))
    o, lse = stream.cache_attention(c, q, causal)
    k, v = (np.stack([c.tokens(0, h)[i] for h in (0, 0, 1, 1)])[None] for i in (0, 1))
    mask = np.arange(150)[None] <= (150 - 3 + np.arange(3))[:, None] if causal else np.ones((3, 150), bool)
    want = torch.nn.functional.scaled_dot_product_attention(*map(torch.from_numpy, (q, k, v)), attn_mask=torch.from_numpy(mask))
    assert np.allclose(o, want.numpy(), atol=1e-12)
    s = np.where(mask, q @ k.transpose(0, 1, 3, 2) / math.sqrt(8), -np.inf)
    assert np.allclose(lse, torch.logsumexp(torch.from_numpy(s), -1).numpy(), atol=1e-12)


def test_queries_that_see_nothing_give_zeros():
    rng = np.random.default_rng(8)
    c = _empty(rng, 1, 1, 8, np.array([[0]]), [0], "i8")
    kv = rng.standard_normal((2, 1, 1, 2, 8))
    c.append(kv[0], kv[1], [2])
    o, lse = stream.cache_attention(c, rng.standard_normal((1, 1, 4, 8)), True)
    assert np.all(o[0, 0, :2] == 0) and np.all(lse[0, 0, :2] == -np.inf) and np.all(np.isfinite(lse[0, 0, 2:]))
    assert np.allclose(o[0, 0, 2], c.tokens(0, 0)[1][0])   # one key: its value
