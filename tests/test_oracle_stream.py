"""Pins of the streaming operators' fp64 oracle (oracle/stream.py) against
closed forms, invariants and brute force."""
import numpy as np
import pytest
import torch

from oracle import stream as so


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("ladder", ["axis", "shared"])
def test_rope_is_a_rotation_that_sees_position_differences(pairing, ladder):
    rng = np.random.default_rng(3)
    dims = (48, 40, 24)
    q, k = rng.standard_normal((2, 5, 2, 128))
    pos = rng.integers(-50, 50, (5, 3))
    kw = dict(dims=dims, pairing=pairing, ladder=ladder)
    rq, rk = so.rope(q, pos, **kw), so.rope(k, pos, **kw)
    np.testing.assert_allclose((rq ** 2).sum(-1), (q ** 2).sum(-1), rtol=1e-12)
    np.testing.assert_array_equal(rq[..., 112:], q[..., 112:])          # channels behind the rotated ones
    np.testing.assert_allclose(so.rope(rq, pos, inverse=True, **kw), q, atol=1e-12)
    # scores between two positions depend on their difference alone
    a = (so.rope(q, pos, **kw)[0, 0] * so.rope(k, pos, **kw)[1, 0]).sum()
    far = pos + np.array([1000, -77, 5])
    np.testing.assert_allclose((so.rope(q, far, **kw)[0, 0] * so.rope(k, far, **kw)[1, 0]).sum(), a, rtol=1e-9)
    # a quarter turn of the first pair: frequency 1
    x = np.zeros((1, 1, 128))
    x[0, 0, 0] = 1.0
    b = 1 if pairing == "interleaved" else 56
    y = so.rope(x, np.array([[np.pi / 2, 0, 0]]), **kw)
    assert abs(y[0, 0, 0]) < 1e-15 and abs(y[0, 0, b] - 1) < 1e-15


def test_e4m3_rounding_against_torch_and_brute_force():
    v = so.e4m3_values()
    assert v[126] == 448.0 and v[1] == 2.0 ** -9 and np.isnan(v[127]) and np.isnan(v[255])
    torch_v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(np.nan_to_num(torch_v, nan=1e9), np.nan_to_num(v, nan=1e9))
    rng = np.random.default_rng(4)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 8, 4000), v[:127],
                        (v[:126] + v[1:127]) / 2, -(v[:126] + v[1:127]) / 2, [0.0, -0.0]])
    x = x[np.abs(x) <= 448]
    got = so.round_e4m3(x)
    ref = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    same32 = x.astype(np.float32).astype(np.float64) == x
    np.testing.assert_array_equal(got[same32], ref[same32])
    assert so.round_e4m3([np.inf, np.nan, -np.inf]).tolist() == [127] * 3


def test_page_exponent_is_the_least_that_fits():
    for a, e in ((448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (1.0, -8), (0.0, -117), (2.0 ** -130, -117)):
        assert so.page_exponent(a) == e
        assert a <= 448 * 2.0 ** e and (e == -117 or a > 448 * 2.0 ** (e - 1))


def test_cache_write_in_parts_and_whole():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((300, 2, 128)) * np.exp(rng.standard_normal((300, 1, 1)))
    one = np.zeros((4, 2, 128, 128), np.uint8), np.zeros((4, 2), np.float32)
    two = np.zeros((4, 2, 128, 128), np.uint8), np.zeros((4, 2), np.float32)
    table = np.array([[2, 0, 3]])
    so.cache_write(x, *one, [0, 300], [300], table)
    done = 0
    for m in (1, 59, 140, 100):
        so.cache_write(x[done:done + m], *two, [0, m], [done + m], table)
        done += m
    np.testing.assert_array_equal(one[1], two[1])
    a, b = so.e4m3_values()[one[0]], so.e4m3_values()[two[0]]
    # the same but for what a larger exponent pushed into the subnormals: one more rounding of at most 2^-10
    assert np.all(np.abs(a - b) <= 2.0 ** -9) and np.mean(a != b) < 1e-3
    assert np.all(one[0][1] == 0)  # the page that no table names


def test_cache_attention_closed_forms():
    c = np.zeros((3, 1, 128, 128), np.uint8)
    v = so.round_e4m3(np.random.default_rng(6).standard_normal((3, 1, 128, 128)))
    s = np.full((3, 1), 0.5, np.float32)
    q = np.random.default_rng(7).standard_normal((2, 4, 128))
    table = np.array([[1, 2, 0]])
    # keys of zero: the mean of the visible values, lse = ln of their count
    o, lse, _ = so.cache_attention(q, c, v, s, s, [0, 4], [200], table, 1.0, unit=1)
    vals = (so.e4m3_values()[v[[1, 2, 0], 0]] * 0.5).reshape(-1, 128)
    for i in range(4):
        np.testing.assert_allclose(o[1, i], vals[:197 + i].mean(0), atol=1e-13)
        np.testing.assert_allclose(lse[1, i], np.log(197 + i))
    # frames of 50: the last four tokens share the frame 150 .. 199
    np.testing.assert_allclose(so.cache_attention(q, c, v, s, s, [0, 4], [200], table, 1.0, unit=50)[1], np.log(200))
    # more tokens than cached: the first ones see nothing
    o, lse, _ = so.cache_attention(q, c, v, s, s, [0, 4], [2], table, 1.0, unit=1)
    assert np.isneginf(lse[0, :2]).all() and (o[0, :2] == 0).all() and np.allclose(lse[0, 2:], np.log([1, 2]))
