"""Streaming operators on the GPU against the fp64 oracle: rotary positions
(forward, gradient), writing the paged 8-bit cache, attention over it, and the
three together as a frame-by-frame generator uses them."""
import math

import numpy as np
import pytest
import torch

from gpu_util import bf16_to_f64, require_gpu

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module")
def binding():
    return require_gpu()


@pytest.fixture(scope="module")
def so():
    from oracle import stream
    return stream


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g).bfloat16()


# ---------------------------------------------------------------------------- rotary positions

def _grid_pos(n, H, W, start):
    t = np.arange(n)
    return np.stack([start[0] + t // (H * W), start[1] + t % (H * W) // W, start[2] + t % W], 1)


def _rope_close(got, ref, x):
    """One rounding to bf16 (2^-8 of the value), and fp32 before it: the fraction of a turn (2^-26), its
    sine and cosine (2 units of 2^-24), two products and a sum (1.5 units): under 2^-21 of |x_a| + |x_b|,
    taken here as twice the token's largest value."""
    tol = BF16 * np.abs(ref) + 2.0 ** -20 * np.abs(x).max(-1, keepdims=True)
    assert got.shape == ref.shape
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))


@pytest.mark.parametrize("pairing,dims", [("interleaved", (44, 42, 42)), ("interleaved", (0, 30, 32)),
                                          ("interleaved", (2, 0, 0)), ("halves", (44, 42, 42)),
                                          ("halves", (16, 0, 16)), ("halves", (48, 40, 24))])
@pytest.mark.parametrize("ladder", ["axis", "shared"])
@pytest.mark.parametrize("n,hq,hk", [(1, 1, 0), (1, 40, 8), (3, 5, 1), (129, 3, 3), (1000, 2, 1)])
def test_rope_matches_oracle(binding, so, pairing, dims, ladder, n, hq, hk):
    g = _gen(n + hq)
    q, k = _randn(g, n, hq, 128), _randn(g, n, hk, 128)
    plan = binding.rope_plan(dims, pairing=pairing, ladder=ladder)
    kw = dict(dims=dims, pairing=pairing, ladder=ladder)
    H, W, start = 7, 9, (123456, 3, -2)
    pos = _grid_pos(n, H, W, start)
    qr, kr = binding.rope_fwd(q.cuda(), k.cuda() if hk else None, plan, grid=(H, W), start=start)
    assert qr.shape == (hq, n, 128) and qr.is_contiguous()
    _rope_close(bf16_to_f64(qr).transpose(1, 0, 2), so.rope(bf16_to_f64(q), pos, **kw), bf16_to_f64(q))
    if hk:
        _rope_close(bf16_to_f64(kr).transpose(1, 0, 2), so.rope(bf16_to_f64(k), pos, **kw), bf16_to_f64(k))
    else:
        assert kr is None
    # explicit positions, far and negative ones
    pos = np.random.default_rng(n).integers(-2 ** 31, 2 ** 31, (n, 3))
    pos[n // 2:] = np.random.default_rng(n).integers(-500, 500, (n - n // 2, 3))
    dpos = torch.from_numpy(pos.astype(np.int32)).cuda()
    qr, _ = binding.rope_fwd(q.cuda(), None, plan, pos=dpos)
    # the oracle's own angle is a product rounded to 2^-53 of up to 2^31 radians: 2^-22; the kernel's likewise
    ref = so.rope(bf16_to_f64(q), pos, **kw)
    tol = BF16 * np.abs(ref) + 2.0 ** -19 * np.abs(bf16_to_f64(q)).max(-1, keepdims=True)
    assert np.all(np.abs(bf16_to_f64(qr).transpose(1, 0, 2) - ref) <= tol)
    # gradient: the oracle's inverse rotation
    dq = _randn(g, hq, n, 128)
    got, _ = binding.rope_bwd(dq.cuda(), None, plan, pos=dpos)
    ref = so.rope(bf16_to_f64(dq).transpose(1, 0, 2), pos, inverse=True, **kw)
    assert got.shape == (n, hq, 128)
    tol = BF16 * np.abs(ref) + 2.0 ** -19 * np.abs(bf16_to_f64(dq)).transpose(1, 0, 2).max(-1, keepdims=True)
    assert np.all(np.abs(bf16_to_f64(got) - ref) <= tol)


def test_rope_gradient_against_differences(binding, so):
    """d/dx of sum(w * rope(x)): the rotation is linear, so a difference over any step is the derivative."""
    g = _gen(5)
    x, w = _randn(g, 6, 2, 128), _randn(g, 2, 6, 128)
    pos = np.array([[i, 2 * i, 5 - i] for i in range(6)])
    plan = binding.rope_plan()
    dx, _ = binding.rope_bwd(w.cuda(), None, plan, pos=torch.from_numpy(pos.astype(np.int32)).cuda())
    f = lambda y: (bf16_to_f64(w).transpose(1, 0, 2) * so.rope(y, pos, (44, 42, 42))).sum()  # noqa: E731
    base = bf16_to_f64(x)
    rng = np.random.default_rng(1)
    for _ in range(40):
        at = tuple(rng.integers(0, s) for s in x.shape)
        up, down = base.copy(), base.copy()
        up[at] += 1.0
        down[at] -= 1.0
        ref = (f(up) - f(down)) / 2
        assert abs(bf16_to_f64(dx)[at] - ref) <= BF16 * abs(ref) + 2.0 ** -19 * float(w.abs().max())


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
def test_rope_strides_in_place_and_broadcast(binding, pairing):
    g = _gen(8)
    n, hq, hk = 70, 4, 2
    plan = binding.rope_plan((48, 40, 24), pairing=pairing)
    fused = _randn(g, n, hq + 2 * hk, 128).cuda()  # a fused projection: queries, keys, values
    q, k = fused[:, :hq], fused[:, hq:hq + hk]
    kw = dict(grid=(5, 7), start=(2, 1, 0))
    want = binding.rope_fwd(q.contiguous(), k.contiguous(), plan, **kw)
    got = binding.rope_fwd(q, k, plan, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # head-major views as inputs
    hm = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(binding.rope_fwd(hm, None, plan, **kw)[0], want[0])
    # in place, inside the fused buffer: the values are not touched
    values = fused[:, hq + hk:].clone()
    binding.rope_fwd(q, k, plan, q_out=q.transpose(0, 1), k_out=k.transpose(0, 1), **kw)
    assert torch.equal(q.transpose(0, 1), want[0]) and torch.equal(k.transpose(0, 1), want[1])
    assert torch.equal(fused[:, hq + hk:], values)
    # partly overlapping outputs are refused
    with pytest.raises(binding.CalibattError):
        binding.rope_fwd(fused[:-1, :hq], None, plan, q_out=fused[1:, :hq].transpose(0, 1), **kw)
    # a gradient that one row stands for
    row = _randn(g, 1, 1, 128).cuda()
    a = binding.rope_bwd(row.expand(hq, n, 128), None, plan, **kw)[0]
    b = binding.rope_bwd(row.expand(hq, n, 128).contiguous(), None, plan, **kw)[0]
    assert torch.equal(a, b)


def test_rope_nonfinite_values_stay_in_their_pair(binding):
    plan = binding.rope_plan((30, 30, 2))
    x = torch.ones((2, 1, 128), dtype=torch.bfloat16)
    x[0, 0, 4], x[0, 0, 70], x[1, 0, 127] = math.inf, math.nan, -math.inf
    y = binding.rope_fwd(x.cuda(), None, plan, grid=(1, 2), start=(3, 3, 3))[0][0].float().cpu()
    bad = ~torch.isfinite(y)
    assert bad[0].nonzero().flatten().tolist() == [4, 5, 70] and bad[1].nonzero().flatten().tolist() == [127]


def test_rope_empty(binding):
    x = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    assert binding.rope_fwd(x, None, binding.rope_plan(), grid=(2, 2))[0].shape == (4, 0, 128)


# ---------------------------------------------------------------------------- writing the cache

class Cache:
    """Pages in a scrambled order, full of earlier values; host copies for the oracle."""

    def __init__(self, batch, heads, width, seed, spare=2):
        rng = np.random.default_rng(seed)
        pages = batch * width + spare
        self.table_h = rng.permutation(pages)[:batch * width].reshape(batch, width).astype(np.int32)
        e = rng.integers(-9, -4, (2, pages, heads))
        bits = rng.integers(0, 256, (2, pages, heads, 128, 128)).astype(np.uint8)
        bits[(bits & 127) > 118] &= 0x47  # no NaN, and nothing near 448
        self.k_h, self.v_h = bits
        self.ks_h, self.vs_h = (2.0 ** e).astype(np.float32)
        self.up()

    def up(self):
        dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
        self.k, self.v = (dev(x).view(torch.float8_e4m3fn) for x in (self.k_h, self.v_h))
        self.ks, self.vs, self.table = dev(self.ks_h), dev(self.vs_h), dev(self.table_h)

    @property
    def dev(self):
        return self.k, self.v, self.ks, self.vs

    def poison(self, lens):
        """NaN into the slots that no token has reached."""
        for b, n in enumerate(lens):
            if n % 128:
                for c in (self.k_h, self.v_h):
                    c[self.table_h[b, n // 128], :, n % 128:] = 127
        self.up()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _starts(new):
    return [0] + np.cumsum(new).tolist()


def _write_both(binding, so, c, k, v, new, lens, **kw):
    start = _starts(new)
    binding.cache_write(k, v, *c.dev, _i32(start), _i32(lens), c.table, **kw)
    so.cache_write(bf16_to_f64(k), c.k_h, c.ks_h, start, lens, c.table_h)
    so.cache_write(bf16_to_f64(v), c.v_h, c.vs_h, start, lens, c.table_h)
    for got, ref in ((c.ks, c.ks_h), (c.vs, c.vs_h)):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)
    for got, ref in ((c.k, c.k_h), (c.v, c.v_h)):
        got = got.view(torch.uint8).cpu().numpy()
        nan = (got & 127 == 127) & (ref & 127 == 127)  # the sign of a NaN says nothing
        np.testing.assert_array_equal(np.where(nan, 0, got), np.where(nan, 0, ref))
    assert binding.get_status() == 0


@pytest.mark.parametrize("heads,new,old", [(1, [1], [0]), (3, [1, 1, 1], [5, 127, 128]), (2, [128], [0]),
                                           (2, [129, 0, 64], [127, 30, 64]), (5, [300, 7], [250, 0]),
                                           (1, [1000], [3])])
def test_cache_write_matches_oracle(binding, so, heads, new, old):
    g = _gen(sum(new))
    lens = [a + b for a, b in zip(new, old)]
    c = Cache(len(new), heads, -(-max(lens) // 128) + 1, seed=heads)
    n = sum(new)
    behind = 3  # tokens that no stream owns
    size = torch.exp(torch.randn((n + behind, heads, 1), generator=g))
    k = (torch.randn((n + behind, heads, 128), generator=g) * size).bfloat16().cuda()
    v = (torch.randn((n + behind, heads, 128), generator=g) * 3).bfloat16().cuda()
    _write_both(binding, so, c, k, v, new, lens, max_new=max(new))


def test_cache_write_grows_scales_and_reencodes(binding, so):
    g = _gen(2)
    c = Cache(1, 2, 2, seed=9)
    done = 0
    for m, size in ((60, 1.0), (1, 50.0), (1, 0.001), (70, 400.0), (1, 1e30), (1, 1e-30)):
        k, v = (_randn(g, m, 2, 128) * size for _ in range(2))
        done += m
        _write_both(binding, so, c, k.cuda(), v.cuda(), [m], [done])


def test_cache_write_special_values(binding, so):
    c = Cache(1, 4, 1, seed=1)
    k = torch.ones((5, 4, 128), dtype=torch.bfloat16)
    k[:, 0] = 0.0
    k[0, 1, 3], k[1, 1, 4], k[2, 1, 5] = math.inf, math.nan, -math.inf
    k[:, 2] = torch.finfo(torch.bfloat16).max
    k[:, 3] = torch.finfo(torch.bfloat16).smallest_normal / 4
    v = torch.linspace(-448, 448, 5 * 4 * 128).reshape(5, 4, 128).bfloat16()
    _write_both(binding, so, c, k.cuda(), v.cuda(), [5], [5])
    again = torch.full((1, 4, 128), math.nan, dtype=torch.bfloat16)
    _write_both(binding, so, c, again.cuda(), again.cuda(), [1], [6])


def test_cache_write_strided_inputs(binding, so):
    g = _gen(3)
    c = Cache(2, 2, 2, seed=4)
    fused = _randn(g, 150, 6, 128).cuda()
    _write_both(binding, so, c, fused[:, 2:4], fused[:, 4:6], [100, 50], [101, 150])
    hm = _randn(g, 2, 150, 128).cuda()
    _write_both(binding, so, c, hm.transpose(0, 1), hm.transpose(0, 1), [100, 50], [100, 50])


def test_malformed_lists_are_reported_and_nothing_is_written(binding):
    c = Cache(2, 2, 2, seed=6)
    k = torch.ones((20, 2, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((2, 20, 128), dtype=torch.bfloat16, device="cuda")
    good = dict(start=[0, 10, 20], lens=[30, 40], table=c.table_h.tolist())
    bad = [dict(start=[0, 12, 10]), dict(start=[-1, 10, 20]), dict(start=[0, 10, 21]), dict(lens=[-1, 40]),
           dict(lens=[300, 40]), dict(table=[[-1, 5], [2, 3]]), dict(table=[[10 ** 6, 1], [2, 3]])]
    before = c.k.view(torch.uint8).clone()
    for b in bad:
        a = {**good, **b}
        page0 = torch.tensor(a["table"], dtype=torch.int32).flatten().tolist()
        binding.cache_write(k, k, *c.dev, _i32(a["start"]), _i32(a["lens"]), _i32(a["table"]), max_new=10)
        assert binding.get_status() == -2, b
        assert binding.get_status() == 0
        o, lse = torch.full_like(q, 7.0), torch.full((2, 20), 7.0, device="cuda")
        binding.cache_attn_fwd(q, *c.dev, _i32(a["start"]), _i32(a["lens"]), _i32(a["table"]), max_new=10, max_kv=100,
                               o=o, lse=lse)
        assert binding.get_status() == -2, b
        touched = (c.k.view(torch.uint8) != before).flatten(1).any(1).nonzero().flatten().tolist()
        assert set(touched) <= set(p for p in page0 if 0 <= p < before.shape[0]), (b, touched)
        c.up()
    # fewer cached than new tokens; more new tokens than the host's bound
    for start, lens, most in (([0, 10, 20], [5, 9], 10), ([0, 10, 20], [30, 40], 9)):
        binding.cache_write(k, k, *c.dev, _i32(start), _i32(lens), c.table, max_new=most)
        assert binding.get_status() == -2
        assert torch.equal(c.k.view(torch.uint8), before)


# ---------------------------------------------------------------------------- attention over the cache

def _p_err(new, hq, hk):
    """Half a step of P's type, fp16 in every kernel (for up to 16 rows a sum of four 8-bit values, within 2^-12)."""
    return 2.0 ** -11


def _attn_close(o, lse, ref, q, c, lens, scale, p_err):
    """Roundings: q's row in fp16 (2^-25 of the row's power of two, an absolute error of the products), the fp32
    sum of 128 products (128 * 2^-24 of their magnitudes), the score's multiplies and the exponential
    (|score| 2^-22 + 2^-21): ds in all, in the exponent. Then P (p_err relative, and 2^-25 absolute below fp16's
    normal range, for up to 2^5 weights' worth of keys), the sums over keys, the output (2^-8)."""
    o_ref, lse_ref, av = ref
    used = np.unique(np.concatenate([c.table_h[b, :-(-m // 128)] for b, m in enumerate(lens)]))
    vals = np.abs(np.nan_to_num(c_vals(c.k_h[used], c.ks_h[used]))).max(initial=0)
    qmax = np.abs(bf16_to_f64(q)).max()
    ds = scale * 128 * qmax * vals * (2.0 ** -24 + 128 * 2.0 ** -24) + 2.0 ** -20
    ds += 2.0 ** -22 * np.abs(np.where(np.isfinite(lse_ref), lse_ref, 0)).max()
    assert ds < 2.0 ** -6, ds
    vmax = np.abs(np.nan_to_num(c_vals(c.v_h[used], c.vs_h[used]))).max(initial=0)
    rel = 2 * ds + p_err + 2.0 ** -12
    tol = BF16 * np.abs(o_ref) + rel * av * (1 + BF16) + 2.0 ** -20 * vmax
    got = bf16_to_f64(o)
    bad = np.isnan(o_ref)
    np.testing.assert_array_equal(np.isnan(got), bad)
    off = np.where(bad, 0, np.abs(got - o_ref) - tol)
    assert np.all(off <= 0), float(off.max())
    got = lse.double().cpu().numpy()
    inf = np.isneginf(lse_ref)
    np.testing.assert_array_equal(np.isneginf(got), inf)
    ok = np.isfinite(lse_ref)
    assert np.all(np.abs(got[ok] - lse_ref[ok]) <= 2 * ds + 2.0 ** -20)


def c_vals(bits, scale):
    from oracle import stream
    return stream.e4m3_values()[bits] * scale[..., None, None].astype(np.float64)


SHAPES = [
    # heads_q, heads_kv, new, cached (new ones included), causal unit
    (1, 1, [1], [1], 0), (2, 2, [1], [129], 1), (8, 2, [1, 1, 1], [5, 128, 700], 0), (5, 1, [3], [300], 1),
    (4, 4, [2, 0, 5], [2, 77, 900], 1), (40, 8, [1], [2500], 0), (3, 3, [17], [1000], 1), (2, 1, [40], [333], 7),
    (2, 2, [129], [140], 1), (1, 1, [300], [300], 64), (4, 2, [70, 33], [513, 64], 0), (6, 2, [100], [1300], 25),
    (1, 1, [260, 1], [770, 128], 0), (2, 2, [513], [600], 128), (8, 1, [31], [4000], 0), (2, 2, [128], [4096], 1),
    # the borders of the kernels' row counts, 1 to 16 rows in every layout
    (1, 1, [16], [1500], 1), (4, 2, [8, 3, 1], [1500, 40, 700], 3), (8, 2, [1, 2], [2000, 128], 0),
    (3, 1, [2, 1, 0, 2], [900, 6, 50, 129], 1), (7, 1, [1], [1300], 0), (10, 2, [1, 1, 1], [130, 2600, 384], 1),
    # 17 to 128, one copy or two of the rows
    (1, 1, [17], [1400], 1), (5, 1, [7, 1], [640, 2300], 2), (2, 1, [32], [900], 0),
    (3, 1, [11, 21, 4], [700, 90, 5], 9),
    (1, 1, [64, 65, 1, 0, 128], [64, 3000, 1, 7, 400], 1), (16, 2, [12], [1025], 4),
    # more: tiles of 256, of which one or both halves are used, split or not
    (1, 1, [129, 5], [129, 1000], 1), (3, 3, [256], [2000], 0), (1, 1, [257], [5000], 16),
    (4, 1, [65, 70], [900, 71], 1),
    (2, 2, [700, 300, 40], [2500, 300, 700], 100), (8, 8, [384], [1100], 128),
    # more tiles than the SMs of any GPU take at once: the ones behind are split, or under the causal mask not
    (80, 80, [300], [1280], 0), (160, 40, [70], [1300], 30), (20, 20, [300, 257, 40, 290], [1000, 1280, 640, 1290], 1),
    (80, 80, [300], [420], 1), (40, 40, [1024], [2000], 1),
]


@pytest.mark.parametrize("hq,hk,new,lens,unit", SHAPES)
def test_cache_attention_matches_oracle(binding, so, hq, hk, new, lens, unit):
    g = _gen(sum(lens))
    c = Cache(len(new), hk, -(-max(lens) // 128) + 1, seed=sum(new))
    c.poison(lens)
    n = sum(new) + 2
    q = _randn(g, hq, n, 128) * 0.5
    scale = 0.05
    o, lse = torch.full((hq, n, 128), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((hq, n), 7.0, device="cuda")
    binding.cache_attn_fwd(q.cuda(), *c.dev, _i32(_starts(new)), _i32(lens), c.table, max_new=max(new),
                           max_kv=max(lens), causal_unit=unit, o=o, lse=lse, scale=scale)
    assert binding.get_status() == 0
    assert torch.all(o[:, -2:] == 7.0) and torch.all(lse[:, -2:] == 7.0)  # tokens of no stream
    ref = so.cache_attention(bf16_to_f64(q), c.k_h, c.v_h, c.ks_h, c.vs_h, _starts(new), lens, c.table_h, scale, unit)
    cut = slice(0, n - 2)
    _attn_close(o[:, cut], lse[:, cut], [r[:, cut] for r in ref], q, c, lens, scale, _p_err(new, hq, hk))


@pytest.mark.parametrize("new,lens", [([4, 3], [2, 0]), ([200], [150]), ([150, 1], [0, 0]), ([16, 9], [7, 0]),
                                      ([30], [11]), ([60, 50], [0, 45])])
@pytest.mark.parametrize("unit", [0, 1, 5])
def test_rows_that_see_nothing(binding, so, new, lens, unit):
    c = Cache(len(new), 2, 2, seed=3)
    c.poison(lens)
    q = _randn(_gen(1), 4, sum(new), 128)
    o, lse = binding.cache_attn_fwd(q.cuda(), *c.dev, _i32(_starts(new)), _i32(lens), c.table, causal_unit=unit,
                                    scale=0.05)
    ref = so.cache_attention(bf16_to_f64(q), c.k_h, c.v_h, c.ks_h, c.vs_h, _starts(new), lens, c.table_h, 0.05, unit)
    assert np.isneginf(ref[1]).any() or unit == 0
    empty = torch.from_numpy(np.isneginf(ref[1])).cuda()
    assert torch.all(o[empty] == 0) and torch.all(lse[empty] == -math.inf)
    _attn_close(o, lse, ref, q, c, lens, 0.05, _p_err(new, 4, 2))
    assert binding.get_status() == 0


@pytest.mark.parametrize("hq,new,unit", [(2, 3, 1), (2, 20, 1), (2, 40, 1), (2, 100, 9), (1, 300, 128), (1, 200, 1)])
def test_nan_in_later_tokens_does_not_reach_earlier_rows(binding, so, hq, new, unit):
    lens = 300 + new
    c = Cache(1, hq, -(-lens // 128), seed=5)
    at = lens - new // 2 - 1  # a new token whose key and value hold NaN
    for x in (c.k_h, c.v_h):
        x[c.table_h[0, at // 128], 0, at % 128, 11] = 127
    c.up()
    q = _randn(_gen(2), hq, new, 128)
    o, lse = binding.cache_attn_fwd(q.cuda(), *c.dev, _i32([0, new]), _i32([lens]), c.table, causal_unit=unit,
                                    scale=0.05)
    ref = so.cache_attention(bf16_to_f64(q), c.k_h, c.v_h, c.ks_h, c.vs_h, [0, new], [lens], c.table_h, 0.05, unit)
    seen = np.isnan(ref[1][0])
    assert seen.any() and (not seen.all() or unit == 128)
    assert torch.all(torch.isnan(o[0]).all(-1).cpu() == torch.from_numpy(seen))
    keep = [(0, ~seen)] + [(h, np.ones(new, bool)) for h in range(1, hq)]
    for h, rows in keep:
        if rows.any():
            idx = torch.from_numpy(rows.nonzero()[0]).cuda()
            _attn_close(o[h:h + 1, idx], lse[h:h + 1, idx], [r[h:h + 1][:, rows] for r in ref], q, c, [lens], 0.05,
                        _p_err([new], 1, 1))


@pytest.mark.parametrize("hq,new,unit", [(2, 3, 1), (2, 30, 1), (1, 60, 4), (2, 100, 1), (1, 200, 1), (1, 260, 7)])
def test_nan_in_a_value_alone_reaches_its_channel_of_the_rows_that_see_it(binding, so, hq, new, unit):
    lens = 200 + new
    c = Cache(1, hq, -(-lens // 128), seed=15)
    at = lens - new // 2 - 1
    c.v_h[c.table_h[0, at // 128], 0, at % 128, 11] = 127
    c.up()
    q = _randn(_gen(3), hq, new, 128)
    o, lse = binding.cache_attn_fwd(q.cuda(), *c.dev, _i32([0, new]), _i32([lens]), c.table, causal_unit=unit,
                                    scale=0.05)
    ref = so.cache_attention(bf16_to_f64(q), c.k_h, c.v_h, c.ks_h, c.vs_h, [0, new], [lens], c.table_h, 0.05, unit)
    assert np.isnan(ref[0]).any() and np.isnan(ref[0]).sum() < new  # one channel of some rows
    _attn_close(o, lse, ref, q, c, [lens], 0.05, _p_err([new], 1, 1))


@pytest.mark.parametrize("rows", [6, 20, 50, 100, 140])
@pytest.mark.parametrize("lens", [128, 256, 384])
def test_extreme_queries_and_scales(binding, so, rows, lens):
    """Rows of very large and very small queries, pages whose scales lie far apart, infinities in one row."""
    c = Cache(1, 1, 3, seed=8)
    c.vs_h[c.table_h[0], 0] = [2.0 ** -60, 2.0 ** -90, 2.0 ** 20]
    c.up()
    q = _randn(_gen(4), 1, rows, 128)
    q[0, 1] *= 2.0 ** -100
    q[0, 2] = 0.0
    q[0, 3, 5] = 2.0 ** -40
    q[0, rows - 2] *= 2.0 ** 100
    q[0, rows - 1, 7] = math.inf
    o, lse = binding.cache_attn_fwd(q.cuda(), *c.dev, _i32([0, rows]), _i32([lens]), c.table, scale=0.05)
    m = rows - 2
    args = (c.k_h, c.v_h, c.ks_h, c.vs_h)
    ref = so.cache_attention(bf16_to_f64(q[:, :m]), *args, [0, m], [lens], c.table_h, 0.05)
    _attn_close(o[:, :m], lse[:, :m], ref, q[:, :m], c, [lens], 0.05, _p_err([rows], 1, 1))
    # the huge row: one key takes everything
    big = so.cache_attention(bf16_to_f64(q[:, m:m + 1]), *args, [0, 1], [lens], c.table_h, 0.05)
    np.testing.assert_allclose(bf16_to_f64(o[:, m:m + 1]), big[0], rtol=2.0 ** -7)
    assert torch.isnan(o[0, m + 1]).all()


@pytest.mark.parametrize("hq,hk,new,lens,unit", [(4, 2, [1, 1], [3000, 9000], 1), (4, 2, [20, 30], [3000, 9000], 1),
                                                 (2, 1, [90, 200], [3000, 9000], 50)])
def test_wild_pages_are_left_out(binding, so, hq, hk, new, lens, unit):
    """A table entry outside the pool in the middle of a stream: reported, and its keys are not seen."""
    g = _gen(77)
    c = Cache(2, hk, -(-max(lens) // 128), seed=31)
    q = _randn(g, hq, sum(new), 128) * 0.5
    table = c.table.clone()
    table[0, 5], table[1, 40] = -7, 1 << 30
    o, lse = binding.cache_attn_fwd(q.cuda(), *c.dev, _i32(_starts(new)), _i32(lens), table, max_new=max(new),
                                    max_kv=max(lens), causal_unit=unit, scale=0.05)
    assert binding.get_status() == -2 and binding.get_status() == 0
    # the oracle on streams without that page: the order of keys does not matter where all are seen
    for b, (wild, m) in enumerate(zip((5, 40), new)):
        tab = np.delete(c.table_h[b], wild)[None]
        ln = lens[b] - 128
        rows = slice(_starts(new)[b], _starts(new)[b] + m)
        ref = so.cache_attention(bf16_to_f64(q[:, rows]), c.k_h, c.v_h, c.ks_h, c.vs_h, [0, m], [ln], tab, 0.05, unit)
        if unit > 1:  # positions moved with the page: take the same visible ends
            ref = so.cache_attention(bf16_to_f64(q[:, rows]), c.k_h, c.v_h, c.ks_h, c.vs_h, [0, m], [ln], tab, 0.05,
                                     unit, shift=128)
        part = Cache.__new__(Cache)
        part.k_h, part.v_h, part.ks_h, part.vs_h, part.table_h = c.k_h, c.v_h, c.ks_h, c.vs_h, tab
        _attn_close(o[:, rows], lse[:, rows], ref, q[:, rows], part, [ln], 0.05, _p_err(new, hq, hk))


def test_a_long_stream_past_32_bit_offsets(binding):
    """A cache of more than 2^32 bytes: the last pages are read where they are."""
    heads, pages = 40, 7000
    k8 = torch.zeros((pages, heads, 128, 128), dtype=torch.uint8, device="cuda")
    v8 = torch.zeros_like(k8)
    assert k8.numel() > 2 ** 32
    ks = torch.ones((pages, heads), device="cuda")
    v8[-1] = 0x38  # 1.0
    v8[0] = 0x40   # 2.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    table[0, 1] = pages - 1
    q = torch.ones((heads, 1, 128), dtype=torch.bfloat16, device="cuda")
    o, lse = binding.cache_attn_fwd(q, k8, v8, ks, ks, _i32([0, 1]), _i32([256]), table, max_kv=256)
    assert torch.all(o == 1.5) and torch.all((lse - math.log(256)).abs() < 1e-5)
    k = torch.ones((1, heads, 128), dtype=torch.bfloat16, device="cuda")
    binding.cache_write(k, k, k8, v8, ks, ks.clone(), _i32([0, 1]), _i32([129]), table)
    assert torch.all(k8[pages - 1, :, 0].view(torch.float8_e4m3fn).float() * ks[pages - 1][:, None] == 1.0)
    assert torch.all(k8[pages - 1, :, 1:] == 0)
    assert binding.get_status() == 0


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("hq,hk", [(2, 2), (4, 1)])
@pytest.mark.parametrize("unit", [0, 35])
def test_frames_rotated_appended_and_attended(binding, so, hq, hk, unit):
    """Five frames of 5 x 7 tokens: each is rotated, appended to the cache and attends to all so far."""
    g = _gen(21)
    H, W, frames = 5, 7, 5
    plan = binding.rope_plan()
    c = Cache(1, hk, 2, seed=2)
    scale = 1 / math.sqrt(128)
    for f in range(frames):
        n = H * W
        x = _randn(g, n, hq + 2 * hk, 128).cuda()
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
        pos = _grid_pos(n, H, W, (f, 0, 0))
        qr, kr = binding.rope_fwd(q, k, plan, grid=(H, W), start=(f, 0, 0))
        _rope_close(bf16_to_f64(qr).transpose(1, 0, 2), so.rope(bf16_to_f64(q), pos, (44, 42, 42)), bf16_to_f64(q))
        lens = [(f + 1) * n]
        _write_both(binding, so, c, kr.transpose(0, 1), v, [n], lens)
        o, lse = binding.cache_attn_fwd(qr, *c.dev, _i32([0, n]), _i32(lens), c.table, causal_unit=unit)
        ref = so.cache_attention(bf16_to_f64(qr), c.k_h, c.v_h, c.ks_h, c.vs_h, [0, n], lens, c.table_h, scale, unit)
        _attn_close(o, lse, ref, qr, c, lens, scale, _p_err([n], hq, hk))


def test_rotated_queries_feed_block_sparse_attention(binding, so, oracle):
    """The rotation's output is the layout of the framework's other attention calls."""
    g = _gen(22)
    n, heads = 300, 2
    q, k, v = (_randn(g, n, heads, 128) for _ in range(3))
    qr, kr = binding.rope_fwd(q.cuda(), k.cuda(), binding.rope_plan(), grid=(10, 10))
    vh = v.cuda().transpose(0, 1).contiguous()
    mask = (np.random.default_rng(0).random((heads, 3, 3)) < 0.6).astype(np.uint8)
    rp, ci = oracle.mask_to_csr(mask)
    work = torch.from_numpy(binding.build_plan(rp, heads, 3)).cuda()
    o, _ = binding.sparse_attn_fwd(qr, kr, vh, torch.from_numpy(rp).cuda(), torch.from_numpy(ci).cuda(), work)
    bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    ref, _ = oracle.masked_attention(bits(qr), bits(kr), bits(vh), mask)
    assert np.max(np.abs(bf16_to_f64(o) - ref)) <= 1e-2 * np.abs(ref).max() + 1e-3


def test_a_captured_step_replays_with_new_lengths(binding, so):
    """Rotation, writing and attention captured once; positions, lengths and inputs change between replays."""
    g = _gen(23)
    hq, hk, n = 4, 2, 3
    plan = binding.rope_plan()
    c, ref = Cache(2, hk, 12, seed=7), Cache(2, hk, 12, seed=7)
    x = torch.zeros((n, hq + 2 * hk, 128), dtype=torch.bfloat16, device="cuda")
    pos, start, lens = _i32([[0, 0, 0]] * n), _i32([0, 2, 3]), _i32([2, 1])
    bufs = [torch.empty((h, n, 128), dtype=torch.bfloat16, device="cuda") for h in (hq, hk, hq)]
    lse = torch.empty((hq, n), device="cuda")
    ws = binding.cache_attn_workspace(bufs[0], c.k, c.table, max_new=2)
    assert ws is not None  # the cache is split

    def step(c, x, pos, lens, bufs, lse, ws):
        binding.rope_fwd(x[:, :hq], x[:, hq:hq + hk], plan, pos=pos, q_out=bufs[0], k_out=bufs[1])
        binding.cache_write(bufs[1].transpose(0, 1), x[:, hq + hk:], *c.dev, start, lens, c.table, max_new=2)
        binding.cache_attn_fwd(bufs[0], *c.dev, start, lens, c.table, max_new=2, causal_unit=1, o=bufs[2], lse=lse,
                               ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c, x, pos, lens, bufs, lse, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, x, pos, lens, bufs, lse, ws)
    for t in (c.k, c.v):
        t.view(torch.uint8).copy_(torch.from_numpy(ref.k_h if t is c.k else ref.v_h))
    c.ks.copy_(torch.from_numpy(ref.ks_h))
    c.vs.copy_(torch.from_numpy(ref.vs_h))
    eager = [torch.empty_like(b) for b in bufs]
    elens, else_ = lens.clone(), torch.empty_like(lse)
    for at in ([2, 1], [400, 1], [1500, 1536]):
        x.copy_(_randn(g, *x.shape))
        pos.copy_(torch.randint(-9, 900, (n, 3), generator=g).int())
        lens.copy_(torch.tensor(at))
        graph.replay()
        elens.copy_(lens)
        step(ref, x, pos, elens, eager, else_, None)
        for a, b in zip(bufs + [lse], eager + [else_]):
            assert torch.equal(a, b)
        assert torch.equal(c.k.view(torch.uint8), ref.k.view(torch.uint8)) and torch.equal(c.vs, ref.vs)
    assert binding.get_status() == 0


def test_frame_streams_match_the_calls_and_the_oracle(binding, so):
    """The package's own path: two ragged streams, frames begun in one step and ended in the next."""
    from calibrated_block_sparse_b200.stream import FrameStreams
    g = _gen(91)
    H, W, hq, hk = 4, 9, 4, 2
    st = FrameStreams(batch=2, heads=hq, kv_heads=hk, H=H, W=W, pages=12, max_tokens=600)
    c = Cache(2, hk, 5, seed=3, spare=2)
    for x in (c.k_h, c.v_h):
        x[:] = 0
    scale, done = 1 / math.sqrt(128), [0, 0]
    for new in ([36, 20], [1, 300], [0, 16], [130, 1]):
        n = sum(new)
        x = _randn(g, n, hq + 2 * hk, 128).cuda()
        o, lse = st.step(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], new=new, causal_unit=H * W)
        t = np.concatenate([np.arange(a, a + m) for a, m in zip(done, new)])
        pos = torch.from_numpy(np.stack([t // 36, t % 36 // W, t % W], 1).astype(np.int32)).cuda()
        done = [a + m for a, m in zip(done, new)]
        assert st.lengths == done
        qr, kr = binding.rope_fwd(x[:, :hq], x[:, hq:hq + hk], st.plan, pos=pos)
        start = _starts(new)
        so.cache_write(bf16_to_f64(kr.transpose(0, 1)), c.k_h, c.ks_h, start, done, c.table_h)
        so.cache_write(bf16_to_f64(x[:, hq + hk:]), c.v_h, c.vs_h, start, done, c.table_h)
        ref = so.cache_attention(bf16_to_f64(qr), c.k_h, c.v_h, c.ks_h, c.vs_h, start, done, c.table_h, scale, H * W)
        _attn_close(o, lse, ref, qr, c, done, scale, _p_err(new, hq, hk))
    assert binding.get_status() == 0
    # refusals change nothing
    free = st.free_pages
    big = torch.zeros((2000, hq + 2 * hk, 128), dtype=torch.bfloat16, device="cuda")
    for new in ([2000, 0], [400, 600]):
        y = big[:sum(new)]
        with pytest.raises((ValueError, RuntimeError)):
            st.step(y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:], new=new)
    y = big[:3]
    for q, k, v, new in ((y[:, :hq], y[:, hq:hq + hk], y[:, hq:], [3, 0]),
                         (y[:, :hq].float(), y[:, hq:hq + hk], y[:, hq + hk:], [3, 0]),
                         (y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:].cpu(), [3, 0]),
                         (y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:], [4, -1]),
                         (y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:], None)):
        with pytest.raises(ValueError):
            st.step(q, k, v, new=new)
    assert st.lengths == done and st.free_pages == free
    st.drop(0)
    assert st.lengths == [0, done[1]] and st.free_pages > free


def test_dropped_pages_are_used_anew(binding):
    """A stream on pages that another one has left, at far larger scales, gives what it gives on fresh pages."""
    from calibrated_block_sparse_b200.stream import FrameStreams
    g = _gen(92)
    made = [FrameStreams(batch=2, heads=2, kv_heads=2, H=5, W=6, pages=5) for _ in range(2)]
    big = (_randn(g, 530, 6, 128) * 1000).cuda()
    made[0].step(big[:, :2], big[:, 2:4], big[:, 4:], new=[330, 200])
    made[0].drop(0)
    made[0].drop(1)
    for new in ([140, 0], [1, 257], [30, 2]):
        x = _randn(g, sum(new), 6, 128).cuda()
        got = [st.step(x[:, :2], x[:, 2:4], x[:, 4:], new=new, causal_unit=30) for st in made]
        for a, b in zip(*got):
            assert torch.equal(a, b)
    assert made[0].free_pages == made[1].free_pages == 0
    assert binding.get_status() == 0


def test_the_compiled_calls_and_ctypes_give_the_same(binding, monkeypatch):
    g = _gen(61)
    x = _randn(g, 40, 6, 128).cuda()
    plan = binding.rope_plan()
    out = []
    fast, made = binding._load_fast(), []
    assert fast is not binding._NoFast  # build() made them

    class Fast:  # the compiled calls, counted
        def __getattr__(self, name):
            def call(*args):
                done = getattr(fast, name)(*args)
                made.append(done is not None)
                return done
            return call

    for calls in (Fast(), binding._NoFast):
        monkeypatch.setattr(binding, "_fast", calls)
        c = Cache(1, 2, 2, seed=5)
        q, k = binding.rope_fwd(x[:, :2], x[:, 2:4], plan, grid=(4, 5), start=(3, 1, 2))
        back, _ = binding.rope_bwd(q, None, plan, grid=(4, 5), start=(3, 1, 2))
        binding.cache_write(k.transpose(0, 1), x[:, 4:], *c.dev, _i32([0, 40]), _i32([100]), c.table)
        o, lse = binding.cache_attn_fwd(q, *c.dev, _i32([0, 40]), _i32([100]), c.table, causal_unit=7, scale=0.1)
        out.append([q, k, back, c.k.view(torch.uint8), c.ks, o, lse])
        with pytest.raises(TypeError):
            binding.cache_attn_fwd(q, *c.dev, _i32([0, 40]), _i32([100]), c.table, max_new=2.5)
    assert made == [True] * 4 + [False]
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert binding.get_status() == 0


def test_two_streams_at_once_and_a_repeat_give_the_same(binding):
    """Calls on two streams with workspaces of their own; the same call twice is bit for bit the same."""
    g = _gen(24)
    c = Cache(2, 2, 30, seed=11)
    qs = [(_randn(g, 8, m, 128) * 0.5).cuda() for m in (2, 260)]
    lens = _i32([3800, 3700])
    starts = [_i32([0, 1, 2]), _i32([0, 130, 260])]
    want = [binding.cache_attn_fwd(q, *c.dev, s, lens, c.table, causal_unit=1) for q, s in zip(qs, starts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = [binding.cache_attn_fwd(q, *c.dev, s, lens, c.table, causal_unit=1, stream=st)
               for q, s, st in zip(qs, starts, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_results_do_not_depend_on_the_bounds(binding):
    """max_new and max_kv plan the launch; a stream longer than max_kv is attended to in full."""
    c = Cache(1, 2, 20, seed=12)
    q = (_randn(_gen(25), 2, 1, 128) * 0.5).cuda()
    args = (q, *c.dev, _i32([0, 1]), _i32([2500]), c.table)
    a = binding.cache_attn_fwd(*args)
    b = binding.cache_attn_fwd(*args, max_new=1, max_kv=100)
    assert (a[0].float() - b[0].float()).abs().max() <= 2.0 ** -7 * a[0].float().abs().max()
    assert (a[1] - b[1]).abs().max() < 1e-5
