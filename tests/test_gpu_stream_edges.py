"""Streaming operators on the GPU where an ordering of warps, a border of the
number formats or an unusual call decides the result."""
import numpy as np
import pytest
import torch

from gpu_util import bf16_to_f64
from test_gpu_stream import (Cache, _attn_close, _gen, _grid_pos, _i32, _p_err, _randn, _rope_close, _starts,  # noqa: F401
                             binding, so)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------- repeats

@pytest.mark.parametrize("rows", [17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("lens", [[1], [128], [100, 128, 1], [300], [129, 2000, 60], [700, 700]])
def test_mid_rows_repeat_bit_for_bit(binding, so, rows, lens):
    """Stretches of one page, where one of the two slots has no work, and of several: the same call many times."""
    g = _gen(rows + sum(lens))
    hk = 3
    c = Cache(len(lens), hk, -(-max(lens) // 128), seed=rows)
    new = [rows] * len(lens)
    q = _randn(g, hk, sum(new), 128) * 0.5
    args = (q.cuda(), *c.dev, _i32(_starts(new)), _i32(lens), c.table)
    kw = dict(max_new=rows, max_kv=max(lens), scale=0.05)
    o, lse = binding.cache_attn_fwd(*args, **kw)
    ref = so.cache_attention(bf16_to_f64(q), c.k_h, c.v_h, c.ks_h, c.vs_h, _starts(new), lens, c.table_h, 0.05)
    _attn_close(o, lse, ref, q, c, lens, 0.05, _p_err(new, hk, hk))
    outs = [binding.cache_attn_fwd(*args, **kw) for _ in range(300)]
    assert all(torch.equal(o, a) and torch.equal(lse, b) for a, b in outs)
    # shares that leave single pages: the plan is made for another length, and every CTA gets a page or two
    if max(lens) > 128:
        kw["max_kv"] = 128 * 40
        many = [binding.cache_attn_fwd(*args, **kw) for _ in range(100)]
        assert all(torch.equal(many[0][0], a) and torch.equal(many[0][1], b) for a, b in many)
        _attn_close(*many[0], ref, q, c, lens, 0.05, _p_err(new, hk, hk))
    assert binding.get_status() == 0


@pytest.mark.parametrize("rows", [(17, 1), (40, 33), (90, 128)])
def test_mid_rows_at_once_with_others(binding, rows):
    """One-page stretches on two streams at the same time, each with outputs of its own: as one after the other."""
    g = _gen(sum(rows))
    c = Cache(4, 8, 2, seed=9)
    lens, calls = _i32([100, 128, 256, 129]), []
    for m in rows:
        q = (_randn(g, 8, 4 * m, 128) * 0.5).cuda()
        calls.append((q, *c.dev, _i32(_starts([m] * 4)), lens, c.table))
    want = [binding.cache_attn_fwd(*a, max_new=m) for a, m in zip(calls, rows)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in rows]
    for _ in range(50):
        got = [binding.cache_attn_fwd(*a, max_new=m, stream=st) for a, m, st in zip(calls, rows, streams)]
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert binding.get_status() == 0


@pytest.mark.parametrize("rows", [20, 40, 100])
def test_one_page_wait_runs_out_then_context_is_usable(binding, rows):
    """A slot without pages waits for the other one: that wait has its limit too, and ends by it alone."""
    k8 = torch.zeros((1, 2, 128, 128), dtype=torch.uint8, device="cuda")
    args = (torch.ones((2, rows, 128), dtype=torch.bfloat16, device="cuda"), k8, torch.full_like(k8, 0x38),
            *[torch.ones((1, 2), device="cuda")] * 2, _i32([0, rows]), _i32([100]), _i32([[0]]))
    try:
        binding.set_wait_limit(1e-9)
        status = 0
        for _ in range(200):  # a wait inside one tick of the timer is not seen to take time
            binding.cache_attn_fwd(*args)
            status = binding.get_status()
            if status != 0:
                break
        assert status == -6
    finally:
        binding.set_wait_limit(0.0)
    o, lse = binding.cache_attn_fwd(*args)
    assert binding.get_status() == 0
    assert torch.all(o == 1.0) and torch.all((lse - np.log(100)).abs() < 1e-5)


# ---------------------------------------------------------------------------- lengths next to 2^31

MOST = 2 ** 31 - 256  # tokens of one stream


@pytest.fixture(scope="module")
def longest():
    """A pool of two pages, named by a table that is wide enough for 2^31 tokens."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    k8 = torch.zeros((2, 1, 128, 128), dtype=torch.uint8, device="cuda")
    v8 = torch.full_like(k8, 0x38)  # 1.0
    scales = [torch.ones((2, 1), device="cuda") for _ in range(2)]
    return k8, v8, *scales, torch.zeros((1, 1 << 24), dtype=torch.int32, device="cuda")


def test_writing_next_to_2_31_tokens(binding):
    """One token at the last position of a stream, beside another stream with so many new ones that the grid's pages
    would reach behind 2^31 tokens for the first."""
    n = 1 + 599
    pool = [torch.zeros((8, 1, 128, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    cache = pool + [torch.ones((8, 1), device="cuda") for _ in range(2)]
    table = torch.zeros((2, 1 << 24), dtype=torch.int32, device="cuda")
    table[0, MOST // 128 - 1] = 1
    table[1, :5] = torch.arange(2, 7, dtype=torch.int32)
    x = torch.full((n, 1, 128), 2.0, dtype=torch.bfloat16, device="cuda")
    binding.cache_write(x, x, *cache, _i32([0, 1, n]), _i32([MOST, n - 1]), table, max_new=n - 1)
    assert binding.get_status() == 0
    for c, s in (cache[::2], cache[1::2]):
        value = c.view(torch.float8_e4m3fn).float()[:, 0, :, 0] * s
        want = torch.zeros((8, 128), device="cuda")
        want[1, 127] = 2.0
        want[2:7].view(-1)[:n - 1] = 2.0
        assert torch.equal(value, want)
    for much in (MOST + 1, 2 ** 31 - 128, 2 ** 31 - 1):
        before = [y.clone() for y in cache]
        binding.cache_write(x[:1], x[:1], *cache, _i32([0, 1, 1]), _i32([much, 0]), table)
        assert binding.get_status() == -2
        assert all(torch.equal(y, z) for y, z in zip(cache, before))


@pytest.mark.parametrize("rows", [1, 20, 140])
def test_attention_next_to_2_31_tokens(binding, longest, rows):
    """Equal scores and values of 1: o = 1, lse = ln of the length (21.5, to a few steps of 2^-19 in fp32)."""
    *cache, table = longest
    q = torch.ones((1, rows, 128), dtype=torch.bfloat16, device="cuda")
    o, lse = binding.cache_attn_fwd(q, *cache, _i32([0, rows]), _i32([MOST]), table, max_kv=MOST)
    assert binding.get_status() == 0
    assert torch.all(o == 1.0) and torch.all((lse.double() - np.log(MOST)).abs() < 2.0 ** -16)
    for much in (MOST + 1, 2 ** 31 - 1):
        o.fill_(7.0)
        binding.cache_attn_fwd(q, *cache, _i32([0, rows]), _i32([much]), table, max_kv=MOST, o=o)
        assert binding.get_status() == -2 and torch.all(o == 7.0)


# ---------------------------------------------------------------------------- borders of the value scales

ROWS = [1, 6, 15, 20, 50, 100, 140, 300]  # every kernel and variant


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("exps", [(-117, 100, -8), (100, -117, -8), (-8, 100, -117), (100, -8, -117),
                                  (-117, -117, 60), (110, 0, -110), (20, -100, 20), (30, -12, -60),
                                  (119, -117, -117), (119, 119, 119)])
@pytest.mark.parametrize("unit", [0, 1])
def test_value_scales_far_apart(binding, so, rows, exps, unit):
    """Pages whose value scales lie up to 2^236 apart (a page of zeros has 2^-117): the weights of all of them count
    in the sum, and no output becomes NaN or infinite."""
    lens = 384
    c = Cache(1, 1, 3, seed=rows)
    c.vs_h[c.table_h[0], 0] = [2.0 ** e for e in exps]
    for page, e in zip(c.table_h[0], exps):
        if e == -117:
            c.v_h[page] = 0
    c.up()
    q = _randn(_gen(rows), 1, rows, 128)
    ref = so.cache_attention(bf16_to_f64(q), c.k_h, c.v_h, c.ks_h, c.vs_h, [0, rows], [lens], c.table_h, 0.05, unit)
    args = (q.cuda(), *c.dev, _i32([0, rows]), _i32([lens]), c.table)
    for max_kv in (lens, 4096):  # in one piece, and split
        o, lse = binding.cache_attn_fwd(*args, max_kv=max_kv, causal_unit=unit, scale=0.05)
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        _attn_close(o, lse, ref, q, c, [lens], 0.05, _p_err([rows], 1, 1))
    assert binding.get_status() == 0


@pytest.mark.parametrize("rows", ROWS)
def test_values_next_to_the_largest(binding, rows):
    """1000 values of 2^127 and of -2^127 each: their mean is inside bf16's range, their sum is not inside fp32's."""
    x = torch.full((1000, 1, 128), 2.0 ** 127, dtype=torch.bfloat16, device="cuda")
    x[:, :, 1::2] = -2.0 ** 127
    k8, v8 = (torch.zeros((8, 1, 128, 128), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((8, 1), device="cuda") for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    binding.cache_write(torch.zeros_like(x), x, k8, v8, ks, vs, _i32([0, 1000]), _i32([1000]), table)
    q = _randn(_gen(1), 1, rows, 128).cuda()
    for max_kv in (128, 1000, 1 << 16):
        o, lse = binding.cache_attn_fwd(q, k8, v8, ks, vs, _i32([0, rows]), _i32([1000]), table, max_kv=max_kv)
        assert torch.equal(o, x[:1, 0].expand(1, rows, 128))
        assert torch.all((lse - np.log(1000)).abs() < 1e-5)
    assert binding.get_status() == 0


# ---------------------------------------------------------------------------- unusual calls

def test_numbers_beyond_32_bits_are_refused(binding):
    """They would reach the library without their upper bits: a causal unit of 2^32 as none at all."""
    c = Cache(1, 1, 2, seed=1)
    x = torch.zeros((3, 1, 128), dtype=torch.bfloat16, device="cuda")
    q, lists = x.transpose(0, 1).contiguous(), (_i32([0, 3]), _i32([200]), c.table)
    before = [t.clone() for t in c.dev]
    for kw in (dict(causal_unit=1 << 32), dict(max_new=(1 << 32) + 3), dict(max_kv=(1 << 32) + 256),
               dict(causal_unit=-(1 << 32) + 1)):
        with pytest.raises(ValueError):
            binding.cache_attn_fwd(q, *c.dev, *lists, **kw)
    with pytest.raises(ValueError):
        binding.cache_write(x, x, *c.dev, *lists, max_new=(1 << 32) + 3)
    with pytest.raises(ValueError):
        binding.cache_attn_workspace(q, c.k, c.table, max_kv=(1 << 32) + 256)
    for grid, start in ((((1 << 32) + 2, 2), (0, 0, 0)), ((2, (1 << 32) + 2), (0, 0, 0)), ((2, 2), (1 << 32, 0, 0))):
        with pytest.raises(ValueError):
            binding.rope_fwd(x, None, binding.rope_plan(), grid=grid, start=start)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c.dev, before))
    # numpy's numbers are taken like Python's
    a = binding.cache_attn_fwd(q, *c.dev, *lists, max_new=np.int64(3), max_kv=np.int32(256), causal_unit=np.int64(2))
    b = binding.cache_attn_fwd(q, *c.dev, *lists, max_new=3, max_kv=256, causal_unit=2)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    a = binding.rope_fwd(x, None, binding.rope_plan(), grid=np.array([2, 2]), start=np.array([1, 2, 3]))
    b = binding.rope_fwd(x, None, binding.rope_plan(), grid=(2, 2), start=(1, 2, 3))
    assert torch.equal(a[0], b[0])
    assert binding.get_status() == 0


def test_default_bound_of_a_table_for_2_31_tokens(binding, longest):
    """A table that names more tokens than 32 bits count is no reason to refuse a short stream."""
    *cache, table = longest
    q = torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    o, lse = binding.cache_attn_fwd(q, *cache, _i32([0, 1]), _i32([300]), table)
    assert torch.all(o == 1.0) and torch.all((lse - np.log(300)).abs() < 1e-5)
    ws = binding.cache_attn_workspace(q, cache[0], table)
    again, _ = binding.cache_attn_fwd(q, *cache, _i32([0, 1]), _i32([300]), table, ws=ws)
    assert torch.equal(o, again) and binding.get_status() == 0


# ---------------------------------------------------------------------------- rotary positions and autograd

@pytest.fixture(params=["compiled", "ctypes"])
def calls(request, binding, monkeypatch):
    monkeypatch.setattr(binding, "_fast", binding._load_fast() if request.param == "compiled" else binding._NoFast)
    return binding


@pytest.mark.parametrize("pairing", ["interleaved", "halves"])
@pytest.mark.parametrize("given", ["grid", "pos"])
def test_rope_under_autograd(calls, so, pairing, given):
    """Slices of a fused projection that asks for a gradient: the formula's gradient, bit for bit rope_bwd's."""
    g = _gen(31)
    n, hq, hk, plan = 77, 4, 2, calls.rope_plan(pairing=pairing)
    pos = torch.randint(-50, 5000, (n, 3), generator=g).int()
    where = dict(pos=pos.cuda()) if given == "pos" else dict(grid=(5, 7), start=(3, 0, 1))
    if given == "grid":
        pos = torch.from_numpy(_grid_pos(n, 5, 7, (3, 0, 1)))
    x = _randn(g, n, hq + hk, 128).cuda().requires_grad_()
    qo, ko = calls.rope_fwd(x[:, :hq], x[:, hq:], plan, **where)
    plain = calls.rope_fwd(x[:, :hq].detach(), x[:, hq:].detach(), plan, **where)
    assert torch.equal(qo, plain[0]) and torch.equal(ko, plain[1])
    assert qo.requires_grad and ko.requires_grad and not plain[0].requires_grad
    dq, dk = _randn(g, hq, n, 128).cuda(), _randn(g, hk, n, 128).cuda()
    before = bytes(plan)
    plan.turns[0] = 0.25  # the gradient is that of the call, whatever becomes of its plan
    torch.autograd.backward([qo, ko], [dq, dk])
    plan = type(plan).from_buffer_copy(before)
    want = torch.cat(calls.rope_bwd(dq, dk, plan, **where), 1)
    assert torch.equal(x.grad, want)
    both = bf16_to_f64(torch.cat([dq, dk]).transpose(0, 1))
    _rope_close(bf16_to_f64(x.grad), so.rope(both, pos.numpy(), (44, 42, 42), pairing=pairing, inverse=True), both)


def test_rope_autograd_of_one_output_and_odd_gradients(calls):
    g = _gen(32)
    plan = calls.rope_plan()
    q, k = (_randn(g, 9, h, 128).cuda().requires_grad_() for h in (3, 2))
    ones = lambda h: torch.ones((h, 9, 128), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    back = calls.rope_bwd(ones(3), ones(2), plan, grid=(3, 3))
    fwd = lambda *a, **kw: calls.rope_fwd(*a, plan, grid=(3, 3), **kw)  # noqa: E731
    # one output alone is used; gradients that are one expanded number, or lie channel by channel
    assert torch.equal(torch.autograd.grad(fwd(q, k)[1].sum(), k)[0], back[1])
    assert torch.equal(torch.autograd.grad(fwd(q, k)[0].sum(), q)[0], back[0])
    assert torch.autograd.grad(fwd(q, k)[1].sum(), q, allow_unused=True)[0] is None
    assert torch.equal(torch.autograd.grad(fwd(q, None)[0].sum(), q)[0], back[0])
    assert torch.equal(torch.autograd.grad(fwd(q.detach(), k)[1].sum(), k)[0], back[1])
    odd = _randn(g, 128, 9, 3).cuda().permute(2, 1, 0)
    got, = torch.autograd.grad(fwd(q, k)[0], q, odd)
    assert torch.equal(got, calls.rope_bwd(odd.contiguous(), None, plan, grid=(3, 3))[0])
    shifted = torch.empty(3 * 9 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(3, 9, 128).copy_(odd)
    got2, = torch.autograd.grad(fwd(q, k)[0], q, shifted)
    assert torch.equal(got, got2)
    # the gradient's own gradient is the rotation
    dq = ones(3).requires_grad_()
    gq, = torch.autograd.grad(fwd(q, None)[0], q, dq, create_graph=True)
    w = _randn(g, 9, 3, 128).cuda()
    assert torch.equal(torch.autograd.grad(gq, dq, w)[0], fwd(w, None)[0])
    direct, _ = calls.rope_bwd(dq, None, plan, grid=(3, 3))
    assert torch.equal(torch.autograd.grad(direct, dq, w)[0], fwd(w, None)[0])


def test_rope_autograd_refusals_streams_and_no_grad(calls):
    g = _gen(33)
    plan = calls.rope_plan()
    q = _randn(g, 6, 2, 128).cuda().requires_grad_()
    out = torch.empty((2, 6, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="gradient"):
        calls.rope_fwd(q, None, plan, grid=(2, 3), q_out=out)
    with torch.no_grad():
        want = calls.rope_fwd(q, None, plan, grid=(2, 3), q_out=out)[0]
        assert want is out or want.data_ptr() == out.data_ptr()
        assert not calls.rope_fwd(q, None, plan, grid=(2, 3))[0].requires_grad
    with torch.inference_mode():
        assert torch.equal(calls.rope_fwd(q, None, plan, grid=(2, 3))[0], out)
    # positions that are changed between the rotation and its gradient
    pos = torch.ones((6, 3), dtype=torch.int32, device="cuda")
    y, _ = calls.rope_fwd(q, None, plan, pos=pos)
    pos += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y.sum(), q)
    # on a stream of its own: the gradient follows it there
    q = q.detach().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, _ = calls.rope_fwd(q, None, plan, grid=(2, 3), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, out)
    dy = _randn(g, 2, 6, 128).cuda()
    got, = torch.autograd.grad(y, q, dy)
    assert torch.equal(got, calls.rope_bwd(dy, None, plan, grid=(2, 3))[0])


def test_rope_autograd_in_a_captured_graph(calls):
    g = _gen(34)
    plan = calls.rope_plan()
    q, k = (_randn(g, 8, h, 128).cuda().requires_grad_() for h in (3, 1))
    pos = torch.zeros((8, 3), dtype=torch.int32, device="cuda")
    dq, dk = (torch.empty((h, 8, 128), dtype=torch.bfloat16, device="cuda") for h in (3, 1))

    def step():
        outs = calls.rope_fwd(q, k, plan, pos=pos)
        return tuple(y.detach() for y in outs) + torch.autograd.grad(outs, (q, k), (dq, dk))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        with torch.no_grad():
            for t in (q, k, dq, dk):
                t.copy_(_randn(g, *t.shape))
            pos.copy_(torch.randint(0, 99, (8, 3), generator=g).int())
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


# ---------------------------------------------------------------------------- refused steps

def test_a_refused_step_leaves_the_cache_as_it_was(binding):
    from calibrated_block_sparse_b200.stream import FrameStreams
    g = _gen(41)
    made = [FrameStreams(batch=2, heads=2, kv_heads=1, H=4, W=5, pages=8) for _ in range(2)]
    x = _randn(g, 100, 4, 128).cuda()
    for st in made:
        st.step(x[:, :2], x[:, 2:3], x[:, 3:], new=[60, 40])
    st = made[0]
    free, was = st.free_pages, [t.clone() for t in (st.k8, st.v8, st.k_scale, st.v_scale, st.table)]
    y = (_randn(g, 300, 4, 128) * 1000).cuda()  # larger: the scales of the begun pages would grow
    wide = torch.zeros((300, 4, 132), dtype=torch.bfloat16, device="cuda")[:, :, :128]
    odd = torch.zeros(300 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(300, 1, 128)
    refused = [dict(causal_unit=-1), dict(causal_unit=1 << 32), dict(causal_unit=0.5), dict(v=odd), dict(k=wide[:, :1]),
               dict(q=wide[:, :2]), dict(v=wide[:, :1])]
    for kw in refused:
        a = {**dict(q=y[:, :2], k=y[:, 2:3], v=y[:, 3:]), **kw}
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            st.step(**a, new=[200, 100])
        assert st.lengths == [60, 40] and st.free_pages == free, kw
    st.plan.pairs = 65
    with pytest.raises(binding.CalibattError):
        st.step(y[:, :2], y[:, 2:3], y[:, 3:], new=[200, 100])
    st.plan.pairs = 64
    assert st.lengths == [60, 40] and st.free_pages == free
    for a, b in zip(was, (st.k8, st.v8, st.k_scale, st.v_scale, st.table)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    outs = [s.step(x[:, :2], x[:, 2:3], x[:, 3:], new=[70, 30], causal_unit=20) for s in made]
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert binding.get_status() == 0
