"""Host-side tests of the streaming entry points: plans, sizes and refusals
(nothing is launched: every refused call returns before it enqueues work)."""
import ctypes

import numpy as np
import pytest
import torch

P = ctypes.c_void_p
FAKE, ODD = 0x10000000, 0x10000008  # never dereferenced
OK, ARG, ALIGN, UNSUPPORTED = 0, -1, -3, -4


@pytest.fixture(scope="module")
def binding():
    from calibrated_block_sparse_b200 import binding as b, build
    build.build()
    b.load()
    return b


@pytest.mark.parametrize("dims", [(44, 42, 42), (16, 0, 0), (0, 64, 64), (48, 40, 24), (2, 0, 0)])
@pytest.mark.parametrize("ladder", ["axis", "shared"])
def test_rope_plan_matches_the_oracle(binding, dims, ladder):
    from oracle import stream as so
    plan = binding.rope_plan(dims, theta=10000.0, ladder=ladder)
    freq, axis = so.rope_frequencies(dims, 10000.0, ladder)
    assert plan.pairs == len(freq)
    assert list(plan.axis[:plan.pairs]) == axis.tolist()
    np.testing.assert_allclose(np.array(plan.turns[:plan.pairs]) * 2 * np.pi, freq, rtol=4e-16 * 4)


@pytest.mark.parametrize("dims,kw,code", [((43, 42, 42), {}, ARG), ((0, 0, 0), {}, ARG), ((64, 64, 2), {}, ARG),
                                          ((-2, 64, 64), {}, ARG), ((44, 42, 42), {"theta": 0.0}, ARG),
                                          ((44, 42, 42), {"theta": float("nan")}, ARG),
                                          ((44, 42, 40), {"pairing": "halves"}, UNSUPPORTED)])
def test_rope_plan_refusals(binding, dims, kw, code):
    with pytest.raises(binding.CalibattError) as e:
        binding.rope_plan(dims, **kw)
    assert e.value.code == code
    with pytest.raises(ValueError):
        binding.rope_plan(pairing="neighbours")


def _rope(binding, fn="calibatt_rope_fwd", **kw):
    plan = kw.pop("plan", None) or binding.rope_plan()
    a = dict(q=FAKE, qts=512, qhs=128, hq=4, k=0, kts=0, khs=0, hk=0, n=10, d=128, pos=0, H=2, W=5, start=None,
             qo=FAKE + (1 << 24), qots=128, qohs=1280, ko=0, kots=0, kohs=0)
    a.update(kw)
    v = list(a.values())
    return getattr(binding.load(), fn)(ctypes.byref(plan), *v, None)


@pytest.mark.parametrize("fn", ["calibatt_rope_fwd", "calibatt_rope_bwd"])
def test_rope_refusals(binding, fn):
    call = lambda **kw: _rope(binding, fn, **kw)  # noqa: E731
    assert call(n=0) == OK
    assert call(d=64) == UNSUPPORTED
    for bad in (dict(q=0), dict(qo=0), dict(hq=0), dict(n=-1), dict(H=0), dict(W=0), dict(hk=2), dict(qts=-8),
                dict(n=1 << 40), dict(qts=1 << 60)):
        assert call(**bad) == ARG, bad
    for bad in (dict(q=ODD), dict(qo=ODD), dict(qts=516), dict(qohs=1284), dict(pos=FAKE + 2)):
        assert call(**bad) == ALIGN, bad
    # outputs that name an element twice, or that another tensor of the call overlaps
    for bad in (dict(qots=0), dict(qohs=0), dict(qots=64), dict(qohs=1024), dict(qo=FAKE),
                dict(qo=FAKE + 256), dict(hk=1, k=FAKE, kts=512, khs=128, ko=FAKE + (1 << 24), kots=128, kohs=1280),
                dict(hk=1, k=FAKE + (1 << 24) + 256, kts=512, khs=128, ko=FAKE + (1 << 25), kots=128, kohs=1280)):
        assert call(**bad) == ARG, bad
    plan = binding.rope_plan()
    plan.pairs = 65
    assert call(plan=plan) == ARG
    plan = binding.rope_plan()
    plan.axis[3] = 3
    assert call(plan=plan) == ARG
    plan = binding.rope_plan(pairing="halves")
    plan.pairs = 60
    assert call(plan=plan) == UNSUPPORTED


def test_compiled_calls_leave_what_is_not_plain_to_the_binding(binding):
    """Nothing is enqueued for tensors that are not CUDA tensors, or no tensors at all."""
    fast = binding._load_fast()
    assert fast is not binding._NoFast  # build() made them
    x, plan = torch.zeros((3, 2, 128), dtype=torch.bfloat16), ctypes.addressof(binding.rope_plan())
    for q in (x, None, 3, "q", [1.0], torch.nn.Parameter(x)):
        assert fast.rope(True, q, None, plan, (1, 3), (0, 0, 0), None, None, None) is None
        assert fast.cache_write(q, q, *[q] * 7, None) is None
        assert fast.cache_attn(q, *[q] * 7, None, None, 0, None, None, None, None, True) is None
    for wrong in ((), (True,), (x,) * 40):
        assert fast.rope(*wrong) is None and fast.cache_write(*wrong) is None and fast.cache_attn(*wrong) is None


def _write(binding, **kw):
    a = dict(k=FAKE, kts=512, khs=128, v=FAKE, vts=512, vhs=128, heads=4, n=10, d=128, start=FAKE, kv=FAKE, batch=2,
             max_new=5, table=FAKE, ts=3, pages=9, k8=FAKE, v8=FAKE + 4096, ks=FAKE, vs=FAKE + 64)
    a.update(kw)
    return binding.load().calibatt_cache_write(*a.values(), None)


def test_cache_write_refusals(binding):
    for fine in (dict(n=0), dict(batch=0), dict(max_new=0)):
        assert _write(binding, **fine) == OK, fine
    assert _write(binding, d=64) == UNSUPPORTED
    assert _write(binding, batch=70000) == UNSUPPORTED
    for bad in (dict(k=0), dict(v=0), dict(start=0), dict(kv=0), dict(table=0), dict(k8=0), dict(v8=0), dict(ks=0),
                dict(vs=0), dict(heads=0), dict(n=-1), dict(batch=-1), dict(max_new=-1), dict(ts=0), dict(pages=0),
                dict(kts=-8), dict(v8=FAKE), dict(vs=FAKE)):
        assert _write(binding, **bad) == ARG, bad
    for bad in (dict(k=ODD), dict(v8=ODD), dict(khs=4), dict(start=FAKE + 2)):
        assert _write(binding, **bad) == ALIGN, bad


def _attn(binding, **kw):
    a = dict(q=FAKE, hq=8, hk=4, n=10, d=128, scale=0.1, unit=0, start=FAKE, kv=FAKE, batch=2, max_new=5, max_kv=300,
             table=FAKE, ts=3, pages=9, k8=FAKE, v8=FAKE, ks=FAKE, vs=FAKE, o=FAKE, lse=0, ws=0, wsb=0)
    a.update(kw)
    return binding.load().calibatt_cache_attn_fwd(*a.values(), None)


def test_cache_attn_refusals(binding):
    for fine in (dict(n=0), dict(batch=0), dict(max_new=0)):
        assert _attn(binding, **fine) == OK, fine
    for bad in (dict(d=64), dict(batch=70000), dict(hq=70000, hk=1),
                dict(batch=65535, hq=65535, hk=65535),  # more CTAs than a grid takes: few rows, and many
                dict(batch=65535, hq=60000, hk=60000, n=400, max_new=400)):
        assert _attn(binding, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=0), dict(o=0), dict(hq=7), dict(hk=0), dict(n=-1), dict(scale=0.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(unit=-1), dict(start=0), dict(kv=0), dict(table=0), dict(k8=0),
                dict(vs=0), dict(max_kv=-1), dict(max_new=-2), dict(ts=-1), dict(pages=-1)):
        assert _attn(binding, **bad) == ARG, bad
    for bad in (dict(q=ODD), dict(o=ODD), dict(k8=ODD), dict(ws=ODD), dict(lse=FAKE + 1), dict(kv=FAKE + 2)):
        assert _attn(binding, **bad) == ALIGN, bad
    # a split cache needs its workspace
    need = binding.cache_attn_workspace_size(2, 8, 4, 10, 5, 100000)
    assert need > 0
    assert _attn(binding, max_kv=100000) == ARG
    assert _attn(binding, max_kv=100000, ws=FAKE, wsb=need - 1) == ARG


def test_workspace_size_of_bad_shapes_is_zero(binding):
    for bad in ((-1, 8, 4, 10, 5, 100), (1, 8, 3, 10, 5, 100000), (1, 0, 1, 10, 5, 100000), (0, 8, 4, 0, 0, 100000)):
        assert binding.cache_attn_workspace_size(*bad) == 0


def test_binding_wants_cuda_tensors(binding):
    x = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        binding.rope_fwd(x, x, binding.rope_plan(), grid=(1, 3))
    for call in (binding.rope_fwd, binding.rope_bwd):
        for plan in (None, 7, ctypes.c_int32(1)):
            with pytest.raises(TypeError):
                call(x, x, plan, grid=(1, 3))
    with pytest.raises(TypeError):
        binding.cache_write(x, x, None, None, None, None, None, None, None)
    with pytest.raises(TypeError):
        binding.cache_attn_fwd(x, None, None, None, None, None, None, None)


def test_frame_streams_refuse_bad_shapes():
    from calibrated_block_sparse_b200.stream import FrameStreams
    for bad in (dict(batch=0), dict(heads=3), dict(kv_heads=0), dict(H=0), dict(pages=0)):
        with pytest.raises(ValueError):
            FrameStreams(**{**dict(batch=1, heads=4, kv_heads=2, H=2, W=3, pages=4), **bad})


def test_cache_attn_refuses_outputs_over_its_inputs(binding):
    """Parts of a stream are read by several CTAs while others already write: o and lse have memory of their own."""
    size = 2 * 8 * 10 * 128  # bytes of q and o
    apart = dict(q=FAKE, o=FAKE + (1 << 20), lse=FAKE + (2 << 20))
    for bad in (dict(o=FAKE), dict(o=FAKE + size - 16), dict(q=FAKE + 256, o=FAKE), dict(lse=FAKE + size - 4),
                dict(lse=FAKE + (1 << 20) + 64), dict(lse=FAKE - 4 * 8 * 10 + 4), dict(k8=FAKE + (1 << 20) - 16),
                dict(v8=FAKE + (1 << 20) + size - 16), dict(v8=FAKE + (2 << 20))):
        a = {**apart, **dict(k8=FAKE + (3 << 20), v8=FAKE + (3 << 20)), **bad}
        assert _attn(binding, **a) == ARG, bad
    # and the workspace
    need = binding.cache_attn_workspace_size(2, 8, 4, 10, 5, 100000)
    for ws in (FAKE, FAKE + (1 << 20), FAKE + (2 << 20), FAKE + (1 << 20) - need + 16):
        assert _attn(binding, max_kv=100000, k8=FAKE + (3 << 28), v8=FAKE + (3 << 28), ws=ws, wsb=need, **apart) == ARG


def test_numbers_beyond_32_bits_are_refused(binding):
    """They would reach the library without their upper bits."""
    for dims in (((1 << 32) + 44, 42, 42), (44, 42, 42 - (1 << 32)), (44, 42.5, 42)):
        with pytest.raises(ValueError):
            binding.rope_plan(dims)
    for i in range(6):
        a = [2, 8, 4, 10, 5, 100000]
        a[i] += 1 << 32
        with pytest.raises(ValueError):
            binding.cache_attn_workspace_size(*a)
    with pytest.raises(TypeError):
        binding.cache_attn_workspace_size(2, 8, 4, 10, 5.5, 100000)


def _streams(**kw):
    from calibrated_block_sparse_b200.stream import FrameStreams
    return FrameStreams(**{**dict(batch=2, heads=4, kv_heads=2, H=2, W=3, pages=6, device="cpu"), **kw})


def _state(st):
    return ([t.view(torch.uint8).clone() for t in (st.k8, st.v8, st.k_scale, st.v_scale, st.table)], list(st.lengths),
            st.free_pages, [list(p) for p in st._owned], list(st._free))


def _unchanged(st, was):
    now = _state(st)
    return all(torch.equal(a, b) for a, b in zip(now[0], was[0])) and now[1:] == was[1:]


def _tokens(n, odd=None):
    """q, k, v of n tokens; odd: the one that does not begin on 16 bytes."""
    make = lambda h, o: torch.zeros(n * h * 128 + 1, dtype=torch.bfloat16)[int(o):][:n * h * 128].view(n, h, 128)  # noqa: E731
    return [make(h, name == odd) for h, name in ((4, "q"), (2, "k"), (2, "v"))]


def test_a_refused_step_changes_nothing(binding, monkeypatch):
    st = _streams()
    fake = lambda *a, **kw: None  # noqa: E731
    monkeypatch.setattr(binding, "rope_fwd", lambda q, k, plan, **kw: (q.transpose(0, 1), k.transpose(0, 1)))
    monkeypatch.setattr(binding, "cache_write", fake)
    monkeypatch.setattr(binding, "cache_attn_fwd", fake)
    st.step(*_tokens(200), new=[130, 70])
    assert st.lengths == [130, 70] and st.free_pages == 3
    was = _state(st)
    for unit in (-1, 1 << 31, 1.5, "6", None):
        with pytest.raises((TypeError, ValueError)):
            st.step(*_tokens(200), new=[130, 70], causal_unit=unit)
        assert _unchanged(st, was), unit
    for odd in "qkv":
        with pytest.raises(ValueError):
            st.step(*_tokens(200, odd), new=[130, 70])
        assert _unchanged(st, was), odd
    # whatever the rotation, the write or an allocation raises
    for name, error in (("rope_fwd", binding.CalibattError(-1)), ("cache_write", binding.CalibattError(-5)),
                        ("cache_attn_fwd", MemoryError())):
        with monkeypatch.context() as m:
            def fail(*a, **kw):
                raise error
            m.setattr(binding, name, fail)
            with pytest.raises(type(error)):
                st.step(*_tokens(200), new=[130, 70])
        now = _state(st)
        assert now[1:] == was[1:], name
    # and the next one goes on as if nothing had been
    st.step(*_tokens(200), new=[130, 70])
    assert st.lengths == [260, 140] and st.free_pages == 1
    assert sorted(sum(st._owned, st._free)) == list(range(6))
    assert st.table[0, :3].tolist() == st._owned[0] and st.table[1, :2].tolist() == st._owned[1]


def test_frame_streams_refuse_more_than_the_library_takes():
    for bad in (dict(batch=65536), dict(heads=65536, kv_heads=65536)):
        with pytest.raises(ValueError):
            _streams(**{**dict(pages=1), **bad})


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build of one small source into a folder of its own."""
    from calibrated_block_sparse_b200 import build
    src = tmp_path / "small.cu"
    src.write_text("extern \"C\" int small(void) { return 1; }\n")
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    for name in ("LIB", "PYCALLS"):
        path = tmp_path / (name + ".so")
        path.write_text("old")
        monkeypatch.setattr(build, name, str(path))
    return build, tmp_path, src


def _module(build, path, code):
    """In the place of the module's compiler: a process that writes the module, or fails."""
    import subprocess
    import sys
    text = f"open({str(path)!r}, 'w').write('new'); raise SystemExit({code})"
    return lambda cc: (subprocess.Popen([sys.executable, "-c", text]), str(path))


@pytest.mark.parametrize("made", [True, False, None])
def test_a_module_of_another_build_does_not_stay(tree, monkeypatch, made):
    """The compiled calls call the library by address: an old module beside a new library would pass old arguments."""
    build, path, _ = tree
    monkeypatch.setattr(build, "start_pycalls",
                        (lambda cc: None) if made is None else _module(build, path / "tmp.so", 0 if made else 1))
    build.build(force=True)
    assert (path / "LIB.so").read_bytes()[:4] == b"\x7fELF"
    if made:
        assert (path / "PYCALLS.so").read_text() == "new"
    else:
        assert not (path / "PYCALLS.so").exists()
    assert not (path / "tmp.so").exists()


def test_a_failed_build_leaves_both_as_they_were(tree, monkeypatch):
    build, path, src = tree
    src.write_text("this is no source\n")
    monkeypatch.setattr(build, "start_pycalls", _module(build, path / "tmp.so", 0))
    with pytest.raises(RuntimeError):
        build.build(force=True)
    assert (path / "LIB.so").read_text() == (path / "PYCALLS.so").read_text() == "old"
    assert not (path / "tmp.so").exists()


def test_a_missing_module_is_built(binding, monkeypatch):
    from calibrated_block_sparse_b200 import build
    assert not build.needs_build()
    monkeypatch.setattr(build, "PYCALLS", build.PYCALLS + ".none")
    assert build.needs_build()
    monkeypatch.setattr(build.shutil, "which", lambda name: None)  # no compiler: the calls go through ctypes
    assert not build.needs_build()


def test_a_module_that_does_not_fit_is_not_used(binding, tmp_path, monkeypatch):
    from calibrated_block_sparse_b200 import build
    monkeypatch.setattr(binding, "_fast", None)
    with monkeypatch.context() as m:
        broken = tmp_path / "broken.so"
        broken.write_text("no module")
        m.setattr(build, "PYCALLS", str(broken))
        with pytest.warns(RuntimeWarning):
            assert binding._load_fast() is binding._NoFast
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.0")
        with pytest.warns(RuntimeWarning):
            assert binding._load_fast() is binding._NoFast
    with monkeypatch.context() as m:
        m.setattr(build, "PYCALLS", str(tmp_path / "none.so"))
        assert binding._load_fast() is binding._NoFast
    # a library of another version
    fast = binding._load_fast()
    assert fast is not binding._NoFast
    other = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: binding.load().calibatt_version() + 1)
    assert fast.bind(*[ctypes.cast(other, P).value] * 6) is False
    assert binding._load_fast() is not binding._NoFast  # bound again
