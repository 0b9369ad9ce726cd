"""Measured cases of the streaming-attention operators: rotary positions over several axes
(forward and gradient), writing keys and values into a paged 8-bit cache with one scale per
page of 128 tokens and head, and attention over that cache.

A video stream is generated frame by frame: the new tokens' queries and keys are rotated by
their (time, height, width) position, keys and values are appended to the cache, and the new
queries attend to everything cached. `run` computes one of these operators: in elementary
torch operations (own = False) or through the package's entry points (own = True).
"""
import math

import torch

own = False

PAGE = 128  # tokens per cache page
D = 128     # head size
E_MIN = -117  # smallest exponent of a page's scale


# ---------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a 40-head model: what a call costs at the least
        _rope("rope one token", n=1, heads=40, kv_heads=40, H=30, W=52, t0=400),
        # queries and keys of a whole 480p clip, 21 x 30 x 52 tokens and 40 heads
        _rope("rope 480p clip", n=32760, heads=40, kv_heads=40, H=30, W=52, t0=0),
        # packed clips and text with explicit positions, shared key heads, halves paired, odd length
        _rope("rope packed positions", n=7421, heads=24, kv_heads=8, H=0, W=0, t0=1000000, pairing="halves",
              ladder="shared"),
        # gradient of three latent frames of a 480p clip
        _rope("rope gradient", n=4680, heads=40, kv_heads=40, H=30, W=52, t0=18, back=True),
        # eight streams, one token each, pages partly filled
        _write("write one token each", batch=8, heads=8, new=1, kv=5000),
        # one latent frame of 30 x 52 tokens, starting inside a page
        _write("write one 480p frame", batch=1, heads=40, new=1560, kv=10001),
        # four ragged streams with three latent 720p frames of 45 x 80 tokens
        _write("write 720p frames", batch=4, heads=40, new=10800, kv=21600),
        # one token of one short stream
        _attn("attend one token, short", batch=1, heads=40, kv_heads=40, new=1, kv=333, unit=0),
        # one token of one stream over a whole 480p clip
        _attn("attend one token, long", batch=1, heads=40, kv_heads=40, new=1, kv=32760, unit=0),
        # sixteen ragged streams with shared key heads, a few tokens each
        _attn("attend few tokens, shared", batch=16, heads=40, kv_heads=8, new=3, kv=20000, unit=1),
        # one latent 480p frame over the clip so far: the step of a frame-by-frame generator
        _attn("attend 480p frame", batch=1, heads=40, kv_heads=40, new=1560, kv=32760, unit=0),
        # three short clips of 16 heads taken in at once, each frame sees itself and earlier ones
        _attn("attend frame by frame", batch=3, heads=16, kv_heads=16, new=6240, kv=6240, unit=1560),
    ]


def _rope(name, n, heads, kv_heads, H, W, t0, pairing="interleaved", ladder="axis", back=False):
    return {"name": name, "op": "rope", "n": n, "heads": heads, "kv_heads": kv_heads, "H": H, "W": W, "t0": t0,
            "pairing": pairing, "ladder": ladder, "back": back}


def _write(name, batch, heads, new, kv):
    return {"name": name, "op": "write", "batch": batch, "heads": heads, "new": new, "kv": kv}


def _attn(name, batch, heads, kv_heads, new, kv, unit):
    return {"name": name, "op": "attn", "batch": batch, "heads": heads, "kv_heads": kv_heads, "new": new, "kv": kv,
            "unit": unit}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "attn", "attn"])
    if op == "rope":
        kv_heads = rng.randint(1, 40)
        group = rng.choice([1, 1, 2, 4, 5, 8])
        heads = min(40, kv_heads * group)
        if heads % kv_heads:
            heads = kv_heads
        H, W = (rng.randint(1, 60), rng.randint(1, 90)) if rng.random() < 0.6 else (0, 0)
        c = _rope("", n=_log(rng, 1, 32760), heads=heads, kv_heads=kv_heads, H=H, W=W, t0=_log(rng, 1, 1000000),
                  pairing=rng.choice(["interleaved", "halves"]), ladder=rng.choice(["axis", "shared"]),
                  back=rng.random() < 0.4)
    elif op == "write":
        batch, heads = _log(rng, 1, 16), rng.randint(1, 40)
        new = _log(rng, 1, max(1, 43200 // batch))
        c = _write("", batch=batch, heads=heads, new=new, kv=new + _log(rng, 1, 20000))
    else:
        kv_heads = rng.choice([1, 2, 5, 8, 16, 24, 40])
        group = rng.choice([1, 1, 1, 2, 4, 5, 8])
        heads = kv_heads * group if kv_heads * group <= 40 else kv_heads
        batch, kv = _log(rng, 1, 16), _log(rng, 1, 75600)
        kv = max(1, min(kv, 40 * 32760 // (batch * kv_heads)))
        new = min(kv, _log(rng, 1, 1560))
        new = max(1, min(new, 40 * 1560 * 32760 // (heads * batch * kv)))
        c = _attn("", batch=batch, heads=heads, kv_heads=kv_heads, new=new, kv=kv,
                  unit=rng.choice([0, 1, rng.randint(2, 1560)]))
    del c["name"]
    return c


def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of each stream: the first as the
    case says, the others shorter."""
    new = [max(1, c["new"] - (c["new"] * 3 * b) // (5 * c["batch"])) for b in range(c["batch"])]
    old = c["kv"] - c["new"]
    return new, [m + old - (old * 5 * b) // (7 * c["batch"]) for b, m in enumerate(new)]


def _pages(length):
    return -(-length // PAGE)


# ---------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    st = {"case": case}
    if case["op"] == "rope":
        n, hq, hk = case["n"], case["heads"], case["kv_heads"]
        # projections write token by token, attention reads head by head
        shape = (lambda h: (h, n, D)) if case["back"] else (lambda h: (n, h, D))
        st["q"], st["k"] = randn(*shape(hq)).bfloat16(), randn(*shape(hk)).bfloat16()
        if case["H"] == 0:
            # packed clips of 16 x 24 patches with text tokens (equal positions on all axes) in between
            t = torch.arange(n, device="cuda")
            clip, at = t // 500, t % 500
            text = at >= 384
            pos = torch.stack([case["t0"] + clip, at // 24, at % 24], 1)
            st["pos"] = torch.where(text[:, None], (at - 384 + case["t0"])[:, None], pos).to(torch.int32)
        return st
    new, lens = _lengths(case)
    batch, heads = case["batch"], case.get("kv_heads", case["heads"])
    st["max_new"], st["max_kv"] = max(new), max(lens)
    width = _pages(max(lens))
    n_pages = batch * width + 1
    st["table"] = torch.randperm(n_pages, generator=g, device="cuda")[: batch * width].reshape(batch, width).to(torch.int32)
    st["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["start"] = torch.tensor([0] + [sum(new[: b + 1]) for b in range(batch)], dtype=torch.int32, device="cuda")
    # what is cached: pages of normal values whose sizes differ from page to page and head to head;
    # slots that no token has reached hold NaN
    shape = (n_pages, heads, PAGE, D)
    for name in ("k", "v"):
        e = torch.randint(-9, -5, (n_pages, heads), generator=g, device="cuda")
        x = (torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) * 80).clamp(-448, 448).to(torch.float8_e4m3fn)
        for b in range(batch):
            held = lens[b] if case["op"] == "attn" else lens[b] - new[b]
            if held % PAGE:
                x.view(torch.uint8)[st["table"][b, held // PAGE].long(), :, held % PAGE:] = 127
        st[name + "8"], st[name + "_scale"] = x, torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    total = sum(new)
    if case["op"] == "write":
        # keys have channels that are larger than the others
        size = torch.exp(randn(heads, D) * 0.5)
        st["k"] = (randn(total, heads, D) * size).bfloat16()
        st["v"] = randn(total, heads, D).bfloat16()
    else:
        st["q"] = randn(case["heads"], total, D).bfloat16()
    return st


# ---------------------------------------------------------------------------------- a pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    if case["op"] == "rope":
        return _plain_rope(state, case)
    return _plain_write(state, case) if case["op"] == "write" else _plain_attn(state, case)


def _own(st, case):
    from calibrated_block_sparse_b200 import binding
    if case["op"] == "rope":
        if "plan" not in st:  # a program makes its plan once
            st["plan"] = binding.rope_plan((44, 42, 42), theta=10000.0, pairing=case["pairing"], ladder=case["ladder"])
        grid = (case["H"], case["W"]) if case["H"] else None
        fn = binding.rope_bwd if case["back"] else binding.rope_fwd
        return fn(st["q"], st["k"], st["plan"], grid=grid, start=(case["t0"], 0, 0), pos=st.get("pos"))
    if case["op"] == "write":
        binding.cache_write(st["k"], st["v"], st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["start"],
                            st["kv_len"], st["table"], max_new=st["max_new"])
        return [st[x] for x in ("k8", "v8", "k_scale", "v_scale")]
    if "ws" not in st:  # a program keeps its workspace
        st["ws"] = binding.cache_attn_workspace(st["q"], st["k8"], st["table"], max_new=st["max_new"],
                                                max_kv=st["max_kv"])
    return binding.cache_attn_fwd(st["q"], st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["start"], st["kv_len"],
                                  st["table"], max_new=st["max_new"], max_kv=st["max_kv"], causal_unit=case["unit"],
                                  ws=st["ws"])


def _plain_rope(st, case):
    """x cos + partner(x) sin per channel pair, the angle position * frequency in 64 bits."""
    dims, n, dev = (44, 42, 42), case["n"], st["q"].device
    axis = torch.repeat_interleave(torch.arange(3, device=dev), torch.tensor([d // 2 for d in dims], device=dev),
                                   output_size=64)
    i = torch.arange(64, device=dev, dtype=torch.float64)
    if case["ladder"] == "axis":
        first = torch.tensor([0, 22, 43], device=dev)[axis]
        expo = 2 * (i - first) / torch.tensor(dims, device=dev, dtype=torch.float64)[axis]
    else:
        expo = 2 * i / 128
    freq = 10000.0 ** -expo
    if case["H"]:
        t = torch.arange(n, device=dev)
        hw = case["H"] * case["W"]
        pos = torch.stack([case["t0"] + t // hw, t % hw // case["W"], t % case["W"]], 1)
    else:
        pos = st["pos"]
    angle = pos[:, axis].double() * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    if case["back"]:
        sin = -sin
    at = (lambda a: a[None]) if case["back"] else (lambda a: a[:, None])

    def turn(x):
        x = x.float()
        a, b = (x[..., 0::2], x[..., 1::2]) if case["pairing"] == "interleaved" else (x[..., :64], x[..., 64:])
        c, d = a * at(cos) - b * at(sin), a * at(sin) + b * at(cos)
        y = torch.stack([c, d], -1).flatten(-2) if case["pairing"] == "interleaved" else torch.cat([c, d], -1)
        return y.to(torch.bfloat16).transpose(0, 1).contiguous()

    return turn(st["q"]), turn(st["k"])


def _places(st, total):
    """Stream and position of every packed new token."""
    t = torch.arange(total, device=st["start"].device, dtype=torch.int32)
    b = torch.searchsorted(st["start"], t, right=True) - 1
    new = st["start"][1:] - st["start"][:-1]
    return b, (st["kv_len"] - new)[b] + t - st["start"][b]


def _plain_write(st, case):
    """Each page and head keeps q = round_e4m3(x / 2^e), 2^e the least power of two with max|x| <= 448 * 2^e;
    a page that was begun earlier keeps the larger of its old and new exponent."""
    b, pos = _places(st, st["k"].shape[0])
    page, slot = st["table"][b, pos // PAGE].long(), pos % PAGE
    old_pos = st["kv_len"] - (st["start"][1:] - st["start"][:-1])
    first = st["table"].gather(1, (old_pos // PAGE).long()[:, None])[:, 0].long()  # page that each stream goes on with
    begun = (old_pos % PAGE > 0)[:, None]
    for x, c, s in ((st["k"], st["k8"], st["k_scale"]), (st["v"], st["v8"], st["v_scale"])):
        x = x.float()
        most = torch.zeros_like(s).index_reduce_(0, page, x.abs().amax(-1), "amax")
        m, e = torch.frexp(most)
        e = torch.where(most > 0, e - 9 + (m > 0.875).int(), E_MIN).clamp_min(E_MIN)
        scale = torch.ldexp(torch.ones_like(most), e)
        scale[first] = torch.where(begun, torch.maximum(scale[first], s[first]), scale[first])
        ratio = torch.where(begun, s[first] / scale[first], 1.0)
        c[first] = (c[first].float() * ratio[:, :, None, None]).to(torch.float8_e4m3fn)
        q = (x / scale[page][..., None]).to(torch.float8_e4m3fn)
        c.view(torch.uint8)[page, :, slot] = q.view(torch.uint8)
        s[page] = scale[page]
    return [st[x] for x in ("k8", "v8", "k_scale", "v_scale")]


def _plain_attn(st, case):
    """softmax(q k / sqrt(d)) v over the cached tokens that each query sees, all streams padded to the longest."""
    hq, total, _ = st["q"].shape
    hk, batch, dev = case["kv_heads"], case["batch"], st["q"].device
    group, table = hq // hk, st["table"].long()
    longest = table.shape[1] * PAGE
    held = torch.arange(longest, device=dev) < st["kv_len"][:, None]                     # [batch][longest]

    def cached(c, s):
        x = c[table].float() * s[table][..., None, None]                                 # [batch][pages][hk][128][d]
        x = x.transpose(1, 2).reshape(batch, hk, longest, D)
        return x.masked_fill_(~held[:, None, :, None], 0.0)

    b, pos = _places(st, total)
    i = torch.arange(total, device=dev) - st["start"][b]
    q = torch.zeros((batch, st["max_new"], hq, D), device=dev)
    q[b, i] = st["q"].transpose(0, 1).float()
    q = q.transpose(1, 2).reshape(batch, hk, group * st["max_new"], D)
    sees = st["kv_len"][b] if case["unit"] == 0 else torch.minimum((pos // case["unit"] + 1) * case["unit"], st["kv_len"][b])
    upto = torch.zeros((batch, st["max_new"]), device=dev, dtype=torch.int64)
    upto[b, i] = sees.long()
    hidden = torch.arange(longest, device=dev) >= upto[:, :, None]                       # [batch][max_new][longest]
    s = torch.matmul(q, cached(st["k8"], st["k_scale"]).transpose(2, 3)).mul_(1 / math.sqrt(D))
    s.view(batch, hk, group, st["max_new"], longest).masked_fill_(hidden[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, cached(st["v8"], st["v_scale"])) / torch.where(l > 0, l, 1.0)
    o = o.reshape(batch, hq, st["max_new"], D)[b, :, i].transpose(0, 1).to(torch.bfloat16).contiguous()
    lse = (m + l.log()).reshape(batch, hq, st["max_new"])[b, :, i].transpose(0, 1).contiguous()
    return o, lse


# ---------------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "rope":
        values = case["n"] * (case["heads"] + case["kv_heads"]) * D
        return {"bytes": 4 * values + (12 * case["n"] if case["H"] == 0 else 0), "flops": 3 * values}
    new, lens = _lengths(case)
    if case["op"] == "write":
        values = 2 * sum(new) * case["heads"] * D
        touched = sum(_pages(k) - (k - m) // PAGE for m, k in zip(new, lens))
        return {"bytes": 3 * values + 8 * touched * case["heads"], "flops": 2 * values}
    hq, hk, unit = case["heads"], case["kv_heads"], case["unit"]
    pairs = 0
    for m, k in zip(new, lens):
        pairs += m * k if unit == 0 else sum(min(k, (p // unit + 1) * unit) for p in range(k - m, k))
    moved = 4 * sum(new) * hq * D + 4 * sum(new) * hq + 2 * sum(lens) * hk * D + 8 * hk * sum(_pages(k) for k in lens)
    return {"bytes": moved, "flops": 4 * D * hq * pairs}


# ---------------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st, case)
    return _exact_write(st, case) if case["op"] == "write" else _exact_attn(st, case)


def _exact_rope(st, case):
    """Each pair as a complex number times exp(i * angle), in its place."""
    n = case["n"]
    owner = [0] * 22 + [1] * 21 + [2] * 21
    within = list(range(22)) + list(range(21)) + list(range(21))
    width = [44] * 22 + [42] * 42
    outs = []
    for x in (st["q"], st["k"]):
        y = x.transpose(0, 1) if not case["back"] else x   # [heads][n][d]
        y = y.double()
        out = torch.empty_like(y)
        t = torch.arange(n, device=y.device, dtype=torch.float64)
        for j in range(64):
            if case["H"]:
                hw = float(case["H"] * case["W"])
                f = torch.floor(t / hw)
                r = torch.floor((t - f * hw) / case["W"])
                p = (f + case["t0"], r, t - f * hw - r * case["W"])[owner[j]]
            else:
                p = st["pos"][:, owner[j]].double()
            w = math.pow(10000.0, -2.0 * within[j] / width[j] if case["ladder"] == "axis" else -j / 64.0)
            a, b = (2 * j, 2 * j + 1) if case["pairing"] == "interleaved" else (j, j + 64)
            z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones_like(p), -p * w if case["back"] else p * w)
            out[..., a], out[..., b] = z.real, z.imag
        outs.append(out.transpose(0, 1).contiguous() if case["back"] else out)
    return tuple(outs)


def _round8(x):
    """The e4m3 value next to x, ties to even, for |x| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _exact_write(st, case):
    new, lens = _lengths(case)
    done = {}
    for name in ("k", "v"):
        c, s = st[name + "8"].double(), st[name + "_scale"].double()
        at = 0
        for m, k in zip(new, lens):
            b = len(done.setdefault(name, []))
            done[name].append(b)
            p = k - m
            while p < k:
                page, lo = int(st["table"][b, p // PAGE]), p % PAGE
                hi = min(PAGE, lo + k - p)
                x = st[name][at: at + hi - lo].double().transpose(0, 1)      # [heads][tokens][d]
                big = x.abs().amax((1, 2))
                e = torch.full_like(big, E_MIN)
                for step in range(E_MIN, 121):
                    e = torch.where(big > 448.0 * 2.0 ** step, float(step + 1), e)
                scale = torch.exp2(e)
                if lo:
                    scale = torch.maximum(scale, s[page])
                    r = (s[page] / scale)[:, None, None]
                    c[page, :, :lo] = _round8(c[page, :, :lo] * r)
                s[page] = scale
                c[page, :, lo:hi] = _round8(x / scale[:, None, None])
                p, at = p + hi - lo, at + hi - lo
        done[name] = (c, s)
    return [done["k"][0], done["v"][0], done["k"][1], done["v"][1]]


def _exact_attn(st, case):
    new, lens = _lengths(case)
    hq, hk = case["heads"], case["kv_heads"]
    o = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    at = 0
    for b, (m, n) in enumerate(zip(new, lens)):
        token = torch.arange(n, device="cuda")
        page, slot = st["table"][b, : _pages(n)].long()[token // PAGE], token % PAGE
        own_pos = torch.arange(n - m, n, device="cuda")
        last = torch.full_like(own_pos, n) if case["unit"] == 0 else (own_pos // case["unit"] + 1) * case["unit"]
        for h in range(hq):
            g = h // (hq // hk)
            k = st["k8"][:, g][page, slot].double() * st["k_scale"][page, g].double()[:, None]
            v = st["v8"][:, g][page, slot].double() * st["v_scale"][page, g].double()[:, None]
            s = (st["q"][h, at: at + m].double() @ k.T) / math.sqrt(D)
            s = torch.where(token[None, :] < last[:, None], s, -math.inf)
            z = torch.logsumexp(s, 1)
            o[h, at: at + m] = torch.exp(s - z[:, None]) @ v
            lse[h, at: at + m] = z
        at += m
    return o, lse
