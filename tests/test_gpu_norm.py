"""The norms around a block on the GPU against 64-bit forms.

Bounds, in fp32 half steps U = 2^-24: a row sum of a group goes through at most 32 additions in a
thread, 5 in a warp and 16 over warps, so its error is at most 53 U of the sum of magnitudes; the
centred values, rstd and the products add a few roundings each; the output is rounded once. The
backward is compared with the definition at the statistics it was given."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PAIRS = [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp32")]
DEPTH = 53
EPS = 1e-6


@pytest.fixture(scope="module")
def V():
    from block_sparse_attention_max_b200 import build
    build.build()
    from block_sparse_attention_max_b200 import veda
    yield veda
    veda.check_device_status()


def _rand(*shape, seed=0, dtype=torch.float32, scale=1.0, shift=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device=DEV) + shift).to(dtype)


def _params(B, C, pdt, seed=50):
    return dict(weight=_rand(C, seed=seed, dtype=pdt, scale=0.3, shift=1.0), bias=_rand(C, seed=seed + 1, dtype=pdt),
                gain=_rand(B, C, seed=seed + 2, dtype=pdt, scale=0.4),
                shift=_rand(B, C, seed=seed + 3, dtype=pdt, scale=0.5))


def _d(t):
    return None if t is None else t.double()


def _forward(x, kind, w, b, G, S, r, res, eps=EPS):
    """Reference and its arithmetic bound. G [B, C] full gain; S shift or None."""
    xd = x.double()
    mean, rstd = R.stats(xd, kind, eps)
    xh = (xd - mean) * rstd
    one = torch.ones(x.shape[-1], device=DEV, dtype=torch.float64)
    A = (G if G is not None else one[None])[:, None] * (w if w is not None else one)
    T = torch.zeros_like(A)
    T = T + ((G if G is not None else one[None])[:, None] * b if b is not None else 0)
    T = T + (S[:, None] if S is not None else 0)
    y = xh * A + T + (r * res if res is not None else 0)
    spread = xd.abs().mean(-1, keepdim=True) * rstd if kind == "layer" else 0.0
    e = A.abs() * ((DEPTH + 2) * spread + (DEPTH / 2 + 8) * xh.abs()) + 4 * T.abs() + 3 * (xh * A).abs()
    if kind == "none":
        e = 4 * (A * xh).abs() + 4 * T.abs()
    mag = 3 * (r * res).abs() if res is not None else 0.0
    # the shift's own sum may cancel: count its terms
    if b is not None and S is not None:
        e = e + 2 * ((G if G is not None else one[None])[:, None] * b).abs() + 2 * S[:, None].abs()
    return y, R.U32 * (e + mag)


SIZES = [(1, 1, 1), (2, 3, 8), (1, 7, 63), (3, 5, 128), (2, 9, 256), (1, 40, 264), (2, 6, 512), (2, 5, 1000),
         (1, 65, 1023), (1, 11, 1024), (2, 3, 1032), (1, 33, 4096), (1, 9, 5120), (1, 4, 5121), (1, 3, 7168), (2, 2, 8192),
         (1, 6, 2047), (2, 3, 3001)]
# enough rows for every slice to take several (the rings go round)
LONG = [(2, 1500, 200), (1, 3000, 1280), (5, 400, 96), (1, 2500, 1023), (2, 1700, 5120), (1, 1300, 8190)]


@pytest.mark.parametrize("kind", ["layer", "rms", "none"])
@pytest.mark.parametrize("B,N,C", SIZES + LONG)
def test_forward(V, kind, B, N, C):
    for i, (ti, to) in enumerate(PAIRS):
        dti, dto = TYPES[ti], TYPES[to]
        x = _rand(B, N, C, seed=i, dtype=dti, shift=0.5)
        p = _params(B, C, [torch.float32, torch.bfloat16, torch.float16][i % 3])
        y = V.norm_modulate(x, p["gain"], p["shift"], p["weight"], p["bias"], kind, EPS, dto)
        ref, e = _forward(x, kind, _d(p["weight"]), _d(p["bias"]), 1 + _d(p["gain"]), _d(p["shift"]), 0, None)
        assert y.dtype == dto and R.worst(y, ref, e, dto) <= 1, (ti, to)
        # after the block: gate, residual
        res = _rand(B, N, C, seed=30 + i, dtype=dto)
        h = V.norm_gate_add(x, res, p["gain"], p["weight"], p["bias"], kind, EPS, 0.75)
        ref, e = _forward(x, kind, _d(p["weight"]), _d(p["bias"]), _d(p["gain"]), None, 0.75, res.double())
        assert h.dtype == dto and R.worst(h, ref, e, dto) <= 1, (ti, to)
    # no parameter at all, statistics
    y, st = V.norm_modulate(x, kind=kind, eps=EPS, want_stats=True)
    ref, e = _forward(x, kind, None, None, None, None, 0, None)
    assert R.worst(y, ref, e, x.dtype) <= 1
    mean, rstd = (t[..., 0] for t in R.stats(x.double(), kind, EPS))
    assert ((st.mean.double() - mean).abs() <= (DEPTH + 2) * R.U32 * x.double().abs().mean(-1)).all()
    spread = x.double().abs().mean(-1) * rstd if kind == "layer" else 0.0
    assert ((st.rstd.double() / rstd - 1).abs() <= R.U32 * (DEPTH / 2 + 8) * (1 + 2 * spread)).all()


def test_forward_far_from_zero_mean(V):
    """Rows whose mean is 1000 deviations away: the variance comes from centred values, so only the
    mean's own rounding counts (E[x^2] - mean^2 would lose everything)."""
    x = _rand(1, 5, 4096, seed=1, shift=1000.0)
    y = V.norm_modulate(x, kind="layer", eps=0.0)
    ref, e = _forward(x, "layer", None, None, None, None, 0, None, eps=0.0)
    assert R.worst(y, ref, e, torch.float32) <= 1


def test_strided_rows_and_slices(V):
    B, N, C = 3, 20, 320
    big = _rand(B, N + 7, 2 * C, seed=2, dtype=torch.bfloat16)
    mod = _rand(B, 6 * C, seed=3, dtype=torch.float32)
    x, sc, sh, gate = big[:, 4:4 + N, C:], mod[:, :C], mod[:, C:2 * C], mod[:, 5 * C:]
    y = V.norm_modulate(x, sc, sh)
    assert torch.equal(y, V.norm_modulate(x.contiguous(), sc.contiguous(), sh.contiguous()))
    res = big[:, 4:4 + N, :C]
    keep = big.clone()
    h = V.norm_gate_add(x.contiguous(), res, gate)
    V.norm_gate_add(x.contiguous(), res, gate, out=res)                       # the stream, in place
    assert torch.equal(res, h)
    keep[:, 4:4 + N, :C] = h
    assert torch.equal(big, keep)                                             # nothing beside it
    odd = _rand(B, N, C + 1, seed=4, dtype=torch.bfloat16)[..., 1:]           # unaligned rows
    assert torch.equal(V.norm_modulate(odd, sc, sh), V.norm_modulate(odd.contiguous(), sc, sh))
    flat = x[0].contiguous()
    assert torch.equal(V.norm_modulate(flat, sc[0], sh[0]), y[0])             # [N, C] with [C] vectors


@pytest.mark.parametrize("C", [64, 1016, 1023, 2048])
def test_two_slices_of_one_buffer(V, C):
    """Block output and stream side by side in the rows of one buffer, the result in the stream's place
    and in a third slice: nothing else changes."""
    B, N = 2, 37
    big = _rand(B, N, 3 * C, seed=60, dtype=torch.bfloat16)
    gate, dy = _rand(B, C, seed=61), _rand(B, N, C, seed=62, dtype=torch.bfloat16)
    keep = big.clone()
    res, o, other = big[..., :C], big[..., C:2 * C], big[..., 2 * C:]
    want, st = V.norm_gate_add(o.contiguous(), res.contiguous(), gate, want_stats=True)
    assert torch.equal(V.norm_gate_add(o, res, gate, out=other), want)
    assert torch.equal(big[..., :2 * C], keep[..., :2 * C])
    V.norm_gate_add(o, res, gate, out=res)
    assert torch.equal(res, want) and torch.equal(o, keep[..., C:2 * C]) and torch.equal(other, want)
    ref = V.norm_gate_add_bwd(dy, o.contiguous(), st, gate)
    got = V.norm_gate_add_bwd(dy, o, st, gate, out=other)
    assert torch.equal(got.dx, ref.dx) and torch.equal(big[..., :C], want) and torch.equal(o, keep[..., C:2 * C])


def test_in_place_and_empty(V):
    x = _rand(2, 30, 640, seed=5, dtype=torch.bfloat16)
    ref = V.norm_modulate(x)
    assert V.norm_modulate(x, out=x) is x and torch.equal(x, ref)
    e = torch.empty((2, 0, 64), device=DEV)
    assert V.norm_modulate(e).shape == (2, 0, 64)
    y, st = V.norm_modulate(e, want_stats=True)
    sc = torch.zeros((2, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    g = V.norm_modulate_bwd(e, e, st, sc, weight=w, bias=w)
    assert g.dx.shape == e.shape
    assert all((t == 0).all() for t in (g.dscale, g.dshift, g.dweight, g.dbias))


def test_constant_and_nonfinite_rows(V):
    x = _rand(1, 6, 512, seed=6)
    x[0, 1] = 3.0                                        # variance 0: xh = 0
    x[0, 2, 7] = float("nan")
    x[0, 3, 7] = float("inf")
    b = _rand(512, seed=7)
    w = torch.ones(512, device=DEV)
    y = V.norm_modulate(x, weight=w, bias=b)
    assert torch.equal(y[0, 1], b) and torch.isnan(y[0, 2]).all() and not torch.isfinite(y[0, 3]).any()
    clean = x.clone()
    clean[0, 2:4] = 0
    yc = V.norm_modulate(clean, weight=w, bias=b)
    assert torch.equal(y[0, [0, 1, 4, 5]], yc[0, [0, 1, 4, 5]])               # other rows untouched


def _backward(dy, x, mean, rstd, kind, w, b, G):
    dy, xd = dy.double(), x.double()
    C = x.shape[-1]
    xh = (xd - mean) * rstd
    one = torch.ones(C, device=DEV, dtype=torch.float64)
    G = G if G is not None else one.expand(x.shape[0], C)
    g = dy * G[:, None] * (w if w is not None else one)
    if kind == "none":
        dx, e = g, 4 * g.abs()
    else:
        c1 = g.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(g[..., :1])
        c2 = (g * xh).mean(-1, keepdim=True)
        dx = (g - c1 - xh * c2) * rstd
        e = rstd * (8 * g.abs() + (DEPTH + 6) * (g.abs().mean(-1, keepdim=True)
                                                  + xh.abs() * (g * xh).abs().mean(-1, keepdim=True)))
    a = xh * (w if w is not None else one) + (b if b is not None else 0)
    mag = (xh * (w if w is not None else one)).abs() + (b.abs() if b is not None else 0)
    n = x.shape[1]
    sums = {"gain": ((dy * a).sum(1), (n + 40) * R.U32 * (dy.abs() * mag).sum(1)),
            "shift": (dy.sum(1), (n + 40) * R.U32 * dy.abs().sum(1)),
            "weight": ((dy * G[:, None] * xh).sum((0, 1)), (n + 60) * R.U32 * (dy * G[:, None] * xh).abs().sum((0, 1))),
            "bias": ((dy * G[:, None]).sum((0, 1)), (n + 60) * R.U32 * (dy * G[:, None]).abs().sum((0, 1)))}
    return dx, R.U32 * e, sums


@pytest.mark.parametrize("kind", ["layer", "rms", "none"])
@pytest.mark.parametrize("B,N,C", SIZES + LONG)
def test_backward(V, kind, B, N, C):
    for i, (ti, to) in enumerate(PAIRS):
        dti, dto = TYPES[ti], TYPES[to]
        x = _rand(B, N, C, seed=i, dtype=dti, shift=0.5)
        dy = _rand(B, N, C, seed=70 + i, dtype=dto)
        dres = _rand(B, N, C, seed=80 + i, dtype=dti)
        p = _params(B, C, [torch.float32, torch.bfloat16, torch.float16][i % 3])
        _, st = V.norm_modulate(x, p["gain"], p["shift"], p["weight"], p["bias"], kind, EPS, dto, want_stats=True)
        m, r = st.mean.double()[..., None], st.rstd.double()[..., None]
        w, b = _d(p["weight"]), _d(p["bias"])
        g = V.norm_modulate_bwd(dy, x, st, p["gain"], p["weight"], p["bias"], kind, residual_grad=dres,
                                residual_scale=0.625)
        dx, e, sums = _backward(dy, x, m, r, kind, w, b, 1 + _d(p["gain"]))
        dx, e = dx + 0.625 * dres.double(), e + 2 * R.U32 * (dx.abs() + dres.double().abs())
        assert g.dx.dtype == dti and R.worst(g.dx, dx, e, dti) <= 1, (ti, to)
        for name, got in (("gain", g.dscale), ("shift", g.dshift), ("weight", g.dweight), ("bias", g.dbias)):
            assert R.worst(got, *sums[name], torch.float32) <= 1, (name, ti, to)
        g = V.norm_gate_add_bwd(dy, x, st, p["gain"], p["weight"], p["bias"], kind)
        dx, e, sums = _backward(dy, x, m, r, kind, w, b, _d(p["gain"]))
        assert R.worst(g.dx, dx, e, dti) <= 1, (ti, to)
        for name, got in (("gain", g.dgate), ("weight", g.dweight), ("bias", g.dbias)):
            assert R.worst(got, *sums[name], torch.float32) <= 1, (name, ti, to)
        assert g.dshift is None and g.dscale is None
    # without parameters
    g = V.norm_modulate_bwd(dy, x, st, kind=kind, want_dshift=False)
    dx, e, _ = _backward(dy, x, m, r, kind, None, None, None)
    assert R.worst(g.dx, dx, e, dti) <= 1
    assert g.dscale is g.dshift is g.dweight is g.dbias is None


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_backward_against_differences(V, kind):
    """Directional difference quotients of the 64-bit forward (central, step h): error h^2 times
    third derivatives of order one, far above the kernels' rounding."""
    B, N, C = 2, 7, 48
    x, dy, dirn = _rand(B, N, C, seed=1), _rand(B, N, C, seed=2), _rand(B, N, C, seed=3)
    p = _params(B, C, torch.float32)
    f = lambda xx, gg, ww, bb: (_forward(xx, kind, ww, bb, 1 + gg, _d(p["shift"]), 0, None)[0] * dy.double()).sum()
    _, st = V.norm_modulate(x, p["gain"], p["shift"], p["weight"], p["bias"], kind, EPS, want_stats=True)
    g = V.norm_modulate_bwd(dy, x, st, p["gain"], p["weight"], p["bias"], kind)
    args = [x.double(), _d(p["gain"]), _d(p["weight"]), _d(p["bias"])]
    h = 1e-4
    for i, grad in enumerate((g.dx, g.dscale, g.dweight, g.dbias)):
        d = torch.randn(args[i].shape, device=DEV, dtype=torch.float64)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * d, args[i] - h * d
        num = (f(*up) - f(*dn)) / (2 * h)
        ana = (grad.double() * d).sum()
        assert abs(num - ana) <= 1e-5 * (grad.double() * d).abs().sum() + 1e-5, i


def test_backward_in_place_repeatable_and_strided(V):
    B, N, C = 2, 700, 1280
    x, dy = _rand(B, N, C, seed=1, dtype=torch.bfloat16), _rand(B, N, C, seed=2, dtype=torch.bfloat16)
    sc = _rand(B, C, seed=3)
    w = _rand(C, seed=4)
    _, st = V.norm_modulate(x, sc, weight=w, want_stats=True)
    a = V.norm_modulate_bwd(dy, x, st, sc, weight=w)
    b = V.norm_modulate_bwd(dy, x, st, sc, weight=w)
    for n in ("dx", "dscale", "dshift", "dweight"):
        assert torch.equal(getattr(a, n), getattr(b, n))                       # bit for bit
    big = _rand(B, N, 2 * C, seed=5, dtype=torch.bfloat16)
    big[..., :C], big[..., C:] = x, dy
    c = V.norm_modulate_bwd(big[..., C:], big[..., :C], st, sc, weight=w)
    assert torch.equal(c.dx, a.dx) and torch.equal(c.dweight, a.dweight)
    d = dy.clone()
    e = V.norm_modulate_bwd(d, x, st, sc, weight=w, out=d)
    assert e.dx is d and torch.equal(d, a.dx) and torch.equal(e.dscale, a.dscale)


def test_stream_and_graph(V):
    B, N, C = 2, 90, 2048
    x, res, dy = (_rand(B, N, C, seed=i, dtype=torch.bfloat16) for i in range(3))
    sc = _rand(B, C, seed=3)
    run = lambda **k: (V.norm_gate_add(x, res, sc, want_stats=True, **k), )
    (ref, st), = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    (h, st2), = run(stream=s)
    g2 = V.norm_gate_add_bwd(dy, x, st2, sc, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g1 = V.norm_gate_add_bwd(dy, x, st, sc)
    assert torch.equal(h, ref) and torch.equal(g1.dx, g2.dx) and torch.equal(g1.dgate, g2.dgate)
    # two captured graphs that are replayed one beside the other keep their own workspaces
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    xs = [x.clone(), (x * 0.5).contiguous()]
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            hh, ss = V.norm_gate_add(xs[i], res, sc, want_stats=True)
            outs.append((hh, V.norm_gate_add_bwd(dy, xs[i], ss, sc)))
        graphs.append(g)
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        hh, ss = V.norm_gate_add(xs[i], res, sc, want_stats=True)
        gg = V.norm_gate_add_bwd(dy, xs[i], ss, sc)
        assert torch.equal(outs[i][0], hh) and torch.equal(outs[i][1].dx, gg.dx)
        assert torch.equal(outs[i][1].dgate, gg.dgate)


def test_many_sequences(V):
    """More sequences than slices of work, one token each (conditioning tokens)."""
    B, C = 1500, 160
    x, dy = _rand(B, 1, C, seed=1), _rand(B, 1, C, seed=2)
    sc = _rand(B, C, seed=3)
    w = _rand(C, seed=4)
    y, st = V.norm_modulate(x, sc, weight=w, want_stats=True)
    ref, e = _forward(x, "layer", _d(w), None, 1 + _d(sc), None, 0, None)
    assert R.worst(y, ref, e, torch.float32) <= 1
    g = V.norm_modulate_bwd(dy, x, st, sc, weight=w)
    dx, e, sums = _backward(dy, x, st.mean.double()[..., None], st.rstd.double()[..., None], "layer", _d(w), None,
                            1 + _d(sc))
    assert R.worst(g.dx, dx, e, torch.float32) <= 1
    assert R.worst(g.dscale, *sums["gain"], torch.float32) <= 1
    # dweight: B sequences are added up one after the other
    ref, b = sums["weight"]
    assert R.worst(g.dweight, ref, b * (B + 60) / 61, torch.float32) <= 1


@pytest.mark.parametrize("B,N,C", [(3, 200, 5120), (5, 190, 5120), (7, 400, 1024), (40, 33, 1016), (150, 130, 640),
                                   (200, 17, 2048), (297, 5, 1023)])
def test_sequence_counts_that_do_not_divide_the_places(V, B, N, C):
    """Sequences cut into slices whose counts are rounded down or up: rows as in calls of one sequence
    (bit for bit: a row's result does not depend on its slice), parameter gradients against 64 bits."""
    x, dy = _rand(B, N, C, seed=90, dtype=torch.bfloat16), _rand(B, N, C, seed=91, dtype=torch.bfloat16)
    sc, w, res = _rand(B, C, seed=92), _rand(C, seed=93), _rand(B, N, C, seed=94)
    y, st = V.norm_modulate(x, sc, sc, w, want_stats=True)
    h = V.norm_gate_add(x, res, sc, w)
    g = V.norm_modulate_bwd(dy, x, st, sc, w)
    for b in (0, B // 2, B - 1):
        one = slice(b, b + 1)
        yb, sb = V.norm_modulate(x[one], sc[one], sc[one], w, want_stats=True)
        assert torch.equal(y[one], yb) and torch.equal(st.rstd[one], sb.rstd)
        assert torch.equal(h[one], V.norm_gate_add(x[one], res[one], sc[one], w))
        assert torch.equal(g.dx[one], V.norm_modulate_bwd(dy[one], x[one], sb, sc[one], w).dx)
    _, _, sums = _backward(dy, x, st.mean.double()[..., None], st.rstd.double()[..., None], "layer", _d(w), None, 1 + _d(sc))
    assert R.worst(g.dscale, *sums["gain"], torch.float32) <= 1
    assert R.worst(g.dshift, *sums["shift"], torch.float32) <= 1
    ref, b = sums["weight"]
    assert R.worst(g.dweight, ref, b * (N + 60 + B) / (N + 60), torch.float32) <= 1      # the sequences' sums are added up


def test_refuses_types_and_shapes(V):
    x, res = _rand(2, 3, 64, dtype=torch.bfloat16), _rand(2, 3, 64)
    with pytest.raises(TypeError, match="float64"):
        V.norm_modulate(x, out_dtype=torch.float64)
    with pytest.raises(TypeError, match="float64"):
        V.norm_gate_add(x, res.double())
    with pytest.raises(V.VedaError, match="types"):
        V.norm_modulate(x, out_dtype=torch.float16)
    with pytest.raises(V.VedaError, match="8192"):
        V.norm_modulate(_rand(1, 2, 8193))
    with pytest.raises(ValueError, match="scale: expected shape"):
        V.norm_modulate(x, _rand(3, 64))
    with pytest.raises(TypeError, match="one type"):
        V.norm_modulate(x, _rand(2, 64), _rand(2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="stats"):
        V.norm_modulate_bwd(x, x, None)
    with pytest.raises(ValueError, match="overlaps"):
        big = _rand(2, 4, 64, dtype=torch.bfloat16)
        V.norm_modulate(big[:, 1:], out=big[:, :3])
    with pytest.raises(ValueError, match="overlap in memory"):
        V.norm_modulate(x, out=_rand(1, 3, 64, dtype=torch.bfloat16).expand(2, 3, 64))
    with pytest.raises(ValueError, match="residual: expected shape"):
        V.norm_gate_add(x, res[:1])
    with pytest.raises(ValueError, match="kind"):
        V.norm_modulate(x, kind="batch")
