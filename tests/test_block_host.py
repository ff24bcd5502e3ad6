"""Block operators without a GPU: argument checks at the C ABI (before any CUDA call) and in the
binding, and the host-side rotary frequencies and positions."""
import ctypes
import math

import numpy as np
import pytest
import torch

veda = pytest.importorskip("block_sparse_attention_max_b200.veda")
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from block_sparse_attention_max_b200 import build
    build.build()
    return veda.lib()


def _i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


def test_rotary_table_refusals(L):
    inv, ax = (ctypes.c_double * 4)(1, .1, .01, .001), (ctypes.c_int32 * 4)(0, 0, 1, 1)
    call = lambda pos=16, axes=2, rows=8, i=inv, a=ax, pairs=4, amp=1.0, out=16: L.veda_rotary_table(
        pos, axes, rows, ctypes.addressof(i) if i is not None else None, ctypes.addressof(a) if a is not None else None,
        pairs, amp, out, None)
    for bad in (dict(axes=0), dict(axes=9), dict(axes=1), dict(rows=-1), dict(pairs=0), dict(pairs=257), dict(i=None),
                dict(a=None), dict(amp=math.inf), dict(pos=None), dict(out=None), dict(out=8), dict(pos=2),
                dict(i=(ctypes.c_double * 4)(1, math.nan, 0, 0)), dict(a=(ctypes.c_int32 * 4)(0, 0, 0, -1))):
        assert call(**bad) == INVALID, bad
        assert L.veda_last_error()
    assert call(rows=0) == OK and call(rows=0, pos=None, out=None) == OK


def test_rotary_refusals(L):
    st = _i64(4096, 512, 128)

    def call(x=256, y=512, dtype=0, cs=16, trows=8, rows=None, rot=128, B=1, N=8, H=4, D=128, xs=st, ys=st):
        return L.veda_rotary(x, ctypes.addressof(xs) if xs is not None else None, y,
                             ctypes.addressof(ys) if ys is not None else None, dtype, cs, trows, rows, rot, 1, 0, B,
                             N, H, D, None)
    for bad in (dict(x=None), dict(y=None), dict(cs=None), dict(cs=8), dict(dtype=3), dict(dtype=-1), dict(trows=7),
                dict(trows=9), dict(B=-1), dict(N=-1), dict(H=-1), dict(D=0), dict(xs=None), dict(ys=None),
                dict(x=255), dict(rows=6), dict(rows=16, trows=0), dict(dtype=2, x=258)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(rot=0), dict(rot=130), dict(rot=63), dict(D=1032), dict(D=640, rot=514)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(N=0, trows=0, x=None, y=None) == OK and call(H=0) == OK


def test_rotary_tile_refusals(L):
    def pool(x=256, xt=512, cs=16, trows=256, rot=128, m=16, v=16, p=16, B=1, N=256, H=1, D=128, Npad=256):
        return L.veda_rotary_permute_pool(x, xt, cs, trows, rot, 1, m, v, p, B, N, H, D, Npad, None)

    def back(x=256, xt=512, cs=16, trows=256, rot=128, m=16, B=1, N=256, H=1, D=128, Npad=256):
        return L.veda_rotary_unpermute(xt, x, cs, trows, rot, 1, 1, m, B, N, H, D, Npad, None)
    for f in (pool, back):
        for bad in (dict(x=None), dict(xt=None), dict(m=None), dict(cs=None), dict(cs=4), dict(x=8), dict(xt=8),
                    dict(trows=255), dict(trows=512), dict(B=0), dict(N=0), dict(H=0), dict(Npad=100), dict(m=2)):
            assert f(**bad) == INVALID, bad
        for bad in (dict(D=64), dict(rot=8), dict(rot=144), dict(rot=24)):
            assert f(**bad) == UNSUPPORTED, bad
    assert pool(v=None) == INVALID and pool(p=None) == INVALID and pool(p=8) == INVALID


def _rows(data=256, b=640, r=64, dtype=0):
    return veda._ROWS.pack(data or 0, b, r, dtype)


def _params(weight=0, bias=0, gain=0, shift=0, weight_dtype=2, mod_dtype=2):
    return veda._NORM_PARAMS.pack(weight, bias, gain, shift, 0, 0, weight_dtype, mod_dtype, 1.0)


def test_norm_refusals(L):
    def fwd(x=None, res=None, y=None, p=None, mean=None, rstd=None, B=1, N=10, C=64, kind=0, eps=1e-6):
        return L.veda_norm_fwd(x or _rows(), res, y or _rows(512), p or _params(), 1.0, mean, rstd, B, N, C, kind, eps,
                               None)
    for bad in (dict(B=-1), dict(N=-1), dict(N=2**31 - 1), dict(C=0), dict(kind=3), dict(kind=-1), dict(eps=-1.0),
                dict(eps=math.nan), dict(x=_rows(dtype=5)), dict(x=_rows(None)), dict(x=_rows(257)), dict(y=_rows(None)),
                dict(mean=16), dict(rstd=2), dict(res=_rows(256, dtype=2)), dict(res=_rows(None)),
                dict(p=_params(weight=16, weight_dtype=7)), dict(p=_params(gain=18))):
        assert fwd(**bad) == INVALID, bad
    assert fwd(C=8193) == UNSUPPORTED
    assert fwd(x=_rows(dtype=1)) == UNSUPPORTED and fwd(y=_rows(dtype=1)) == UNSUPPORTED   # fp16 with another type
    assert fwd(B=0) == OK and fwd(N=0, x=_rows(None), y=_rows(None)) == OK
    assert L.veda_norm_fwd(None, None, _rows(), _params(), 1.0, None, None, 1, 1, 8, 0, 1e-6, None) == INVALID

    need = L.veda_norm_bwd_workspace_bytes(1, 10, 64)
    assert need > 0 and L.veda_norm_bwd_workspace_bytes(0, 1, 1) == 0 == L.veda_norm_bwd_workspace_bytes(1, 1, 8193)

    def bwd(dy=None, x=None, mean=16, rstd=16, res=None, dx=None, dg=None, ws=16, nws=need, B=1, N=10, C=64, kind=0):
        return L.veda_norm_bwd(dy or _rows(), x or _rows(), mean, rstd, res, dx or _rows(512), _params(), 1.0, dg,
                               None, None, None, ws, nws, B, N, C, kind, None)
    for bad in (dict(mean=None), dict(rstd=None), dict(kind=1, rstd=None), dict(ws=None), dict(ws=8),
                dict(nws=need - 1), dict(dx=_rows(dtype=2)), dict(res=_rows(dtype=2)), dict(dg=2), dict(dy=_rows(None)),
                dict(x=_rows(None)), dict(C=0), dict(kind=7)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(B=70000, nws=2**60) == UNSUPPORTED


def test_norm_workspace_covers_every_slice_count(L):
    """B sequences are cut into ceil(160 SMs * 4 / B) slices at most, none of them empty."""
    for B in (1, 2, 3, 7, 64, 639, 640, 641, 1500, 65535):
        for N in (1, 2, 5, 1000, 100000):
            slices = max(1, min(-(-640 // B), N))
            assert L.veda_norm_bwd_workspace_bytes(B, N, 100) >= (B * slices + B) * 2 * 100 * 4


def test_int8_refusals(L):
    q = lambda x=256, st=64, dt=0, c=16, s=16, rows=4, K=64: L.veda_quantize_int8(x, st, dt, c, s, rows, K, None)
    for bad in (dict(x=None), dict(c=None), dict(s=None), dict(c=8), dict(s=2), dict(x=255), dict(dt=3), dict(rows=-1),
                dict(rows=2**31), dict(K=0), dict(K=2**30 + 1)):
        assert q(**bad) == INVALID, bad
    assert q(rows=0, x=None) == OK

    def mm(a=16, sa=16, w=16, sw=16, bias=None, y=16, ys=32, dt=0, M=4, N=32, K=64):
        return L.veda_int8_matmul(a, sa, w, sw, bias, y, ys, dt, M, N, K, None)
    for bad in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(a=8), dict(w=8),
                dict(sa=2), dict(sw=1), dict(bias=2), dict(y=17), dict(dt=4), dict(M=-1), dict(N=-1), dict(K=0),
                dict(ys=31), dict(ys=-1)):
        assert mm(**bad) == INVALID, bad
    assert mm(K=131072) == mm(M=2**30 + 1) == mm(N=2**30 + 1, ys=2**31) == UNSUPPORTED
    assert mm(M=0) == OK and mm(N=0) == OK

    need = L.veda_int8_linear_workspace_bytes(9, 60)
    assert need >= 9 * 64 + 9 * 4 and L.veda_int8_linear_workspace_bytes(0, 60) == 0
    assert L.veda_int8_linear_workspace_bytes(4, 4096) == 0 < L.veda_int8_linear_workspace_bytes(4, 4097)

    def lin(x=256, st=64, xdt=0, w=16, sw=16, bias=None, y=16, ys=32, dt=0, ws=16, nws=need, M=9, N=32, K=60):
        return L.veda_int8_linear(x, st, xdt, w, sw, bias, y, ys, dt, ws, nws, M, N, K, None)
    for bad in (dict(x=None), dict(w=None), dict(sw=None), dict(y=None), dict(x=255), dict(w=8), dict(xdt=3),
                dict(dt=-1), dict(M=-1), dict(K=0), dict(ys=31), dict(bias=2)):   # with a workspace, and without
        assert lin(**bad) == INVALID and lin(**{**dict(M=4, ws=None, nws=0), **bad}) == INVALID, bad
    for bad in (dict(ws=None), dict(ws=8), dict(nws=need - 1)):
        assert lin(**bad) == INVALID, bad
    assert lin(K=131072, nws=2**40) == UNSUPPORTED
    assert lin(M=0, x=None, ws=None, nws=0) == OK and lin(N=0) == OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
def test_no_device_means_error(L):
    st = _i64(4096, 512, 128)
    assert L.veda_rotary(256, ctypes.addressof(st), 512, ctypes.addressof(st), 0, 16, 8, None, 128, 1, 0, 1, 8, 4, 128,
                         None) in (2, 3)
    assert L.veda_int8_matmul(16, 16, 16, 16, None, 16, 32, 0, 4, 32, 64, None) in (2, 3)
    assert L.veda_norm_fwd(_rows(), None, _rows(512), _params(), 1.0, None, None, 1, 10, 64, 0, 1e-6, None) in (2, 3)


def test_binding_checks():
    f = torch.float32
    x = torch.zeros(1, 4, 2, 64)
    for call in (lambda: veda.rotary(x, veda.RotaryTable(torch.zeros(4, 32, 2), True)),
                 lambda: veda.norm_modulate(x[0, 0]), lambda: veda.quantize_int8(x),
                 lambda: veda.rotary_table(torch.zeros(3, dtype=torch.int32), np.ones(2))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        veda._need_strided(torch.zeros(2, 2, dtype=torch.float64), "x", 2)
    with pytest.raises(ValueError, match="dimensions"):
        veda._need_strided(torch.zeros(2, 2), "x", 3)
    with pytest.raises(ValueError, match="contiguous"):
        veda._need_strided(torch.zeros(4, 4).t(), "x", 2)
    with pytest.raises(ValueError, match="rows of one stride"):
        veda._matrix(torch.zeros(4, 6, 8)[:, :3], "x")
    assert veda._matrix(torch.zeros(4, 6, 16)[..., :8], "x").stride(0) == 16
    a = torch.zeros(64)
    with pytest.raises(ValueError, match="overlaps"):
        veda._separate(a[1:33], a[:32], "x", True)
    veda._separate(a[:32], a[32:], "x", True)
    veda._separate(a[:32], a[:32], "x", True)
    with pytest.raises(ValueError, match="must not be"):
        veda._separate(a[:32], a[:32], "x", False)
    with pytest.raises(ValueError, match="kind"):
        veda._norm_kind("group")
    with pytest.raises(TypeError):
        veda.Int8Rows.from_codes(torch.zeros(2, 3), torch.ones(2))
    with pytest.raises(ValueError, match="scale"):
        veda.Int8Rows.from_codes(torch.zeros(2, 3, dtype=torch.int8), torch.ones(3))
    r = veda.Int8Rows.from_codes(torch.ones(2, 3, dtype=torch.int8), torch.ones(2, dtype=f))
    assert r.codes.shape == (2, 16) and r.codes.sum() == 6 and r.K == 3


def test_frequencies():
    f = veda.rotary_frequencies(128)
    assert np.allclose(f.inv_freq, 10000.0 ** (-np.arange(64) / 64), rtol=1e-14) and (f.axis == 0).all()
    f3 = veda.rotary_frequencies((44, 42, 42), theta=256.0)
    assert len(f3.inv_freq) == 64 and list(np.bincount(f3.axis)) == [22, 21, 21]
    assert f3.inv_freq[0] == f3.inv_freq[22] == f3.inv_freq[43] == 1.0 and f3.amplitude == 1.0
    assert np.allclose(veda.rotary_frequencies(64, scaling="linear", factor=4).inv_freq,
                       veda.rotary_frequencies(64).inv_freq / 4, rtol=1e-15)
    base, ntk = veda.rotary_frequencies(64), veda.rotary_frequencies(64, scaling="ntk", factor=8)
    assert ntk.inv_freq[0] == 1.0 and np.isclose(ntk.inv_freq[-1], base.inv_freq[-1] / 8, rtol=1e-12)
    y = veda.rotary_frequencies(128, scaling="yarn", factor=4, original_length=4096)
    base = veda.rotary_frequencies(128).inv_freq
    turns = 4096 * base / (2 * np.pi)
    ratio = y.inv_freq / base
    assert (ratio[turns > 40] == 1).all() and np.allclose(ratio[turns < 0.8], 0.25)
    assert (np.diff(ratio) <= 1e-15).all() and np.isclose(y.amplitude, 0.1 * math.log(4) + 1)
    for scaling in ("linear", "ntk", "yarn"):                          # factor 1 changes nothing
        g = veda.rotary_frequencies(128, scaling=scaling, factor=1.0, original_length=4096)
        assert np.allclose(g.inv_freq, base, rtol=1e-14) and g.amplitude == 1.0
    for bad in (dict(dims=3), dict(dims=()), dict(dims=(0, 0)), dict(dims=(4, -2)), dict(dims=8, theta=1.0),
                dict(dims=8, scaling="x"), dict(dims=8, factor=0.5), dict(dims=2, scaling="ntk", factor=2),
                dict(dims=8, scaling="yarn", factor=2), dict(dims=8, scaling="yarn", original_length=8, beta_slow=40)):
        with pytest.raises(ValueError):
            veda.rotary_frequencies(**bad)


def test_positions():
    p = veda.rotary_positions((2, 3, 4), 2)
    assert p.shape == (3, 26) and p.dtype == np.int32
    for n, thw in ((0, (0, 0, 0)), (5, (0, 1, 1)), (12, (1, 0, 0)), (23, (1, 2, 3)), (24, (4, 4, 4)), (25, (5, 5, 5))):
        assert tuple(p[:, n]) == thw


def test_sizes_past_32_bits_are_refused():
    """Sizes that the library takes in 32 bits must not wrap: 2^32 + 5 rows would pass as 5."""
    many = 2 ** 32 + 5
    cs = veda.RotaryTable(torch.ones(1, 1, 2), True)
    wide = torch.zeros(1, 16).expand(many, 16)
    w = veda.Int8Rows(torch.zeros(1, 16, dtype=torch.int8), torch.ones(1), 16)
    for call in (lambda: veda.rotary(torch.zeros(1, 1, 1, 2).expand(1, many, 1, 2), cs),
                 lambda: veda.norm_modulate(wide),
                 lambda: veda.norm_gate_add(wide, wide),
                 lambda: veda.norm_modulate_bwd(wide, wide, None, kind="none"),
                 lambda: veda.norm_gate_add_bwd(wide, wide, None, kind="none"),
                 lambda: veda.int8_linear(wide, w),
                 lambda: veda.quantize_int8(wide), lambda: veda.quantize_int8(wide.t()),
                 lambda: veda.int8_matmul(veda.Int8Rows(torch.zeros(1, 16, dtype=torch.int8).expand(many, 16),
                                                        torch.ones(1).expand(many), 16), w)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.parametrize("d,theta,length", [(128, 1e4, 4096), (128, 1e4, 1 << 20), (64, 1e4, 131072), (44, 256.0, 8192),
                                            (128, 1e4, 54000), (128, 1e4, 1 << 17), (8, 1e4, 100), (128, 1e4, 64)])
@pytest.mark.parametrize("fast,slow,factor", [(32.0, 1.0, 4.0), (8.0, 2.0, 16.0)])
def test_yarn_ramp(d, theta, length, fast, slow, factor):
    """Every pair against the ramp: linear in the pair index between the whole pairs around those that
    turn beta_fast and beta_slow times within the length, also where one of them lies outside the head
    (the slowest pair turns 1 to 32 times; the fastest fewer than 32)."""
    f = veda.rotary_frequencies(d, theta, "yarn", factor, length, fast, slow)
    base = veda.rotary_frequencies(d, theta).inv_freq
    # the pair index, a real number, whose frequency turns t times within the length
    index = lambda t: math.log(length / (2 * math.pi * t)) * d / (2 * math.log(theta))
    low, high = math.floor(index(fast)), math.ceil(index(slow))
    for i in range(d // 2):
        ramp = min(max((i - low) / (high - low), 0.0), 1.0)
        assert math.isclose(f.inv_freq[i], base[i] * (1 - ramp + ramp / factor), rel_tol=1e-12), i
        turns = length * base[i] / (2 * math.pi)
        if turns < slow and i >= high:
            assert math.isclose(f.inv_freq[i], base[i] / factor, rel_tol=1e-12)
        if i <= low:
            assert f.inv_freq[i] == base[i] and turns > fast * (1 - 1e-12)
        if turns > slow * (1 + 1e-12):                     # only slower pairs get the whole factor
            assert f.inv_freq[i] > base[i] / factor


class _FakeStream:
    made: list = []

    def __init__(self, device=None):
        self.after = []                                     # streams whose work so far comes before this one's
        _FakeStream.made.append(self)

    def wait_stream(self, s):
        self.after.append(s)


def test_host_pipeline_waits_for_the_stream_it_is_made_on(L, monkeypatch):
    """The table, the tile maps and the buffers come from the stream that is current when the pipeline is
    made: the pipeline's own streams must not read or write them before that stream's work has run."""
    monkeypatch.setattr(_FakeStream, "made", [])
    current = _FakeStream()
    monkeypatch.setattr(torch.cuda, "Stream", _FakeStream)
    monkeypatch.setattr(torch.cuda, "Event", lambda *a, **k: object())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: None)
    maps = veda.build_tile_map((2, 8, 16), [(1, 8, 16)]).to("cpu")
    table = veda.RotaryTable(torch.ones(256, 64, 2), True)
    pipe = veda.HostPipeline(1, 256, 1, maps, [(1, 10)], 0.1, "cpu", rotary=table)
    for s in (pipe.h2d, pipe.comp):
        assert s.after == [current]


def test_host_pipeline_keeps_its_memory_until_its_streams_are_done(L, monkeypatch):
    """A pipeline that is dropped before its last clips are done must not give its buffers, the maps or
    the table back to the current stream while its own streams still use them."""
    kept = []
    monkeypatch.setattr(_FakeStream, "made", [])
    monkeypatch.setattr(torch.cuda, "Stream", _FakeStream)
    monkeypatch.setattr(torch.cuda, "Event", lambda *a, **k: object())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((id(t), s)))
    maps = veda.build_tile_map((2, 8, 16), [(1, 8, 16)]).to("cpu")
    table = veda.RotaryTable(torch.ones(256, 64, 2), True)
    pipe = veda.HostPipeline(1, 256, 1, maps, [(1, 10)], 0.1, "cpu", rotary=table)
    b, ls = pipe.bufs, pipe.bufs.lists
    used = {pipe.comp: [b.q_t, b.k_t, b.v_t, b.pooled_q, b.pooled_k, b.scores, b.workspace, b.o_t, b.lse, ls.full_cnt,
                        ls.full_idx, ls.part_cnt, ls.part_idx, maps.tile_map, maps.tile_valid, maps.tile_segment,
                        maps.nT_per_head, table.cos_sin, *pipe.outputs, *(t for i in pipe.inputs for t in i.values())],
            pipe.h2d: [t for i in pipe.inputs for t in i.values()], pipe.d2h: pipe.outputs}
    for s, ts in used.items():
        assert {id(t) for t in ts} <= {i for i, st in kept if st is s}


def test_path_buffers_come_from_the_launching_stream(L, monkeypatch):
    """sparse_attention(stream=s) without buffers: memory and the lists' zeros on s, not on the current
    stream, and every buffer kept from reuse while the current stream still reads it."""
    import contextlib
    current, other, kept, active = _FakeStream(), _FakeStream(), [], []

    @contextlib.contextmanager
    def on(s):
        active.append(s)
        yield
        active.pop()
    made = []
    real = torch.empty, torch.zeros
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: active[-1] if active else current)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append((real[0](*a, **k), active[-1:])) or made[-1][0])
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: made.append((real[1](*a, **k), active[-1:])) or made[-1][0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((t, s)))
    monkeypatch.setattr(veda, "permute_pool", lambda *a, **k: (_ for _ in ()).throw(StopIteration))
    maps = veda.build_tile_map((2, 8, 16), [(1, 8, 16)]).to("cpu")
    q = real[1]((1, 256, 1, 128), dtype=torch.bfloat16)
    with pytest.raises((StopIteration, RuntimeError)):
        veda.sparse_attention(q, q, q, None, None, maps, [(1, 10)], 0.1, stream=other)
    assert len(made) == 14 and all(s == [other] for _, s in made)
    assert {id(t) for t, _ in made} == {id(t) for t, s in kept if s is current}


def _bytes_of(t):
    idx = np.zeros(tuple(t.shape), np.int64)
    for d, (n, st) in enumerate(zip(t.shape, t.stride())):
        idx += (np.arange(n) * st).reshape([-1 if i == d else 1 for i in range(t.dim())])
    first = (t.data_ptr() + idx.reshape(-1) * t.element_size())[:, None]
    return set((first + np.arange(t.element_size())).reshape(-1).tolist())


def _refused(out, t, same_ok=True):
    try:
        veda._separate(out, t, "x", same_ok)
        return False
    except ValueError:
        return True


def test_slices_of_one_buffer_do_not_overlap():
    big, even = torch.zeros(3, 5, 40), torch.zeros(3, 6, 40)
    a, b = big[..., :16], big[..., 16:32]
    for x, y in ((a, b), (b, a), (a, big[..., 24:]), (even[:, ::2], even[:, 1::2]), (big[:2], big[2:]),
                 (big[:, :2, :16], big[:, 3:, :16]), (big.view(3, 5, 4, 10)[:, :, :2], big.view(3, 5, 4, 10)[:, :, 2:]),
                 (a, big.view(torch.float16)[..., 32:64]), (a[0], b[0])):
        assert not _refused(x, y)
    for x, y in ((a, big[..., 15:31]), (big[..., 15:31], a), (big[:, :3], big[:, 2:]), (a, big), (a, big[..., 1:17]),
                 (big[..., ::2], big[..., 1:]), (a, big.view(torch.float16)[..., 31:63]), (a, big[1:2, 1:2, 3:4])):
        assert _refused(x, y)
    # one place for both is an in-place call, whatever the strides of dimensions of one element are
    assert not _refused(a, big[..., :16]) and _refused(a, big[..., :16], same_ok=False)
    one = big[1:2]
    assert not _refused(one, one.as_strided((1, 5, 40), (7, 40, 1)))


def test_overlap_check_against_the_bytes():
    """Random strided views of one buffer: two that share a byte are never let through."""
    rng = np.random.default_rng(3)
    base = torch.zeros(4096, dtype=torch.uint8)
    accepted = 0
    for _ in range(4000):
        views = []
        for _ in range(2):
            dt = [torch.uint8, torch.float16, torch.float32][rng.integers(3)]
            t = base.view(dt)
            shape = rng.integers(1, 5, 3).tolist()
            inner = int(rng.choice([1, 1, 2]))
            s1 = shape[2] * inner + int(rng.integers(0, 9))
            s0 = s1 * shape[1] + int(rng.integers(0, 9))
            views.append(t.as_strided(shape, (s0, s1, inner), int(rng.integers(0, 60))))
        same = views[0].data_ptr() == views[1].data_ptr() and views[0].dtype == views[1].dtype
        if not _refused(*views, same_ok=False):
            accepted += 1
            assert same is False and not (_bytes_of(views[0]) & _bytes_of(views[1]))
    assert accepted > 500


def test_written_buffers_must_not_share_memory(monkeypatch):
    """Every buffer that a call writes against everything that the call reads or writes besides."""
    monkeypatch.setattr(veda, "_here", lambda t: True)                   # the checks, on CPU tensors
    monkeypatch.setattr(veda, "lib", lambda: pytest.fail("the library was reached"))
    f, bf = torch.float32, torch.bfloat16
    pool = torch.zeros(1 << 20, dtype=torch.uint8)

    def at(byte, dtype, *shape):
        n = math.prod(shape) * dtype.itemsize
        return pool[byte:byte + n].view(dtype).view(shape)

    def refused(call, match):
        with pytest.raises(ValueError, match=match):
            call()
    far = 1 << 19
    inv = np.ones(8)
    pos = at(0, torch.int32, 1, 64)
    refused(lambda: veda.rotary_table(pos, inv, out=at(128, f, 64, 8, 2)), "positions")

    x = at(0, f, 1, 4, 2, 16)
    table = veda.RotaryTable(at(4096, f, 8, 8, 2), True)
    rows = at(8192, torch.int32, 1, 4)
    refused(lambda: veda.rotary(x, table, rows=rows, out=at(8192 - 64, f, 1, 4, 2, 16)), "rows")
    refused(lambda: veda.rotary(x, table, rows=rows, out=at(4096, f, 1, 4, 2, 16)), "table")

    maps = veda.DeviceMaps(at(65536, torch.int32, 1, 128), at(66560, torch.int32, 1, 1), at(67584, torch.int32, 1, 1),
                           at(68608, torch.int32, 1), 4, 1, 128)
    x = at(0, bf, 1, 4, 1, 128)
    t = veda.RotaryTable(at(4096, f, 4, 64, 2), True)
    tiles, pooled = at(far, bf, 1, 1, 128, 128), at(131072, f, 1, 1, 1, 3, 128)
    for given, match in ((dict(out=at(4096, bf, 1, 1, 128, 128)), "table"), (dict(out=at(65536, bf, 1, 1, 128, 128)), "map"),
                         (dict(out=at(512, bf, 1, 1, 128, 128)), "x"), (dict(pooled=at(512, f, 1, 1, 1, 3, 128)), "x"),
                         (dict(pooled=at(4096, f, 1, 1, 1, 3, 128)), "table"),
                         (dict(pooled=at(66560, f, 1, 1, 1, 3, 128)), "valid"),
                         (dict(pooled=at(far + 16, f, 1, 1, 1, 3, 128)), "out")):
        refused(lambda: veda.rotary_permute_pool(x, t, maps, **{**dict(out=tiles, pooled=pooled), **given}), match)
    for place, match in ((4096, "table"), (65536, "map"), (far, "x_t")):
        refused(lambda: veda.rotary_unpermute(tiles, t, maps, 4, out=at(place, bf, 1, 4, 1, 128)), match)

    x = at(0, bf, 2, 4, 64)
    w, b, g, sh = (at(4096 + 1024 * i, bf, 2, 64) for i in range(4))
    for i, n in enumerate(("weight", "bias", "scale", "shift")):
        refused(lambda: veda.norm_modulate(x, g, sh, w[0], b[0], out=at(4096 + 1024 * i - 512, bf, 2, 4, 64)), n)
    refused(lambda: veda.norm_gate_add(x, at(far, bf, 2, 4, 64), g, out=at(4096 + 2048 - 512, bf, 2, 4, 64)), "gate")
    st = veda.NormStats(at(16384, f, 2, 4), at(20480, f, 2, 4))
    dy = at(far, bf, 2, 4, 64)
    for place, n in ((4096, "weight"), (5120, "bias"), (6144, "scale"), (16384, "stats.mean"), (20480, "stats.rstd")):
        refused(lambda: veda.norm_modulate_bwd(dy, x, st, g, w[0], b[0], out=at(place, bf, 2, 4, 64)), n)

    x = at(0, bf, 4, 32)
    refused(lambda: veda.quantize_int8(x, out=veda.Int8Rows(at(far, torch.int8, 4, 32), at(64, f, 4), 32)), "x")
    refused(lambda: veda.quantize_int8(x, out=veda.Int8Rows(at(far, torch.int8, 4, 32), at(far + 16, f, 4), 32)), "codes")


def test_token_count_of_the_tile_map(L, monkeypatch):
    """Tokens that the tile map does not have would come back as whatever their memory held."""
    monkeypatch.setattr(veda, "_here", lambda t: True)
    maps = veda.build_tile_map((2, 8, 16), [(1, 8, 16)]).to("cpu")
    monkeypatch.setattr(veda, "lib", lambda: pytest.fail("the library was reached"))
    table = lambda n: veda.RotaryTable(torch.ones(n, 64, 2), True)
    tiles = torch.zeros(1, 1, 256, 128, dtype=torch.bfloat16)
    for n in (255, 257):
        with pytest.raises(ValueError, match="tile map has 256 tokens"):
            veda.rotary_unpermute(tiles, table(n), maps, n)
        rows = veda.Int8Rows(torch.zeros(128, 64, dtype=torch.int8), torch.ones(128), 64)
        w = veda.BlockWeights(rows, rows, rows, rows, torch.zeros(1, 128, 384), torch.zeros(1, 128, 384))
        with pytest.raises(ValueError, match="tile map has 256 tokens"):
            veda.attention_block(torch.zeros(1, n, 64), w, None, None, None, table(n), maps, [(1, 10)], 0.1)


def test_axis_is_taken_as_it_is(monkeypatch):
    """An axis of another type or past 32 bits must not arrive as another axis."""
    monkeypatch.setattr(veda, "_here", lambda t: True)
    monkeypatch.setattr(veda, "lib", lambda: pytest.fail("the library was reached"))
    pos, inv = torch.zeros(2, 4, dtype=torch.int32), np.ones(3)
    for bad in (np.array([0, 2 ** 32, 1]), np.array([0, -2 ** 32, 1]), np.array([0, 2, 1]), np.array([0, -1, 1])):
        with pytest.raises(ValueError, match="axis"):
            veda.rotary_table(pos, inv, bad)
    for bad in (np.array([0.0, 0.7, 1.0]), np.array([False, True, False])):
        with pytest.raises(TypeError, match="axis"):
            veda.rotary_table(pos, inv, bad)


def test_the_status_word_has_one_translation_unit():
    """Kernels of a second unit that included the device helpers would flag a word that nothing reads."""
    import os
    import re
    from block_sparse_attention_max_b200 import build

    def reaches(name, seen):
        if name in seen or not os.path.exists(os.path.join(build.CSRC, name)):
            return set()
        seen.add(name)
        text = open(os.path.join(build.CSRC, name)).read()
        below = re.findall(r'#include "([^"]+)"', text)
        return {name}.union(*(reaches(n, seen) for n in below))
    users = [n for n in build.SOURCES if "veda_ptx.cuh" in reaches(n, set())]
    assert users == ["veda_lib.cu"]
    assert "#error" in open(os.path.join(build.CSRC, "veda_ptx.cuh")).read().split("g_status")[0]
