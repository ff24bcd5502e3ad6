"""Rotary positions on the GPU against 64-bit forms.

Bounds: the products and the sum of a turned channel are fp32 (three roundings of terms no larger
than (|x1| + |x2|)(|c| + |s|)), then one rounding to the output type; the table is one rounding of
an fp64 value."""
import numpy as np
import pytest
import torch

import block_ref as R
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def V():
    from block_sparse_attention_max_b200 import build
    build.build()
    from block_sparse_attention_max_b200 import veda
    yield veda
    veda.check_device_status()


def _rand(*shape, seed=0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def _table(V, rows, rot, interleaved, seed=1, amplitude=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    pos = torch.randint(-1000, 1_000_000, (1, rows), generator=g, device=DEV, dtype=torch.int32)
    f = V.rotary_frequencies(rot)
    return V.rotary_table(pos, f.inv_freq, f.axis, amplitude, interleaved)


@pytest.mark.parametrize("rows,dims,amp", [(1, (2,), 1.0), (1000, (128,), 1.25), (777, (44, 42, 42), 1.0),
                                           (33, (0, 2, 510), 0.5), (50220, (16, 24, 24), 1.0)])
def test_table(V, rows, dims, amp):
    rng = np.random.default_rng(rows)
    pos = rng.integers(-2**31, 2**31, (len(dims), rows), dtype=np.int64).astype(np.int32)
    if rows == 50220:
        pos = V.rotary_positions((31, 30, 54))
    f = V.rotary_frequencies(dims)
    t = V.rotary_table(torch.from_numpy(pos).to(DEV), f.inv_freq, f.axis, amp)
    ang = pos.astype(np.float64)[f.axis].T * f.inv_freq
    ref = amp * np.stack([np.cos(ang), np.sin(ang)], -1)
    err = np.abs(t.cos_sin.double().cpu().numpy() - ref)
    # one rounding to fp32 and, before it, two fp64 sines that may differ by a few fp64 steps
    assert (err <= R.U32 * np.abs(ref) + 1e-15 * amp).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,N,H,D,rot", [(1, 1, 1, 2, 2), (1, 1, 40, 128, 128), (2, 37, 8, 128, 64), (3, 5, 1, 96, 30),
                                         (2, 130, 3, 80, 80), (1, 300, 17, 256, 256), (1, 3, 2, 640, 512),
                                         (2, 9, 5, 33, 18), (1, 1025, 12, 64, 48), (1, 1300, 1, 256, 86),
                                         (1, 1300, 40, 64, 20), (2, 700, 33, 72, 24), (1, 2000, 17, 36, 14), (3, 50, 2, 128, 2)])
def test_rotary_matches_definition(V, dtype, layout, B, N, H, D, rot):
    dt, inter = TYPES[dtype], layout == "interleaved"
    x = _rand(B, N, H, D, seed=D + rot, dtype=dt)
    t = _table(V, N, rot, inter)
    for inverse in (False, True):
        y = V.rotary(x, t, inverse=inverse)
        ref, mag = R.rotate(x.double(), t.cos_sin.double()[None, :, None], rot, inter, inverse)
        assert R.worst(y, ref, 3 * R.U32 * mag, dt) <= 1.0
        if rot < D:
            assert torch.equal(y[..., rot:], x[..., rot:])
    assert torch.equal(V.rotary(x.clone(), t, out=None), V.rotary(x, t))
    z = x.clone()
    assert V.rotary(z, t, out=z) is z and torch.equal(z, V.rotary(x, t))       # in place


def test_strided_slices_and_offsets(V):
    B, N, H, D = 2, 77, 6, 64
    packed = _rand(B, N, 3 * H, D, seed=3, dtype=torch.bfloat16)
    t = _table(V, N, 64, False)
    keep = packed.clone()
    for i in range(3):
        x = packed[:, :, i * H:(i + 1) * H]
        assert torch.equal(V.rotary(x, t), V.rotary(x.contiguous(), t))
    q = packed[:, :, :H]
    V.rotary(q, t, out=q)                                                     # a slice in place
    assert torch.equal(q, V.rotary(keep[:, :, :H], t)) and torch.equal(packed[:, :, H:], keep[:, :, H:])
    head_major = _rand(B, H, N, D, seed=4, dtype=torch.bfloat16).transpose(1, 2)
    assert torch.equal(V.rotary(head_major, t), V.rotary(head_major.contiguous(), t))
    # rows that start on no 16-byte boundary, channels cut out of a wider head
    odd = _rand(B, N, H, D + 1, seed=5, dtype=torch.float16)[..., 1:]
    assert torch.equal(V.rotary(odd, t), V.rotary(odd.contiguous(), t))
    one = _rand(1, N, H, D, seed=6, dtype=torch.bfloat16).expand(3, N, H, D)   # broadcast batch
    assert torch.equal(V.rotary(one, t), V.rotary(one.contiguous(), t))


def test_table_rows_own_and_given(V):
    B, N, H, D = 4, 6, 3, 64
    x = _rand(B, N, H, D, seed=7, dtype=torch.bfloat16)
    t = _table(V, B * N, D, True)
    rows = torch.randperm(B * N, device=DEV).view(B, N).int()
    y_own = V.rotary(x, t)                                                     # row b N + n
    y_rows = V.rotary(x, t, rows=rows)
    for b in range(B):
        sub = lambda r: V.RotaryTable(t.cos_sin[r].contiguous(), True)
        assert torch.equal(y_own[b:b + 1], V.rotary(x[b:b + 1], sub(slice(b * N, (b + 1) * N))))
        assert torch.equal(y_rows[b:b + 1], V.rotary(x[b:b + 1], sub(rows[b].long())))


@pytest.mark.parametrize("rot", [64, 40])
def test_row_outside_the_table_is_flagged(V, rot):
    x = _rand(1, 3, 2, 64, seed=8, dtype=torch.bfloat16)
    t = _table(V, 5, rot, False)
    V.check_device_status()
    for bad in (-1, 5, 2**31 - 1, -2**31):
        y = V.rotary(x, t, rows=torch.tensor([[0, bad, 4]], dtype=torch.int32, device=DEV))
        with pytest.raises(V.VedaError):
            V.check_device_status()
        assert (y[:, 1] == 0).all()
        good = V.rotary(x, t, rows=torch.tensor([[0, 0, 4]], dtype=torch.int32, device=DEV))
        assert torch.equal(y[:, ::2], good[:, ::2])


def test_empty_and_nonfinite(V):
    t = _table(V, 0, 64, True)
    assert V.rotary(_rand(2, 0, 3, 64), t).shape == (2, 0, 3, 64)
    assert V.rotary(_rand(0, 4, 3, 64), _table(V, 4, 64, True)).shape == (0, 4, 3, 64)
    x = _rand(1, 4, 2, 64, seed=9)
    x[0, 1, 0, 5], x[0, 2, 1, 8] = float("nan"), float("inf")
    y = V.rotary(x, _table(V, 4, 64, True))
    ok = torch.ones_like(y, dtype=torch.bool)
    ok[0, 1, 0, 4:6] = ok[0, 2, 1, 8:10] = False                                # their pairs only
    assert torch.isfinite(y[ok]).all() and not torch.isfinite(y[~ok]).any()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_channels_behind_the_turned_ones_keep_their_bits(V, layout):
    """A vector may hold turned and other channels: NaN, infinities and signs of the others stay."""
    x = _rand(2, 40, 3, 64, seed=20, dtype=torch.bfloat16)
    x[..., 22:26] = torch.tensor([float("nan"), float("-inf"), -0.0, float("inf")], device=DEV)
    t = _table(V, 40, 22, layout == "interleaved")
    for y in (V.rotary(x, t), V.rotary(x.clone(), t, out=None)):
        assert torch.equal(y[..., 22:].view(torch.int16), x[..., 22:].view(torch.int16))
        assert torch.isfinite(y[..., :22]).all()


SPECIAL = [float("nan"), float("-inf"), -0.0, float("inf")]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,N,H,D,rot", [(2, 40, 3, 64, 22), (1, 600, 17, 64, 24), (1, 9, 2, 33, 18), (3, 5, 1, 96, 30),
                                         (1, 300, 40, 128, 96)])
def test_in_place_keeps_the_other_channels(V, dtype, layout, B, N, H, D, rot):
    """In place only the turned channels' vectors are written, and those may hold others: turned
    channels as out of place, the others bit for bit, whether table rows are given or not."""
    bits = torch.int32 if dtype == "fp32" else torch.int16
    x = _rand(B, N, H, D, seed=30, dtype=TYPES[dtype])
    x[..., rot:rot + 4] = torch.tensor(SPECIAL, device=DEV)[:min(4, D - rot)]
    t = _table(V, B * N, rot, layout == "interleaved")
    rows = torch.randperm(B * N, device=DEV).view(B, N).int()
    for inverse in (False, True):
        for r in (None, rows):
            want = V.rotary(x, t, rows=r, inverse=inverse)
            z = x.clone()
            assert V.rotary(z, t, rows=r, inverse=inverse, out=z) is z
            assert torch.equal(z.view(bits), want.view(bits))
            assert torch.equal(z[..., rot:].contiguous().view(bits), x[..., rot:].contiguous().view(bits))
            assert torch.isfinite(z[..., :rot]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("H,D,rot", [(3, 64, 22), (40, 128, 96), (2, 33, 18)])
def test_in_place_row_outside_the_table(V, layout, H, D, rot):
    """In place too, a token whose row is outside the table becomes zeros, all of its channels."""
    x = _rand(2, 7, H, D, seed=31, dtype=torch.bfloat16)
    t = _table(V, 9, rot, layout == "interleaved")
    rows = torch.arange(14, device=DEV, dtype=torch.int32).view(2, 7) % 9
    want = V.rotary(x, t, rows=rows)
    V.check_device_status()
    for b, n, bad in ((0, 3, 9), (1, 6, -1)):
        given, z = rows.clone(), x.clone()
        given[b, n] = bad
        V.rotary(z, t, rows=given, out=z)
        with pytest.raises(V.VedaError):
            V.check_device_status()
        assert (z[b, n] == 0).all()
        z[b, n] = want[b, n]
        assert torch.equal(z, want)


def test_gradient_is_the_transpose(V):
    """<R x, g> = <x, R^T g>, and the turn's difference quotient along a direction."""
    x, g = _rand(2, 11, 3, 96, seed=10), _rand(2, 11, 3, 96, seed=11)
    t = _table(V, 11, 64, False, amplitude=1.5)
    y, gx = V.rotary(x, t).double(), V.rotary(g, t, inverse=True).double()
    a, b = (y * g.double()).sum(), (x.double() * gx).sum()
    # each side sums 6336 products of values rounded in fp32
    assert abs(a - b) <= 8 * R.U32 * ((y * g).abs().sum() + (x * gx).abs().sum())
    h = 2.0 ** -4
    d = (V.rotary(x + h * g, t).double() - V.rotary(x - h * g, t).double()) / (2 * h)
    ref, mag = R.rotate(g.double(), t.cos_sin.double()[None, :, None], 64, False)
    full = (x.abs() + h * g.abs()).amax() * 4
    assert (d - ref).abs().max() <= 16 * R.U32 * float(full) / h


GEOMS = [((4, 8, 16), [(1, 8, 16)] * 2, 0, False, 1), ((3, 7, 13), [(1, 8, 16), (2, 8, 8), (4, 4, 8)], 5, True, 2),
         ((5, 9, 17), [(2, 8, 8)] * 3, 131, True, 1), ((1, 1, 1), [(1, 8, 16)], 0, False, 1)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("grid,shapes,tail,shuffle,B", GEOMS)
@pytest.mark.parametrize("rot", [128, 112, 16])
def test_tiles_and_back(V, layout, grid, shapes, tail, shuffle, B, rot):
    inter, H = layout == "interleaved", len(shapes)
    order = None
    if shuffle:
        rng = np.random.default_rng(5)
        n = [int(np.prod([-(-g // s) for g, s in zip(grid, sh)])) for sh in shapes]
        order = np.zeros((H, max(n)), np.int32)
        for h in range(H):
            order[h, :n[h]] = rng.permutation(n[h])
    maps = V.build_tile_map(grid, shapes, tail, order).to(DEV)
    N = maps.N
    f = V.rotary_frequencies([2 * (rot // 6)] * 2 + [rot - 4 * (rot // 6)])
    pos = torch.from_numpy(V.rotary_positions(grid, tail)).to(DEV)
    tables = [V.rotary_table(pos, f.inv_freq, f.axis, interleaved=inter)]
    if B > 1:
        tables.append(_table(V, B * N, rot, inter))
    x = _rand(B, N, H, 128, seed=12, dtype=torch.bfloat16)
    for t in tables:
        xt, pooled = V.rotary_permute_pool(x, t, maps)
        turned = V.rotary(x, t)
        assert torch.equal(xt, V.permute_tiles(turned, maps))                   # bit for bit
        cs = t.cos_sin.double().view(-1, N, 1, rot // 2, 2)
        ref, mag = R.rotate(x.double(), cs, rot, inter)
        for h in range(H):
            for j in range(maps.nT):
                tok = maps.tile_map[h, 128 * j:128 * j + 128]
                tok = tok[tok >= 0].long()
                got = pooled[:, h, j]
                if len(tok) == 0:
                    assert (got == 0).all()
                    continue
                r, m = ref[:, tok, h], mag[:, tok, h]
                arith = 3 * R.U32 * m.amax(1)
                assert R.worst(got[:, 0], r.mean(1), arith + 130 * R.U32 * r.abs().mean(1), torch.float32) <= 1
                assert R.worst(got[:, 1], r.amax(1), arith, torch.float32) <= 1
                assert R.worst(got[:, 2], r.amin(1), arith, torch.float32) <= 1
        g_t = _rand(B, H, maps.Npad, 128, seed=13, dtype=torch.bfloat16)
        raster = V.unpermute(g_t, maps, N)
        for inverse in (True, False):
            assert torch.equal(V.rotary_unpermute(g_t, t, maps, N, inverse=inverse),
                               V.rotary(raster, t, inverse=inverse))
    V.check_device_status()


def test_tile_map_entry_out_of_range_is_flagged(V):
    maps = V.build_tile_map((2, 8, 16), [(1, 8, 16)], 0).to(DEV)
    x = _rand(1, 256, 1, 128, seed=14, dtype=torch.bfloat16)
    t = _table(V, 256, 128, True)
    good, _ = V.rotary_permute_pool(x, t, maps)
    maps.tile_map[0, 3] = 256
    xt, _ = V.rotary_permute_pool(x, t, maps)
    with pytest.raises(V.VedaError):
        V.check_device_status()
    assert (xt[0, 0, 3] == 0).all() and torch.equal(xt[0, 0, 4:], good[0, 0, 4:])
    out = torch.full((1, 256, 1, 128), 7.0, device=DEV, dtype=torch.bfloat16)
    V.rotary_unpermute(good, t, maps, 256, out=out)
    with pytest.raises(V.VedaError):
        V.check_device_status()
    assert (out[0, 3] == 7).all() and not (out[0, 4] == 7).all()                 # the token has no slot now


def test_other_stream_and_graph(V):
    x = _rand(2, 50, 4, 128, seed=15, dtype=torch.bfloat16)
    t = _table(V, 50, 128, True)
    ref = V.rotary(x, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = V.rotary(x, t, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, ref)
    f = V.rotary_frequencies(128)
    pos = torch.arange(50, device=DEV, dtype=torch.int32)
    out = torch.empty_like(x)
    cs = torch.empty((50, 64, 2), device=DEV)
    V.rotary(x, V.rotary_table(pos, f.inv_freq, f.axis, out=cs), out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        V.rotary(x, V.rotary_table(pos, f.inv_freq, f.axis, out=cs), out=out)
    x2 = _rand(2, 50, 4, 128, seed=16, dtype=torch.bfloat16)
    x.copy_(x2)
    pos += 100
    g.replay()
    assert torch.equal(out, V.rotary(x2, V.rotary_table(pos, f.inv_freq, f.axis)))


def test_full_clip_rows(V):
    """The 16:9 clip's shape: sampled tokens against the definition."""
    w = synth.CLIP16x9
    x = _rand(1, w.N, w.H, 128, seed=17, dtype=torch.bfloat16)
    f = V.rotary_frequencies((44, 42, 42))
    t = V.rotary_table(torch.from_numpy(V.rotary_positions(w.grid)).to(DEV), f.inv_freq, f.axis)
    y = V.rotary(x, t)
    tok = torch.randint(0, w.N, (500,), device=DEV)
    ref, mag = R.rotate(x[:, tok].double(), t.cos_sin[tok].double()[None, :, None], 128, True)
    assert R.worst(y[:, tok], ref, 3 * R.U32 * mag, torch.bfloat16) <= 1.0


def test_refuses_types_and_shapes(V):
    x, t = _rand(2, 6, 3, 64, dtype=torch.bfloat16), _table(V, 6, 64, True)
    with pytest.raises(TypeError, match="float64"):
        V.rotary(x.double(), t)
    with pytest.raises(ValueError, match="dimensions"):
        V.rotary(x[0], t)
    with pytest.raises(V.VedaError, match="rot_dim"):
        V.rotary(x[..., :32].contiguous(), t)                     # a table of more channels than the head
    with pytest.raises(V.VedaError, match="rows"):
        V.rotary(x[:, :5], t)
    with pytest.raises(ValueError, match="rows: expected shape"):
        V.rotary(x, t, rows=torch.zeros((2, 5), dtype=torch.int32, device=DEV))
    with pytest.raises(TypeError, match="rows"):
        V.rotary(x, t, rows=torch.zeros((2, 6), dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="overlaps"):
        y = _rand(2, 7, 3, 64, dtype=torch.bfloat16)
        V.rotary(y[:, 1:], t, out=y[:, :6])
    with pytest.raises(ValueError, match="contiguous"):
        V.rotary(x.transpose(2, 3), t)
    with pytest.raises(ValueError, match="cos_sin"):
        V.rotary(x, V.RotaryTable(t.cos_sin[..., 0], True))
    with pytest.raises(ValueError, match="current device|CUDA"):
        V.rotary(x, V.RotaryTable(t.cos_sin.cpu(), True))
