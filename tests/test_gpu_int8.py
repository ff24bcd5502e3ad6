"""8-bit integer rows and products on the GPU against their definition.

Codes and scales are exact. A product's integer sum is exact; its conversion to fp32, the product of
the scales and the fused multiply-add are one rounding each, then one rounding to the output type."""
import numpy as np
import pytest
import torch

import block_ref as R

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


def _codes(rows, K, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-128, 128, (rows, K), generator=g, device=DEV, dtype=torch.int8)


def _check_rows(got, x):
    codes, scale = R.quantize(x)
    K = x.shape[1]
    assert torch.equal(got.scale.nan_to_num(-1.0), scale.nan_to_num(-1.0))
    assert torch.equal(got.codes[:, :K], codes)
    assert (got.codes[:, K:] == 0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 7), (9, 16), (17, 100), (5, 1024), (6, 1025), (3, 1032), (4, 4101),
                                    (2, 5120), (3, 8192), (2, 8200), (2, 20001), (9000, 200),
                                    (3000, 1040), (2500, 5120), (2000, 1025)])
def test_quantize(V, dtype, rows, K):
    x = _rand(rows, K, seed=K, dtype=TYPES[dtype])
    _check_rows(V.quantize_int8(x), x)
    wide = _rand(rows, K + 3, seed=K + 1, dtype=TYPES[dtype])[:, 1:K + 1]       # unaligned, strided rows
    _check_rows(V.quantize_int8(wide), wide)


def test_quantize_borders(V):
    """Quotients that lie on a rounding border or next to one: scale 2^e with amax 127 2^e makes
    every half-integer a tie; other scales put values one fp32 step beside the border."""
    k = torch.arange(-127, 128, device=DEV, dtype=torch.float32)
    ties = torch.cat([torch.tensor([127.0], device=DEV), k[:-1] + 0.5])
    rows = [ties * s for s in (1.0, 2.0 ** -20, 2.0 ** 40, 2.0 ** -90)]
    g = torch.Generator(device=DEV).manual_seed(1)
    for _ in range(60):
        amax = torch.rand(1, generator=g, device=DEV) * 10 + 0.1
        s = (amax.double() / 127).float()
        near = ((k[:-1].double() + 0.5) * s.double()).float()
        for d in (-1, 0, 1):
            v = near if d == 0 else torch.nextafter(near, torch.full_like(near, d * 1e9))
            rows.append(torch.cat([amax, v.clamp(-float(amax), float(amax))]))
    x = torch.stack(rows)
    _check_rows(V.quantize_int8(x), x)
    for dt in (torch.bfloat16, torch.float16):
        xb = x.to(dt)
        _check_rows(V.quantize_int8(xb), xb)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_scales_are_the_rounded_quotients(V, dtype):
    """amax / 127 rounded once to fp32, as IEEE division on the CPU gives it (a product with a rounded
    1 / 127 is a step off for one row in twenty), for every 16-bit mantissa and many of fp32; a row of two
    tokens as for the fused product of a few tokens."""
    dt = TYPES[dtype]
    if dt == torch.float32:
        a = 1 + torch.arange(4096, dtype=torch.float64) * 2.0 ** -12 + 3 * 2.0 ** -23
    else:
        a = 1 + torch.arange(round(1 / torch.finfo(dt).eps), dtype=torch.float64) * torch.finfo(dt).eps
    a = torch.cat([a * 2.0 ** e for e in (-9, 0, 7)]).to(dt).to(DEV)
    x = torch.stack([a, -a / 3, a / 7], 1)
    scale = torch.from_numpy(a.float().cpu().numpy() / np.float32(127))
    got = V.quantize_int8(x)
    assert torch.equal(got.scale.cpu(), scale)
    _check_rows(got, x)
    one = V.Int8Rows.from_codes(torch.tensor([[1, 0, 0]], device=DEV, dtype=torch.int8), torch.ones(1, device=DEV))
    for i in range(0, len(a), 97):
        y = V.int8_linear(x[i:i + 2], one, out_dtype=torch.float32)                  # code 127 times the scale
        assert torch.equal(y[:, 0].cpu(), (scale[i:i + 2].double() * 127).float())


def test_quantize_special_rows(V):
    x = _rand(10, 300, seed=2)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 5] = float("-inf")
    x[3] *= 2.0 ** -103                               # amax near 2^-101: a zero row
    x[4] *= 2.0 ** -98
    x[5] = 0
    x[5, 299] = 3.0e38
    x[6] = 2.0 ** -149
    got = V.quantize_int8(x)
    _check_rows(got, x)
    assert got.scale[0] == 1 and torch.isnan(got.scale[1:3]).all()
    w = V.quantize_int8(_rand(20, 300, seed=3))
    y = V.int8_matmul(got, w, out_dtype=torch.float32)
    assert torch.isnan(y[1:3]).all() and torch.isfinite(y[[0, 3, 4, 6, 7]]).all() and (y[0] == 0).all()


def _product(a, sa, w, sw, bias):
    acc = a.double() @ w.double().t()                 # exact: below 2^53
    y = acc * sa.double()[:, None] * sw.double()[None]
    e = 3 * R.U32 * y.abs()
    if bias is not None:
        e = e + R.U32 * (y + bias.double()).abs()
        y = y + bias.double()
    return y, e


SIZES = [(1, 1, 1), (1, 5, 17), (1, 257, 5120), (2, 100, 333), (2, 3000, 64), (3, 127, 16), (4, 129, 5000), (7, 5200, 130),
         (17, 600, 1100), (33, 128, 2000), (65, 1000, 700), (100, 70, 4097), (128, 2049, 384), (3, 64, 48), (5, 1000, 640), (8, 130, 4101), (9, 1, 1),
         (9, 33, 50), (16, 256, 128), (31, 300, 127), (64, 511, 1040), (127, 255, 129), (128, 256, 512), (129, 257, 513),
         (200, 640, 256), (300, 1030, 2064), (777, 515, 4101), (1000, 2600, 100), (2049, 96, 130), (256, 5120, 200), (20000, 64, 256), (20000, 128, 384)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(V, M, N, K):
    a, w = _codes(M, K, seed=M), _codes(N, K, seed=N + 7)
    sa, sw = _rand(M, seed=3).abs() + 0.1, _rand(N, seed=4).abs() * 0.01
    bias = _rand(N, seed=5)
    ar, wr = V.Int8Rows.from_codes(a, sa), V.Int8Rows.from_codes(w, sw)
    for b in (bias, None):
        ref, e = _product(a, sa, w, sw, b)
        for dt in TYPES.values():
            if dt == torch.float16 and ref.abs().max() > 60000:
                continue
            assert R.worst(V.int8_matmul(ar, wr, b, dt), ref, e, dt) <= 1, dt
    # a slice of a wider output, nothing beside it touched
    wide = torch.full((M, N + 5), 9.0, device=DEV)
    V.int8_matmul(ar, wr, bias, out=wide[:, 2:2 + N])
    ref, e = _product(a, sa, w, sw, bias)
    assert R.worst(wide[:, 2:2 + N], ref, e, torch.float32) <= 1
    assert (wide[:, :2] == 9).all() and (wide[:, 2 + N:] == 9).all()


def test_largest_sum(V):
    """K at its limit with codes of -128 throughout: 2^14 * 131071, next to 2^31."""
    K = 131071
    a = torch.full((9, K), -128, device=DEV, dtype=torch.int8)
    w = torch.full((3, K), -128, device=DEV, dtype=torch.int8)
    one = lambda n: torch.ones(n, device=DEV)
    for rows in (1, 9):
        y = V.int8_matmul(V.Int8Rows.from_codes(a[:rows], one(rows)), V.Int8Rows.from_codes(w, one(3)),
                          out_dtype=torch.float32)
        assert (y == torch.tensor(16384.0 * K, dtype=torch.float64).float().item()).all()
    big = V.Int8Rows(torch.zeros((2, 131072), device=DEV, dtype=torch.int8), one(2), 131072)
    with pytest.raises(V.VedaError, match="131071"):
        V.int8_matmul(big, big)


def test_many_tiles_repeat_exactly(V):
    """More tiles than SMs (every CTA takes several): equal to a few columns of the definition, and
    the same bits twice."""
    M, N, K = 4100, 2600, 640
    a, w = _codes(M, K, seed=1), _codes(N, K, seed=2)
    sa, sw = _rand(M, seed=3).abs(), _rand(N, seed=4).abs()
    ar, wr = V.Int8Rows.from_codes(a, sa), V.Int8Rows.from_codes(w, sw)
    y = V.int8_matmul(ar, wr, out_dtype=torch.float32)
    ref, e = _product(a, sa, w, sw, None)
    assert R.worst(y, ref, e, torch.float32) <= 1
    assert torch.equal(y, V.int8_matmul(ar, wr, out_dtype=torch.float32))


def test_linear_shapes_streams_graph(V):
    w = V.quantize_int8(_rand(96, 200, seed=1))
    bias = _rand(96, seed=2)
    for shape in ((200,), (4, 200), (2, 3, 200), (0, 200), (2, 0, 200)):
        x = _rand(*shape, seed=3, dtype=torch.bfloat16)
        y = V.int8_linear(x, w, bias)
        assert y.shape == shape[:-1] + (96,) and y.dtype == torch.bfloat16
        if x.numel():
            q, s = R.quantize(x.reshape(-1, 200))
            ref, e = _product(q, s, w.codes[:, :200], w.scale, bias)
            assert R.worst(y.reshape(-1, 96), ref, e, torch.bfloat16) <= 1
    # one call equals the two: rounded by the product itself (few short rows) or beforehand
    for rows, K, dt, ydt in ((1, 5120, "bf16", "bf16"), (3, 4101, "fp16", "fp32"), (4, 4096, "fp32", "bf16"),
                             (4, 4097, "bf16", "bf16"), (2, 9000, "bf16", "fp16"), (1, 7, "fp32", "fp32"),
                             (5, 100, "bf16", "bf16")):
        x = _rand(rows, K + 1, seed=K, dtype=TYPES[dt])[:, K % 2:K % 2 + K]
        wk = V.quantize_int8(_rand(70, K, seed=K + 1))
        a = V.int8_linear(x, wk, out_dtype=TYPES[ydt])
        assert torch.equal(a, V.int8_matmul(V.quantize_int8(x), wk, out_dtype=TYPES[ydt]))
        x[0, K // 2] = float("nan")
        y = V.int8_linear(x, wk, out_dtype=torch.float32)
        assert torch.isnan(y[0]).all() and torch.isfinite(y[1:]).all()
    for rows in (1, 40):
        x = _rand(rows, 200, seed=4, dtype=torch.bfloat16)
        ref = V.int8_linear(x, w, bias)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        y = V.int8_linear(x, w, bias, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, ref)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = V.int8_linear(x, w, bias)
        x2 = _rand(rows, 200, seed=5, dtype=torch.bfloat16)
        x.copy_(x2)
        for _ in range(3):
            g.replay()
        assert torch.equal(y, V.int8_linear(x2, w, bias))


def test_refuses_types_and_shapes(V):
    x, w = _rand(4, 64, dtype=torch.bfloat16), V.quantize_int8(_rand(8, 64))
    with pytest.raises(TypeError, match="float64"):
        V.quantize_int8(x.double())
    with pytest.raises(TypeError, match="out_dtype"):
        V.int8_linear(x, w, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="rows of 32"):
        V.int8_linear(x[:, :32], w)
    with pytest.raises(ValueError, match="a has rows"):
        V.int8_matmul(V.quantize_int8(x[:, :32]), w)
    with pytest.raises(ValueError, match="bias: expected shape"):
        V.int8_linear(x, w, _rand(7))
    with pytest.raises(TypeError, match="bias"):
        V.int8_linear(x, w, _rand(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="rows of one stride"):
        V.int8_linear(_rand(2, 4, 128, dtype=torch.bfloat16)[:, :3, :64], w)
    with pytest.raises(ValueError, match="expected 4 rows"):
        V.quantize_int8(x, out=w)
    with pytest.raises(ValueError, match="overlap in memory"):
        V.int8_matmul(V.quantize_int8(x), w, out=_rand(1, 8).expand(4, 8))
