"""The block operators run together with the sparse path, as a model's attention block runs them:
inference through ``attention_block`` stage by stage, and a training step's gradients."""
import math

import numpy as np
import pytest
import torch

import block_ref as R
import parity as P
import synth
from oracle import veda_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def V():
    from block_sparse_attention_max_b200 import build
    build.build()
    from block_sparse_attention_max_b200 import veda
    yield veda
    veda.check_device_status()


def _rand(*shape, seed=0, dtype=torch.float32, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device=DEV)).to(dtype)


def _setup(V, w):
    maps = V.build_tile_map(w.grid, w.head_shapes, w.n_tail, synth.tile_orders(w)).to(DEV)
    f = V.rotary_frequencies((44, 42, 42))
    table = V.rotary_table(torch.from_numpy(V.rotary_positions(w.grid, w.n_tail)).to(DEV), f.inv_freq, f.axis)
    return maps, table


def test_sparse_attention_with_positions(V):
    """The path with ``rotary`` equals turning Q and K first, tile for tile; the lists may differ only
    through the pooled features, which the fused step takes before rounding."""
    w = synth.SMALL
    maps, table = _setup(V, w)
    q, k, v = (_rand(w.B, w.N, w.H, 128, seed=i, dtype=torch.bfloat16) for i in range(3))
    wq, wk = _rand(w.H, 128, 384, seed=4, scale=0.02), _rand(w.H, 128, 384, seed=5, scale=0.02)
    scale = 1 / math.sqrt(128)
    a = V.sparse_attention(q, k, v, wq, wk, maps, w.rho, scale, rotary=table)
    b = V.sparse_attention(V.rotary(q, table), V.rotary(k, table), v, wq, wk, maps, w.rho, scale)
    assert torch.equal(a.q_t, b.q_t) and torch.equal(a.k_t, b.k_t) and torch.equal(a.v_t, b.v_t)
    # one bf16 rounding of a maximum or minimum
    assert (a.pooled_q - b.pooled_q).abs().max() <= 2.0 ** -8 * b.pooled_q.abs().max()
    o, _ = V.block_sparse_attn_fwd(b.q_t, b.k_t, b.v_t, maps, a.lists, scale)
    assert torch.equal(V.unpermute(o, maps, w.N), a.o)
    V.check_device_status()


@pytest.mark.parametrize("w,xdt", [(synth.TINY, torch.bfloat16), (synth.TINY, torch.float32)])
def test_attention_block(V, w, xdt):
    B, N, H = w.B, w.N, w.H
    C = 192                                       # the stream is narrower than the heads
    maps, table = _setup(V, w)
    lin = lambda rows, K, seed: V.quantize_int8(_rand(rows, K, seed=seed, scale=1 / math.sqrt(K)))
    wt = V.BlockWeights(lin(H * 128, C, 1), lin(H * 128, C, 2), lin(H * 128, C, 3), lin(C, H * 128, 4),
                        _rand(H, 128, 384, seed=5, scale=0.02), _rand(H, 128, 384, seed=6, scale=0.02),
                        q_bias=_rand(H * 128, seed=7), o_bias=_rand(C, seed=8), pre_weight=_rand(C, seed=9),
                        pre_bias=_rand(C, seed=10), post_weight=_rand(C, seed=11), post_kind="rms")
    x = _rand(B, N, C, seed=12, dtype=xdt)
    mod = _rand(B, 3 * C, seed=13, scale=0.3)
    sc, sh, gate = mod[:, :C], mod[:, C:2 * C], mod[:, 2 * C:]
    scale = 1 / math.sqrt(128)
    h = V.attention_block(x, wt, sc, sh, gate, table, maps, w.rho, scale, residual_scale=0.5)
    assert h.shape == x.shape and h.dtype == xdt
    # the stages by hand, each against its definition on the stage's own input
    a = V.norm_modulate(x, sc, sh, wt.pre_weight, wt.pre_bias, "layer", wt.eps, torch.bfloat16)
    xd = x.double()
    mean, rstd = R.stats(xd, "layer", wt.eps)
    ref = ((xd - mean) * rstd * wt.pre_weight + wt.pre_bias) * (1 + sc.double()[:, None]) + sh[:, None]
    assert R.worst(a, ref, 100 * R.U32 * (ref.abs() + 8 * (1 + sc.double().abs()[:, None]) * wt.pre_weight.abs().max()
                                          + 4), torch.bfloat16) <= 1
    a8 = V.quantize_int8(a)
    codes, s = R.quantize(a.view(-1, C))
    assert torch.equal(a8.codes[:, :C], codes) and torch.equal(a8.scale, s)
    qkv = []
    for r, b in ((wt.q, wt.q_bias), (wt.k, None), (wt.v, None)):
        y = V.int8_matmul(a8, r, b)
        ref = (codes.double() @ r.codes[:, :C].double().t()) * s.double()[:, None] * r.scale.double()
        ref = ref + b.double() if b is not None else ref
        assert R.worst(y, ref, 4 * R.U32 * (ref.abs() + (b.double().abs() if b is not None else 0)), torch.bfloat16) <= 1
        qkv.append(y.view(B, N, H, 128))
    bufs = V.sparse_attention(*qkv, wt.pred_q, wt.pred_k, maps, w.rho, scale, rotary=table)
    n_valid = maps.tile_valid.cpu().numpy()
    lists = O.select(bufs.scores.double().cpu().numpy(), n_valid, maps.tile_segment.cpu().numpy(),
                     list(maps.nT_per_head.cpu().numpy()), w.rho)
    o_ref, _ = O.attention(P.f64(bufs.q_t), P.f64(bufs.k_t), P.f64(bufs.v_t), n_valid, lists, scale)
    mx, mean_err = P.attn_errors(P.f64(bufs.o_t), o_ref)
    top = max(1.0, float(bufs.v_t.abs().max()) / 4)             # the rule is stated for V ~ N(0, 1)
    assert mx <= P.ATTN_MAX_ABS * top and mean_err <= P.ATTN_MEAN_ABS * top
    o = V.int8_linear(bufs.o.view(B, N, H * 128), wt.o, wt.o_bias)
    assert torch.equal(h, V.norm_gate_add(o, x, gate, wt.post_weight, None, "rms", wt.eps, 0.5))
    # on another stream, with its own buffers
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    h2 = V.attention_block(x, wt, sc, sh, gate, table, maps, w.rho, scale, residual_scale=0.5, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(h, h2)
    V.check_device_status()


def test_training_step_gradients(V):
    """Norm, rotary, sparse attention, gated residual and their backward against automatic
    differentiation in 64 bits over the same block lists. The attention's rule is 2e-2 (max) and 2e-3
    (mean) of the gradient's scale; the chain rounds to bf16 six more times, by at most 2^-8 each; half of
    that sum is allowed."""
    w = synth.TINY
    B, N, H = w.B, w.N, w.H
    C = H * 128
    maps, table = _setup(V, w)
    scale = 1 / math.sqrt(128)
    x = _rand(B, N, C, seed=1, dtype=torch.bfloat16)
    sc, sh, gate = (_rand(B, C, seed=2 + i, scale=0.3) for i in range(3))
    wn = 1 + _rand(C, seed=6, scale=0.1)
    dh = _rand(B, N, C, seed=7, dtype=torch.bfloat16)
    wq, wk = _rand(H, 128, 384, seed=8, scale=0.02), _rand(H, 128, 384, seed=9, scale=0.02)
    # forward
    a, st1 = V.norm_modulate(x, sc, sh, weight=wn, kind="rms", want_stats=True)
    heads = a.view(B, N, H, 128)
    bufs = V.sparse_attention(heads, heads, heads, wq, wk, maps, w.rho, scale, rotary=table)
    o = bufs.o.view(B, N, C)
    h, st2 = V.norm_gate_add(o, x, gate, kind="layer", residual_scale=0.5, want_stats=True)
    # backward
    g2 = V.norm_gate_add_bwd(dh, o, st2, gate, kind="layer")
    do_t = V.permute_tiles(g2.dx.view(B, N, H, 128), maps)
    tl = V.transpose_lists(bufs.lists, maps)
    dq, dk, dv = V.block_sparse_attn_bwd(bufs.q_t, bufs.k_t, bufs.v_t, bufs.o_t, do_t, bufs.lse, maps, bufs.lists, tl,
                                         scale)
    da = (V.rotary_unpermute(dq, table, maps, N).float() + V.rotary_unpermute(dk, table, maps, N).float()
          + V.unpermute(dv, maps, N).float()).to(torch.bfloat16).view(B, N, C)
    g1 = V.norm_modulate_bwd(da, x, st1, sc, weight=wn, kind="rms", residual_grad=dh, residual_scale=0.5)
    V.check_device_status()
    # 64-bit reference with a token mask from the same lists
    mask = torch.zeros((H, N, N), dtype=torch.bool, device=DEV)
    for hd in range(H):
        for r in range(maps.nT):
            qt = maps.tile_map[hd, r * 128:r * 128 + 128].long()
            for cnt, idx in ((bufs.lists.full_cnt, bufs.lists.full_idx), (bufs.lists.part_cnt, bufs.lists.part_idx)):
                for j in idx[0, hd, r, :int(cnt[0, hd, r])].tolist():
                    kt = maps.tile_map[hd, j * 128:j * 128 + 128].long()
                    kt = kt[kt >= 0]
                    mask[hd, qt[qt >= 0][:, None], kt[None]] = True
    leaf = lambda t: t.double().requires_grad_()
    X, SC, SH, G, W = leaf(x), leaf(sc), leaf(sh), leaf(gate), leaf(wn)
    _, rstd = R.stats(X, "rms", 1e-6)
    A = (X * rstd * W * (1 + SC[:, None]) + SH[:, None]).view(B, N, H, 128)
    cs = table.cos_sin.double()[None, :, None]
    c, s = cs[..., 0], cs[..., 1]
    turn = lambda t: torch.stack([t[..., 0::2] * c - t[..., 1::2] * s, t[..., 1::2] * c + t[..., 0::2] * s], -1).flatten(-2)
    S = torch.einsum("bnhd,bmhd->bhnm", turn(A), turn(A)) * scale
    Pm = S.masked_fill(~mask[None], -math.inf).softmax(-1)
    Ov = torch.einsum("bhnm,bmhd->bnhd", Pm, A).reshape(B, N, C)
    mu, rs = R.stats(Ov, "layer", 1e-6)
    Hh = 0.5 * X + G[:, None] * (Ov - mu) * rs
    Hh.backward(dh.double())
    six = 6 * 2.0 ** -9
    for name, got, ref in (("h", h, Hh.detach()), ("dx", g1.dx, X.grad), ("dscale", g1.dscale, SC.grad),
                           ("dshift", g1.dshift, SH.grad), ("dweight", g1.dweight, W.grad), ("dgate", g2.dgate, G.grad)):
        e, top = (got.double() - ref).abs(), ref.abs().max()
        assert e.max() <= (2e-2 + six) * top and e.mean() <= (2e-3 + six / 2) * top, (name, float(e.max() / top))


def test_block_refuses_bad_shapes(V):
    w = synth.TINY
    maps, table = _setup(V, w)
    lin = lambda rows, K: V.quantize_int8(_rand(rows, K))
    wt = V.BlockWeights(lin(256, 64), lin(256, 64), lin(128, 64), lin(64, 256), _rand(2, 128, 384), _rand(2, 128, 384))
    x = _rand(1, w.N, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="v: expected 256"):
        V.attention_block(x, wt, None, None, None, table, maps, w.rho, 0.1)
    with pytest.raises(ValueError, match="expected shape"):
        V.attention_block(x[0], wt, None, None, None, table, maps, w.rho, 0.1)
    short = V.RotaryTable(table.cos_sin[:-1].contiguous(), True)
    q = _rand(1, w.N, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(V.VedaError, match="rows"):
        V.rotary_permute_pool(q, short, maps)
    with pytest.raises(V.VedaError, match="rows"):
        V.rotary(q, short)


def test_host_pipeline_with_positions(V):
    w = synth.SMALL
    maps, table = _setup(V, w)
    scale = 1 / math.sqrt(128)
    pipe = V.HostPipeline(w.B, w.N, w.H, maps, w.rho, scale, DEV, rotary=table)
    pin = lambda t: t.cpu().pin_memory()
    clips, outs = [], []
    for i in range(3):
        clips.append([pin(_rand(w.B, w.N, w.H, 128, seed=10 * i + j, dtype=torch.bfloat16)) for j in range(3)]
                     + [pin(_rand(w.H, 128, 384, seed=10 * i + j, scale=0.02)) for j in (4, 5)])
        outs.append(torch.empty((w.B, w.N, w.H, 128), dtype=torch.bfloat16).pin_memory())
        pipe.submit(*clips[-1], outs[-1])
    pipe.synchronize()
    for c, o in zip(clips, outs):
        ref = V.sparse_attention(*[t.to(DEV) for t in c], maps, w.rho, scale, rotary=table)
        assert torch.equal(o, ref.o.cpu())


def test_host_pipeline_made_behind_queued_work(V):
    """A table that the current stream has still to make when the pipeline is built and the first clips
    are submitted: about 0.1 s of copies are queued ahead of it."""
    w = synth.SMALL
    maps, table = _setup(V, w)
    scale = 1 / math.sqrt(128)
    pin = lambda t: t.cpu().pin_memory()
    clip = [pin(_rand(w.B, w.N, w.H, 128, seed=j, dtype=torch.bfloat16)) for j in range(3)]
    clip += [pin(_rand(w.H, 128, 384, seed=j, scale=0.02)) for j in (4, 5)]
    ref = V.sparse_attention(*[t.to(DEV) for t in clip], maps, w.rho, scale, rotary=table).o.cpu()
    outs = [torch.empty((w.B, w.N, w.H, 128), dtype=torch.bfloat16).pin_memory() for _ in range(3)]
    f = V.rotary_frequencies((44, 42, 42))
    pos = torch.from_numpy(V.rotary_positions(w.grid, w.n_tail)).to(DEV)
    cs = torch.zeros_like(table.cos_sin)
    a, b = torch.zeros(1 << 30, device=DEV, dtype=torch.uint8), torch.zeros(1 << 30, device=DEV, dtype=torch.uint8)
    torch.cuda.synchronize()
    for _ in range(300):
        b.copy_(a)
    late = V.rotary_table(pos, f.inv_freq, f.axis, out=cs)
    pipe = V.HostPipeline(w.B, w.N, w.H, maps, w.rho, scale, DEV, rotary=late)
    for o in outs:
        pipe.submit(*clip, o)
    pipe.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


def test_two_threads_on_their_own_streams(V):
    """Calls enqueued from two host threads at once, each on its stream: bit for bit the results of
    calls one after the other."""
    import threading
    N, C = 3000, 1280
    f = V.rotary_frequencies(128)
    table = V.rotary_table(torch.arange(N, device=DEV, dtype=torch.int32), f.inv_freq, f.axis)
    wt = V.quantize_int8(_rand(640, C, seed=1))

    def chain(seed, stream):
        x, dy = _rand(1, N, C, seed=seed, dtype=torch.bfloat16), _rand(1, N, C, seed=seed + 1, dtype=torch.bfloat16)
        sc = _rand(1, C, seed=seed + 2)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out = []
        for _ in range(4):
            y, st = V.norm_modulate(x, sc, sc, want_stats=True, stream=stream)
            g = V.norm_modulate_bwd(dy, x, st, sc, stream=stream)
            r = V.rotary(y.view(1, N, C // 128, 128), table, stream=stream)
            m = V.int8_linear(y, wt, stream=stream)
            t = V.int8_linear(y[:, :40], wt, stream=stream)
            out = [y, g.dx, g.dscale, g.dshift, r, m, t]
        return out
    serial = [chain(100 * i, None) for i in range(2)]
    torch.cuda.synchronize()
    got = [None, None]

    def run(i):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        got[i] = chain(100 * i, s)
        s.synchronize()
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(serial, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_offsets_past_32_bits(V):
    """Tensors of more than 2^31 elements: their last rows against calls on those rows alone."""
    tail = 300
    f = V.rotary_frequencies(128)
    N, H = 140_000, 128
    x = torch.empty((1, N, H, 128), device=DEV, dtype=torch.bfloat16)
    assert x.numel() > 2**31
    x[:, -tail:] = _rand(1, tail, H, 128, seed=1, dtype=torch.bfloat16)
    x[:, :-tail] = 1
    pos = torch.arange(N, device=DEV, dtype=torch.int32)
    table = V.rotary_table(pos, f.inv_freq, f.axis)
    y = V.rotary(x, table)
    small = V.RotaryTable(table.cos_sin[-tail:].contiguous(), True)
    assert torch.equal(y[:, -tail:], V.rotary(x[:, -tail:], small))
    # the same memory as rows of 8,192 channels
    rows = x.view(1, -1, 8192)
    sc = _rand(1, 8192, seed=2)
    h, st = V.norm_modulate(rows, sc, kind="rms", out=y.view(1, -1, 8192), want_stats=True)
    n = tail * H * 128 // 8192
    ref, st1 = V.norm_modulate(rows[:, -n:], sc, kind="rms", want_stats=True)
    assert torch.equal(h[:, -n:], ref) and torch.equal(st.rstd[:, -n:], st1.rstd)
    big = V.norm_modulate_bwd(rows, rows, st, sc, kind="rms", out=y.view(1, -1, 8192))
    part = V.norm_modulate_bwd(rows[:, -n:], rows[:, -n:], st1, sc, kind="rms")
    assert torch.equal(big.dx[:, -n:], part.dx)
    del big, part, ref, h
    q = V.quantize_int8(rows[0])
    q1 = V.quantize_int8(rows[0, -n:])
    assert torch.equal(q.codes[-n:], q1.codes) and torch.equal(q.scale[-n:], q1.scale)
    del y, x, rows, q
    # a product with more than 2^31 outputs
    M, No, K = 70_000, 32_768, 48
    a, w = V.quantize_int8(_rand(M, K, seed=3)), V.quantize_int8(_rand(No, K, seed=4))
    out = V.int8_matmul(a, w)
    assert out.numel() > 2**31
    last = V.Int8Rows(a.codes[-300:].contiguous(), a.scale[-300:].contiguous(), K)
    assert torch.equal(out[-300:], V.int8_matmul(last, w))
    V.check_device_status()
