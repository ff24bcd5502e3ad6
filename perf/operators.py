"""The operators of the transformer block around the sparse attention: measured cases.

Three families, as a block uses them one after the other:

* rotary positions of Q and K (interleaved and half layouts, part of the head, three position
  axes or one, a fresh or a kept table), alone and on the way into the 3D tiles, and the way
  back of their gradients;
* the norms before and after a block, fused with the block's scale / shift, gate and residual
  scale, forward and backward;
* the product of 8-bit integers with a scale for every token and every output channel.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded
once at the end), or, with ``own`` set, through the package's entry points. ``exact`` computes
the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
THETA = 10000.0


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one new token of each of eight sequences, every sequence at its own position of a kept
        # table (the call whose cost is its latency)
        dict(name="rotary_tokens", op="rotary", B=8, N=1, H=40, Hk=8, D=128, rot=128, layout="half",
             dtype="bf16", packed=False, table="rows", inverse=False),
        # prompt of two sequences: the table of its positions is built in the call, Q and K are
        # slices of one packed projection output, and half of each head is rotated
        dict(name="rotary_prompt_part", op="rotary", B=2, N=4095, H=32, Hk=32, D=128, rot=64,
             layout="half", dtype="fp16", packed=True, table="built", inverse=False),
        # Q and K of the 16:9 clip rotated on their way into 3D tiles, with the tiles' pooling
        dict(name="rotary_tiles_clip", op="rotary_tiles", B=1, H=40, grid_t=31, grid_h=30, grid_w=54,
             tile_t=1, tile_h=8, tile_w=16, tail=0, rot=128, layout="interleaved", shuffle=False),
        # dQ and dK of the mixed workload (a different tile order in every head, 1D tail tokens)
        # back to raster order and through the rotation's transpose
        dict(name="rotary_grads_mixed", op="rotary_grads", B=1, H=32, grid_t=16, grid_h=32, grid_w=56,
             tile_t=2, tile_h=8, tile_w=8, tail=640, rot=128, layout="half", shuffle=True),
        # the norm before the block on a handful of conditioning tokens (latency)
        dict(name="pre_norm_few", op="pre", B=2, N=3, C=1024, kind="layer", dtype="bf16", out="bf16",
             pdtype="fp32", affine=False),
        # the norm before the block on the 16:9 clip's tokens, 40 heads of 128 channels
        dict(name="pre_norm_clip", op="pre", B=1, N=50220, C=5120, kind="layer", dtype="bf16", out="bf16",
             pdtype="bf16", affine=False),
        # its backward in training, with the gradient that flows around the block
        dict(name="pre_norm_clip_bwd", op="pre_bwd", B=1, N=50220, C=5120, kind="rms", dtype="bf16",
             out="bf16", pdtype="bf16", affine=True),
        # the norm after the block, its gate and the residual sum, residual stream in fp32
        dict(name="post_norm_mixed", op="post", B=2, N=14657, C=4096, kind="rms", dtype="bf16", out="fp32",
             pdtype="fp32", affine=True),
        # its backward; an odd channel count, which has no 16-byte rows
        dict(name="post_norm_odd_bwd", op="post_bwd", B=3, N=2049, C=1023, kind="layer", dtype="fp16",
             out="fp16", pdtype="fp32", affine=True),
        # the modulation vectors (scale, shift, gate of two sub-blocks) of one conditioning token
        dict(name="int8_one_token", op="int8", M=1, N=30720, K=5120, dtype="bf16", bias=True),
        # a ragged prompt: no size is a multiple of a tile, rows of K bytes are not 16-byte aligned
        dict(name="int8_ragged", op="int8", M=777, N=4099, K=4101, dtype="fp16", bias=True),
        # one projection of the 16:9 clip's tokens
        dict(name="int8_clip", op="int8", M=50220, N=5120, K=5120, dtype="bf16", bias=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "rotary_tiles", "rotary_grads", "pre", "pre_bwd", "post", "post_bwd",
                     "int8", "int8"])
    if op == "rotary":
        D = rng.choice([32, 64, 80, 96, 128, 192, 256])
        H = rng.randint(1, 40)
        table = rng.choice(["rows", "built", "kept"])
        B = _log(rng, 1, 64)
        rot = D if rng.random() < 0.5 else 2 * rng.randint(1, D // 2)
        N = _log(rng, 1, max(1, min(65536, 200_000_000 // (B * (H + 8) * D))))
        return dict(op=op, B=B, N=N, H=H, Hk=rng.choice([H, max(1, H // 4), 1]), D=D, rot=rot,
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    packed=rng.random() < 0.5, table=table, inverse=rng.random() < 0.5)
    if op in ("rotary_tiles", "rotary_grads"):
        tt, th, tw = rng.choice([(1, 8, 16), (2, 8, 8), (4, 4, 8), (8, 4, 4), (1, 16, 8)])
        H = rng.randint(1, 40)
        T, Hg, Wg = rng.randint(1, 27), rng.randint(4, 32), rng.randint(4, 56)
        return dict(op=op, B=1 if H > 12 else rng.randint(1, 2), H=H, grid_t=T, grid_h=Hg, grid_w=Wg,
                    tile_t=tt, tile_h=th, tile_w=tw, tail=rng.choice([0, 0, rng.randint(1, 700)]),
                    rot=rng.choice([128, 128, 16 * rng.randint(1, 8)]),
                    layout=rng.choice(["half", "interleaved"]), shuffle=rng.random() < 0.5)
    if op in ("pre", "pre_bwd", "post", "post_bwd"):
        C = _log(rng, 64, 8192)
        C = C if rng.random() < 0.4 else max(64, C // 64 * 64)
        C = C if rng.random() < 0.3 or C < 512 else 128 * rng.choice([8, 16, 32, 40, 56, 64])
        B = _log(rng, 1, 16)
        N = _log(rng, 1, max(1, 150_000_000 // (B * C)))
        dtype, out = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"),
                                 ("fp32", "bf16") if op.startswith("pre") else ("bf16", "fp32")])
        kind = rng.choice(["layer", "rms"] + (["none"] if op.startswith("post") else []))
        return dict(op=op, B=B, N=N, C=C, kind=kind, dtype=dtype, out=out,
                    pdtype=rng.choice(["fp32", "bf16"]), affine=kind != "none" and rng.random() < 0.6)
    M = _log(rng, 1, 50220)
    K = _log(rng, 64, 8192)
    K = K if rng.random() < 0.4 else max(64, K // 64 * 64)
    N = _log(rng, 64, 30720)
    N = max(64, min(N, 1_000_000_000_000 // (M * K)))
    return dict(op=op, M=M, N=N, K=K, dtype=rng.choice(["bf16", "bf16", "fp16"]), bias=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=DEV, dtype=dtype)


def _activations(g, shape, dtype):
    """Hidden activations: normal, with channels of larger spread and a common offset, as a
    transformer's residual stream has them."""
    C = shape[-1]
    spread = torch.exp(0.5 * _randn(g, C))
    offset = 0.3 * _randn(g, C)
    x = torch.empty(shape, device=DEV, dtype=dtype)
    flat = x.reshape(-1, C)
    for r in range(0, flat.shape[0], 8192):
        n = min(8192, flat.shape[0] - r)
        flat[r:r + n] = (_randn(g, n, C) * spread + offset).to(dtype)
    return x


def _frequencies(rot, axes):
    """Inverse frequencies and position axis of each pair: the pairs are split over the axes,
    each with the geometric series theta^(-2 i / d) of its own part d of the head."""
    P = rot // 2
    per = [P // axes + (1 if a < P % axes else 0) for a in range(axes)]
    inv = np.concatenate([THETA ** (-np.arange(p) / max(p, 1)) for p in per])
    axis = np.concatenate([np.full(p, a, np.int32) for a, p in enumerate(per)])
    return inv.astype(np.float64), axis.astype(np.int32)


def _angles(pos, inv, axis):
    """[rows, P] angles in 64 bits from positions [axes, rows]."""
    p = pos.double()[torch.from_numpy(axis.astype(np.int64)).to(pos.device)]
    return (p * torch.from_numpy(inv).to(pos.device)[:, None]).t().contiguous()


def _table(pos, inv, axis):
    a = _angles(pos, inv, axis)
    return torch.stack([a.cos(), a.sin()], -1).float()


def _grid_positions(T, Hg, Wg, tail):
    """(t, h, w) of the video tokens in raster order; a tail token j has the position
    max(T, Hg, Wg) + j on all three axes."""
    t, h, w = np.meshgrid(np.arange(T), np.arange(Hg), np.arange(Wg), indexing="ij")
    video = np.stack([t.ravel(), h.ravel(), w.ravel()])
    extra = np.tile(max(T, Hg, Wg) + np.arange(tail), (3, 1))
    return np.concatenate([video, extra], 1).astype(np.int32)


def _tile_map(case, rng):
    """[H, Npad] raster token of each tile slot (-1 for a pad slot) and [H, nT] valid slots: the
    valid tokens of a tile come first, in local raster order; tail tokens fill 1D tiles."""
    T, Hg, Wg = case["grid_t"], case["grid_h"], case["grid_w"]
    tt, th, tw = case["tile_t"], case["tile_h"], case["tile_w"]
    t, h, w = np.meshgrid(np.arange(T), np.arange(Hg), np.arange(Wg), indexing="ij")
    nh, nw = -(-Hg // th), -(-Wg // tw)
    tile = (((t // tt) * nh + h // th) * nw + w // tw).ravel()
    nvt = -(-T // tt) * nh * nw
    n_tail_tiles = -(-case["tail"] // 128)
    nT = nvt + n_tail_tiles
    first = np.argsort(tile, kind="stable")          # raster order inside a tile
    count = np.bincount(tile, minlength=nvt)
    start = np.concatenate([[0], np.cumsum(count)[:-1]])
    slot = np.arange(len(first)) - start[tile[first]]
    base = np.full((nT, 128), -1, np.int32)
    base[tile[first], slot] = first
    tail = np.full(n_tail_tiles * 128, -1, np.int32)
    tail[:case["tail"]] = T * Hg * Wg + np.arange(case["tail"])
    base[nvt:] = tail.reshape(n_tail_tiles, 128)
    maps = []
    for _ in range(case["H"]):
        order = rng.permutation(nvt) if case["shuffle"] else np.arange(nvt)
        maps.append(np.concatenate([base[:nvt][order], base[nvt:]]).reshape(-1))
    m = np.stack(maps)
    valid = (m.reshape(case["H"], nT, 128) >= 0).sum(-1).astype(np.int32)
    return m, valid, nvt


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "rotary":
        B, N, H, Hk, D = case["B"], case["N"], case["H"], case["Hk"], case["D"]
        dt = DTYPES[case["dtype"]]
        if case["packed"]:
            packed = _activations(g, (B, N, H + 2 * Hk, D), dt)     # Q, K, V of one projection
            s["q"], s["k"] = packed[:, :, :H], packed[:, :, H:H + Hk]
        else:
            s["q"], s["k"] = _activations(g, (B, N, H, D), dt), _activations(g, (B, N, Hk, D), dt)
        axes = 3 if case["rot"] >= 6 and case["table"] == "built" else 1
        s["inv"], s["axis"] = _frequencies(case["rot"], axes)
        if case["table"] == "rows":
            R = max(4096, N)
            s["cos_sin"] = _table(torch.arange(R, device=DEV, dtype=torch.int32)[None], s["inv"], s["axis"])
            s["rows"] = torch.randint(0, R, (B, N), generator=g, device=DEV, dtype=torch.int32)
        else:
            far = torch.randint(0, 1_000_000, (axes, 1), generator=g, device=DEV, dtype=torch.int32)
            s["pos"] = far + torch.arange(N, device=DEV, dtype=torch.int32)[None]
            if case["table"] == "kept":
                s["cos_sin"] = _table(s["pos"], s["inv"], s["axis"])
    elif op in ("rotary_tiles", "rotary_grads"):
        B, H = case["B"], case["H"]
        m, valid, nvt = _tile_map(case, np.random.default_rng(int(seed) + 5))
        N = case["grid_t"] * case["grid_h"] * case["grid_w"] + case["tail"]
        s["N"], s["nT"], s["Npad"] = N, valid.shape[1], m.shape[1]
        s["tile_map"], s["tile_valid"] = torch.from_numpy(m).to(DEV), torch.from_numpy(valid).to(DEV)
        seg = np.zeros_like(valid)
        seg[:, nvt:] = 1
        s["tile_segment"] = torch.from_numpy(seg).to(DEV)
        s["nT_per_head"] = torch.full((H,), valid.shape[1], dtype=torch.int32, device=DEV)
        pos = _grid_positions(case["grid_t"], case["grid_h"], case["grid_w"], case["tail"])
        inv, axis = _frequencies(case["rot"], 3 if case["rot"] >= 6 else 1)
        s["cos_sin"] = _table(torch.from_numpy(pos).to(DEV), inv, axis)
        shape = (B, N, H, 128) if op == "rotary_tiles" else (B, H, s["Npad"], 128)
        s["q"], s["k"] = _activations(g, shape, torch.bfloat16), _activations(g, shape, torch.bfloat16)
    elif op in ("pre", "pre_bwd", "post", "post_bwd"):
        B, N, C = case["B"], case["N"], case["C"]
        dt, dto, dtp = DTYPES[case["dtype"]], DTYPES[case["out"]], DTYPES[case["pdtype"]]
        s["x"] = _activations(g, (B, N, C), dt)
        s["weight"] = (1 + 0.2 * _randn(g, C)).to(dtp) if case["affine"] else None
        s["bias"] = (0.1 * _randn(g, C)).to(dtp) if case["affine"] and case["kind"] == "layer" else None
        if op.startswith("pre"):
            s["scale"], s["shift"] = (0.3 * _randn(g, B, C)).to(dtp), (0.3 * _randn(g, B, C)).to(dtp)
        else:
            s["gate"] = (0.5 * _randn(g, B, C)).to(dtp)
            s["residual_scale"] = 0.875
        if op == "post":
            s["residual"] = _activations(g, (B, N, C), dto)
        if op.endswith("bwd"):
            s["dy"] = _randn(g, B, N, C, dtype=torch.float32).to(dto)
            if op == "pre_bwd":
                s["dres"], s["residual_scale"] = _randn(g, B, N, C, dtype=torch.float32).to(dt), 0.875
            # what the forward kept: mean and reciprocal deviation of every row
            mean = torch.zeros((B, N), device=DEV)
            rstd = torch.ones((B, N), device=DEV)
            if case["kind"] != "none":
                flat = s["x"].reshape(-1, C)
                for r in range(0, B * N, 16384):
                    v = flat[r:r + 16384].double()
                    mu = v.mean(1) if case["kind"] == "layer" else torch.zeros(v.shape[0], device=DEV).double()
                    var = (v - mu[:, None]).square().mean(1)
                    mean.view(-1)[r:r + 16384] = mu.float()
                    rstd.view(-1)[r:r + 16384] = (1.0 / (var + EPS).sqrt()).float()
            s["mean"], s["rstd"] = mean, rstd
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _activations(g, (M, K), DTYPES[case["dtype"]])
        w = _randn(g, N, K) * (0.02 * torch.exp(0.3 * _randn(g, N)))[:, None]
        s["w_codes"], s["w_scale"] = _quantize(w)
        s["bias"] = 0.1 * _randn(g, N) if case["bias"] else None
        if own:
            # a program lays its weights out once
            from block_sparse_attention_max_b200 import veda as V
            s["w"] = V.Int8Rows.from_codes(s["w_codes"], s["w_scale"])
    return s


EPS = 1e-6


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _rotated(x, cs, rot, half, inverse):
    """x [..., D] (32 or 64 bits) rotated by cos / sin [..., P, 2]."""
    c, sn = cs[..., 0], cs[..., 1]
    if inverse:
        sn = -sn
    P = rot // 2
    y = x.clone()
    if half:
        a, b = x[..., :P], x[..., P:rot]
        y[..., :P], y[..., P:rot] = a * c - b * sn, b * c + a * sn
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * sn, b * c + a * sn
    return y


def _plain_rotary(s):
    case = s["case"]
    cs = _table(s["pos"], s["inv"], s["axis"]) if case["table"] == "built" else s["cos_sin"]
    cs = cs[s["rows"].long()][:, :, None] if case["table"] == "rows" else cs[None, :, None]
    half = case["layout"] == "half"
    return {n: _rotated(s[n].float(), cs, case["rot"], half, case["inverse"]).to(s[n].dtype) for n in ("q", "k")}


def _plain_tiles(s):
    case = s["case"]
    half = case["layout"] == "half"
    out = {}
    m = s["tile_map"].long()
    pad = m < 0
    heads = torch.arange(case["H"], device=m.device)[:, None]
    for n in ("q", "k"):
        r = _rotated(s[n].float(), s["cos_sin"][None, :, None], case["rot"], half, False)
        t = r[:, m.clamp(min=0), heads]                        # [B, H, Npad, 128]
        t = t.masked_fill(pad[None, :, :, None], 0.0)
        B, H, Npad, D = t.shape
        v = t.view(B, H, Npad // 128, 128, D)
        gone = pad.view(1, H, Npad // 128, 128, 1)
        cnt = s["tile_valid"][None, :, :, None].float()
        some = cnt > 0
        mean = v.sum(3) / cnt.clamp(min=1)
        mx = v.masked_fill(gone, -math.inf).amax(3)
        mn = v.masked_fill(gone, math.inf).amin(3)
        zero = torch.zeros_like(mean)
        pooled = torch.stack([torch.where(some, a, zero) for a in (mean, mx, mn)], 3)
        out[n], out["pooled_" + n] = t.to(torch.bfloat16), pooled
        del r, t, v, mx, mn
    return out


def _plain_grads(s):
    case = s["case"]
    half = case["layout"] == "half"
    m = s["tile_map"].long()
    H = case["H"]
    # slot of every raster token of every head
    where = torch.empty((H, s["N"] + 1), dtype=torch.long, device=m.device)
    slots = torch.arange(s["Npad"], device=m.device)[None].expand(H, -1)
    where.scatter_(1, torch.where(m < 0, s["N"], m), slots)
    where = where[:, :s["N"]]
    heads = torch.arange(H, device=m.device)[:, None]
    out = {}
    for n in ("q", "k"):
        x = s[n][:, heads, where].transpose(1, 2).float()       # [B, N, H, 128]
        out[n] = _rotated(x, s["cos_sin"][None, :, None], case["rot"], half, True).to(torch.bfloat16)
    return out


def _stats(x, kind):
    if kind == "none":
        return None, None
    mean = x.mean(-1, keepdim=True) if kind == "layer" else None
    d = x - mean if kind == "layer" else x
    return mean, 1.0 / (d.square().mean(-1, keepdim=True) + EPS).sqrt()


def _normed(x, mean, rstd):
    if rstd is None:
        return x
    return (x - mean) * rstd if mean is not None else x * rstd


def _affine(xh, s, cast):
    if s["weight"] is not None:
        xh = xh * cast(s["weight"])
    if s["bias"] is not None:
        xh = xh + cast(s["bias"])
    return xh


def _norm_forward(s, cast):
    case = s["case"]
    x = cast(s["x"])
    a = _affine(_normed(x, *_stats(x, case["kind"])), s, cast)
    if case["op"] == "pre":
        return a * (1 + cast(s["scale"])[:, None]) + cast(s["shift"])[:, None]
    return s["residual_scale"] * cast(s["residual"]) + cast(s["gate"])[:, None] * a


def _norm_backward(s, cast, mean, rstd):
    case = s["case"]
    x, dy = cast(s["x"]), cast(s["dy"])
    pre = case["op"] == "pre_bwd"
    gain = (1 + cast(s["scale"]) if pre else cast(s["gate"]))[:, None]
    xh = _normed(x, mean, rstd)
    out = {}
    out["dscale" if pre else "dgate"] = (dy * _affine(xh, s, cast)).sum(1)
    if pre:
        out["dshift"] = dy.sum(1)
    da = dy * gain
    if s["weight"] is not None:
        out["dweight"] = (da * xh).sum((0, 1))
        if s["bias"] is not None:
            out["dbias"] = da.sum((0, 1))
        da = da * cast(s["weight"])
    if rstd is None:
        dx = da
    else:
        c2 = (da * xh).mean(-1, keepdim=True)
        dx = da - xh * c2
        if mean is not None:
            dx = dx - da.mean(-1, keepdim=True)
        dx = dx * rstd
    if pre:
        dx = dx + s["residual_scale"] * cast(s["dres"])
    out["dx"] = dx
    return out


def _plain_norm(s):
    return {"y": _norm_forward(s, lambda t: t.float()).to(DTYPES[s["case"]["out"]])}


def _plain_norm_bwd(s):
    kind = s["case"]["kind"]
    mean = s["mean"][..., None] if kind == "layer" else None
    rstd = s["rstd"][..., None] if kind != "none" else None
    out = _norm_backward(s, lambda t: t.float(), mean, rstd)
    out["dx"] = out["dx"].to(s["x"].dtype)
    return out


def _quantize(x):
    """Codes (int8) and scale (fp32) of every row: scale = amax / 127 rounded to fp32, code =
    x / scale rounded to the nearest integer, ties to even (in 64 bits: values next to a
    rounding border). A row whose amax is below 2^-100 counts as zero: scale 1, codes 0."""
    amax = x.abs().amax(-1).float()
    tiny = amax < 2.0 ** -100
    scale = torch.where(tiny, torch.ones_like(amax), amax / 127.0)
    codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    for r in range(0, x.shape[0], 16384):
        q = (x[r:r + 16384].double() / scale[r:r + 16384, None].double()).round()
        codes[r:r + 16384] = q.masked_fill(tiny[r:r + 16384, None], 0.0).to(torch.int8)
    return codes, scale


def _plain_int8(s):
    codes, scale = _quantize(s["x"])
    y = (codes.float() @ s["w_codes"].float().t()) * (scale[:, None] * s["w_scale"][None])
    if s["bias"] is not None:
        y = y + s["bias"]
    return {"y": y.to(s["x"].dtype)}


_PLAIN = {"rotary": _plain_rotary, "rotary_tiles": _plain_tiles, "rotary_grads": _plain_grads,
          "pre": _plain_norm, "post": _plain_norm, "pre_bwd": _plain_norm_bwd, "post_bwd": _plain_norm_bwd,
          "int8": _plain_int8}


# ---------------------------------------------------------------------------------------
# the package's own calls
# ---------------------------------------------------------------------------------------

def _own_rotary(s):
    from block_sparse_attention_max_b200 import veda as V
    case = s["case"]
    inter = case["layout"] == "interleaved"
    if case["table"] == "built":
        t = V.rotary_table(s["pos"], s["inv"], s["axis"], interleaved=inter)
    else:
        t = V.RotaryTable(s["cos_sin"], inter)
    return {n: V.rotary(s[n], t, rows=s.get("rows"), inverse=case["inverse"]) for n in ("q", "k")}


def _maps(s):
    from block_sparse_attention_max_b200 import veda as V
    return V.DeviceMaps(s["tile_map"], s["tile_valid"], s["tile_segment"], s["nT_per_head"], s["N"], s["nT"],
                        s["Npad"])


def _own_tiles(s):
    from block_sparse_attention_max_b200 import veda as V
    t = V.RotaryTable(s["cos_sin"], s["case"]["layout"] == "interleaved")
    out = {}
    for n in ("q", "k"):
        out[n], out["pooled_" + n] = V.rotary_permute_pool(s[n], t, _maps(s))
    return out


def _own_grads(s):
    from block_sparse_attention_max_b200 import veda as V
    t = V.RotaryTable(s["cos_sin"], s["case"]["layout"] == "interleaved")
    return {n: V.rotary_unpermute(s[n], t, _maps(s), s["N"]) for n in ("q", "k")}


def _own_pre(s):
    from block_sparse_attention_max_b200 import veda as V
    return {"y": V.norm_modulate(s["x"], s["scale"], s["shift"], weight=s["weight"], bias=s["bias"],
                                 kind=s["case"]["kind"], eps=EPS, out_dtype=DTYPES[s["case"]["out"]])}


def _own_post(s):
    from block_sparse_attention_max_b200 import veda as V
    return {"y": V.norm_gate_add(s["x"], s["residual"], s["gate"], weight=s["weight"], bias=s["bias"],
                                 kind=s["case"]["kind"], eps=EPS, residual_scale=s["residual_scale"])}


def _named(grads, names):
    out = {}
    for n in names:
        v = getattr(grads, n)
        if v is not None:
            out[n] = v
    return out


def _own_pre_bwd(s):
    from block_sparse_attention_max_b200 import veda as V
    stats = V.NormStats(s["mean"], s["rstd"])
    gr = V.norm_modulate_bwd(s["dy"], s["x"], stats, s["scale"], weight=s["weight"], bias=s["bias"],
                             kind=s["case"]["kind"], residual_grad=s["dres"], residual_scale=s["residual_scale"])
    return _named(gr, ("dscale", "dshift", "dweight", "dbias", "dx"))


def _own_post_bwd(s):
    from block_sparse_attention_max_b200 import veda as V
    stats = V.NormStats(s["mean"], s["rstd"])
    gr = V.norm_gate_add_bwd(s["dy"], s["x"], stats, s["gate"], weight=s["weight"], bias=s["bias"],
                             kind=s["case"]["kind"])
    return _named(gr, ("dgate", "dweight", "dbias", "dx"))


def _own_int8(s):
    from block_sparse_attention_max_b200 import veda as V
    return {"y": V.int8_linear(s["x"], s["w"], bias=s["bias"])}


_OWN = {"rotary": _own_rotary, "rotary_tiles": _own_tiles, "rotary_grads": _own_grads, "pre": _own_pre,
        "post": _own_post, "pre_bwd": _own_pre_bwd, "post_bwd": _own_post_bwd, "int8": _own_int8}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------

def _turn(x, angle_cos, angle_sin, rot, half):
    """The rotation as a product of complex numbers, in 64 bits."""
    x = x.double()
    z = torch.complex(angle_cos, angle_sin)
    part = x[..., :rot]
    if half:
        v = torch.complex(part[..., :rot // 2].contiguous(), part[..., rot // 2:].contiguous()) * z
        turned = torch.cat([v.real, v.imag], -1)
    else:
        v = torch.complex(part[..., 0::2].contiguous(), part[..., 1::2].contiguous()) * z
        turned = torch.view_as_real(v).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rotary":
        if case["table"] == "built":
            a = _angles(s["pos"], s["inv"], s["axis"])
            c, sn = a.cos()[None, :, None], a.sin()[None, :, None]
        else:
            cs = s["cos_sin"].double()
            cs = cs[s["rows"].long()][:, :, None] if case["table"] == "rows" else cs[None, :, None]
            c, sn = cs[..., 0].contiguous(), cs[..., 1].contiguous()
        sn = -sn if case["inverse"] else sn
        return {n: _turn(s[n], c, sn, case["rot"], case["layout"] == "half") for n in ("q", "k")}
    if op in ("rotary_tiles", "rotary_grads"):
        half = case["layout"] == "half"
        c, sn = s["cos_sin"][..., 0].double(), s["cos_sin"][..., 1].double()
        B, H, N, nT = case["B"], case["H"], s["N"], s["nT"]
        out = {}
        for n in ("q", "k"):
            heads_t, heads_p = [], []
            for h in range(H):
                slot = (s["tile_map"][h] >= 0).nonzero()[:, 0]
                tok = s["tile_map"][h][slot].long()
                if op == "rotary_grads":
                    back = torch.zeros((B, N, 128), dtype=torch.float64, device=DEV)
                    back[:, tok] = s[n][:, h, slot].double()
                    heads_t.append(_turn(back, c[None], -sn[None], case["rot"], half))
                    continue
                y = _turn(s[n][:, :, h], c[None], sn[None], case["rot"], half)
                t = torch.zeros((B, s["Npad"], 128), dtype=torch.float64, device=DEV)
                t[:, slot] = y[:, tok]
                big = torch.full_like(t, -math.inf)
                big[:, slot] = y[:, tok]
                low = torch.full_like(t, math.inf)
                low[:, slot] = y[:, tok]
                cnt = s["tile_valid"][h].double()
                pooled = torch.stack([t.view(B, nT, 128, 128).sum(2) / cnt.clamp(min=1)[None, :, None],
                                      big.view(B, nT, 128, 128).amax(2), low.view(B, nT, 128, 128).amin(2)], 2)
                pooled[:, cnt == 0] = 0.0
                heads_t.append(t)
                heads_p.append(pooled)
            if op == "rotary_grads":
                out[n] = torch.stack(heads_t, 2)
            else:
                out[n], out["pooled_" + n] = torch.stack(heads_t, 1), torch.stack(heads_p, 1)
        return out
    if op in ("pre", "post"):
        return {"y": _norm_exact(s)}
    if op in ("pre_bwd", "post_bwd"):
        return _norm_exact_bwd(s)
    # the integer product: codes from the definition, exact sums
    x = s["x"].double()
    amax = x.abs().amax(1)
    scale = (amax / 127.0).float().double()            # the scale is an fp32 value by definition
    zero = amax < 2.0 ** -100
    scale = torch.where(zero, torch.ones_like(scale), scale)
    wt = s["w_codes"].double().t().contiguous()
    y = torch.empty((case["M"], case["N"]), dtype=torch.float64, device=DEV)
    for r in range(0, case["M"], 8192):
        codes = (x[r:r + 8192] / scale[r:r + 8192, None]).round()
        codes = torch.where(zero[r:r + 8192, None], torch.zeros_like(codes), codes)
        y[r:r + 8192] = (codes @ wt) * scale[r:r + 8192, None] * s["w_scale"].double()[None]
        if s["bias"] is not None:
            y[r:r + 8192] += s["bias"].double()
    return {"y": y}


def _row_blocks(s):
    """Batches of a norm case, a few thousand rows at a time."""
    B, N, C = s["x"].shape
    step = max(1, 40_000_000 // C)
    for b in range(B):
        for r in range(0, N, step):
            yield b, slice(r, min(N, r + step))


def _row_stats(x, kind):
    if kind == "none":
        return torch.zeros_like(x[:, :1]), torch.ones_like(x[:, :1])
    mu = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    return mu, torch.rsqrt(((x - mu) ** 2).mean(1, keepdim=True) + EPS)


def _norm_exact(s):
    case = s["case"]
    y = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
    w = s["weight"].double() if s["weight"] is not None else 1.0
    b0 = s["bias"].double() if s["bias"] is not None else 0.0
    for b, r in _row_blocks(s):
        x = s["x"][b, r].double()
        mu, rstd = _row_stats(x, case["kind"])
        a = (x - mu) * rstd * w + b0
        if case["op"] == "pre":
            y[b, r] = a + a * s["scale"][b].double() + s["shift"][b].double()
        else:
            y[b, r] = s["residual_scale"] * s["residual"][b, r].double() + s["gate"][b].double() * a
    return y


def _norm_exact_bwd(s):
    case = s["case"]
    pre = case["op"] == "pre_bwd"
    B, N, C = s["x"].shape
    w = s["weight"].double() if s["weight"] is not None else torch.ones(C, dtype=torch.float64, device=DEV)
    b0 = s["bias"].double() if s["bias"] is not None else 0.0
    z = lambda *n: torch.zeros(n, dtype=torch.float64, device=DEV)
    dx = torch.empty(s["x"].shape, dtype=torch.float64, device=DEV)
    dgain, dshift, dw, db = z(B, C), z(B, C), z(C), z(C)
    for b, r in _row_blocks(s):
        x, dy = s["x"][b, r].double(), s["dy"][b, r].double()
        mu, rstd = _row_stats(x, case["kind"])
        xh = (x - mu) * rstd
        gain = 1 + s["scale"][b].double() if pre else s["gate"][b].double()
        dgain[b] += (dy * (xh * w + b0)).sum(0)
        dshift[b] += dy.sum(0)
        dw += (dy * gain * xh).sum(0)
        db += (dy * gain).sum(0)
        g = dy * gain * w
        if case["kind"] != "none":
            g = g - xh * (g * xh).mean(1, keepdim=True) - (g.mean(1, keepdim=True) if case["kind"] == "layer" else 0.0)
            g = g * rstd
        dx[b, r] = g + (s["residual_scale"] * s["dres"][b, r].double() if pre else 0.0)
    out = {"dscale" if pre else "dgate": dgain}
    if pre:
        out["dshift"] = dshift
    if s["weight"] is not None:
        out["dweight"] = dw
        if s["bias"] is not None:
            out["dbias"] = db
    out["dx"] = dx
    return out


# ---------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    op = case["op"]
    if op == "rotary":
        rows = case["B"] * case["N"]
        n = rows * (case["H"] + case["Hk"]) * case["D"]
        table = (rows if case["table"] == "rows" else case["N"]) * case["rot"] * 4
        pos = (case["N"] * 4 * 3 if case["table"] == "built" else table) + (rows * 4 if case["table"] == "rows" else 0)
        return {"bytes": 2 * n * size[case["dtype"]] + pos, "flops": 3 * n * case["rot"] // case["D"]}
    if op in ("rotary_tiles", "rotary_grads"):
        N = case["grid_t"] * case["grid_h"] * case["grid_w"] + case["tail"]
        nT = (-(-case["grid_t"] // case["tile_t"]) * -(-case["grid_h"] // case["tile_h"])
              * -(-case["grid_w"] // case["tile_w"]) + -(-case["tail"] // 128))
        bh = case["B"] * case["H"]
        common = 2 * case["H"] * (nT * 128 if case["shuffle"] else N) * 4 + N * case["rot"] * 4
        if op == "rotary_tiles":
            b = 2 * bh * (N * 256 + nT * 128 * 256 + nT * 3 * 128 * 4)
        else:
            b = 2 * bh * 2 * N * 256
        return {"bytes": b + common, "flops": 2 * bh * N * (3 * case["rot"] + (4 * 128 if op == "rotary_tiles" else 0))}
    if op in ("pre", "post", "pre_bwd", "post_bwd"):
        n = case["B"] * case["N"] * case["C"]
        x, o, p = size[case["dtype"]], size[case["out"]], size[case["pdtype"]]
        params = case["C"] * p * ((2 if op.startswith("pre") else 1) * case["B"] + 2 * case["affine"])
        per = {"pre": x + o, "post": x + 2 * o, "pre_bwd": o + 3 * x, "post_bwd": o + 2 * x}[op]
        grads = 4 * case["C"] * (2 * case["B"] + 2) if op.endswith("bwd") else 0
        return {"bytes": n * per + params + grads, "flops": n * (16 if op.endswith("bwd") else 8)}
    M, N, K, e = case["M"], case["N"], case["K"], size[case["dtype"]]
    return {"bytes": M * K * e + N * K + M * N * e + N * 8, "flops": 2 * M * N * K}
