"""ctypes binding of libveda.so (include/veda.h) -- argument marshalling only.

Every step of the path runs in the library's CUDA kernels; this module only turns
torch tensors into pointers and sizes, allocates outputs with torch, and raises when
a call returns an error. There is no fallback: if the library is missing or the device
is not a B200 (compute capability 10.0), calls raise.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct
from typing import List, Optional, Sequence, Tuple

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libveda.so")

VEDA_OK = 0
STATUS_NAMES = {0: "VEDA_OK", 1: "VEDA_ERR_INVALID_ARG", 2: "VEDA_ERR_UNSUPPORTED",
                3: "VEDA_ERR_CUDA", 4: "VEDA_ERR_TIMEOUT", 5: "VEDA_ERR_DEVICE_CHECK"}

EXPORTED = (
    "veda_abi_version", "veda_status_string", "veda_last_error", "veda_geometry_sizes",
    "veda_build_tile_map", "veda_permute_tiles", "veda_permute_pool", "veda_tile_pool",
    "veda_block_scores_workspace_bytes", "veda_block_scores", "veda_block_scores_noalloc",
    "veda_select_blocks",
    "veda_block_sparse_attn_fwd", "veda_unpermute", "veda_transpose_lists",
    "veda_block_sparse_attn_bwd", "veda_block_heat", "veda_mask_quality", "veda_rel_error",
    "veda_tile_plan_vote",
    "veda_quantize_fp8", "veda_block_sparse_attn_fwd_fp8",
    "veda_rotary_table", "veda_rotary", "veda_rotary_permute_pool", "veda_rotary_unpermute",
    "veda_norm_fwd", "veda_norm_bwd_workspace_bytes", "veda_norm_bwd",
    "veda_quantize_int8", "veda_int8_matmul", "veda_int8_linear_workspace_bytes", "veda_int8_linear",
    "veda_check_device_status", "veda_selftest_wait_timeout",
)


class VedaError(RuntimeError):
    def __init__(self, call: str, status: int, message: str):
        super().__init__(f"{call} -> {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class TileShape(ctypes.Structure):
    _fields_ = [("t", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32)]


class Geometry(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("T", ctypes.c_int32), ("Hg", ctypes.c_int32),
                ("Wg", ctypes.c_int32), ("n_tail", ctypes.c_int32),
                ("head_shape", ctypes.POINTER(TileShape)),
                ("tile_order", ctypes.POINTER(ctypes.c_int32)),
                ("order_stride", ctypes.c_int32)]


# veda_rows and veda_norm_params as packed bytes (a third of a ctypes.Structure's cost per call)
_ROWS = struct.Struct("@Pqqi4x")            # data, batch_stride, row_stride, dtype
_NORM_PARAMS = struct.Struct("@PPPPqqiif4x")  # weight, bias, gain, shift, 2 strides, 2 types, gain_offset
_STRIDES3 = struct.Struct("@qqq")

_lib = None

_P = ctypes.c_void_p
_L = ctypes.c_int64
_D = ctypes.c_double
_Z = ctypes.c_size_t
_I = ctypes.c_int32
_F = ctypes.c_float
_SIG = {
    "veda_abi_version": (_I, []),
    "veda_status_string": (ctypes.c_char_p, [_I]),
    "veda_last_error": (ctypes.c_char_p, []),
    "veda_geometry_sizes": (_I, [ctypes.POINTER(Geometry), _P, _P, _P]),
    "veda_build_tile_map": (_I, [ctypes.POINTER(Geometry), _P, _P, _P, _P]),
    "veda_permute_tiles": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "veda_tile_pool": (_I, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "veda_permute_pool": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "veda_block_scores_workspace_bytes": (ctypes.c_size_t, [_I, _I, _I, _I]),
    "veda_block_scores": (_I, [_P, _P, _P, _P, _P, _P, ctypes.c_size_t, _I, _I, _I, _I, _P]),
    "veda_block_scores_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "veda_select_blocks": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "veda_block_sparse_attn_fwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _F, _P, _P, _I, _I,
                                        _I, _I, _P]),
    "veda_unpermute": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "veda_quantize_fp8": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "veda_block_sparse_attn_fwd_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _F, _P, _P,
                                            _I, _I, _I, _I, _P]),
    "veda_transpose_lists": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P]),
    "veda_block_sparse_attn_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I,
                                        _F, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "veda_rel_error": (_I, [_P, _P, _P, _I, _I, _I, _I, _P]),
    "veda_tile_plan_vote": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "veda_block_heat": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _F, _P, _I, _I, _I, _I, _P]),
    "veda_mask_quality": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _P, _P,
                               _I, _I, _I, _P]),
    "veda_rotary_table": (_I, [_P, _I, _L, _P, _P, _I, _D, _P, _P]),
    "veda_rotary": (_I, [_P, _P, _P, _P, _I, _P, _L, _P, _I, _I, _I, _I, _I, _I, _I, _P]),
    "veda_rotary_permute_pool": (_I, [_P, _P, _P, _L, _I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "veda_rotary_unpermute": (_I, [_P, _P, _P, _L, _I, _I, _I, _P, _I, _I, _I, _I, _I, _P]),
    "veda_norm_fwd": (_I, [_P, _P, _P, _P, _F, _P, _P, _I, _I, _I, _I, _F, _P]),
    "veda_norm_bwd_workspace_bytes": (_Z, [_I, _I, _I]),
    "veda_norm_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _P, _Z, _I, _I, _I, _I, _P]),
    "veda_quantize_int8": (_I, [_P, _L, _I, _P, _P, _L, _I, _P]),
    "veda_int8_matmul": (_I, [_P, _P, _P, _P, _P, _P, _L, _I, _I, _I, _I, _P]),
    "veda_int8_linear_workspace_bytes": (_Z, [_I, _I]),
    "veda_int8_linear": (_I, [_P, _L, _I, _P, _P, _P, _P, _L, _I, _P, _Z, _I, _I, _I, _P]),
    "veda_check_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_uint32)]),
    "veda_selftest_wait_timeout": (_I, [ctypes.c_uint32, _P]),
}


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if libveda.so has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m block_sparse_attention_max_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIG.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(call: str, status: int) -> None:
    if status != VEDA_OK:
        msg = lib().veda_last_error().decode(errors="replace")
        raise VedaError(call, status, msg)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _here(t: torch.Tensor) -> bool:
    """On the calling thread's current device (where the library launches)."""
    return t.is_cuda and t.get_device() == torch._C._cuda_getDevice()


def _need(t: torch.Tensor, dtype: torch.dtype, name: str, cuda: bool = True,
          shape: Optional[Sequence[int]] = None) -> None:
    """Type, shape, layout and device of a tensor handed to the library: a wrong shape would
    send a kernel outside the buffer, so every one is checked before its pointer is passed."""
    if t.dtype is dtype and t.is_contiguous() and (shape is None or t.shape == shape) and (not cuda or _here(t)):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name}: expected shape {tuple(int(x) for x in shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if cuda and t.device.index != torch.cuda.current_device():
        # the library launches on the calling thread's current device
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _need_maps(maps: "DeviceMaps", H: int, Npad: int, cuda: bool = True) -> None:
    """The device tile map of H heads with Npad slots each (and its per-tile arrays)."""
    if maps.Npad != Npad or maps.nT * 128 != Npad:
        raise ValueError(f"tile map of {maps.Npad} slots per head, tensors have {Npad}")
    _need(maps.tile_map, torch.int32, "tile_map", cuda, shape=(H, Npad))
    for t, n in ((maps.tile_valid, "tile_valid"), (maps.tile_segment, "tile_segment")):
        _need(t, torch.int32, n, cuda, shape=(H, Npad // 128))
    _need(maps.nT_per_head, torch.int32, "nT_per_head", cuda, shape=(H,))


def _need_tokens(maps: "DeviceMaps", N: int) -> None:
    """A buffer made for N raster tokens is written where the map has a token and nowhere else."""
    if N != maps.N:
        raise ValueError(f"the tile map has {maps.N} tokens, the call {N}")


def _need_lists(lists: "BlockLists", B: int, H: int, nT: int, name: str = "lists", cuda: bool = True) -> None:
    """Block lists of a [B, H, nT] problem: counts [B, H, nT], indices [B, H, nT, stride]."""
    if not 0 < lists.stride <= nT:
        raise ValueError(f"{name}: stride {lists.stride} outside [1, {nT}]")
    for t, n in ((lists.full_cnt, "full_cnt"), (lists.part_cnt, "part_cnt")):
        _need(t, torch.int32, f"{name}.{n}", cuda, shape=(B, H, nT))
    for t, n in ((lists.full_idx, "full_idx"), (lists.part_idx, "part_idx")):
        _need(t, torch.int32, f"{name}.{n}", cuda, shape=(B, H, nT, lists.stride))


# ---------------------------------------------------------------------------------------
# geometry (host)
# ---------------------------------------------------------------------------------------

@dataclasses.dataclass
class TileMaps:
    """Host tile maps of one geometry (numpy int32)."""
    tile_map: np.ndarray       # [H, Npad]
    tile_valid: np.ndarray     # [H, nT]
    tile_segment: np.ndarray   # [H, nT]
    nT_per_head: np.ndarray    # [H]
    N: int
    nT: int
    Npad: int

    def to(self, device) -> "DeviceMaps":
        f = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
        return DeviceMaps(f(self.tile_map), f(self.tile_valid), f(self.tile_segment),
                          f(self.nT_per_head), self.N, self.nT, self.Npad)


@dataclasses.dataclass
class DeviceMaps:
    tile_map: torch.Tensor
    tile_valid: torch.Tensor
    tile_segment: torch.Tensor
    nT_per_head: torch.Tensor
    N: int
    nT: int
    Npad: int


def _geometry(grid, head_shapes, n_tail, tile_order):
    H = len(head_shapes)
    shapes = (TileShape * H)(*[TileShape(*map(int, s)) for s in head_shapes])
    keep = [shapes]
    g = Geometry(H, int(grid[0]), int(grid[1]), int(grid[2]), int(n_tail), shapes, None, 0)
    if tile_order is not None:
        order = np.ascontiguousarray(np.asarray(tile_order, dtype=np.int32))
        keep.append(order)
        g.tile_order = order.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        g.order_stride = order.shape[1]
    return g, keep


def geometry_sizes(grid, head_shapes, n_tail=0) -> Tuple[int, int, int]:
    g, _keep = _geometry(grid, head_shapes, n_tail, None)
    N, nT, Npad = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check("veda_geometry_sizes", lib().veda_geometry_sizes(
        ctypes.byref(g), ctypes.addressof(N), ctypes.addressof(nT), ctypes.addressof(Npad)))
    return N.value, nT.value, Npad.value


def build_tile_map(grid, head_shapes, n_tail=0, tile_order=None) -> TileMaps:
    g, _keep = _geometry(grid, head_shapes, n_tail, tile_order)
    N, nT, Npad = geometry_sizes(grid, head_shapes, n_tail)
    H = len(head_shapes)
    tm = np.empty((H, Npad), np.int32)
    tv = np.empty((H, nT), np.int32)
    ts = np.empty((H, nT), np.int32)
    nph = np.empty((H,), np.int32)
    _check("veda_build_tile_map", lib().veda_build_tile_map(
        ctypes.byref(g), tm.ctypes.data, tv.ctypes.data, ts.ctypes.data, nph.ctypes.data))
    return TileMaps(tm, tv, ts, nph, N, nT, Npad)


# ---------------------------------------------------------------------------------------
# device steps
# ---------------------------------------------------------------------------------------

def permute_tiles(x: torch.Tensor, maps: DeviceMaps, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    _need(x, torch.bfloat16, "x")
    B, N, H, D = x.shape
    _need_maps(maps, H, maps.Npad)
    if out is None:
        out = torch.empty((B, H, maps.Npad, D), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out", shape=(B, H, maps.Npad, D))
    _check("veda_permute_tiles", lib().veda_permute_tiles(
        _ptr(x), _ptr(out), _ptr(maps.tile_map), B, N, H, D, maps.Npad, _stream(stream)))
    return out


def permute_pool(x: torch.Tensor, maps: DeviceMaps, out: Optional[torch.Tensor] = None,
                 pooled: Optional[torch.Tensor] = None, stream=None):
    """veda_permute_pool: the tile gather and the tile pooling in one pass."""
    _need(x, torch.bfloat16, "x")
    B, N, H, D = x.shape
    _need_maps(maps, H, maps.Npad)
    if out is None:
        out = torch.empty((B, H, maps.Npad, D), dtype=torch.bfloat16, device=x.device)
    if pooled is None:
        pooled = torch.empty((B, H, maps.Npad // 128, 3, D), dtype=torch.float32, device=x.device)
    _need(out, torch.bfloat16, "out", shape=(B, H, maps.Npad, D))
    _need(pooled, torch.float32, "pooled", shape=(B, H, maps.Npad // 128, 3, D))
    _check("veda_permute_pool", lib().veda_permute_pool(
        _ptr(x), _ptr(out), _ptr(maps.tile_map), _ptr(maps.tile_valid), _ptr(pooled), B, N, H, D,
        maps.Npad, _stream(stream)))
    return out, pooled


def tile_pool(x_tiled: torch.Tensor, maps: DeviceMaps, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    _need(x_tiled, torch.bfloat16, "x_tiled")
    B, H, Npad, D = x_tiled.shape
    nT = Npad // 128
    _need_maps(maps, H, Npad)
    if out is None:
        out = torch.empty((B, H, nT, 3, D), dtype=torch.float32, device=x_tiled.device)
    _need(out, torch.float32, "out", shape=(B, H, nT, 3, D))
    _check("veda_tile_pool", lib().veda_tile_pool(
        _ptr(x_tiled), _ptr(maps.tile_valid), _ptr(out), B, H, nT, D, _stream(stream)))
    return out


def block_scores_workspace_bytes(B: int, H: int, nT: int, D: int = 128) -> int:
    return int(lib().veda_block_scores_workspace_bytes(B, H, nT, D))


def block_scores(pooled_q: torch.Tensor, pooled_k: torch.Tensor, wq: torch.Tensor,
                 wk: torch.Tensor, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _need(pooled_q, torch.float32, "pooled_q")
    B, H, nT, three, D = pooled_q.shape
    if three != 3:
        raise ValueError("pooled_q: expected shape [B, H, nT, 3, D]")
    _need(pooled_k, torch.float32, "pooled_k", shape=pooled_q.shape)
    for t, n in ((wq, "wq"), (wk, "wk")):
        _need(t, torch.float32, n, shape=(H, D, 3 * D))
    if out is None:
        out = torch.empty((B, H, nT, nT), dtype=torch.float32, device=pooled_q.device)
    _need(out, torch.float32, "out", shape=(B, H, nT, nT))
    nbytes = block_scores_workspace_bytes(B, H, nT, D)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=pooled_q.device)
    _need(workspace, workspace.dtype, "workspace")
    _check("veda_block_scores", lib().veda_block_scores(
        _ptr(pooled_q), _ptr(pooled_k), _ptr(wq), _ptr(wk), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), B, H, nT, D, _stream(stream)))
    return out


def block_scores_noalloc(pooled_q: torch.Tensor, pooled_k: torch.Tensor, wq: torch.Tensor,
                         wk: torch.Tensor, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """veda_block_scores_noalloc: same result as block_scores, scratch built into the library.

    For callers that may not allocate device memory (see include/veda.h); ``out`` should
    then be passed in. Calls sharing a device must not overlap on the GPU.
    """
    for t, n in ((pooled_q, "pooled_q"), (pooled_k, "pooled_k"), (wq, "wq"), (wk, "wk")):
        _need(t, torch.float32, n)
    B, H, nT, three, D = pooled_q.shape
    if three != 3 or tuple(pooled_k.shape) != tuple(pooled_q.shape):
        raise ValueError("pooled_q / pooled_k: expected equal shapes [B, H, nT, 3, D]")
    for t, n in ((wq, "wq"), (wk, "wk")):
        if tuple(t.shape) != (H, D, 3 * D):
            raise ValueError(f"{n}: expected shape {(H, D, 3 * D)}, got {tuple(t.shape)}")
    if out is None:
        out = torch.empty((B, H, nT, nT), dtype=torch.float32, device=pooled_q.device)
    _need(out, torch.float32, "out")
    if tuple(out.shape) != (B, H, nT, nT):
        raise ValueError(f"out: expected shape {(B, H, nT, nT)}, got {tuple(out.shape)}")
    _check("veda_block_scores_noalloc", lib().veda_block_scores_noalloc(
        _ptr(pooled_q), _ptr(pooled_k), _ptr(wq), _ptr(wk), _ptr(out), B, H, nT, D,
        _stream(stream)))
    return out


def list_stride_for(nT: int, rho: Sequence[Tuple[int, int]]) -> int:
    """Smallest list_stride veda_select_blocks accepts for these densities."""
    bound = 1 + sum(-(-nT * p // q) for p, q in rho)
    return min(nT, bound)


@dataclasses.dataclass
class BlockLists:
    full_cnt: torch.Tensor    # [B, H, nT] int32
    full_idx: torch.Tensor    # [B, H, nT, stride] int32
    part_cnt: torch.Tensor
    part_idx: torch.Tensor
    stride: int


def select_blocks(scores: torch.Tensor, maps: DeviceMaps, rho: Sequence[Tuple[int, int]],
                  list_stride: Optional[int] = None, out: Optional[BlockLists] = None,
                  stream=None) -> BlockLists:
    _need(scores, torch.float32, "scores")
    B, H, nT, nT2 = scores.shape
    if nT2 != nT:
        raise ValueError("scores: expected shape [B, H, nT, nT]")
    _need_maps(maps, H, nT * 128)
    stride = list_stride or list_stride_for(nT, rho)
    if out is None:
        dev = scores.device
        out = BlockLists(torch.empty((B, H, nT), dtype=torch.int32, device=dev),
                         torch.zeros((B, H, nT, stride), dtype=torch.int32, device=dev),
                         torch.empty((B, H, nT), dtype=torch.int32, device=dev),
                         torch.zeros((B, H, nT, stride), dtype=torch.int32, device=dev), stride)
    _need_lists(out, B, H, nT, "out")
    num = (ctypes.c_int32 * len(rho))(*[int(p) for p, _ in rho])
    den = (ctypes.c_int32 * len(rho))(*[int(q) for _, q in rho])
    _check("veda_select_blocks", lib().veda_select_blocks(
        _ptr(scores), _ptr(maps.tile_valid), _ptr(maps.tile_segment), _ptr(maps.nT_per_head),
        len(rho), ctypes.addressof(num), ctypes.addressof(den), _ptr(out.full_cnt),
        _ptr(out.full_idx), _ptr(out.part_cnt), _ptr(out.part_idx), out.stride, B, H, nT,
        _stream(stream)))
    return out


def block_sparse_attn_fwd(q_t: torch.Tensor, k_t: torch.Tensor, v_t: torch.Tensor,
                          maps: DeviceMaps, lists: BlockLists, scale: float,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          want_lse: bool = True, stream=None):
    _need(q_t, torch.bfloat16, "q")
    B, H, Npad, D = q_t.shape
    nT = Npad // 128
    for t, n in ((k_t, "k"), (v_t, "v")):
        _need(t, torch.bfloat16, n, shape=q_t.shape)
    _need_maps(maps, H, Npad)
    _need_lists(lists, B, H, nT)
    if out is None:
        out = torch.empty_like(q_t)
    if lse is None and want_lse:
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=q_t.device)
    _need(out, torch.bfloat16, "out", shape=q_t.shape)
    if lse is not None:
        _need(lse, torch.float32, "lse", shape=(B, H, Npad))
    _check("veda_block_sparse_attn_fwd", lib().veda_block_sparse_attn_fwd(
        _ptr(q_t), _ptr(k_t), _ptr(v_t), _ptr(maps.tile_valid), _ptr(lists.full_cnt),
        _ptr(lists.full_idx), _ptr(lists.part_cnt), _ptr(lists.part_idx), lists.stride,
        float(scale), _ptr(out), _ptr(lse), B, H, nT, D, _stream(stream)))
    return out, lse


def quantize_fp8(x_t: torch.Tensor, transpose_tiles: bool = False, codes: Optional[torch.Tensor] = None,
                 scale: Optional[torch.Tensor] = None, stream=None):
    """Tiled bf16 [B, H, Npad, 128] -> (e4m3 codes uint8 [B, H, Npad, 128], scale fp32 [B, H]);
    with transpose_tiles every 128 x 128 tile of the codes is stored transposed, keys in the
    order veda_quantize_fp8 documents (V of the FP8 attention)."""
    _need(x_t, torch.bfloat16, "x_t")
    B, H, Npad, D = x_t.shape
    if codes is None:
        codes = torch.empty((B, H, Npad, D), dtype=torch.uint8, device=x_t.device)
    if scale is None:
        scale = torch.empty((B, H), dtype=torch.float32, device=x_t.device)
    _need(codes, torch.uint8, "codes", shape=(B, H, Npad, D))
    _need(scale, torch.float32, "scale", shape=(B, H))
    _check("veda_quantize_fp8", lib().veda_quantize_fp8(
        _ptr(x_t), _ptr(codes), _ptr(scale), B, H, Npad // 128, D, 1 if transpose_tiles else 0, _stream(stream)))
    return codes, scale


def block_sparse_attn_fwd_fp8(q8: torch.Tensor, k8: torch.Tensor, vt8: torch.Tensor, q_scale: torch.Tensor,
                              k_scale: torch.Tensor, v_scale: torch.Tensor, maps: DeviceMaps, lists: BlockLists,
                              scale: float, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                              want_lse: bool = True, stream=None):
    """FP8 variant of the attention step: e4m3 codes of Q, K and (transposed tiles) V with
    their per-(batch, head) scales -> bf16 O [B, H, Npad, 128] and fp32 LSE."""
    _need(q8, torch.uint8, "q8")
    B, H, Npad, D = q8.shape
    nT = Npad // 128
    for t, n in ((k8, "k8"), (vt8, "vt8")):
        _need(t, torch.uint8, n, shape=q8.shape)
    for t, n in ((q_scale, "q_scale"), (k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, torch.float32, n, shape=(B, H))
    _need_maps(maps, H, Npad)
    _need_lists(lists, B, H, nT)
    if out is None:
        out = torch.empty((B, H, Npad, D), dtype=torch.bfloat16, device=q8.device)
    if lse is None and want_lse:
        lse = torch.empty((B, H, Npad), dtype=torch.float32, device=q8.device)
    _need(out, torch.bfloat16, "out", shape=(B, H, Npad, D))
    if lse is not None:
        _need(lse, torch.float32, "lse", shape=(B, H, Npad))
    _check("veda_block_sparse_attn_fwd_fp8", lib().veda_block_sparse_attn_fwd_fp8(
        _ptr(q8), _ptr(k8), _ptr(vt8), _ptr(q_scale), _ptr(k_scale), _ptr(v_scale), _ptr(maps.tile_valid),
        _ptr(lists.full_cnt), _ptr(lists.full_idx), _ptr(lists.part_cnt), _ptr(lists.part_idx), lists.stride,
        float(scale), _ptr(out), _ptr(lse), B, H, nT, D, _stream(stream)))
    return out, lse


@dataclasses.dataclass
class TransposedLists:
    cnt: torch.Tensor    # [B, H, nT] int32: query tiles per key tile
    idx: torch.Tensor    # [B, H, nT, stride] int32, ascending
    stride: int


def transpose_lists(lists: BlockLists, maps: DeviceMaps, stream=None) -> TransposedLists:
    """veda_transpose_lists: the query tiles of every key tile (the backward's lists)."""
    B, H, nT = lists.full_cnt.shape
    _need_lists(lists, B, H, nT)
    _need_maps(maps, H, nT * 128)
    dev = lists.full_cnt.device
    t = TransposedLists(torch.empty((B, H, nT), dtype=torch.int32, device=dev),
                        torch.zeros((B, H, nT, nT), dtype=torch.int32, device=dev), nT)
    _check("veda_transpose_lists", lib().veda_transpose_lists(
        _ptr(lists.full_cnt), _ptr(lists.full_idx), _ptr(lists.part_cnt), _ptr(lists.part_idx),
        lists.stride, _ptr(maps.nT_per_head), _ptr(t.cnt), _ptr(t.idx), t.stride, B, H, nT,
        _stream(stream)))
    return t


def block_sparse_attn_bwd(q_t: torch.Tensor, k_t: torch.Tensor, v_t: torch.Tensor, o_t: torch.Tensor,
                          do_t: torch.Tensor, lse: torch.Tensor, maps: DeviceMaps, lists: BlockLists,
                          tlists: TransposedLists, scale: float, stream=None):
    """veda_block_sparse_attn_bwd: dQ, dK, dV (tile order, bf16) over the forward's lists."""
    _need(q_t, torch.bfloat16, "q")
    B, H, Npad, D = q_t.shape
    nT = Npad // 128
    for t, n in ((k_t, "k"), (v_t, "v"), (o_t, "o"), (do_t, "dout")):
        _need(t, torch.bfloat16, n, shape=q_t.shape)
    _need(lse, torch.float32, "lse", shape=(B, H, Npad))
    _need_maps(maps, H, Npad)
    _need_lists(lists, B, H, nT)
    if tlists.stride != nT:
        raise ValueError(f"tlists: stride {tlists.stride}, expected {nT}")
    _need(tlists.cnt, torch.int32, "tlists.cnt", shape=(B, H, nT))
    _need(tlists.idx, torch.int32, "tlists.idx", shape=(B, H, nT, nT))
    dq, dk, dv = torch.empty_like(q_t), torch.empty_like(k_t), torch.empty_like(v_t)
    delta = torch.empty(B * H * Npad + 4, dtype=torch.float32, device=q_t.device)   # D + work counters
    _check("veda_block_sparse_attn_bwd", lib().veda_block_sparse_attn_bwd(
        _ptr(q_t), _ptr(k_t), _ptr(v_t), _ptr(o_t), _ptr(do_t), _ptr(lse), _ptr(maps.tile_valid),
        _ptr(lists.full_cnt), _ptr(lists.full_idx), _ptr(lists.part_cnt), _ptr(lists.part_idx),
        lists.stride, _ptr(tlists.cnt), _ptr(tlists.idx), tlists.stride, float(scale), _ptr(dq),
        _ptr(dk), _ptr(dv), _ptr(delta), B, H, nT, D, _stream(stream)))
    return dq, dk, dv


def block_heat(q_t: torch.Tensor, k_t: torch.Tensor, maps: DeviceMaps, lists: BlockLists,
               lse: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """veda_block_heat: per-block attention mass against the given (dense) LSE."""
    _need(q_t, torch.bfloat16, "q")
    B, H, Npad, D = q_t.shape
    nT = Npad // 128
    _need(k_t, torch.bfloat16, "k", shape=q_t.shape)
    _need(lse, torch.float32, "lse", shape=(B, H, Npad))
    _need_maps(maps, H, Npad)
    _need_lists(lists, B, H, nT)
    if out is None:
        out = torch.empty((B, H, nT, nT), dtype=torch.float32, device=q_t.device)
    _need(out, torch.float32, "out", shape=(B, H, nT, nT))
    _check("veda_block_heat", lib().veda_block_heat(
        _ptr(q_t), _ptr(k_t), _ptr(maps.tile_valid), _ptr(lists.full_cnt), _ptr(lists.full_idx),
        _ptr(lists.part_cnt), _ptr(lists.part_idx), lists.stride, _ptr(lse), float(scale),
        _ptr(out), B, H, nT, D, _stream(stream)))
    return out


@dataclasses.dataclass
class MaskQuality:
    mass_rows: torch.Tensor     # [B, H, nT] heat kept per query tile
    recall_rows: torch.Tensor   # [B, H, nT] |pred & oracle| / |oracle|
    totals: torch.Tensor        # [4] see veda_mask_quality

    @property
    def mass(self) -> float:
        """Attention mass the mask keeps, over valid query slots."""
        t = self.totals.tolist()
        return t[0] / t[1] if t[1] else 0.0

    @property
    def recall(self) -> float:
        """Mean block recall against the oracle mask."""
        t = self.totals.tolist()
        return t[2] / t[3] if t[3] else 0.0


def mask_quality(heat: torch.Tensor, maps: DeviceMaps, pred: BlockLists, oracle: BlockLists,
                 stream=None) -> MaskQuality:
    """veda_mask_quality: kept attention mass of `pred` and its recall against `oracle`."""
    _need(heat, torch.float32, "heat")
    B, H, nT, nT2 = heat.shape
    if nT2 != nT:
        raise ValueError("heat: expected shape [B, H, nT, nT]")
    _need_maps(maps, H, nT * 128)
    _need_lists(pred, B, H, nT, "pred")
    _need_lists(oracle, B, H, nT, "oracle")
    dev = heat.device
    q = MaskQuality(torch.empty((B, H, nT), dtype=torch.float32, device=dev),
                    torch.empty((B, H, nT), dtype=torch.float32, device=dev),
                    torch.empty(4, dtype=torch.float32, device=dev))
    _check("veda_mask_quality", lib().veda_mask_quality(
        _ptr(heat), _ptr(maps.tile_valid), _ptr(maps.nT_per_head), _ptr(pred.full_cnt),
        _ptr(pred.full_idx), _ptr(pred.part_cnt), _ptr(pred.part_idx), pred.stride,
        _ptr(oracle.full_cnt), _ptr(oracle.full_idx), _ptr(oracle.part_cnt), _ptr(oracle.part_idx),
        oracle.stride, _ptr(q.mass_rows), _ptr(q.recall_rows), _ptr(q.totals), B, H, nT,
        _stream(stream)))
    return q


def rel_error(o: torch.Tensor, o_ref: torch.Tensor, stream=None) -> torch.Tensor:
    """veda_rel_error: [H, 2] sums of |o - o_ref|^2 and |o_ref|^2 per head (raster bf16)."""
    _need(o, torch.bfloat16, "o")
    _need(o_ref, torch.bfloat16, "o_ref", shape=o.shape)
    B, N, H, D = o.shape
    sums = torch.empty((H, 2), dtype=torch.float32, device=o.device)
    _check("veda_rel_error", lib().veda_rel_error(_ptr(o), _ptr(o_ref), _ptr(sums), B, N, H, D,
                                                  _stream(stream)))
    return sums


def tile_plan_vote(errors: np.ndarray, max_shapes: int = 2) -> Tuple[List[int], np.ndarray]:
    """veda_tile_plan_vote (host): the kept candidates (ascending) and each head's candidate
    from an [H, C] matrix of relative output errors."""
    err = np.ascontiguousarray(errors, dtype=np.float64)
    if err.ndim != 2:
        raise ValueError("errors: expected [H, C]")
    H, C = err.shape
    kept = np.zeros(max(1, min(max_shapes, C)), np.int32)
    n_kept = np.zeros(1, np.int32)
    assign = np.zeros(H, np.int32)
    _check("veda_tile_plan_vote", lib().veda_tile_plan_vote(
        err.ctypes.data, H, C, max_shapes, kept.ctypes.data, n_kept.ctypes.data, assign.ctypes.data))
    return [int(c) for c in kept[:int(n_kept[0])]], assign


def unpermute(o_t: torch.Tensor, maps: DeviceMaps, N: int, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    _need(o_t, torch.bfloat16, "o_tiled")
    B, H, Npad, D = o_t.shape
    _need_maps(maps, H, Npad)
    if out is None:
        out = torch.empty((B, N, H, D), dtype=torch.bfloat16, device=o_t.device)
    _need(out, torch.bfloat16, "out", shape=(B, N, H, D))
    _check("veda_unpermute", lib().veda_unpermute(
        _ptr(o_t), _ptr(out), _ptr(maps.tile_map), B, N, H, D, Npad, _stream(stream)))
    return out


# ---------------------------------------------------------------------------------------
# the block around the attention: rotary positions, norms, 8-bit integer projections
# ---------------------------------------------------------------------------------------

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_KIND = {"layer": 0, "rms": 1, "none": 2}


def _fits(name: str, shape: Sequence[int]) -> None:
    """Sizes the library takes in 32 bits: a larger one would arrive as its remainder."""
    if max(shape, default=0) > 0x7fffffff:
        raise ValueError(f"{name}: sizes of 2^31 and more are not supported, got {tuple(shape)}")


def _need_strided(t: torch.Tensor, name: str, ndim: int, dtype: Optional[torch.dtype] = None,
                  shape: Optional[Sequence[int]] = None, written: bool = False) -> None:
    """Checks of a tensor whose leading dimensions may have any stride: type, shape, device,
    contiguous channels, and, where the library writes it, no two elements in one place."""
    if ((t.dtype is dtype or dtype is None and t.dtype in _DTYPE) and t.dim() == ndim and (shape is None or t.shape == shape)
            and (t.is_contiguous() or not written and t.stride(-1) == 1) and _here(t)):
        return
    if dtype is None and t.dtype not in _DTYPE:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got shape {tuple(t.shape)}")
    if shape is not None and tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name}: expected shape {tuple(int(x) for x in shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    if written and t.numel() > 0 and not t.is_contiguous():
        extent = 1
        for st, n in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n > 1):
            if st < extent:
                raise ValueError(f"{name}: elements overlap in memory")
            extent = st * (n - 1) + extent


def _separate(out: torch.Tensor, t: Optional[torch.Tensor], name: str, same_ok: bool, what: str = "out") -> None:
    """out may be t itself (where same_ok), else they must not share memory."""
    if t is None or out.numel() == 0 or t.numel() == 0:
        return
    if (out.data_ptr() == t.data_ptr() and out.shape == t.shape and out.dtype == t.dtype
            and all(a == b for a, b, n in zip(out.stride(), t.stride(), out.shape) if n > 1)):
        if same_ok:
            return
        raise ValueError(f"{what} must not be {name}")
    a, b = _span(out), _span(t)
    if a[0] < b[1] and b[0] < a[1] and not _apart(out, t):
        raise ValueError(f"{what} overlaps {name} in memory")


def _separate_all(out: torch.Tensor, what: str, *others: Tuple[Optional[torch.Tensor], str]) -> None:
    """A written buffer against the named others (None: not there)."""
    for t, name in others:
        _separate(out, t, name, False, what)


def _span(t: torch.Tensor) -> Tuple[int, int]:
    """First byte and one past the last byte of a tensor's elements."""
    n = t.numel() if t.is_contiguous() else 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + t.element_size() * n


def _apart(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether two tensors are seen to share no byte although their spans meet, as slices of one buffer
    do: for some stride S of either, dimensions whose stride is a multiple of S leave an address's
    remainder by S alone, and the others' extents are two separate pieces of the circle of remainders."""
    dims = [[(n, st * t.element_size()) for n, st in zip(t.shape, t.stride()) if n > 1] for t in (a, b)]
    for S in {st for d in dims for _, st in d if st > 0}:
        ea, eb = (t.element_size() + sum((n - 1) * st for n, st in d if st % S) for t, d in zip((a, b), dims))
        gap = (b.data_ptr() - a.data_ptr()) % S
        if gap >= ea and gap + eb <= S:
            return True
    return False


def _new(like: torch.Tensor, shape, dtype: torch.dtype, stream) -> torch.Tensor:
    """A buffer beside `like` for work on `stream` (None: the current one): taken from that stream's
    memory, and kept from reuse until what the current stream does with it later has run."""
    if stream is None:
        if dtype is not like.dtype:
            return like.new_empty(shape, dtype=dtype)
        return torch.empty_like(like) if shape == like.shape and like.is_contiguous() else like.new_empty(shape)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream())
    return t


@dataclasses.dataclass
class RotaryFrequencies:
    """Pairs of a rotated head: inverse frequency (fp64) and position axis of each, and the
    amplitude of the turned vectors."""
    inv_freq: np.ndarray
    axis: np.ndarray
    amplitude: float = 1.0


def rotary_frequencies(dims, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0) -> RotaryFrequencies:
    """Frequencies theta^(-2 i / d), i < d / 2, for the d channels of each position axis (``dims``:
    an even count per axis, e.g. (44, 42, 42) for time, height and width; an int for one axis).

    Scalings for contexts ``factor`` times as long as trained on: ``linear`` divides every
    frequency by the factor (position interpolation); ``ntk`` raises theta to
    theta * factor^(d / (d - 2)), which keeps the fastest pair and slows the slowest by the factor;
    ``yarn`` (Peng et al., "YaRN: Efficient Context Window Extension of Large Language Models")
    keeps the pairs that turn more than beta_fast times within original_length, divides those that
    turn less than beta_slow times by the factor, and scales the turned vectors by
    0.1 ln(factor) + 1. Between the two it goes linearly in the pair index (the paper's formula is
    linear in the number of turns), from the last whole pair before the one that turns beta_fast
    times to the first whole pair behind the one that turns beta_slow times; either may lie outside
    the head, and the ramp is then cut off there, not bent.
    """
    dims = [int(dims)] if isinstance(dims, (int, np.integer)) else [int(d) for d in dims]
    if not dims or any(d < 0 or d % 2 for d in dims) or sum(dims) == 0:
        raise ValueError("dims: expected even channel counts")
    if not (theta > 1.0) or not (factor >= 1.0):
        raise ValueError("theta must be above 1 and factor at least 1")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError("scaling must be none, linear, ntk or yarn")
    if scaling == "yarn" and (original_length <= 0 or not beta_fast > beta_slow > 0):
        raise ValueError("yarn needs original_length > 0 and beta_fast > beta_slow > 0")
    inv, axis, amplitude = [], [], 1.0
    for a, d in enumerate(dims):
        if d == 0:
            continue
        i = np.arange(d // 2, dtype=np.float64)
        base = float(theta)
        if scaling == "ntk":
            if d <= 2:
                raise ValueError("ntk scaling needs more than 2 channels per axis")
            base *= float(factor) ** (d / (d - 2))
        f = base ** (-2.0 * i / d)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            pair = lambda turns: d * np.log(original_length / (2 * np.pi * turns)) / (2 * np.log(theta))
            low, high = np.floor(pair(beta_fast)), np.ceil(pair(beta_slow))
            ramp = np.clip((i - low) / max(high - low, 1.0), 0.0, 1.0)
            f = f * (1.0 - ramp) + f / factor * ramp
            amplitude = 0.1 * float(np.log(factor)) + 1.0
        inv.append(f)
        axis.append(np.full(d // 2, a, np.int32))
    return RotaryFrequencies(np.concatenate(inv), np.concatenate(axis), amplitude)


def rotary_positions(grid, n_tail: int = 0) -> np.ndarray:
    """[3, N] int32 (t, h, w) of a geometry's raster tokens; appended 1D token j has the position
    max(T, Hg, Wg) + j on all three axes (behind every video position)."""
    T, Hg, Wg = (int(x) for x in grid)
    t, h, w = np.meshgrid(np.arange(T), np.arange(Hg), np.arange(Wg), indexing="ij")
    tail = np.tile(max(T, Hg, Wg) + np.arange(int(n_tail)), (3, 1))
    return np.concatenate([np.stack([t.ravel(), h.ravel(), w.ravel()]), tail], 1).astype(np.int32)


@dataclasses.dataclass
class RotaryTable:
    """cos / sin of every (row, pair): fp32 [rows, P, 2]; rot_dim = 2 P channels are turned, in
    interleaved pairs (2p, 2p + 1) or, in the half layout, (p, p + P)."""
    cos_sin: torch.Tensor
    interleaved: bool

    @property
    def rows(self) -> int:
        return self.cos_sin.shape[0]

    @property
    def rot_dim(self) -> int:
        return 2 * self.cos_sin.shape[1]

    def _check(self) -> None:
        t = self.cos_sin
        if t.dtype is torch.float32 and t.dim() == 3 and t.shape[2] == 2 and t.is_contiguous() and _here(t):
            return
        if self.cos_sin.dim() != 3 or self.cos_sin.shape[2] != 2:
            raise ValueError("cos_sin: expected shape [rows, P, 2]")
        _need(self.cos_sin, torch.float32, "cos_sin")


def rotary_table(positions: torch.Tensor, inv_freq: np.ndarray, axis: Optional[np.ndarray] = None,
                 amplitude: float = 1.0, interleaved: bool = True, out: Optional[torch.Tensor] = None,
                 stream=None) -> RotaryTable:
    """veda_rotary_table: positions int32 [rows] or [axes, rows] on the device; inv_freq / axis
    [P] on the host (see ``rotary_frequencies``; axis defaults to 0)."""
    if positions.dim() == 1:
        positions = positions.unsqueeze(0)
    if positions.dim() != 2:
        raise ValueError("positions: expected shape [rows] or [axes, rows]")
    _need(positions, torch.int32, "positions")
    inv = np.ascontiguousarray(inv_freq, dtype=np.float64)
    ax = np.zeros(inv.shape, np.int32) if axis is None else np.asarray(axis)
    if inv.ndim != 1 or ax.shape != inv.shape:
        raise ValueError("inv_freq / axis: expected equal shapes [P]")
    axes, rows = positions.shape
    if ax.dtype != np.int32:                       # the library checks the values that it gets
        if ax.dtype.kind not in "iu":
            raise TypeError(f"axis: expected integers, got {ax.dtype}")
        if ax.size and not 0 <= int(ax.min()) <= int(ax.max()) < axes:
            raise ValueError(f"axis: outside the {axes} axes of positions")
    ax = np.ascontiguousarray(ax, dtype=np.int32)
    if out is None:
        out = _new(positions, (rows, len(inv), 2), torch.float32, stream)
    else:
        _need(out, torch.float32, "out", shape=(rows, len(inv), 2))
        _separate(out, positions, "positions", False)
    _check("veda_rotary_table", lib().veda_rotary_table(
        _ptr(positions), axes, rows, inv.ctypes.data, ax.ctypes.data, len(inv), float(amplitude), _ptr(out),
        _stream(stream)))
    return RotaryTable(out, bool(interleaved))


def rotary(x: torch.Tensor, table: RotaryTable, rows: Optional[torch.Tensor] = None, inverse: bool = False,
           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """veda_rotary: x [B, N, H, D] (bf16, fp16 or fp32; any strides, channels contiguous) turned by
    the table's row of each token -- row n, row b N + n (a table of B N rows), or rows[b, n]
    (int32). ``inverse`` is the transpose, which the gradient takes. ``out`` may be x."""
    _fits("x", x.shape)
    _need_strided(x, "x", 4)
    B, N, H, D = x.shape
    table._check()
    if rows is not None:
        _need(rows, torch.int32, "rows", shape=(B, N))
    if out is None:
        out = _new(x, (B, N, H, D), x.dtype, stream)
    else:
        _need_strided(out, "out", 4, x.dtype, x.shape, written=True)
        _separate(out, x, "x", True)
        _separate_all(out, "out", (table.cos_sin, "the table"), (rows, "rows"))
    cs = table.cos_sin
    _check("veda_rotary", lib().veda_rotary(
        x.data_ptr(), _STRIDES3.pack(*x.stride()[:3]), out.data_ptr(), _STRIDES3.pack(*out.stride()[:3]),
        _DTYPE[x.dtype], cs.data_ptr(), cs.shape[0], _ptr(rows), 2 * cs.shape[1], int(table.interleaved),
        int(bool(inverse)), B, N, H, D, _stream(stream)))
    return out


def rotary_permute_pool(x: torch.Tensor, table: RotaryTable, maps: DeviceMaps, out: Optional[torch.Tensor] = None,
                        pooled: Optional[torch.Tensor] = None, stream=None):
    """veda_rotary_permute_pool: ``permute_pool`` with the rotation of ``rotary`` on the way (the
    pooled features are those of the turned values before they are rounded to bf16)."""
    _need(x, torch.bfloat16, "x")
    if x.dim() != 4:
        raise ValueError("x: expected shape [B, N, H, 128]")
    B, N, H, D = x.shape
    _need_maps(maps, H, maps.Npad)
    table._check()
    read = ((x, "x"), (table.cos_sin, "the table"), (maps.tile_map, "the tile map"), (maps.tile_valid, "tile_valid"))
    if out is None:
        out = _new(x, (B, H, maps.Npad, D), torch.bfloat16, stream)
    else:
        _need(out, torch.bfloat16, "out", shape=(B, H, maps.Npad, D))
        _separate_all(out, "out", *read)
    if pooled is None:
        pooled = _new(x, (B, H, maps.Npad // 128, 3, D), torch.float32, stream)
    else:
        _need(pooled, torch.float32, "pooled", shape=(B, H, maps.Npad // 128, 3, D))
        _separate_all(pooled, "pooled", *read, (out, "out"))
    _check("veda_rotary_permute_pool", lib().veda_rotary_permute_pool(
        _ptr(x), _ptr(out), _ptr(table.cos_sin), table.rows, table.rot_dim, int(table.interleaved),
        _ptr(maps.tile_map), _ptr(maps.tile_valid), _ptr(pooled), B, N, H, D, maps.Npad, _stream(stream)))
    return out, pooled


def rotary_unpermute(x_t: torch.Tensor, table: RotaryTable, maps: DeviceMaps, N: int, inverse: bool = True,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """veda_rotary_unpermute: tiles back to raster order through the transposed rotation -- dQ / dK
    of the attention's backward to the gradients of the unturned Q / K. Tokens that the tile map does not
    have stay as they are in ``out``; without it, N is the map's."""
    _need(x_t, torch.bfloat16, "x_t")
    if x_t.dim() != 4:
        raise ValueError("x_t: expected shape [B, H, Npad, 128]")
    B, H, Npad, D = x_t.shape
    _need_maps(maps, H, Npad)
    table._check()
    if out is None:
        _need_tokens(maps, N)
        out = _new(x_t, (B, N, H, D), torch.bfloat16, stream)
    else:
        _need(out, torch.bfloat16, "out", shape=(B, N, H, D))
        _separate_all(out, "out", (x_t, "x_t"), (table.cos_sin, "the table"), (maps.tile_map, "the tile map"))
    _check("veda_rotary_unpermute", lib().veda_rotary_unpermute(
        _ptr(x_t), _ptr(out), _ptr(table.cos_sin), table.rows, table.rot_dim, int(table.interleaved),
        int(bool(inverse)), _ptr(maps.tile_map), B, N, H, D, Npad, _stream(stream)))
    return out


@dataclasses.dataclass
class NormStats:
    """What a norm's backward needs of its forward: mean (layer norm) and 1 / deviation of every
    row, fp32 [B, N]."""
    mean: torch.Tensor
    rstd: torch.Tensor


@dataclasses.dataclass
class NormGrads:
    """Gradients of a norm and of what is fused with it; None where there is no such parameter.
    dx: of the normed input; the parameters' in fp32."""
    dx: torch.Tensor
    dweight: Optional[torch.Tensor] = None   # [C]
    dbias: Optional[torch.Tensor] = None     # [C]
    dscale: Optional[torch.Tensor] = None    # [B, C]
    dshift: Optional[torch.Tensor] = None    # [B, C]
    dgate: Optional[torch.Tensor] = None     # [B, C]


def _rows3(t: torch.Tensor, name: str, dtype=None, shape=None, written=False) -> torch.Tensor:
    """[N, C] as [1, N, C], checked."""
    t = t.unsqueeze(0) if t.dim() == 2 else t
    if shape is None:
        _fits(name, t.shape)
    _need_strided(t, name, 3, dtype, shape, written)
    return t


def _rows(t: Optional[torch.Tensor]):
    if t is None:
        return None
    sb, sn, _ = t.stride()
    return _ROWS.pack(t.data_ptr(), sb, sn, _DTYPE[t.dtype])


def _vectors(B: int, C: int, weight, bias, gain, shift, gain_name: str, offset: float):
    """Checked parameters of a norm: weight / bias [C] of one type, gain / shift [B, C] ([C] for
    one sequence) of one type with any batch stride."""
    wd = md = 2
    if weight is not None or bias is not None:
        for t, n in ((weight, "weight"), (bias, "bias")):
            if t is not None:
                _need_strided(t, n, 1, None, (C,))
                wd = _DTYPE[t.dtype]
        if weight is not None and bias is not None and weight.dtype != bias.dtype:
            raise TypeError(f"weight and bias: expected one type, got {weight.dtype} and {bias.dtype}")
    if gain is not None:
        gain = gain.unsqueeze(0) if gain.dim() == 1 else gain
        _need_strided(gain, gain_name, 2, None, (B, C))
        md = _DTYPE[gain.dtype]
    if shift is not None:
        shift = shift.unsqueeze(0) if shift.dim() == 1 else shift
        _need_strided(shift, "shift", 2, None, (B, C))
        md = _DTYPE[shift.dtype]
        if gain is not None and gain.dtype != shift.dtype:
            raise TypeError(f"{gain_name} and shift: expected one type, got {gain.dtype} and {shift.dtype}")
    return _NORM_PARAMS.pack(_ptr(weight) or 0, _ptr(bias) or 0, _ptr(gain) or 0, _ptr(shift) or 0,
                             gain.stride(0) if gain is not None else 0, shift.stride(0) if shift is not None else 0,
                             wd, md, offset)


def _norm_kind(kind: str) -> int:
    if kind not in _KIND:
        raise ValueError(f"kind must be one of {sorted(_KIND)}, got {kind!r}")
    return _KIND[kind]


def _norm_fwd(x, x3, residual, params, read, residual_scale, kind, eps, out_dtype, out, want_stats, stream):
    """``read``: the parameters and their names, which out must not overlap."""
    B, N, C = x3.shape
    if out_dtype not in _DTYPE:
        raise TypeError(f"out_dtype: expected bfloat16, float16 or float32, got {out_dtype}")
    if residual is not None:
        residual = _rows3(residual, "residual", out_dtype, x3.shape)
    if out is None:
        out = _new(x, x.shape, out_dtype, stream)
        out3 = out if out.dim() == 3 else out.unsqueeze(0)
    else:
        out3 = _rows3(out, "out", out_dtype, x3.shape, written=True)
        _separate(out3, x3, "x", True)
        _separate(out3, residual, "the residual", True)
        _separate_all(out3, "out", *read)
    stats = mean = rstd = None
    if want_stats:
        stats = NormStats(_new(x, (B, N), torch.float32, stream), _new(x, (B, N), torch.float32, stream))
        mean, rstd = stats.mean.data_ptr(), stats.rstd.data_ptr()
    _check("veda_norm_fwd", lib().veda_norm_fwd(
        _rows(x3), _rows(residual), _rows(out3), params, residual_scale, mean, rstd, B, N, C, _norm_kind(kind), eps,
        _stream(stream)))
    return (out, stats) if want_stats else out


def norm_modulate(x: torch.Tensor, scale: Optional[torch.Tensor] = None, shift: Optional[torch.Tensor] = None,
                  weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, kind: str = "layer",
                  eps: float = 1e-6, out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                  want_stats: bool = False, stream=None):
    """The norm before a block (veda_norm_fwd): (norm(x) weight + bias) (1 + scale) + shift.

    x [B, N, C] or [N, C] (any row strides); weight / bias [C]; scale / shift [B, C], one vector
    per sequence (any batch stride: slices of one modulation vector will do); every one of them
    optional. kind "layer", "rms" or "none". ``want_stats`` also returns the ``NormStats`` of
    ``norm_modulate_bwd``. out_dtype: x's type, or bf16 for fp32 x, or fp32 for bf16 x."""
    x3 = _rows3(x, "x")
    p = _vectors(x3.shape[0], x3.shape[2], weight, bias, scale, shift, "scale", 1.0)
    dt = out_dtype if out_dtype is not None else out.dtype if out is not None else x.dtype
    read = ((weight, "weight"), (bias, "bias"), (scale, "scale"), (shift, "shift"))
    return _norm_fwd(x, x3, None, p, read, 0.0, kind, eps, dt, out, want_stats, stream)


def norm_gate_add(o: torch.Tensor, residual: torch.Tensor, gate: Optional[torch.Tensor] = None,
                  weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, kind: str = "rms",
                  eps: float = 1e-6, residual_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                  want_stats: bool = False, stream=None):
    """The norm after a block and the residual sum (veda_norm_fwd):
    residual_scale residual + gate (norm(o) weight + bias).

    o: the block's output [B, N, C] or [N, C]; residual of the same shape, whose type the result
    has (o's type, or fp32 with bf16 o, or bf16 with fp32 o); gate [B, C]. kind "none" gates o
    itself. ``out`` may be the residual (in place)."""
    o3 = _rows3(o, "o")
    p = _vectors(o3.shape[0], o3.shape[2], weight, bias, gate, None, "gate", 0.0)
    read = ((weight, "weight"), (bias, "bias"), (gate, "gate"))
    return _norm_fwd(o, o3, residual, p, read, residual_scale, kind, eps, residual.dtype, out, want_stats, stream)


def _norm_bwd(dy, x, x3, stats, params, read, want_dshift, residual_grad, residual_scale, kind, out, stream):
    """``read``: weight, bias and gain with their names; which of them is given says which gradients are wanted."""
    B, N, C = x3.shape
    dy3 = _rows3(dy, "dy", None, x3.shape)
    res3 = None if residual_grad is None else _rows3(residual_grad, "residual_grad", x.dtype, x3.shape)
    k = _norm_kind(kind)
    mean = rstd = None
    if stats is not None:
        _need(stats.rstd, torch.float32, "stats.rstd", shape=(B, N))
        _need(stats.mean, torch.float32, "stats.mean", shape=(B, N))
        mean, rstd = stats.mean.data_ptr(), stats.rstd.data_ptr()
    elif k != 2:
        raise ValueError("stats: the forward's statistics are needed (want_stats=True)")
    if out is None:
        out = _new(x, x.shape, x.dtype, stream)
        out3 = out if out.dim() == 3 else out.unsqueeze(0)
    else:
        out3 = _rows3(out, "out", x.dtype, x3.shape, written=True)
        for t, n in ((x3, "x"), (dy3, "dy"), (res3, "residual_grad")):
            _separate(out3, t, n, True)
        _separate_all(out3, "out", *read)
        if stats is not None:
            _separate_all(out3, "out", (stats.mean, "stats.mean"), (stats.rstd, "stats.rstd"))
    f32 = torch.float32
    (weight, _), (bias, _), (gain, _) = read
    dgain = _new(x, (B, C), f32, stream) if gain is not None else None
    dshift = _new(x, (B, C), f32, stream) if want_dshift else None
    dweight = _new(x, (C,), f32, stream) if weight is not None else None
    dbias = _new(x, (C,), f32, stream) if bias is not None else None
    nbytes = lib().veda_norm_bwd_workspace_bytes(B, N, C)
    work = _new(x, (max(nbytes, 16),), torch.uint8, stream)
    _check("veda_norm_bwd", lib().veda_norm_bwd(
        _rows(dy3), _rows(x3), mean, rstd, _rows(res3), _rows(out3), params, residual_scale, _ptr(dgain),
        _ptr(dshift), _ptr(dweight), _ptr(dbias), work.data_ptr(), work.numel(), B, N, C, k, _stream(stream)))
    return out, dgain, dshift, dweight, dbias


def norm_modulate_bwd(dy: torch.Tensor, x: torch.Tensor, stats: Optional[NormStats],
                      scale: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None, kind: str = "layer", want_dshift: bool = True,
                      residual_grad: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
                      out: Optional[torch.Tensor] = None, stream=None) -> NormGrads:
    """Backward of ``norm_modulate``: dx (x's type), dscale, dshift, dweight, dbias.

    residual_grad (x's type) is the gradient of the stream that passes the block by: dx gets
    residual_scale times it added, which saves the separate sum."""
    x3 = _rows3(x, "x")
    p = _vectors(x3.shape[0], x3.shape[2], weight, bias, scale, None, "scale", 1.0)
    read = ((weight, "weight"), (bias, "bias"), (scale, "scale"))
    dx, dg, dt, dw, db = _norm_bwd(dy, x, x3, stats, p, read, bool(want_dshift), residual_grad, residual_scale, kind, out, stream)
    return NormGrads(dx, dw, db, dscale=dg, dshift=dt)


def norm_gate_add_bwd(dh: torch.Tensor, o: torch.Tensor, stats: Optional[NormStats],
                      gate: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      bias: Optional[torch.Tensor] = None, kind: str = "rms", out: Optional[torch.Tensor] = None,
                      stream=None) -> NormGrads:
    """Backward of ``norm_gate_add``: dx is the gradient of the block's output o, and dgate,
    dweight, dbias. The residual's gradient is residual_scale dh, which ``norm_modulate_bwd`` of
    the same block adds on its way (residual_grad=dh)."""
    o3 = _rows3(o, "o")
    p = _vectors(o3.shape[0], o3.shape[2], weight, bias, gate, None, "gate", 0.0)
    read = ((weight, "weight"), (bias, "bias"), (gate, "gate"))
    dx, dg, _, dw, db = _norm_bwd(dh, o, o3, stats, p, read, False, None, 0.0, kind, out, stream)
    return NormGrads(dx, dw, db, dgate=dg)


@dataclasses.dataclass
class Int8Rows:
    """Rows of 8-bit codes with a scale each: codes int8 [rows, kp], kp = K rounded up to a
    multiple of 16 with zeros behind K; scale fp32 [rows]; row r stands for codes * scale[r]."""
    codes: torch.Tensor
    scale: torch.Tensor
    K: int

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @staticmethod
    def from_codes(codes: torch.Tensor, scale: torch.Tensor) -> "Int8Rows":
        """From int8 codes [rows, K] made elsewhere (a checkpoint) and their scales [rows]."""
        if codes.dim() != 2 or codes.dtype != torch.int8:
            raise TypeError("codes: expected int8 [rows, K]")
        rows, K = codes.shape
        if tuple(scale.shape) != (rows,):
            raise ValueError(f"scale: expected shape {(rows,)}, got {tuple(scale.shape)}")
        kp = -(-K // 16) * 16
        padded = codes.contiguous() if kp == K else torch.zeros((rows, kp), dtype=torch.int8, device=codes.device)
        if kp != K:
            padded[:, :K] = codes
        return Int8Rows(padded, scale.float().contiguous(), K)

    def _check(self, name: str) -> None:
        if self.K <= 0:
            raise ValueError(f"{name}: K must be positive")
        _need(self.codes, torch.int8, f"{name}.codes", shape=(self.codes.shape[0], -(-self.K // 16) * 16))
        _need(self.scale, torch.float32, f"{name}.scale", shape=(self.codes.shape[0],))


def _matrix(x: torch.Tensor, name: str) -> torch.Tensor:
    """x [..., K] as a matrix of rows without a copy."""
    if x.dim() == 2:
        return x
    if x.dim() < 1:
        raise ValueError(f"{name}: expected at least one dimension")
    try:
        return x.view(-1, x.shape[-1]) if x.numel() else x.reshape(0, x.shape[-1])
    except RuntimeError:
        raise ValueError(f"{name}: its leading dimensions do not form rows of one stride") from None


def quantize_int8(x: torch.Tensor, out: Optional[Int8Rows] = None, stream=None) -> Int8Rows:
    """veda_quantize_int8: rows of x [..., K] (bf16, fp16 or fp32) to codes with a scale for each
    row -- tokens of an activation, output channels of a weight [N, K]."""
    m = _matrix(x, "x")
    _fits("x", m.shape)
    _need_strided(m, "x", 2)
    rows, K = m.shape
    if out is None:
        out = Int8Rows(_new(x, (rows, -(-K // 16) * 16), torch.int8, stream),
                       _new(x, (rows,), torch.float32, stream), K)
    else:
        if out.K != K or out.rows != rows:
            raise ValueError(f"out: expected {rows} rows of {K} codes")
        out._check("out")
        _separate_all(out.codes, "out.codes", (m, "x"), (out.scale, "out.scale"))
        _separate_all(out.scale, "out.scale", (m, "x"))
    _check("veda_quantize_int8", lib().veda_quantize_int8(
        _ptr(m), m.stride(0), _DTYPE[m.dtype], _ptr(out.codes), _ptr(out.scale), rows, K, _stream(stream)))
    return out


def int8_matmul(a: Int8Rows, w: Int8Rows, bias: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """veda_int8_matmul: y[m, n] = (a[m] . w[n]) a.scale[m] w.scale[n] + bias[n] (bias fp32 [N]);
    y [M, N] in bf16, fp16 or fp32."""
    _fits("a", a.codes.shape)
    _fits("w", w.codes.shape)
    a._check("a")
    w._check("w")
    if a.K != w.K:
        raise ValueError(f"a has rows of {a.K} codes, w of {w.K}")
    M, N = a.rows, w.rows
    if bias is not None:
        _need(bias, torch.float32, "bias", shape=(N,))
    if out is None:
        if out_dtype not in _DTYPE:
            raise TypeError(f"out_dtype: expected bfloat16, float16 or float32, got {out_dtype}")
        out = _new(a.codes, (M, N), out_dtype, stream)
    else:
        _need_strided(out, "out", 2, None, (M, N), written=True)
        _separate_all(out, "out", (a.codes, "a.codes"), (w.codes, "w.codes"), (a.scale, "a.scale"), (w.scale, "w.scale"),
                      (bias, "bias"))
    _check("veda_int8_matmul", lib().veda_int8_matmul(
        _ptr(a.codes), _ptr(a.scale), _ptr(w.codes), _ptr(w.scale), _ptr(bias), _ptr(out),
        out.stride(0), _DTYPE[out.dtype], M, N, a.K, _stream(stream)))
    return out


def int8_linear(x: torch.Tensor, w: Int8Rows, bias: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """veda_int8_linear: x [..., K] W^T + bias in 8-bit integers -- ``quantize_int8`` of x's rows and
    ``int8_matmul`` with the weight's rows in one call; [..., N] in x's type (or out_dtype)."""
    m = _matrix(x, "x")
    _fits("x", m.shape)
    _fits("w", w.codes.shape)
    _need_strided(m, "x", 2)
    w._check("w")
    M, K = m.shape
    N = w.codes.shape[0]
    if K != w.K:
        raise ValueError(f"x has rows of {K} values, w of {w.K}")
    if bias is not None:
        _need(bias, torch.float32, "bias", shape=(N,))
    dt = x.dtype if out_dtype is None else out_dtype
    if dt not in _DTYPE:
        raise TypeError(f"out_dtype: expected bfloat16, float16 or float32, got {dt}")
    out = _new(x, (*x.shape[:-1], N), dt, stream)
    nbytes = lib().veda_int8_linear_workspace_bytes(M, K)
    work = _new(x, (nbytes,), torch.uint8, stream) if nbytes else None
    _check("veda_int8_linear", lib().veda_int8_linear(
        m.data_ptr(), m.stride(0), _DTYPE[m.dtype], w.codes.data_ptr(), w.scale.data_ptr(), _ptr(bias),
        out.data_ptr(), N, _DTYPE[dt], _ptr(work), nbytes, M, N, K, _stream(stream)))
    return out


def check_device_status(stream=None) -> int:
    """Synchronise the stream and raise if a kernel recorded an error. Returns the raw bits."""
    detail = ctypes.c_uint32(0)
    st = lib().veda_check_device_status(_stream(stream), ctypes.byref(detail))
    _check("veda_check_device_status", st)
    return detail.value


def selftest_wait_timeout(limit_us: int = 2000, stream=None) -> None:
    """Launch the bounded-wait self-test (see include/veda.h); check the status afterwards."""
    _check("veda_selftest_wait_timeout", lib().veda_selftest_wait_timeout(int(limit_us), _stream(stream)))


# ---------------------------------------------------------------------------------------
# the whole path
# ---------------------------------------------------------------------------------------

@dataclasses.dataclass
class PathBuffers:
    """Device buffers of one attention call (reusable across calls of the same shape)."""
    q_t: torch.Tensor
    k_t: torch.Tensor
    v_t: torch.Tensor
    pooled_q: torch.Tensor
    pooled_k: torch.Tensor
    scores: torch.Tensor
    workspace: torch.Tensor
    lists: BlockLists
    o_t: torch.Tensor
    lse: torch.Tensor
    o: torch.Tensor

    def tensors(self) -> List[torch.Tensor]:
        ls = self.lists
        return [self.q_t, self.k_t, self.v_t, self.pooled_q, self.pooled_k, self.scores, self.workspace, self.o_t, self.lse,
                self.o, ls.full_cnt, ls.full_idx, ls.part_cnt, ls.part_idx]

    @staticmethod
    def allocate(B: int, N: int, H: int, maps: DeviceMaps, rho, device, stream=None) -> "PathBuffers":
        """Buffers for work on ``stream`` (None: the current one): its memory, and the lists' zeros in
        its order; kept from reuse until what the current stream does with them later has run."""
        if stream is not None:
            with torch.cuda.stream(stream):
                bufs = PathBuffers.allocate(B, N, H, maps, rho, device)
            for t in bufs.tensors():
                t.record_stream(torch.cuda.current_stream())
            return bufs
        nT, Npad, D = maps.nT, maps.Npad, 128
        bf = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        stride = list_stride_for(nT, rho)
        i32 = dict(dtype=torch.int32, device=device)
        lists = BlockLists(torch.zeros((B, H, nT), **i32), torch.zeros((B, H, nT, stride), **i32),
                           torch.zeros((B, H, nT), **i32), torch.zeros((B, H, nT, stride), **i32),
                           stride)
        return PathBuffers(
            torch.empty((B, H, Npad, D), **bf), torch.empty((B, H, Npad, D), **bf),
            torch.empty((B, H, Npad, D), **bf), torch.empty((B, H, nT, 3, D), **f32),
            torch.empty((B, H, nT, 3, D), **f32), torch.empty((B, H, nT, nT), **f32),
            torch.empty(block_scores_workspace_bytes(B, H, nT, D), dtype=torch.uint8, device=device),
            lists, torch.empty((B, H, Npad, D), **bf), torch.empty((B, H, Npad), **f32),
            torch.empty((B, N, H, D), **bf))


def sparse_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, wq: torch.Tensor,
                     wk: torch.Tensor, maps: DeviceMaps, rho: Sequence[Tuple[int, int]],
                     scale: float, buffers: Optional[PathBuffers] = None, stream=None,
                     rotary: Optional[RotaryTable] = None):
    """All six steps on raster Q/K/V [B, N, H, 128] (bf16, on the device).

    Returns the PathBuffers holding every intermediate; ``.o`` is the raster output. Steps 1
    and 2 of Q and K run as one call each (``permute_pool``: the tiles of ``permute_tiles``,
    the pooled features of ``tile_pool`` up to fp32 summation order in the mean), so that the
    tiled Q and K are not read a second time. ``rotary``: positions turned into Q and K on the
    way into the tiles (``rotary_permute_pool``).
    """
    B, N, H, D = q.shape
    bufs = buffers or PathBuffers.allocate(B, N, H, maps, rho, q.device, stream)
    if rotary is None:
        permute_pool(q, maps, bufs.q_t, bufs.pooled_q, stream)
        permute_pool(k, maps, bufs.k_t, bufs.pooled_k, stream)
    else:
        rotary_permute_pool(q, rotary, maps, bufs.q_t, bufs.pooled_q, stream)
        rotary_permute_pool(k, rotary, maps, bufs.k_t, bufs.pooled_k, stream)
    permute_tiles(v, maps, bufs.v_t, stream)
    block_scores(bufs.pooled_q, bufs.pooled_k, wq, wk, bufs.scores, bufs.workspace, stream)
    select_blocks(bufs.scores, maps, rho, bufs.lists.stride, bufs.lists, stream)
    block_sparse_attn_fwd(bufs.q_t, bufs.k_t, bufs.v_t, maps, bufs.lists, scale, bufs.o_t,
                          bufs.lse, stream=stream)
    unpermute(bufs.o_t, maps, N, bufs.o, stream)
    return bufs


@dataclasses.dataclass
class BlockWeights:
    """Weights of one attention block: 8-bit projections (rows are output channels; H * 128 of Q,
    K, V), the predictor's projections, and the norms around the block."""
    q: Int8Rows
    k: Int8Rows
    v: Int8Rows
    o: Int8Rows
    pred_q: torch.Tensor                        # [H, 128, 384] fp32
    pred_k: torch.Tensor
    q_bias: Optional[torch.Tensor] = None       # fp32
    k_bias: Optional[torch.Tensor] = None
    v_bias: Optional[torch.Tensor] = None
    o_bias: Optional[torch.Tensor] = None
    pre_weight: Optional[torch.Tensor] = None   # norm before the block
    pre_bias: Optional[torch.Tensor] = None
    post_weight: Optional[torch.Tensor] = None  # norm after it
    pre_kind: str = "layer"
    post_kind: str = "none"
    eps: float = 1e-6


def attention_block(x: torch.Tensor, w: BlockWeights, scale: Optional[torch.Tensor], shift: Optional[torch.Tensor],
                    gate: Optional[torch.Tensor], table: RotaryTable, maps: DeviceMaps,
                    rho: Sequence[Tuple[int, int]], softmax_scale: float, residual_scale: float = 1.0,
                    buffers: Optional[PathBuffers] = None, stream=None) -> torch.Tensor:
    """One self-attention block on the residual stream x [B, N, C] (bf16 or fp32), for inference:

    ``norm_modulate`` (scale, shift), one ``quantize_int8`` for the three ``int8_matmul`` of Q, K and
    V, ``sparse_attention`` with the rotary positions, ``int8_linear`` back to C channels, and
    ``norm_gate_add`` (gate, residual). Returns the new stream, of x's type. Blocks with other stages (a
    norm of Q and K before the positions, a bias behind the norm after the block) call the operators
    themselves."""
    if x.dim() != 3:
        raise ValueError("x: expected shape [B, N, C]")
    B, N, C = x.shape
    _need_tokens(maps, N)
    H = w.pred_q.shape[0]
    for r, n in ((w.q, "q"), (w.k, "k"), (w.v, "v")):
        if r.rows != H * 128:
            raise ValueError(f"{n}: expected {H * 128} output channels, got {r.rows}")
    a = norm_modulate(x, scale, shift, w.pre_weight, w.pre_bias, w.pre_kind, w.eps, torch.bfloat16, stream=stream)
    a8 = quantize_int8(a, stream=stream)
    q, k, v = (int8_matmul(a8, r, b, stream=stream).view(B, N, H, 128)
               for r, b in ((w.q, w.q_bias), (w.k, w.k_bias), (w.v, w.v_bias)))
    bufs = sparse_attention(q, k, v, w.pred_q, w.pred_k, maps, rho, softmax_scale, buffers, stream, rotary=table)
    o = int8_linear(bufs.o.view(B, N, H * 128), w.o, w.o_bias, stream=stream)
    return norm_gate_add(o, x, gate, w.post_weight, None, w.post_kind, w.eps, residual_scale, stream=stream)


class HostPipeline:
    """Clips from pinned host memory through the whole path, one clip per ``submit``.

    Three CUDA streams overlap the host-to-device copy of clip i + 1, the six steps of clip i
    and the device-to-host copy of clip i - 1's output (the host link carries both directions
    at once). Device copies of the raster inputs and of the raster output are kept per slot
    (``depth`` slots); CUDA events order every reuse of a slot after the work that last read
    it, so a clip's result does not depend on its neighbours. ``rotary``: positions for Q and K of
    every clip. What the current stream holds when the pipeline is made (the table's kernel, the
    maps) comes before the first clip. ``synchronize`` waits for every submitted clip's output to be in
    its host tensor.
    """

    def __init__(self, B: int, N: int, H: int, maps: DeviceMaps, rho: Sequence[Tuple[int, int]],
                 scale: float, device, depth: int = 2, rotary: Optional[RotaryTable] = None):
        if depth < 1:
            raise ValueError("depth must be >= 1")
        self.maps, self.rho, self.scale, self.depth = maps, list(rho), float(scale), depth
        self.rotary = rotary
        bf = dict(dtype=torch.bfloat16, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        self.inputs = [dict(q=torch.empty((B, N, H, 128), **bf), k=torch.empty((B, N, H, 128), **bf),
                            v=torch.empty((B, N, H, 128), **bf), wq=torch.empty((H, 128, 384), **f32),
                            wk=torch.empty((H, 128, 384), **f32)) for _ in range(depth)]
        self.outputs = [torch.empty((B, N, H, 128), **bf) for _ in range(depth)]
        self.bufs = PathBuffers.allocate(B, N, H, maps, rho, device)
        self.h2d, self.comp, self.d2h = (torch.cuda.Stream(device) for _ in range(3))
        # the buffers' memory, the lists' zeros, the maps and the table are the current stream's (d2h
        # follows comp)
        for st in (self.h2d, self.comp):
            st.wait_stream(torch.cuda.current_stream(device))
        # and go back to it, when the pipeline is dropped, only behind what its streams do with them
        copied = [t for i in self.inputs for t in i.values()]
        read = [maps.tile_map, maps.tile_valid, maps.tile_segment, maps.nT_per_head]
        read += [] if rotary is None else [rotary.cos_sin]
        for st, ts in ((self.h2d, copied), (self.comp, copied + self.outputs + self.bufs.tensors() + read),
                       (self.d2h, self.outputs)):
            for t in ts:
                t.record_stream(st)
        ev = lambda: [torch.cuda.Event() for _ in range(depth)]
        self.in_ready, self.in_free, self.out_ready, self.out_free = ev(), ev(), ev(), ev()
        self.n = 0

    def submit(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, wq: torch.Tensor, wk: torch.Tensor,
               out: torch.Tensor) -> None:
        """Enqueue one clip: q / k / v [B, N, H, 128] bf16, wq / wk [H, 128, 384] fp32 and the
        output out [B, N, H, 128] bf16, all pinned host tensors; returns at once."""
        s = self.n % self.depth
        reuse = self.n >= self.depth
        slot = self.inputs[s]
        # inputs of slot s: after the clip that last used them has been computed
        if reuse:
            self.h2d.wait_event(self.in_free[s])
        with torch.cuda.stream(self.h2d):
            for name, src in (("q", q), ("k", k), ("v", v), ("wq", wq), ("wk", wk)):
                slot[name].copy_(src, non_blocking=True)
            self.in_ready[s].record(self.h2d)
        # the six steps, into output slot s once its previous contents have left the device
        self.comp.wait_event(self.in_ready[s])
        if reuse:
            self.comp.wait_event(self.out_free[s])
        bufs = dataclasses.replace(self.bufs, o=self.outputs[s])
        sparse_attention(slot["q"], slot["k"], slot["v"], slot["wq"], slot["wk"], self.maps, self.rho,
                         self.scale, buffers=bufs, stream=self.comp, rotary=self.rotary)
        self.in_free[s].record(self.comp)
        self.out_ready[s].record(self.comp)
        # the output of slot s to the host
        self.d2h.wait_event(self.out_ready[s])
        with torch.cuda.stream(self.d2h):
            out.copy_(self.outputs[s], non_blocking=True)
            self.out_free[s].record(self.d2h)
        self.n += 1

    def synchronize(self) -> None:
        self.d2h.synchronize()
