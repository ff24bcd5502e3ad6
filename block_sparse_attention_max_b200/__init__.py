"""B200-native hot path of Veda block-sparse attention.

The six steps run in ``libveda.so`` (CUDA kernels for sm_100a behind the C ABI of
``include/veda.h``); ``veda`` is its ctypes binding. Build the library with
``python -m block_sparse_attention_max_b200.build``.
"""
from . import veda  # noqa: F401
from .veda import (  # noqa: F401
    BlockWeights, Int8Rows, NormGrads, NormStats, RotaryFrequencies, RotaryTable, attention_block, int8_linear,
    int8_matmul, norm_gate_add, norm_gate_add_bwd, norm_modulate, norm_modulate_bwd, quantize_int8, rotary,
    rotary_frequencies, rotary_permute_pool, rotary_positions, rotary_table, rotary_unpermute,
    VedaError, block_scores, block_sparse_attn_fwd, build_tile_map, check_device_status,
    geometry_sizes, permute_tiles, select_blocks, sparse_attention, tile_pool, unpermute,
)
