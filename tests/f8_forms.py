"""Which kernel an 8-bit product takes, by the library's own rule, and a size for every one."""
from __future__ import annotations

import ctypes

import mixed_gemm_amd as mg

TILES = ("32 x 32", "32 x 64", "64 x 64", "128 x 128", "256 x 256", "192 x 256")     # the first three: few rows


class _Choice(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("time", ctypes.c_double), ("time256", ctypes.c_double)]


def _symbol(name, args, res):
    f = mg.lib()[name]
    f.argtypes, f.restype = args, res
    return f


def tile(M: int, K: int, N: int, out: str) -> str:
    """The kernel of a product [M][K] by [N][K]."""
    f = _symbol("_ZN2mg9f8_choiceEliib", [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_bool], _Choice)
    return TILES[f(M, N, K, out == "f32").tile]


def fused(M: int, F: int, C: int) -> tuple:
    """Whether the gate is formed in the product's epilogue: forward, forward with what is kept, gradient."""
    f = _symbol("_ZN2mg11gated_fusedEliii", [ctypes.c_int64] + 3 * [ctypes.c_int32], ctypes.c_bool)
    return tuple(bool(f(M, F, C, what)) for what in range(3))


def linear_direct(M: int, K: int, N: int) -> bool:
    """Whether a layer goes straight from its activations."""
    f = _symbol("_ZN2mg14f8_direct_paysElii", [ctypes.c_int64] + 2 * [ctypes.c_int32], ctypes.c_bool)
    return bool(f(M, K, N))


def gated_direct(M: int, K: int, F: int, N: int) -> bool:
    """Whether the gated block does."""
    f = _symbol("_ZN2mg20f8_direct_pays_gatedEliii", [ctypes.c_int64] + 3 * [ctypes.c_int32], ctypes.c_bool)
    return bool(f(M, K, F, N))


# (tile, output, M, K, N): ragged in both directions, K over several scale windows where it can be; the
# second size of a large tile has more tiles than workgroups
FORMS = [
    ("32 x 32", "bf16", 260, 4128, 288), ("32 x 64", "bf16", 45, 544, 2080), ("64 x 64", "bf16", 515, 1056, 1056),
    ("128 x 128", "bf16", 1550, 672, 2080), ("128 x 128", "bf16", 8200, 544, 1056),
    ("256 x 256", "bf16", 3000, 1056, 5152), ("256 x 256", "bf16", 8200, 1056, 5152),
    ("192 x 256", "bf16", 2055, 1056, 5152), ("192 x 256", "bf16", 8200, 1056, 4128),
    ("32 x 32", "f32", 260, 5120, 544), ("32 x 64", "f32", 45, 544, 2080), ("64 x 64", "f32", 515, 2080, 1056),
    ("128 x 128", "f32", 2055, 544, 2592), ("128 x 128", "f32", 8200, 1056, 4128),
    ("256 x 256", "f32", 2900, 1056, 4128), ("256 x 256", "f32", 8200, 2080, 5152),
]

# (tile, output, F, tokens, K) of dWg and dWu, rows of two outputs in turn; 192 x 256 is not built for two
# outputs and gives way to another
PAIRS = [
    ("32 x 64", "bf16", 416, 540, 288), ("128 x 128", "bf16", 1952, 1050, 2080), ("256 x 256", "bf16", 2848, 1050, 2592),
    ("192 x 256", "bf16", 2080, 1050, 2592), ("32 x 64", "f32", 2080, 1050, 544), ("128 x 128", "f32", 2336, 1050, 1568),
    ("256 x 256", "f32", 2080, 1050, 2592),
]

# (M, K, F, N) of gated blocks whose gate is formed in the epilogue in every form, K and N over several windows
GATED = [(2900, 1056, 2080, 672), (4100, 1056, 1056, 544)]
