"""Host-side rules of the tile GEMM, evaluated by the library's own code."""
import ctypes

import numpy as np
import pytest

import fp8_weight_only_w4a16_b200 as sk

# Sizes that test_gpu_tile_widths.py runs, with the width that each of them means.
SILU_WIDE = [                                       # F, K, rows per expert
    (1410, 400, [300, 200, 1, 0], 128),             # 23 row tiles: the last pair has one
    (1500, 12000, [385], 128),                      # split along K
    (1030, 400, [400, 390, 5, 7, 300], 192),        # 17 row tiles
    (1000, 8192, [400, 390, 5, 7, 300], 192),       # split along K
    (3000, 2000, [100, 300, 1], 192),
]
STORE_WIDE = [                                      # format, N, K, rows per expert
    (0, 6000, 272, [300, 1, 0, 257], 128),          # several tiles of an expert
    (1, 6000, 272, [300, 1, 0, 257], 128),
    (1, 4000, 400, [400, 390, 5, 7, 300], 192),
    (0, 5003, 400, [385, 0, 577, 1], 192),          # last tiles of one row
]
INT8_LAST_TILE = [(4097, 5120, 256), (257, 40000, 272), (1025, 20000, 144), (4100, 5000, 512)]      # M, N, K


def tile_width(fmt, T, K, N, E, gate_up, workspace, sms):
    w = ctypes.c_int(0)
    status = sk.library().skinny_debug_tile_width(fmt, T, K, N, E, gate_up, workspace, sms, ctypes.byref(w))
    assert status == sk.OK, sk.status_string(status)
    return w.value


@pytest.mark.parametrize("width", [16, 32, 64, 128, 192, 256])
def test_columns_of_the_matrix_instruction(width):
    """One CTA's instruction of 128 rows takes its columns in steps of 16, a pair's of 256 rows in steps of 32."""
    step = 32 if width > 64 else 16
    for rows in range(1, width + 1):
        n = sk.library().skinny_debug_tile_columns(width, rows)
        assert n % step == 0 and n - step < rows <= n <= width


def test_no_such_tile():
    for width, rows in ((0, 1), (48, 1), (512, 1), (16, 0), (16, 17), (256, 257), (64, -1)):
        assert sk.library().skinny_debug_tile_columns(width, rows) == -1


@pytest.mark.parametrize("fmt,T,K,N,E,gate_up,width", [
    # the sizes of tests that mean a tile width, with and without a workspace
    *[(fmt, sum(c), K, 2 * F, len(c), 1, w) for fmt in (0, 1) for F, K, c, w in SILU_WIDE],
    *[(fmt, sum(c), K, N, len(c), 0, w) for fmt, N, K, c, w in STORE_WIDE],
    *[(-1, M, K, N, 1, 0, 256) for M, N, K in INT8_LAST_TILE],
    (0, 64, 5120, 5632, 128, 1, 16), (1, 64, 1408, 5120, 128, 0, 16), (0, 1003, 2048, 2051, 32, 0, 64),
    (0, 16387, 5120, 5632, 32, 1, 192), (-1, 1, 5120, 5120, 1, 0, 16), (-1, 61, 5120, 34816, 1, 0, 64),
    (-1, 2048, 5120, 34816, 1, 0, 256), (-1, 200, 4096, 6000, 1, 0, 128), (-1, 20, 5120, 300, 1, 0, 32),
])
def test_tile_width_on_148_sms(fmt, T, K, N, E, gate_up, width):
    for workspace in (0, 1):
        assert tile_width(fmt, T, K, N, E, gate_up, workspace, 148) == width


@pytest.mark.parametrize("fmt", [-1, 0, 1])
def test_tile_width_is_one_that_exists(fmt):
    rng = np.random.default_rng(fmt + 1)
    for _ in range(2000):
        T, K, N = (int(round(np.exp(rng.uniform(0, np.log(top))))) for top in (1 << 24, 4096, 1 << 16))
        E = 1 if fmt < 0 else int(rng.integers(1, 513))
        w = tile_width(fmt, T, 16 * K, 2 * N, E, int(fmt >= 0 and rng.random() < 0.5), int(rng.integers(2)),
                       int(rng.choice([1, 2, 7, 148, 160])))
        assert w in (16, 32, 64, 128, 256 if fmt < 0 else 192)
        assert w <= 64 or w <= 2 * T                    # no wide tiles for a few tokens


def test_tile_width_refusals():
    w = ctypes.c_int(0)
    call = sk.library().skinny_debug_tile_width
    good = [0, 10, 64, 128, 2, 0, 1, 148]
    assert call(*good, ctypes.byref(w)) == sk.OK and call(*good, None) == sk.ERR_INVALID_ARG
    for i, bad in ((0, 2), (0, -1), (1, 0), (1, -1), (2, 40), (3, 0), (4, 0), (7, 0)):
        assert call(*good[:i], bad, *good[i + 1:], ctypes.byref(w)) == sk.ERR_INVALID_ARG
    assert call(0, 10, 64, 129, 2, 1, 1, 148, ctypes.byref(w)) == sk.ERR_INVALID_ARG
    assert call(0, 10, 64, 128, 513, 0, 1, 148, ctypes.byref(w)) == sk.ERR_UNSUPPORTED
    assert call(-1, 10, 131072, 128, 1, 0, 1, 148, ctypes.byref(w)) == sk.ERR_UNSUPPORTED
