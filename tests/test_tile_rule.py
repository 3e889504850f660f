"""Host-side rules of the tile GEMM, evaluated by the library's own code."""
import pytest

import fp8_weight_only_w4a16_b200 as sk


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
