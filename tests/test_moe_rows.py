"""The rows of W that one buffer of the grouped products covers (csrc/q4k_rows.h),
under the hardware's range check, on the host: nothing behind the matrix is read."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BLOCK_BYTES = 144

SHIM = '''
#include "{header}"
extern "C" void window(int n, int most, int N, int *out) {{
    constexpr q4k::RowWindow at_compile_time = q4k::row_window(5, 8, 9);
    static_assert(at_compile_time.first == 5 && at_compile_time.rows == 4, "");
    const q4k::RowWindow r = q4k::row_window(n, most, N);
    out[0] = r.first;
    out[1] = r.rows;
}}
'''


@pytest.fixture(scope="module")
def row_window(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src, so = str(d / "rows.cpp"), str(d / "librows.so")
    with open(src, "w") as f:
        f.write(SHIM.format(header=os.path.join(ROOT, "gguf_q4_dequant_amd", "csrc", "q4k_rows.h")))
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-o", so, src], check=True)
    lib = ctypes.CDLL(so)

    def window(n, most, N):
        out = (ctypes.c_int * 2)()
        lib.window(n, most, N, out)
        return out[0], out[1]
    return window


def _reads_behind(window, n, most, N, blocks):
    """Bytes behind the matrix's end that a copy of rows n .. n + most - 1 reads:
    lane offsets as the kernels form them, a scalar offset of 144 bytes a block,
    and the range check offset < size - scalar offset in 32 unsigned bits."""
    row_bytes = blocks * BLOCK_BYTES
    first, rows = window(n, most, N)
    size = rows * row_bytes
    piece = np.arange(9 * most)
    offset = (piece // 9) * row_bytes + (piece % 9) * 16
    behind = 0
    for b in range(blocks):
        read = offset < ((size - b * BLOCK_BYTES) & 0xFFFFFFFF)
        end = first * row_bytes + b * BLOCK_BYTES + offset + 16
        behind += int((read & (end > N * row_bytes)).sum())
        # every row that exists is read, each byte of it inside the row
        want = offset // row_bytes < rows
        assert np.array_equal(read, want), (n, most, N, b)
    return behind


@pytest.mark.parametrize("most", [16, 32])
def test_no_row_behind_the_matrix_is_read(row_window, most):
    for N in list(range(1, 70)) + [127, 128, 129, 1999]:
        for n in range(0, (N + 255) // 256 * 256, most):
            first, rows = row_window(n, most, N)
            assert rows >= 1 and 0 <= first and first + rows <= N and rows <= most
            if n < N:
                assert first == n and rows == min(most, N - n)
            for blocks in (1, 2, 5):
                assert _reads_behind(row_window, n, most, N, blocks) == 0, (n, most, N, blocks)


def test_an_empty_buffer_would_read_behind_the_matrix():
    """What the windows must not be: with no row, the check's difference wraps."""
    empty = lambda n, most, N: (min(n, N), max(0, min(most, N - n)))  # noqa: E731
    with pytest.raises(AssertionError):
        _reads_behind(empty, 64, 16, 33, 2)
