"""The layer norm's workspace: as many partial sums as its kernels write, and no more."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_stacked_gb300.build import build_all
    build_all()
    from newton_schulz_stacked_gb300 import _binding
    return _binding.load()


GOOD = 1 << 12      # aligned, never dereferenced: every call below fails its checks first


def _bytes(lib, rows, cols):
    out = ctypes.c_size_t()
    assert lib.mb_layer_norm_workspace_bytes(rows, cols, ctypes.byref(out)) == 0
    return out.value


@pytest.mark.parametrize("cols", [1, 768, 1025, 8192])
def test_rows_that_are_held(lib, cols):
    for rows, parts in ((0, 1), (1, 1), (17, 17), (456, 456), (457, 456), (1 << 20, 456)):
        assert _bytes(lib, rows, cols) == parts * 2 * cols * 4


@pytest.mark.parametrize("cols", [8193, 8200, 33001, 1 << 20, 1 << 30])
def test_wide_rows(lib, cols):
    """Rows that are read again add up in 64 slabs at most: 2^20 columns need 0.54 GB."""
    for rows, parts in ((0, 1), (1, 1), (63, 63), (64, 64), (65, 64), (456, 64), (1 << 20, 64)):
        assert _bytes(lib, rows, cols) == parts * 2 * cols * 4


def test_less_is_refused(lib):
    from newton_schulz_stacked_gb300 import _binding as b
    for cols in (8192, 8200):
        need = _bytes(lib, 300, cols)
        for nbytes in (0, need - 1):
            assert lib.mb_layer_norm_backward(GOOD, cols, GOOD, cols, b.MB_F32, GOOD, b.MB_F32, GOOD, GOOD, GOOD, cols, GOOD,
                                              GOOD, 300, cols, GOOD, nbytes, None) == b.MB_ERR_WORKSPACE
