"""The refusals of the products with bias, activation and residual, none of which needs a device."""
import ctypes

import pytest
import torch

GOOD = 1 << 12      # aligned, never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_stacked_gb300.build import build_all
    build_all()
    from newton_schulz_stacked_gb300 import _binding
    return _binding.load()


@pytest.fixture(scope="module")
def b():
    from newton_schulz_stacked_gb300 import _binding
    return _binding


def _desc(b, **change):
    d = b.MbLinearDesc(GOOD, GOOD, GOOD, GOOD, None, GOOD, GOOD, 64, 32, 32, 32, 10, 64, 32, 1, b.MB_BF16, b.MB_F32,
                       b.MB_ACT_RELU2)
    for k, v in change.items():
        setattr(d, k, v)
    return d


def _back(b, **change):
    d = b.MbLinearBackwardDesc(GOOD, GOOD, GOOD, GOOD, None, GOOD, GOOD, GOOD, 32, 64, 32, 64, 10, 64, 32, 1, b.MB_BF16,
                               b.MB_F32, b.MB_ACT_RELU2)
    for k, v in change.items():
        setattr(d, k, v)
    return d


SHAPES = [{"rows": -1}, {"rows": (1 << 30) + 1}, {"inputs": 0}, {"inputs": (1 << 20) + 1}, {"out": 0}, {"out": -8}, {"groups": 0},
          {"groups": 2}, {"groups": 1025, "ends": GOOD}, {"groups": 1024, "ends": GOOD, "inputs": 1 << 20, "out": 1 << 20}]


def test_forward_statuses(lib, b):
    need = ctypes.c_size_t()

    def size(**change):
        return lib.mb_linear_workspace_bytes(ctypes.byref(_desc(b, **change)), ctypes.byref(need))

    def call(ws=None, nbytes=0, **change):
        return lib.mb_linear(ctypes.byref(_desc(b, **change)), ws, nbytes, None)

    for f in (size, call):
        for name in ("x", "weight", "y"):
            assert f(**{name: None}) == b.MB_ERR_NULL
            assert f(**{name: GOOD + 1}) == b.MB_ERR_ALIGN
        for change in ({"residual": GOOD + 1}, {"z": GOOD + 1}, {"bias": GOOD + 2}, {"ends": GOOD + 2}):
            assert f(**change) == b.MB_ERR_ALIGN
        for change in SHAPES + [{"x_stride": -64}, {"y_stride": 31}, {"z_stride": 31}, {"residual_stride": -1},
                                {"y_stride": 1 << 40}]:
            assert f(**change) == b.MB_ERR_SHAPE, change
        for change in ({"type": b.MB_F32}, {"bias_type": b.MB_F16}, {"activation": 5}, {"activation": -1}):
            assert f(**change) == b.MB_ERR_ARG
    assert lib.mb_linear_workspace_bytes(None, ctypes.byref(need)) == b.MB_ERR_NULL
    assert lib.mb_linear_workspace_bytes(ctypes.byref(_desc(b)), None) == b.MB_ERR_NULL
    assert lib.mb_linear(None, None, 0, None) == b.MB_ERR_NULL
    assert size() == b.MB_OK and need.value == 0
    assert size(x=GOOD + 2) == b.MB_OK and need.value >= 10 * 64 * 2         # x is copied
    assert call(x=GOOD + 2) == b.MB_ERR_WORKSPACE
    assert call(x=GOOD + 2, ws=GOOD, nbytes=need.value - 1) == b.MB_ERR_WORKSPACE
    assert call(x=GOOD + 2, ws=GOOD + 128, nbytes=need.value) == b.MB_ERR_ALIGN
    assert size(inputs=65, x_stride=72) == b.MB_OK and need.value >= 32 * 72 * 2   # the weight is
    assert call(rows=0, x=None, y=None, weight=None) == b.MB_OK


def test_backward_statuses(lib, b):
    need = ctypes.c_size_t()

    def size(**change):
        return lib.mb_linear_backward_workspace_bytes(ctypes.byref(_back(b, **change)), ctypes.byref(need))

    def call(ws=None, nbytes=0, **change):
        return lib.mb_linear_backward(ctypes.byref(_back(b, **change)), ws, nbytes, None)

    for f in (size, call):
        for name in ("dy", "x", "weight", "z"):
            assert f(**{name: None}) == b.MB_ERR_NULL
            assert f(**{name: GOOD + 1}) == b.MB_ERR_ALIGN
        for change in ({"dx": GOOD + 1}, {"dweight": GOOD + 1}, {"dbias": GOOD + 2}, {"ends": GOOD + 1}):
            assert f(**change) == b.MB_ERR_ALIGN
        for change in SHAPES + [{"dy_stride": -1}, {"x_stride": -1}, {"z_stride": -1}, {"dx_stride": 63}]:
            assert f(**change) == b.MB_ERR_SHAPE, change
        for change in ({"type": b.MB_F32}, {"bias_type": b.MB_F16}, {"activation": 5}):
            assert f(**change) == b.MB_ERR_ARG
    assert size() == b.MB_OK and need.value >= 10 * 32 * 2 + 32 * 4           # dz, and the bias's sums
    assert call() == b.MB_ERR_WORKSPACE
    assert size(activation=b.MB_ACT_NONE, z=None, dbias=None) == b.MB_OK and need.value == 0
    assert size(weight=None, dx=None) == b.MB_OK and size(x=None, dweight=None) == b.MB_OK
    assert call(dx=None, dweight=None, dbias=None) == b.MB_OK                 # nothing is wanted


def test_python_refusals_without_a_device(lib):
    import newton_schulz_stacked_gb300 as nss
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(16, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nss.mb_linear(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        nss.mb_linear_backward(torch.zeros(4, 16, dtype=torch.bfloat16), x, w)
