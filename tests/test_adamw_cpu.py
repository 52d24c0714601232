"""AdamW's refusals, none of which needs a device: C statuses and Python errors."""
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


def _call(lib, b, count=1, lr=1e-3, wd=0.1, beta1=0.9, beta2=0.95, eps=1e-8, step=1, grad_scale=None, **change):
    t = b.MbAdamwTensor(GOOD, GOOD, GOOD, GOOD, None, None, None, 8, b.MB_F32, b.MB_F32, b.MB_F32, 1.0, 1.0)
    for k, v in change.items():
        setattr(t, k, v)
    return lib.adamw_multi_step((b.MbAdamwTensor * 1)(t), count, lr, wd, beta1, beta2, eps, step, grad_scale, 0, 0, None)


def test_statuses(lib, b):
    for name in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert _call(lib, b, **{name: None}) == b.MB_ERR_NULL
        assert _call(lib, b, **{name: GOOD + 2}) == b.MB_ERR_ALIGN
    assert _call(lib, b, param_type=b.MB_BF16, param=GOOD + 1) == b.MB_ERR_ALIGN
    assert _call(lib, b, param_type=b.MB_BF16, mantissa=GOOD + 1) == b.MB_ERR_ALIGN
    assert _call(lib, b, grad_scale=GOOD + 2) == b.MB_ERR_ALIGN
    assert _call(lib, b, state_type=b.MB_E4M3) == b.MB_ERR_NULL            # no scales
    assert _call(lib, b, state_type=b.MB_E4M3, avg_scale=GOOD, sq_scale=GOOD + 1) == b.MB_ERR_ALIGN
    for n in (-1, (1 << 40) + 1):
        assert _call(lib, b, n=n) == b.MB_ERR_SHAPE
    for change in ({"param_type": b.MB_I32}, {"grad_type": b.MB_E4M3}, {"state_type": b.MB_BF16}, {"mantissa": GOOD},
                   {"param_type": b.MB_F16, "mantissa": GOOD}, {"lr_mul": float("inf")}, {"wd_mul": float("nan")}):
        assert _call(lib, b, **change) == b.MB_ERR_ARG
    for change in ({"lr": float("nan")}, {"wd": float("inf")}, {"beta1": 1.0}, {"beta1": -0.1}, {"beta2": 1.0},
                   {"beta2": float("nan")}, {"eps": -1e-8}, {"eps": float("inf")}, {"step": 0}, {"step": -1},
                   {"step": (1 << 53) + 2}):
        assert _call(lib, b, **change) == b.MB_ERR_ARG
    for count in (-1, b.MB_ADAMW_MAX_TENSORS + 1):
        assert _call(lib, b, count=count) == b.MB_ERR_TOO_MANY
    assert lib.adamw_multi_step(None, 1, 0, 0, 0, 0, 0, 1, None, 0, 0, None) == b.MB_ERR_NULL
    assert lib.adamw_multi_step(None, 0, 0, 0, 0, 0, 0, 1, None, 0, 0, None) == b.MB_OK


def test_device_scalar_statuses(lib, b):
    t = b.MbAdamwTensor(GOOD, GOOD, GOOD, GOOD, None, None, None, 8, b.MB_F32, b.MB_F32, b.MB_F32, 1.0, 1.0)
    arr, need = (b.MbAdamwTensor * 1)(t), ctypes.c_size_t()
    assert lib.adamw_multi_step_dev_workspace_bytes(1, None) == b.MB_ERR_NULL
    assert lib.adamw_multi_step_dev_workspace_bytes(-1, ctypes.byref(need)) == b.MB_ERR_TOO_MANY
    assert lib.adamw_multi_step_dev_workspace_bytes(1, ctypes.byref(need)) == b.MB_OK

    def call(scalars=GOOD, ws=GOOD, nbytes=None):
        return lib.adamw_multi_step_dev(arr, 1, scalars, None, 0, 0, ws, need.value if nbytes is None else nbytes, None)

    assert call(scalars=None) == b.MB_ERR_NULL
    assert call(scalars=GOOD + 4) == b.MB_ERR_ALIGN
    assert call(ws=None) == b.MB_ERR_WORKSPACE
    assert call(nbytes=need.value - 1) == b.MB_ERR_WORKSPACE
    assert call(ws=GOOD + 8) == b.MB_ERR_ALIGN


def test_python_refusals_without_a_device(lib):
    import newton_schulz_stacked_gb300 as nss
    state = nss.adamw_state(torch.zeros(300), torch.zeros(300), bits=8)
    assert state.avg_scale.shape == (2,) and state.exp_avg.dtype == torch.float8_e4m3fn
    with pytest.raises(ValueError, match="CUDA"):
        nss.adamw_multi_step([state], 1e-3, 0.1)
    with pytest.raises(ValueError, match="no tensors"):
        nss.adamw_multi_step([], 1e-3, 0.1)
    with pytest.raises(ValueError, match="AdamState"):
        nss.adamw_multi_step([(1, 2)], 1e-3, 0.1)
    with pytest.raises(TypeError):
        nss.adamw_multi_step(7, 1e-3, 0.1)
    with pytest.raises(ValueError, match="bits"):
        nss.adamw_state(torch.zeros(3), bits=4)
