"""The block operators' refusals, none of which needs a device: C statuses and Python errors."""
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


def _norm(lib, x=GOOD, xs=64, kind=1, w=GOOD, bias=GOOD, wkind=0, y=GOOD, ys=64, mean=GOOD, rstd=GOOD, rows=4, cols=64,
          eps=1e-5):
    return lib.mb_layer_norm(x, xs, kind, w, bias, wkind, y, ys, mean, rstd, rows, cols, eps, None)


def test_layer_norm_statuses(lib, b):
    assert _norm(lib, x=None) == b.MB_ERR_NULL
    assert _norm(lib, y=None) == b.MB_ERR_NULL
    assert _norm(lib, x=GOOD + 1) == b.MB_ERR_ALIGN                # a bf16 needs 2 bytes
    assert _norm(lib, w=GOOD + 2) == b.MB_ERR_ALIGN                # an fp32 weight needs 4
    assert _norm(lib, mean=GOOD + 2) == b.MB_ERR_ALIGN
    for cols in (0, -1, (1 << 30) + 1):
        assert _norm(lib, cols=cols) == b.MB_ERR_SHAPE
    assert _norm(lib, rows=-1) == b.MB_ERR_SHAPE
    assert _norm(lib, xs=-64) == b.MB_ERR_SHAPE
    assert _norm(lib, ys=63) == b.MB_ERR_SHAPE                     # rows of the result would overlap
    assert _norm(lib, kind=3) == b.MB_ERR_ARG and _norm(lib, kind=9) == b.MB_ERR_ARG
    assert _norm(lib, wkind=2) == b.MB_ERR_ARG                     # neither the activations' type nor fp32
    for eps in (-1e-5, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == b.MB_ERR_ARG
    assert _norm(lib, x=None, y=None, mean=None, rstd=None, rows=0) == b.MB_OK


def _norm_back(lib, dy=GOOD, x=GOOD, xs=64, kind=1, w=GOOD, wkind=0, mean=GOOD, dx=GOOD, dxs=64, dw=GOOD, db=GOOD, rows=4,
               cols=64, ws=GOOD, nbytes=1 << 30):
    return lib.mb_layer_norm_backward(dy, 64, x, xs, kind, w, wkind, mean, GOOD, dx, dxs, dw, db, rows, cols, ws, nbytes,
                                      None)


def test_layer_norm_backward_statuses(lib, b):
    out = ctypes.c_size_t()
    assert lib.mb_layer_norm_workspace_bytes(4, 64, ctypes.byref(out)) == b.MB_OK
    assert out.value >= 2 * 64 * 4
    assert lib.mb_layer_norm_workspace_bytes(4, 0, ctypes.byref(out)) == b.MB_ERR_SHAPE
    assert lib.mb_layer_norm_workspace_bytes(4, 64, None) == b.MB_ERR_NULL
    assert _norm_back(lib, dy=None) == b.MB_ERR_NULL
    assert _norm_back(lib, mean=None) == b.MB_ERR_NULL
    assert _norm_back(lib, dx=GOOD + 1) == b.MB_ERR_ALIGN
    assert _norm_back(lib, dxs=8) == b.MB_ERR_SHAPE
    assert _norm_back(lib, wkind=2) == b.MB_ERR_ARG
    assert _norm_back(lib, ws=None) == b.MB_ERR_WORKSPACE
    assert _norm_back(lib, nbytes=out.value - 1) == b.MB_ERR_WORKSPACE
    assert _norm_back(lib, ws=GOOD + 16) == b.MB_ERR_ALIGN
    # nothing to do: no rows and no parameter gradients wanted
    assert _norm_back(lib, dy=None, x=None, mean=None, dx=None, dw=None, db=None, rows=0, ws=None, nbytes=0) == b.MB_OK


def _rotary_desc(b, **change):
    d = b.MbRotaryDesc()
    for x, heads in ((d.q, 4), (d.k, 2)):
        x.src = x.dst = GOOD
        x.heads = heads
        x.src_head = x.dst_head = 32
        x.src_token = x.dst_token = 32 * heads
        x.src_batch = x.dst_batch = 32 * heads * 5
    d.type, d.batch, d.tokens, d.dim, d.pairs = b.MB_BF16, 2, 5, 32, 16
    d.positions, d.position_type, d.pos_axis, d.pos_batch, d.pos_token = GOOD, b.MB_I32, 10, 5, 1
    d.axes, d.inv_freq = 2, GOOD
    d.sections[0] = d.sections[1] = 8
    for name, v in change.items():
        at, *rest = name.split("__")
        if rest:
            setattr(getattr(d, at), rest[0], v)
        elif at.startswith("section"):
            d.sections[int(at[-1])] = v
        else:
            setattr(d, at, v)
    return ctypes.addressof(d), d


@pytest.mark.parametrize("name", ["mb_rotary", "mb_rotary_backward"])
def test_rotary_statuses(lib, b, name):
    def call(**change):
        at, keep = _rotary_desc(b, **change)
        return getattr(lib, name)(at, None)
    assert getattr(lib, name)(None, None) == b.MB_ERR_NULL
    for change in (dict(q__src=0), dict(k__dst=0), dict(positions=0), dict(inv_freq=0)):
        assert call(**change) == b.MB_ERR_NULL, change
    for change in (dict(q__src=GOOD + 1), dict(k__dst=GOOD + 1), dict(positions=GOOD + 2), dict(inv_freq=GOOD + 2)):
        assert call(**change) == b.MB_ERR_ALIGN, change
    for change in (dict(pairs=0), dict(pairs=17), dict(dim=31), dict(dim=1 << 17), dict(axes=0), dict(axes=5),
                   dict(section0=7), dict(section0=-8, section1=24), dict(batch=-1), dict(tokens=-1),
                   dict(batch=1 << 16, tokens=1 << 15), dict(q__heads=-1), dict(q__heads=0, k__heads=0),
                   dict(q__heads=65535), dict(q__src_token=-1), dict(q__dst_head=0), dict(pos_token=-1)):
        assert call(**change) == b.MB_ERR_SHAPE, change
    for change in (dict(type=b.MB_I32), dict(type=7), dict(position_type=b.MB_BF16)):
        assert call(**change) == b.MB_ERR_ARG, change
    assert call(tokens=0, q__src=0, q__dst=0, k__src=0, k__dst=0, positions=0, inv_freq=0) == b.MB_OK


def _router(lib, logits=GOOD, stride=16, kind=0, valid=None, tokens=8, experts=16, k=2, index=GOOD, gate=GOOD, counts=GOOD,
            loss=GOOD, used=GOOD, ws=GOOD, nbytes=1 << 30):
    return lib.mb_router(logits, stride, kind, valid, tokens, experts, k, 0, index, gate, counts, loss, used, ws, nbytes,
                         None)


def test_router_statuses(lib, b):
    out = ctypes.c_size_t()
    assert lib.mb_router_workspace_bytes(8, 16, ctypes.byref(out)) == b.MB_OK and out.value == 0    # one CTA's work
    many = dict(tokens=100000)
    assert lib.mb_router_workspace_bytes(100000, 16, ctypes.byref(out)) == b.MB_OK and out.value > 0
    assert lib.mb_router_workspace_bytes(8, 1025, ctypes.byref(out)) == b.MB_ERR_SHAPE
    assert lib.mb_router_workspace_bytes(8, 16, None) == b.MB_ERR_NULL
    for name in ("logits", "index", "gate", "counts", "loss", "used"):
        assert _router(lib, **{name: None}) == b.MB_ERR_NULL, name
        assert _router(lib, **{name: GOOD + 1}) == b.MB_ERR_ALIGN, name
    for change in (dict(experts=0), dict(experts=1025), dict(k=0), dict(k=17), dict(experts=64, k=33), dict(tokens=-1),
                   dict(tokens=1 << 31), dict(tokens=1 << 30, k=2), dict(stride=-1)):
        assert _router(lib, **change) == b.MB_ERR_SHAPE, change
    assert _router(lib, kind=4) == b.MB_ERR_ARG
    assert _router(lib, ws=None, **many) == b.MB_ERR_WORKSPACE
    assert lib.mb_router_workspace_bytes(100000, 16, ctypes.byref(out)) == b.MB_OK
    assert _router(lib, nbytes=out.value - 1, **many) == b.MB_ERR_WORKSPACE
    assert _router(lib, ws=GOOD + 4, **many) == b.MB_ERR_ALIGN


def test_router_backward_statuses(lib, b):
    def call(dloss=GOOD, dgate=GOOD, logits=GOOD, stride=16, kind=0, tokens=8, experts=16, k=2, index=GOOD, gate=GOOD,
             counts=GOOD, used=GOOD, dlogits=GOOD, dstride=16):
        return lib.mb_router_backward(dloss, dgate, logits, stride, kind, None, tokens, experts, k, 0, index, gate, counts,
                                      used, dlogits, dstride, None)
    for name in ("logits", "index", "gate", "counts", "used", "dlogits"):
        assert call(**{name: None}) == b.MB_ERR_NULL, name
        assert call(**{name: GOOD + 1}) == b.MB_ERR_ALIGN, name
    assert call(dloss=GOOD + 2) == b.MB_ERR_ALIGN and call(dgate=GOOD + 2) == b.MB_ERR_ALIGN
    for change in (dict(experts=1025), dict(k=17), dict(dstride=15), dict(stride=-1)):
        assert call(**change) == b.MB_ERR_SHAPE, change
    assert call(kind=3) == b.MB_ERR_ARG
    assert call(tokens=0, logits=None, index=None, gate=None, dlogits=None) == b.MB_OK


def test_python_calls_require_cuda_tensors(lib):
    import newton_schulz_stacked_gb300 as nss
    x = torch.zeros(4, 8)
    pos, freq = torch.zeros(1, 4, dtype=torch.int32), torch.ones(4)
    for call in (lambda: nss.mb_layer_norm(x), lambda: nss.mb_layer_norm_backward(x, x, x[:, 0], x[:, 0]),
                 lambda: nss.mb_rotary(x[:, None], None, pos, freq, (4,)),
                 lambda: nss.mb_rotary_backward(x[:, None], None, pos, freq, (4,)), lambda: nss.mb_router(x, 2),
                 lambda: nss.mb_router_backward(None, None, x, pos, x, pos, pos)):
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            call()
