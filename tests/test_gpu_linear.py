"""Products with bias, activation and residual over groups of rows, and their gradients, against the formulas in 64 bits.

Tolerances.  A result's own rounding is half a step of its type (u = 2^-8 for bf16, 2^-11 for fp16, relative).  Products of
operands are exact in fp32 and their sum of K terms is off by at most K 2^-24 of the sum of the terms' magnitudes (and
far less where the signs vary; the tensor cores' own additions keep at least 2^-23 of the largest term): checked as
2^-22 sqrt(K) + 2^-21 of that sum.  dz is rounded to the operands' type (another u of every term of dx and dW).
Activations add 2^-20 of their value and pass on the error of z by their slope, at most 1.13 (silu, gelu) or 2 |z|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
ACTS = ["none", "relu", "relu2", "silu", "gelu"]


@pytest.fixture(scope="module")
def nss():
    from newton_schulz_stacked_gb300.build import build_all
    build_all()
    import newton_schulz_stacked_gb300 as nss
    return nss


def _gen(seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(n, cols, dtype, g, pad=0, shift=0, std=1.0):
    """[n, cols] with rows cols + pad apart, `shift` elements past a 16-byte boundary."""
    flat = (std * torch.randn(n * (cols + pad) + shift, generator=g, device="cuda")).to(dtype)
    return flat[shift:].view(n, cols + pad)[:, :cols]


def _act(z, kind):
    k = 2 * math.sqrt(2 / math.pi)
    return {"none": lambda: z, "relu": lambda: z.clamp(min=0), "relu2": lambda: z.clamp(min=0) ** 2,
            "silu": lambda: z * torch.sigmoid(z), "gelu": lambda: z * torch.sigmoid(k * (z + 0.044715 * z ** 3))}[kind]()


def _slope(z, kind):
    if kind == "relu":                           # 0 at 0
        return (z > 0).to(z.dtype)
    z = z.detach().requires_grad_()
    _act(z, kind).sum().backward()
    return z.grad


def _bounds(ends, rows):
    ends = [rows] if ends is None else ends
    return list(zip([0] + ends[:-1], ends))


def _add(K):
    return 2.0 ** -22 * math.sqrt(K) + 2.0 ** -21


def _near(got, want, slack):
    """|got - want| <= half a step of the result + slack (what the sums may be off by)."""
    u = HALF_STEP[got.dtype]
    floor = 2.0 ** -25 if got.dtype == torch.float16 else 0            # half of the least subnormal
    off = (got.double() - want).abs()
    bad = ~(off <= u * (want.abs() + slack) + slack + floor)
    assert not bad.any(), (bad.sum().item(), off.max().item(), bad.nonzero()[:4].tolist())


def _check_forward(nss, x, w, bias, residual, act, ends, keep=True, **given):
    rows, out = x.shape[0], w.shape[-2]
    dev_ends = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    y, z = nss.mb_linear(x, w, bias, residual, act, dev_ends, keep=keep, **given)
    want_y, want_z, slack = (torch.zeros(rows, out, dtype=torch.double, device="cuda") for _ in range(3))
    ws, bs = (w[None], None if bias is None else bias[None]) if ends is None else (w, bias)
    for g, (a, e) in enumerate(_bounds(ends, rows)):
        zz = x[a:e].double() @ ws[g].double().T
        slack[a:e] = _add(x.shape[1]) * (x[a:e].double().abs() @ ws[g].double().abs().T)
        if bias is not None:
            zz = zz + bs[g].double()
            slack[a:e] += 2.0 ** -23 * bs[g].double().abs()
        want_z[a:e] = zz
        want_y[a:e] = _act(zz, act) + (0 if residual is None else residual[a:e].double())
    if keep:
        _near(z, want_z, slack)
    else:
        assert z is None
    gain = {"none": 1.0, "relu": 1.0, "silu": 1.13, "gelu": 1.13}.get(act)
    slack = slack * (gain if gain else 2 * want_z.abs() + slack) + 2.0 ** -20 * (want_y.abs() + want_z.abs())
    _near(y, want_y, slack)
    return y, z


def _check_backward(nss, dy, x, w, z, act, ends, bias=True, **given):
    rows = x.shape[0]
    dev_ends = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    dx, dw, db = nss.mb_linear_backward(dy, x, w, z, act, dev_ends, bias=bias, **given)
    u = HALF_STEP[x.dtype] if act != "none" else 0
    tiny = 2.0 ** -25 if x.dtype == torch.float16 and act != "none" else 0
    want_dx, slack_dx = torch.zeros(x.shape, dtype=torch.double, device="cuda"), torch.zeros(x.shape, dtype=torch.double, device="cuda")
    ws = w[None] if ends is None else w
    dws, dbs = (None if t is None else t[None] if ends is None else t for t in (dw, db))
    for g, (a, e) in enumerate(_bounds(ends, rows)):
        dz = dy[a:e].double()
        if act != "none":
            dz = dz * _slope(z[a:e].double(), act)
        size = dz.abs()
        W, X = ws[g].double(), x[a:e].double()
        want_dx[a:e] = dz @ W
        slack_dx[a:e] = ((u + 2.0 ** -18) * size + tiny) @ W.abs() + _add(W.shape[0]) * (size @ W.abs())
        n = max(e - a, 1)
        if dws is not None:
            _near(dws[g], dz.T @ X, ((u + 2.0 ** -18) * size + tiny).T @ X.abs() + _add(n) * (size.T @ X.abs()))
        if dbs is not None:
            _near(dbs[g], dz.sum(0), (_add(n) + 2.0 ** -18) * size.sum(0))
    if dx is not None:
        _near(dx, want_dx, slack_dx)
    return dx, dw, db


@pytest.mark.parametrize("rows,cols,out", [(1, 8, 8), (1, 64, 64), (7, 40, 24), (64, 768, 768), (128, 64, 256), (129, 72, 264),
                                           (255, 128, 128), (256, 256, 256), (257, 320, 520), (1000, 200, 1000), (3000, 64, 40), (511, 264, 40), (512, 64, 264),
                                           (513, 64, 264), (520, 8, 8), (600, 768, 768), (769, 72, 264)])
def test_forward_sizes(nss, rows, cols, out):
    g = _gen(rows + cols)
    x, w = _rows(rows, cols, torch.bfloat16, g), _rows(out, cols, torch.bfloat16, g, std=cols ** -0.5)
    _check_forward(nss, x, w, None, None, "none", None)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(None, False), ("own", True), ("f32", False), (None, True)])
@pytest.mark.parametrize("rows", [300, 600])
def test_forward_epilogues(nss, dtype, act, bias, residual, rows):
    g, t = _gen(3), TYPES[dtype]
    cols, out = 136, 392
    x, w = _rows(rows, cols, t, g), _rows(out, cols, t, g, std=cols ** -0.5)
    b = None if bias is None else torch.randn(out, generator=g, device="cuda").to(t if bias == "own" else torch.float32)
    r = _rows(rows, out, t, g) if residual else None
    _check_forward(nss, x, w, b, r, act, None)
    _check_forward(nss, x, w, b, r, act, None, keep=False)


@pytest.mark.parametrize("cols,out,pad,shift", [(7, 5, 0, 0), (65, 67, 0, 0), (64, 64, 8, 0), (64, 64, 3, 0), (64, 64, 0, 1),
                                                (64, 66, 2, 2), (129, 1, 0, 0), (1, 130, 0, 0), (1, 1, 0, 0), (61, 61, 3, 0),
                                                (63, 191, 1, 8), (64, 333, 3, 0)])
@pytest.mark.parametrize("rows", [270, 530])
def test_forward_layouts(nss, cols, out, pad, shift, rows):
    """Odd widths, rows and tensors off 16-byte boundaries, results in wider buffers (whose other columns stay)."""
    g = _gen(5)
    t = torch.bfloat16
    x, w = _rows(rows, cols, t, g, pad, shift), _rows(out, cols, t, g, 0, shift, std=cols ** -0.5)
    r, b = _rows(rows, out, t, g, pad, shift), torch.randn(out, generator=g, device="cuda").to(t)
    whole = [torch.full((rows * (out + pad) + shift,), 7.0, device="cuda", dtype=t) for _ in range(2)]
    y, z = (f[shift:].view(rows, out + pad)[:, :out] for f in whole)
    _check_forward(nss, x, w, b, r, "silu", None, y=y, z=z)
    for f in whole:
        assert (f[:shift] == 7).all() and (f[shift:].view(rows, out + pad)[:, out:] == 7).all()
    want, _ = _check_forward(nss, x, w, b, r, "relu", None)
    y.copy_(r)
    nss.mb_linear(x, w, b, y, "relu", y=y)                                  # over the residual
    assert torch.equal(y, want)


GROUPS = [[10, 10, 300, 301, 690], [0, 0, 0], [256, 512], [700], [1, 2, 3, 4, 5, 6, 7, 700], [0, 700], [63, 64, 128, 193, 650]]


@pytest.mark.parametrize("ends", GROUPS)
@pytest.mark.parametrize("out", [200, 131])
def test_forward_groups(nss, ends, out):
    g, rows, cols, t = _gen(7), 700, 72, torch.bfloat16
    x, w = _rows(rows, cols, t, g), (torch.randn(len(ends), out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    b, r = torch.randn(len(ends), out, generator=g, device="cuda"), _rows(rows, out, t, g)
    y = torch.full((rows, out), 7.0, device="cuda", dtype=t)
    y, z = _check_forward(nss, x, w, b, r, "gelu", ends, y=y)
    assert not y[ends[-1]:].any() and not z[ends[-1]:].any()


@pytest.mark.parametrize("n", [140, 141, 1024])
def test_many_groups(nss, n):
    """Up to the most groups that a call takes, most of them small, some empty; with a residual."""
    g, cols, out, t = _gen(n), 64, 64, torch.bfloat16
    sizes = torch.randint(0, 9, (n,), generator=g, device="cuda")
    sizes[100], sizes[50] = 700, 0
    ends = sizes.cumsum(0).tolist()
    x, w = _rows(ends[-1] + 5, cols, t, g), (torch.randn(n, out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    dev = torch.tensor(ends, dtype=torch.int32, device="cuda")
    r = _rows(ends[-1] + 5, out, t, g)
    y, _ = nss.mb_linear(x, w, residual=r, ends=dev)
    dy = _rows(ends[-1] + 5, out, t, g)
    dx, dw, _ = nss.mb_linear_backward(dy, x, w, ends=dev)
    which = torch.bucketize(torch.arange(ends[-1], device="cuda"), dev, right=True)
    X, D = x[:ends[-1]].double(), dy[:ends[-1]].double()
    W = w.double()[which]
    _near(y[:ends[-1]], torch.einsum("ti,toi->to", X, W) + r[:ends[-1]].double(),
          _add(cols) * torch.einsum("ti,toi->to", X.abs(), W.abs()) + 2.0 ** -23 * r[:ends[-1]].double().abs())
    _near(dx[:ends[-1]], torch.einsum("to,toi->ti", D, W), _add(out) * torch.einsum("to,toi->ti", D.abs(), W.abs()))
    want, size = (torch.zeros(n, out, cols, dtype=torch.double, device="cuda") for _ in range(2))
    want.index_add_(0, which, D[:, :, None] * X[:, None, :])
    size.index_add_(0, which, (D[:, :, None] * X[:, None, :]).abs())
    _near(dw, want, _add(700) * size)
    assert not y[ends[-1]:].any() and not dx[ends[-1]:].any() and not dw[50].any()


@pytest.mark.parametrize("rows,cols,out", [(1, 8, 8), (7, 40, 24), (64, 64, 64), (128, 128, 256), (129, 72, 264), (1000, 200, 520),
                                           (5000, 256, 256)])
def test_backward_sizes(nss, rows, cols, out):
    g, t = _gen(rows + out), torch.bfloat16
    x, w, dy = _rows(rows, cols, t, g), _rows(out, cols, t, g, std=cols ** -0.5), _rows(rows, out, t, g)
    _check_backward(nss, dy, x, w, None, "none", None)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ACTS)
def test_backward_activations(nss, dtype, act):
    g, t, rows, cols, out = _gen(11), TYPES[dtype], 500, 136, 200
    x, w, dy, z = _rows(rows, cols, t, g), _rows(out, cols, t, g, std=cols ** -0.5), _rows(rows, out, t, g), _rows(rows, out, t, g)
    z[0, :40] = 0.0
    z[1, :40], z[2, :40] = 12.0, -12.0
    _check_backward(nss, dy, x, w, z, act, None)
    dbias = torch.empty(out, device="cuda")
    _, _, db = _check_backward(nss, dy, x, w, z, act, None, dbias=dbias)
    assert db is dbias
    for wanted in range(8):                      # any of the three results alone
        which = {"input_grad": bool(wanted & 1), "weight_grad": bool(wanted & 2), "bias": bool(wanted & 4)}
        got = _check_backward(nss, dy, x, w, z, act, None, **which)
        assert [r is not None for r in got] == list(which.values())


@pytest.mark.parametrize("cols,out,pad,shift", [(7, 5, 0, 0), (65, 67, 0, 0), (64, 64, 8, 0), (64, 66, 3, 1), (129, 1, 0, 0),
                                                (1, 130, 0, 0), (1, 1, 0, 0), (61, 61, 3, 0), (191, 63, 1, 8)])
@pytest.mark.parametrize("act", ["none", "relu2"])
def test_backward_layouts(nss, cols, out, pad, shift, act):
    g, rows, t = _gen(13), 270, torch.bfloat16
    x, w = _rows(rows, cols, t, g, pad, shift), _rows(out, cols, t, g, 0, shift, std=cols ** -0.5)
    dy, z = _rows(rows, out, t, g, pad, shift), _rows(rows, out, t, g, pad, shift)
    whole = torch.full((rows * (cols + pad) + shift,), 7.0, device="cuda", dtype=t)
    dx = whole[shift:].view(rows, cols + pad)[:, :cols]
    _check_backward(nss, dy, x, w, z, act, None, dx=dx)
    assert (whole[:shift] == 7).all() and (whole[shift:].view(rows, cols + pad)[:, cols:] == 7).all()


@pytest.mark.parametrize("ends", GROUPS)
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("cols,out", [(72, 200), (131, 77)])
def test_backward_groups(nss, ends, act, cols, out):
    """Nothing crosses from group to group: the rows behind the last group hold NaN, one group holds infinities."""
    g, rows, t = _gen(15), 700, torch.bfloat16
    x, w = _rows(rows, cols, t, g), (torch.randn(len(ends), out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    dy, z = _rows(rows, out, t, g), _rows(rows, out, t, g)
    for tensor in (x, dy, z):
        tensor[ends[-1]:] = math.nan
    dx, dw, db = _check_backward(nss, dy, x, w, z, act, ends)
    assert not dx[ends[-1]:].any()
    for i, (a, e) in enumerate(_bounds(ends, rows)):
        assert e > a or (not dw[i].any() and not db[i].any())
    if len(ends) == 5:                           # what group 2 has of infinities and NaN stays in it
        a, e = _bounds(ends, rows)[2]
        x[a:e] = math.inf
        dy[a:e] = math.nan
        dev = torch.tensor(ends, dtype=torch.int32, device="cuda")
        dx2, dw2, db2 = nss.mb_linear_backward(dy, x, w, z, act, dev, bias=True)
        for i in (0, 1, 3, 4):
            assert torch.equal(dw2[i], dw[i]) and torch.equal(db2[i], db[i])
        assert torch.equal(dx2[:a], dx[:a]) and torch.equal(dx2[e:], dx[e:])
        assert dw2[2].isnan().all() and dx2[a:e].isnan().all()


def test_long_contractions_are_cut(nss):
    """Few tiles and long sums: parts in the workspace, joined in order, the same bits each time."""
    g, t = _gen(17), torch.bfloat16
    x, w, b = _rows(200, 20000, t, g), _rows(96, 20000, t, g, std=20000 ** -0.5), torch.randn(96, generator=g, device="cuda")
    before = nss.mb_launch_count()
    y, z = _check_forward(nss, x, w, b, _rows(200, 96, t, g), "relu2", None)
    assert nss.mb_launch_count() - before == 2
    x, dy, w = _rows(40000, 200, t, g), _rows(40000, 300, t, g), _rows(300, 200, t, g, std=200 ** -0.5)
    first = _check_backward(nss, dy, x, w, None, "none", None)
    again = nss.mb_linear_backward(dy, x, w, bias=True)
    for a, c in zip(first, again):
        assert torch.equal(a, c)
    ends = [39000, 39037]
    w2 = (torch.randn(2, 300, 200, generator=g, device="cuda") * 200 ** -0.5).to(t)
    _check_backward(nss, dy, x, w2, None, "none", ends)


@pytest.mark.parametrize("ends", [None, [6001, 6001, 6100, 19990], [20000], [0, 3]])
@pytest.mark.parametrize("act,dtype", [("relu2", "bf16"), ("gelu", "f16")])
def test_large_backward_forms_dz_under_the_products(nss, ends, act, dtype):
    """dz in pieces by the products' launch; the same bits each time, any of the results alone."""
    g, t, rows, cols, out = _gen(27), TYPES[dtype], 20000, 72, 2528
    x, dy, z = _rows(rows, cols, t, g), _rows(rows, out, t, g), _rows(rows, out, t, g)
    n = 1 if ends is None else len(ends)
    w = (torch.randn(n, out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    w = w[0] if ends is None else w
    for tensor in (x, dy, z):
        if ends is not None:
            tensor[ends[-1]:] = math.nan
    first = _check_backward(nss, dy, x, w, z, act, ends)
    dev = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    workspace = torch.full((1 << 27,), 0xFF, dtype=torch.uint8, device="cuda")          # NaN everywhere
    again = nss.mb_linear_backward(dy, x, w, z, act, dev, bias=True, workspace=workspace)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    for wanted in range(1, 7):
        which = {"input_grad": bool(wanted & 1), "weight_grad": bool(wanted & 2), "bias": bool(wanted & 4)}
        got = _check_backward(nss, dy, x, w, z, act, ends, workspace=workspace, **which)
        assert [r is not None for r in got] == list(which.values())
    assert nss.mb_sync_status() == 0


def test_rows_of_any_shape(nss):
    """More dimensions than two, rows all the same (a stride of 0), every second row."""
    g, t = _gen(29), torch.bfloat16
    w = _rows(96, 64, t, g, std=0.125)
    x = _rows(24, 64, t, g)
    flat, _ = nss.mb_linear(x, w)
    y, _ = nss.mb_linear(x.view(2, 3, 4, 64), w)
    assert y.shape == (2, 3, 4, 96) and torch.equal(y.view(24, 96), flat)
    one, _ = nss.mb_linear(x[0], w)
    assert one.shape == (96,) and torch.equal(one, flat[0])
    y, _ = nss.mb_linear(x[:1].expand(300, 64), w)
    assert torch.equal(y, flat[:1].expand(300, 96))
    y, _ = nss.mb_linear(x[::2], w)
    assert torch.equal(y, flat[::2])
    dy = _rows(24, 96, t, g)
    dx, dw, _ = nss.mb_linear_backward(dy, x, w)
    dx2, dw2, _ = nss.mb_linear_backward(dy.view(4, 6, 96), x.view(4, 6, 64), w)
    assert dx2.shape == (4, 6, 64) and torch.equal(dx2.view(24, 64), dx) and torch.equal(dw2, dw)
    _, dw3, _ = nss.mb_linear_backward(dy[:1].expand(8, 96), x[:8], w, input_grad=False)
    _near(dw3, dy[:1].expand(8, 96).double().T @ x[:8].double(), _add(8) * (dy[:1].expand(8, 96).double().abs().T @ x[:8].double().abs()))


def test_host_threads(nss):
    """Calls of two threads on streams of their own."""
    import threading
    g, t = _gen(31), torch.bfloat16
    x, w, dy = _rows(512, 128, t, g), _rows(256, 128, t, g, std=0.09), _rows(512, 256, t, g)
    want = (*nss.mb_linear(x, w, activation="gelu", keep=True), *nss.mb_linear_backward(dy, x, w))
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(200):
                got = (*nss.mb_linear(x, w, activation="gelu", keep=True), *nss.mb_linear_backward(dy, x, w))
        stream.synchronize()
        wrong.extend(1 for a, b in zip(got, want) if a is not b and not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_nothing(nss):
    w, ends = torch.ones(2, 16, 8, device="cuda", dtype=torch.bfloat16), torch.zeros(2, device="cuda", dtype=torch.int32)
    x, dy = torch.ones(0, 8, device="cuda", dtype=torch.bfloat16), torch.ones(0, 16, device="cuda", dtype=torch.bfloat16)
    y, z = nss.mb_linear(x, w, ends=ends, keep=True)
    assert y.shape == z.shape == (0, 16)
    dx, dw, db = nss.mb_linear_backward(dy, x, w, ends=ends, bias=True)
    assert dx.shape == (0, 8) and not dw.any() and not db.any()


@pytest.mark.parametrize("rows", [300, 600])
def test_values_that_are_no_numbers(nss, rows):
    """A NaN or an infinity of a row stays in the row; through the activations as in torch."""
    g, t = _gen(19), torch.bfloat16
    x, w = _rows(rows, 64, t, g), _rows(128, 64, t, g, std=0.125)
    for act in ACTS:
        x[5, 3], x[6, 3], x[7, 3] = math.nan, math.inf, 1e30
        y, z = nss.mb_linear(x, w, activation=act, keep=True)
        want = _act(z.float(), act).to(t)
        assert torch.equal(y.isnan()[[5, 6]], want.isnan()[[5, 6]])
        assert z[5].isnan().all() and y[5].isnan().all()
        keep = [i for i in range(rows) if i not in (5, 6, 7)]
        assert y[keep].isfinite().all()


def test_bad_ends_are_held_and_reported(nss):
    from newton_schulz_stacked_gb300 import _binding as b
    g, t = _gen(21), torch.bfloat16
    x, w = _rows(100, 64, t, g), (torch.randn(3, 64, 64, generator=g, device="cuda") * 0.125).to(t)
    assert nss.mb_sync_status() == 0
    for bad, held in (([50, 20, 80], [50, 50, 80]), ([10, 20, 300], [10, 20, 100]), ([-5, 20, 60], [0, 20, 60])):
        y, _ = nss.mb_linear(x, w, ends=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert nss.mb_sync_status() == b.MB_ERR_ARG
        want, _ = nss.mb_linear(x, w, ends=torch.tensor(held, dtype=torch.int32, device="cuda"))
        assert nss.mb_sync_status() == 0
        assert torch.equal(y, want)


def test_streams_and_graphs(nss):
    """Several calls at once on streams of their own, and two graphs replayed with new ends and inputs."""
    g, t = _gen(23), torch.bfloat16
    x, w = _rows(2000, 128, t, g), (torch.randn(4, 256, 128, generator=g, device="cuda") * 0.09).to(t)
    dy = _rows(2000, 256, t, g)
    ends = torch.tensor([100, 700, 700, 1990], dtype=torch.int32, device="cuda")
    y, z = nss.mb_linear(x, w, activation="silu", ends=ends, keep=True)
    grads = nss.mb_linear_backward(dy, x, w, z, "silu", ends, bias=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        got.append((nss.mb_linear(x, w, activation="silu", ends=ends, keep=True, stream=s),
                    nss.mb_linear_backward(dy, x, w, z, "silu", ends, bias=True, stream=s)))
    torch.cuda.synchronize()
    for (a, b), back in got:
        assert torch.equal(a, y) and torch.equal(b, z)
        assert all(torch.equal(p, q) for p, q in zip(back, grads))
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o = nss.mb_linear(x, w, activation="silu", ends=ends, keep=True)
            outs.append((*o, *nss.mb_linear_backward(dy, x, w, o[1], "silu", ends, bias=True)))
        graphs.append(graph)
    ends.copy_(torch.tensor([1, 900, 1500, 1500], dtype=torch.int32))
    x.mul_(0.5)
    for graph in graphs:
        graph.replay()
    y, z = nss.mb_linear(x, w, activation="silu", ends=ends, keep=True)
    want = (y, z, *nss.mb_linear_backward(dy, x, w, z, "silu", ends, bias=True))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, want))
    assert nss.mb_sync_status() == 0


def test_autograd(nss):
    """Through torch's autograd: the gradients of a run of products, against the same in 64 bits and against differences."""
    from newton_schulz_stacked_gb300 import autograd
    g, t = _gen(25), torch.bfloat16
    make = lambda *s, std=1.0: (std * torch.randn(*s, generator=g, device="cuda")).to(t).requires_grad_()   # noqa: E731
    x, up, down = make(300, 64), make(3, 128, 64, std=0.125), make(3, 64, 128, std=0.09)
    b1, b2 = torch.randn(3, 128, generator=g, device="cuda").requires_grad_(), make(3, 64)
    ends = torch.tensor([100, 180, 290], dtype=torch.int32, device="cuda")
    leaves = [x, up, b1, down, b2]
    seed = torch.randn(300, 64, generator=g, device="cuda")

    def run(x, up, b1, down, b2, linear):
        h = linear(x, up, b1, None, "relu2", ends)
        return linear(h, down, b2, x, "none", ends)

    def plain(x, w, b, residual, act, ends):
        rows, a = [], 0
        for i, e in enumerate(ends.tolist()):
            y = _act(x[a:e] @ w[i].T + b[i], act)
            rows.append(y if residual is None else y + residual[a:e])
            a = e
        rows.append(x.new_zeros(len(x) - a, w.shape[1]))
        return torch.cat(rows)

    (run(*leaves, autograd.linear).float() * seed).sum().backward()
    wide = [l.detach().double().requires_grad_() for l in leaves]
    out = run(*wide, plain)
    (out * seed).sum().backward()
    for a, b in zip(leaves, wide):
        assert a.grad.dtype == a.dtype
        # five roundings of 2^-8 (h, z, two dz, the result), each at most half a step of a term of a sum of random signs
        assert (a.grad.double() - b.grad).norm() <= 5 * 2.0 ** -8 * b.grad.norm()
    # along a direction: differences of the 64-bit run, which the gradients above must reproduce
    for i, l in enumerate(wide):
        d = torch.randn(l.shape, generator=g, device="cuda", dtype=torch.double)
        h = 1e-6
        ahead = [p.detach() + (h * d if j == i else 0) for j, p in enumerate(wide)]
        behind = [p.detach() - (h * d if j == i else 0) for j, p in enumerate(wide)]
        slope = ((run(*ahead, plain) - run(*behind, plain)) * seed).sum() / (2 * h)
        assert abs(slope - (leaves[i].grad.double() * d).sum()) <= 5 * 2.0 ** -8 * leaves[i].grad.double().norm() * d.norm() / 8 + 1e-3
    # frozen parameters have none; second derivatives are refused
    y = autograd.linear(x, up.detach(), None, None, "gelu", ends)
    (gx,) = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second"):
        torch.autograd.grad(gx.float().sum(), x)


def test_refusals(nss):
    t = torch.bfloat16
    x, w, b = (torch.ones(*s, device="cuda", dtype=t) for s in ((4, 8), (16, 8), (16,)))
    bank, ends = w.expand(2, 16, 8).contiguous(), torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    y, dy = torch.zeros(4, 16, device="cuda", dtype=t), torch.ones(4, 16, device="cuda", dtype=t)

    def refused(match, *args, f=nss.mb_linear, **more):
        with pytest.raises(ValueError, match=match):
            f(*args, **more)

    refused("float32|Float", x.float(), w)
    refused("weight", x, w.half())
    refused("last dimension", x[:, :7], w)
    refused("weight", x, w[:, ::2])
    refused("ends", x, bank)
    refused("ends", x, w, ends=ends)
    refused("ends", x, bank, ends=ends.long())
    refused("ends", x, bank, ends=ends[:1])
    refused("bias", x, w, b[:15])
    refused("bias", x, w, b.half())
    refused("bias", x, bank, b, ends=ends)
    refused("residual", x, w, None, y[:, :15])
    refused("activation", x, w, activation="tanh")
    refused("activation", x, w, activation=1)
    refused("y", x, w, y=y.half())
    refused("contiguous", x.t().contiguous().t(), w)
    refused("cpu", x, w.cpu())
    refused("z", dy, x, w, activation="relu", f=nss.mb_linear_backward)
    refused("dy", dy[:, :8], x, w, f=nss.mb_linear_backward)
    refused("dweight", dy, x, w, dweight=torch.ones(16, 16, device="cuda", dtype=t)[:, :8], f=nss.mb_linear_backward)
    refused("dbias", dy, x, w, dbias=b.half(), f=nss.mb_linear_backward)
    refused("workspace", dy, x, w, torch.ones_like(dy), "relu", workspace=torch.empty(8, device="cuda", dtype=torch.uint8),
            f=nss.mb_linear_backward)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,cols,out,pad", [(1, 1, 1, 0), (1, 8, 8, 0), (1, 2048, 4096, 0), (2, 1000, 2000, 0), (26, 512, 77, 3),
                                               (31, 65, 1000, 0), (200, 72, 10, 0), (256, 8, 300, 8), (2, 2816, 768, 0)])
@pytest.mark.parametrize("groups", [0, 4])
def test_few_rows_keep_dz_in_two_halves(nss, dtype, rows, cols, out, pad, groups):
    """With up to 2048 elements of x or y dz is not rounded to 16 bits: what its halves leave is u^2 of it (fp16: half of the least
    subnormal at least), over twice the terms."""
    g, t = _gen(rows + cols), TYPES[dtype]
    shape = (groups, out, cols) if groups else (out, cols)
    ends = [rows // 3, rows // 3, rows - rows // 5, rows - rows // 8] if groups else None
    bounds, u = _bounds(ends, rows), HALF_STEP[t] ** 2
    x, dy, z = _rows(rows, cols, t, g, pad), _rows(rows, out, t, g, pad), _rows(rows, out, t, g, pad)
    w = (torch.randn(shape, generator=g, device="cuda") * cols ** -0.5).to(t)
    if groups:
        for tensor in (x, dy, z):
            tensor[ends[-1]:] = math.nan
    dev = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    workspace = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device="cuda")          # NaN everywhere
    tiny = 2.0 ** -25 if dtype == "f16" else 0
    for act in ACTS[1:]:
        dx, dw, db = nss.mb_linear_backward(dy, x, w, z, act, dev, bias=True, workspace=workspace)
        _check_backward(nss, dy, x, w, z, act, ends)
        for i, (a, e) in enumerate(bounds):
            W, X, D = (w[i] if groups else w).double(), x[a:e].double(), dy[a:e].double() * _slope(z[a:e].double(), act)
            off = (u + 2.0 ** -18) * D.abs() + tiny
            _near(dx[a:e], D @ W, off @ W.abs() + _add(2 * out) * (D.abs() @ W.abs()))
            _near(dw[i] if groups else dw, D.T @ X, off.T @ X.abs() + _add(2 * max(e - a, 1)) * (D.abs().T @ X.abs()))
        assert not dx[bounds[-1][1]:].any()
        for which in ({"input_grad": False}, {"weight_grad": False}):
            one = nss.mb_linear_backward(dy, x, w, z, act, dev, workspace=workspace, **which)
            for got, want in ((one[0], dx), (one[1], dw)):
                assert got is None or torch.allclose(got.float(), want.float(), rtol=4 * HALF_STEP[t], atol=1e-3)
    assert nss.mb_sync_status() == 0


def test_dz_past_the_type_is_infinite(nss):
    """fp16: a dz past 65504 makes its sums infinite, not NaN, with few rows (two halves) as with many."""
    for rows in (2, 3000):
        x, w = torch.ones(rows, 64, device="cuda", dtype=torch.float16), torch.ones(64, 64, device="cuda", dtype=torch.float16)
        dy, z = torch.ones_like(x), torch.ones_like(x)
        dy[1, 3] = z[1, 3] = 30000.0
        dx, dw, _ = nss.mb_linear_backward(dy, x, w, z, "relu2")
        assert (dx[1] == math.inf).all() and dx[0].eq(128).all()
        assert (dw[3] == math.inf).all() and dw[:3].isfinite().all() and dw[4:].isfinite().all()


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("cols,out,pad,shift", [(1, 1, 0, 0), (8, 8, 0, 0), (768, 768, 0, 0), (4096, 1001, 0, 0), (2056, 130, 8, 0),
                                                (257, 66, 0, 0), (64, 67, 3, 1), (5000, 3, 0, 8), (1000, 1, 0, 0)])
def test_forward_few_rows(nss, rows, cols, out, pad, shift):
    """Single tokens: a pass over W, the tests' other sizes and epilogues with up to 8 rows."""
    for dtype, act in (("bf16", "gelu"), ("f16", "relu2")):
        g, t = _gen(rows + cols), TYPES[dtype]
        x, w = _rows(rows, cols, t, g, pad, shift), _rows(out, cols, t, g, 0, shift, std=cols ** -0.5)
        r, b = _rows(rows, out, t, g, pad, shift), torch.randn(out, generator=g, device="cuda")
        whole = [torch.full((rows * (out + pad) + shift,), 7.0, device="cuda", dtype=t) for _ in range(2)]
        y, z = (f[shift:].view(rows, out + pad)[:, :out] for f in whole)
        _check_forward(nss, x, w, b, r, act, None, y=y, z=z)
        for f in whole:
            assert (f[:shift] == 7).all() and (f[shift:].view(rows, out + pad)[:, out:] == 7).all()
        want, _ = _check_forward(nss, x, w, b.to(t), r, act, None, keep=False)
        y.copy_(r)
        nss.mb_linear(x, w, b.to(t), y, act, y=y)                           # over the residual
        assert torch.equal(y, want)
        _check_forward(nss, x, w, None, None, "silu", None)


@pytest.mark.parametrize("ends", [[0, 0, 0], [8], [3, 3, 7], [0, 1, 2, 3, 4, 5, 6, 7], [1] * 40 + [2] * 30 + [8], [0] * 1023 + [5]])
@pytest.mark.parametrize("out", [200, 131])
def test_forward_few_rows_of_groups(nss, ends, out):
    g, rows, cols, t = _gen(33), 8, 72, torch.bfloat16
    x, w = _rows(rows, cols, t, g), (torch.randn(len(ends), out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    x[ends[-1]:] = math.nan
    b, r = torch.randn(len(ends), out, generator=g, device="cuda"), _rows(rows, out, t, g)
    y, z = (torch.full((rows, out), 7.0, device="cuda", dtype=t) for _ in range(2))
    _check_forward(nss, x, w, b, r, "silu", ends, y=y, z=z)
    assert not y[ends[-1]:].any() and not z[ends[-1]:].any()
    if len(ends) == 3:
        from newton_schulz_stacked_gb300 import _binding as binding
        assert nss.mb_sync_status() == 0
        for bad, held in (([5, 2, 8], [5, 5, 8]), ([1, 2, 30], [1, 2, 8]), ([-5, 2, 6], [0, 2, 6])):
            x = _rows(rows, cols, t, g)
            y, _ = nss.mb_linear(x, w, ends=torch.tensor(bad, dtype=torch.int32, device="cuda"))
            assert nss.mb_sync_status() == binding.MB_ERR_ARG
            want, _ = nss.mb_linear(x, w, ends=torch.tensor(held, dtype=torch.int32, device="cuda"))
            assert nss.mb_sync_status() == 0 and torch.equal(y, want)


def test_narrow_products_with_many_columns(nss):
    """dz of more elements than are formed under the products, with sums so few that it comes in two halves."""
    g, t, rows, cols, out = _gen(35), torch.bfloat16, 1024, 2, 50000
    x, w = _rows(rows, cols, t, g), _rows(out, cols, t, g)
    dy, z = _rows(rows, out, t, g), _rows(rows, out, t, g)
    workspace = torch.full((1 << 29,), 0xFF, dtype=torch.uint8, device="cuda")
    _check_backward(nss, dy, x, w, z, "silu", None, workspace=workspace)


def test_results_over_inputs_are_refused(nss):
    t = torch.bfloat16
    x, w = torch.ones(12, 64, device="cuda", dtype=t), torch.ones(64, 64, device="cuda", dtype=t)
    z, dy = torch.ones_like(x), torch.ones_like(x)
    for given in ({"y": x}, {"z": x}, {"y": z, "z": z}, {"residual": z, "z": z}, {"y": w[:12]}):
        with pytest.raises(ValueError):
            nss.mb_linear(x, w, activation="relu", **given)
    for given in ({"dx": dy}, {"dx": x}, {"dx": z}, {"dweight": w}):
        with pytest.raises(ValueError):
            nss.mb_linear_backward(dy, x, w, z, "relu", **given)
    both = torch.ones(12, 128, device="cuda", dtype=t)                      # side by side is no overlap
    y, _ = nss.mb_linear(both[:, :64], w, y=both[:, 64:])
    assert (both[:, 64:] == 64).all() and (both[:, :64] == 1).all()


@pytest.mark.parametrize("rows", [2, 7, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("cols,out,pad", [(8, 8, 0), (40, 1, 8), (264, 67, 0), (768, 768, 0), (1000, 130, 24), (4096, 333, 0)])
def test_forward_some_rows(nss, rows, cols, out, pad):
    """Up to 64 rows from 16-byte boundaries: the warps' products, and one row more."""
    for dtype, act in (("bf16", "silu"), ("f16", "none")):
        g, t = _gen(rows + cols), TYPES[dtype]
        x, w = _rows(rows, cols, t, g, pad), _rows(out, cols, t, g, std=cols ** -0.5)
        r, b = _rows(rows, out, t, g, 5), torch.randn(out, generator=g, device="cuda").to(t)
        whole = torch.full((rows, out + 3), 7.0, device="cuda", dtype=t)
        _check_forward(nss, x, w, b, r, act, None, y=whole[:, :out])
        assert (whole[:, out:] == 7).all()
        _check_forward(nss, x, w, None, None, "relu2", None, keep=False)


@pytest.mark.parametrize("ends", [[0, 0, 0], [60], [3, 3, 50], [5, 20, 20, 41, 57, 64], [1] * 40 + [30] * 30 + [62],
                                  list(range(1, 65)), [0] * 1023 + [64]])
@pytest.mark.parametrize("out", [200, 131])
def test_forward_some_rows_of_groups(nss, ends, out):
    g, rows, cols, t = _gen(37), 64, 72, torch.bfloat16
    x, w = _rows(rows, cols, t, g), (torch.randn(len(ends), out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    x[ends[-1]:] = math.nan
    b, r = torch.randn(len(ends), out, generator=g, device="cuda"), _rows(rows, out, t, g)
    y, z = (torch.full((rows, out), 7.0, device="cuda", dtype=t) for _ in range(2))
    _check_forward(nss, x, w, b, r, "gelu", ends, y=y, z=z)
    assert not y[ends[-1]:].any() and not z[ends[-1]:].any()
