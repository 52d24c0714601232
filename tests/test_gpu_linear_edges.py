"""The products at the edges of what a call may ask of them: values, layouts, sizes on both sides of the rules that choose a
kernel.  Tolerances are those of test_gpu_linear.py, whose plain forms in 64 bits these tests take."""
import math

import pytest
import torch

from test_gpu_linear import ACTS, TYPES, _add, _bounds, _check_backward, _check_forward, _gen, _near, _rows, _slope, nss  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows", [4, 300])
def test_slopes_of_large_finite_values(nss, act, rows):
    """Values whose powers pass fp32: the slope is finite where the formula's is."""
    g, t, cols, out = _gen(41), torch.bfloat16, 64, 64
    x, w, dy, z = _rows(rows, cols, t, g), _rows(out, cols, t, g, std=cols ** -0.5), _rows(rows, out, t, g), _rows(rows, out, t, g)
    sizes = [15.0, 16.0, 17.0, 1e3, 1e6, 1e12, 1e14, 1e18, 1e20, 1e30, 1e38, 3.3e38]
    z[1, :len(sizes)] = torch.tensor(sizes, device="cuda")
    z[2, :len(sizes)] = -torch.tensor(sizes, device="cuda")
    if act == "relu2":                           # a slope of 2 z: dz of these is infinite in earnest
        z[1:3, sizes.index(1e30):len(sizes)] = 1.0
        dy[1:3] *= 2.0 ** -100
    dx, dw, db = nss.mb_linear_backward(dy, x, w, z, act, bias=True)
    want = dy.double() * (torch.ones_like(z) if act == "none" else _wide_slope(z.double(), act))
    assert dx.isfinite().all() and dw.isfinite().all() and db.isfinite().all()
    _near(db, want.sum(0), (_add(rows) + 2.0 ** -18) * want.abs().sum(0))
    if act != "none":                            # an infinity stays one that shows
        z[3, 5] = math.inf
        dx, _, _ = nss.mb_linear_backward(dy, x, w, z, act)
        shown = not dx[3].isfinite().all()
        assert shown == (act != "relu") and dx[:3].isfinite().all()


def _wide_slope(z, act):
    """The derivative, by its limits where the powers of z pass 64 bits' range too."""
    far = z.abs() > 1e3
    near = _slope(torch.where(far, 1.0, z), act)
    return torch.where(far, 2 * z.clamp(min=0) if act == "relu2" else (z > 0).double(), near)


def _time(call, n=20):
    """us of a call among others: in a graph, the best of five replays."""
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(n):
            call()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = math.inf
    for _ in range(6):
        begin.record()
        graph.replay()
        end.record()
        end.synchronize()
        best = min(best, begin.elapsed_time(end) * 1e3 / n)
    return best


@pytest.mark.parametrize("cols,out,groups", [(8, 8192, 0), (8, 65536, 0), (64, 2816, 0), (64, 8192, 0), (64, 64, 0), (768, 768, 0),
                                             (256, 16384, 0), (16384, 768, 0), (65536, 8, 0), (65536, 64, 0), (33, 20001, 0),
                                             (64, 8192, 64), (1024, 2816, 8), (1024, 2816, 64), (1024, 64, 64), (2816, 1024, 256)])
def test_fewer_rows_take_no_longer(nss, cols, out, groups):
    """Whichever kernels a call's sizes choose, more rows must not be the cheaper call."""
    g, t = _gen(43), torch.bfloat16
    x = _rows(513, cols, t, g)
    w = torch.randn(*((groups,) if groups else ()), out, cols, generator=g, device="cuda").to(t)

    def time(rows):
        ends = None
        if groups:
            ends = torch.tensor([rows * (i + 1) // groups for i in range(groups)], dtype=torch.int32, device="cuda")
        y = torch.empty(rows, out, device="cuda", dtype=t)
        workspace = torch.empty(1 << 28, device="cuda", dtype=torch.uint8)
        return _time(lambda: nss.mb_linear(x[:rows], w, ends=ends, y=y, workspace=workspace))

    most = time(513)
    for rows in (1, 2, 8, 16, 17, 64, 128, 256, 512):
        few = time(rows)
        assert few <= 1.6 * most + 1, (rows, few, most)


@pytest.mark.parametrize("rows,cols,out", [(1, 8, 65536), (1, 65536, 8), (2, 40, 20000), (2, 16384, 72), (5, 33, 9001), (8, 4095, 15),
                                           (16, 32, 40008), (16, 20000, 16), (17, 2056, 1000), (64, 64, 33000), (65, 1024, 4096),
                                           (250, 8, 8200), (256, 256, 1000), (256, 256, 4096), (512, 64, 264), (512, 64, 8192),
                                           (512, 72, 1003), (512, 768, 768), (500, 4096, 130), (512, 4096, 1040)])
def test_forward_on_both_sides_of_the_rule(nss, rows, cols, out):
    """Few rows by the kernels without tiles and by tiles, narrow and wide, with everything around the product."""
    for dtype, act in ((torch.bfloat16, "silu"), (torch.float16, "none")):
        g = _gen(rows + cols)
        x, w = _rows(rows, cols, dtype, g), _rows(out, cols, dtype, g, std=cols ** -0.5)
        r, b = _rows(rows, out, dtype, g), torch.randn(out, generator=g, device="cuda")
        _check_forward(nss, x, w, b, r, act, None)


@pytest.mark.parametrize("rows,cols,out,groups", [(64, 1024, 520, 3), (65, 1024, 520, 3), (64, 64, 8192, 8), (63, 256, 1000, 20),
                                                  (64, 768, 1001, 64), (16, 768, 1000, 9), (9, 64, 8192, 30), (64, 2056, 64, 64)])
def test_groups_on_both_sides_of_the_rule(nss, rows, cols, out, groups):
    g, t = _gen(rows + groups), torch.bfloat16
    sizes = torch.rand(groups, generator=g, device="cuda").cumsum(0)
    ends = (sizes / sizes[-1] * (rows - 2)).int().tolist()
    x, w = _rows(rows, cols, t, g), (torch.randn(groups, out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    x[ends[-1]:] = math.nan
    b, r = torch.randn(groups, out, generator=g, device="cuda"), _rows(rows, out, t, g)
    y, z = (torch.full((rows, out), 7.0, device="cuda", dtype=t) for _ in range(2))
    _check_forward(nss, x, w, b, r, "gelu", ends, y=y, z=z)
    assert not y[ends[-1]:].any() and not z[ends[-1]:].any()


@pytest.mark.parametrize("rows", [300, 1024])
@pytest.mark.parametrize("cols,out", [(64, 96), (768, 2816)])
def test_forward_rows_of_any_shape(nss, rows, cols, out):
    """Rows that are all one (a stride of 0), folded leading dimensions, every second row: by tiles as well as without them.
    Kernels may add in another order: the tolerance is that of the sums."""
    g, t = _gen(47), torch.bfloat16
    w, x = _rows(out, cols, t, g, std=cols ** -0.5), _rows(2 * rows, cols, t, g)
    _check_forward(nss, x[:1].expand(rows, cols), w, None, None, "relu2", None)
    _check_forward(nss, x[::2], w, None, None, "gelu", None)
    flat, _ = nss.mb_linear(x[:rows], w)
    y, _ = nss.mb_linear(x[:rows].view(2, rows // 4, 2, cols), w)
    assert y.shape == (2, rows // 4, 2, out) and torch.equal(y.view(rows, out), flat)
    one, _ = nss.mb_linear(x[0], w)
    _near(one[None], x[:1].double() @ w.double().T, _add(cols) * (x[:1].double().abs() @ w.double().abs().T))


@pytest.mark.parametrize("rows,cols,out", [(1024, 256, 512), (2000, 768, 768)])
def test_threads_with_products_by_tiles(nss, rows, cols, out):
    """Calls of three host threads on streams of their own, forward and backward, by tiles."""
    import threading
    g, t = _gen(53), torch.bfloat16
    x, w, dy = _rows(rows, cols, t, g), _rows(out, cols, t, g, std=cols ** -0.5), _rows(rows, out, t, g)
    y, z = nss.mb_linear(x, w, activation="gelu", keep=True)
    want = (y, z, *nss.mb_linear_backward(dy, x, w, z, "gelu", bias=True))
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(100):
                y, z = nss.mb_linear(x, w, activation="gelu", keep=True)
                got = (y, z, *nss.mb_linear_backward(dy, x, w, z, "gelu", bias=True))
        stream.synchronize()
        wrong.extend(1 for a, b in zip(got, want) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong and nss.mb_sync_status() == 0


def test_results_that_share_memory_are_refused(nss):
    """Any shared byte, not only a shared first one; views side by side are none."""
    t = torch.bfloat16
    g = _gen(59)
    buf, w = _rows(40, 192, t, g), _rows(64, 64, t, g, std=0.125)
    x, side, last = buf[:20, :64], buf[:20, 64:128], buf[:20, 128:]
    ends = torch.tensor([20], dtype=torch.int32, device="cuda")

    def refused(call, *args, **more):
        before = buf.clone()
        with pytest.raises(ValueError, match="may not be written over"):
            call(*args, **more)
        torch.cuda.synchronize()
        assert torch.equal(buf, before)

    flat = buf.view(-1)
    shifted = lambda n: flat[n:n + 20 * 192].view(20, 192)[:, :64]                         # noqa: E731
    for y in (buf[1:21, :64], buf[:20, 63:127], buf[:20, 1:65], shifted(160), flat[64:64 + 20 * 64].view(20, 64),
              buf[19:39, 10:74]):
        refused(nss.mb_linear, x, w, y=y)
        refused(nss.mb_linear, x.clone(), w, y=x, z=y)
        refused(nss.mb_linear, x.clone(), w, residual=x, z=y)
    for y in (side, last, buf[20:, :64], flat[20 * 192:20 * 192 + 20 * 64].view(20, 64)):
        want, _ = nss.mb_linear(x.clone(), w)
        nss.mb_linear(x, w, y=y)
        assert torch.equal(y, want)
    # the residual: over itself, element by element, and no other way
    refused(nss.mb_linear, x, w, residual=side, y=buf[1:21, 64:128])
    refused(nss.mb_linear, x, w, residual=flat[64:64 + 20 * 64].view(20, 64), y=side)
    refused(nss.mb_linear, x, w, residual=side[:1].expand(20, 64), y=side)
    one = last[0:1].expand(20, 64)                                                         # one row for all
    nss.mb_linear(x, w, residual=one, y=side)
    want, _ = nss.mb_linear(x, w, residual=side.clone())
    nss.mb_linear(x, w, residual=side, y=side)
    assert torch.equal(side, want)
    # weights, biases, ends, workspaces
    refused(nss.mb_linear, x, w, y=w[10:30])
    many = torch.zeros(20 * 64 + 64, device="cuda", dtype=t)
    refused(nss.mb_linear, x, w, many[20 * 64 - 8:20 * 64 + 56], y=many[:20 * 64].view(20, 64))
    refused(nss.mb_linear, x, w[None], ends=many[20:22].view(torch.int32), y=many[:20 * 64].view(20, 64))
    odd = flat[1:1 + 20 * 64].view(20, 64)                                                 # copied: a workspace
    refused(nss.mb_linear, odd, w, workspace=buf.view(torch.uint8))
    dy = torch.ones(20, 64, device="cuda", dtype=t)
    refused(nss.mb_linear_backward, dy, x, w, dx=buf[1:21, :64])
    refused(nss.mb_linear_backward, x, dy, w, dx=buf[:20, 32:96])
    refused(nss.mb_linear_backward, dy, x, w, dweight=flat[100:100 + 64 * 64].view(64, 64))
    refused(nss.mb_linear_backward, dy, x, w, dbias=flat[50:114])
    refused(nss.mb_linear_backward, dy, x, w, dx=side, dbias=flat[70:134])
    refused(nss.mb_linear_backward, dy, x, w, torch.ones_like(dy), "relu", workspace=buf.view(torch.uint8))
    want, _, _ = nss.mb_linear_backward(dy, x, w)
    nss.mb_linear_backward(dy, x, w, dx=side, dbias=flat[20 * 192:20 * 192 + 64])
    assert torch.equal(side, want)
    assert nss.mb_sync_status() == 0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ["relu2", "silu"])
@pytest.mark.parametrize("rows,cols,out,groups", [(1, 64, 64, 0), (2, 1000, 72, 0), (30, 65, 130, 0), (1, 8, 20000, 0), (2, 20008, 3, 0),
                                                  (24, 64, 96, 3), (300, 64, 96, 0), (600, 136, 200, 3)])
def test_infinite_operands_of_the_gradient(nss, dtype, act, rows, cols, out, groups):
    """An infinity in x or in a weight makes its sums infinite, and NaN only where the formula has it, with dz in two halves (the
    smallest calls) as in one."""
    g, t = _gen(rows + cols), TYPES[dtype]
    n = max(groups, 1)
    x, dy, z = _rows(rows, cols, t, g), _rows(rows, out, t, g), _rows(rows, out, t, g).abs_().add_(0.5)
    w = (torch.randn(n, out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    dy[0, ::2] = 1.0                             # some of dz fit 16 bits as they are: nothing is left of them
    z[0, ::2] = 2.0
    x[0, 1], x[rows // 2, cols - 1], w[0, 1, 0], w[0, out // 2, cols // 2] = math.inf, -math.inf, math.inf, -math.inf
    ends = [rows // 3, rows // 3, rows - 1] if groups else None
    dev = torch.tensor(ends, dtype=torch.int32, device="cuda") if groups else None
    dx, dw, _ = nss.mb_linear_backward(dy, x, w if groups else w[0], z, act, dev)
    for i, (a, e) in enumerate(_bounds(ends, rows)):
        D, X, W = dy[a:e].double() * _slope(z[a:e].double(), act), x[a:e].double(), w[i].double()
        for got, want in ((dx[a:e], D @ W), (dw[i] if groups else dw, D.T @ X)):
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
            assert torch.equal(got[got.isinf()].double(), want[want.isinf()])


@pytest.mark.parametrize("used", [[1023], [0], [500, 501], []])
@pytest.mark.parametrize("cols,out", [(8, 8), (200, 520)])
def test_runs_of_groups_without_rows(nss, used, cols, out):
    """Most of 1024 experts without a token, so that a pair has many units without blocks in a row: the same result each time."""
    g, t, rows = _gen(67), torch.bfloat16, 700
    sizes = torch.zeros(1024, dtype=torch.int64)
    for i in used:
        sizes[i] = rows // len(used)
    ends = sizes.cumsum(0).tolist()
    x, dy = _rows(rows, cols, t, g), _rows(rows, out, t, g)
    w = (torch.randn(1024, out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    dev = torch.tensor(ends, dtype=torch.int32, device="cuda")
    dx, dw, db = nss.mb_linear_backward(dy, x, w, ends=dev, bias=True)
    for i in range(1024):
        if i not in used:
            continue
        a = ends[i] - int(sizes[i])
        X, D = x[a:ends[i]].double(), dy[a:ends[i]].double()
        _near(dw[i], D.T @ X, _add(rows) * (D.abs().T @ X.abs()))
        _near(dx[a:ends[i]], D @ w[i].double(), _add(out) * (D.abs() @ w[i].double().abs()))
    rest = torch.ones(1024, dtype=torch.bool)
    rest[used] = False
    for turn in range(30):
        given = torch.full_like(dw, 7.0)
        dx2, dw2, db2 = nss.mb_linear_backward(dy, x, w, ends=dev, bias=True, dweight=given)
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
        assert not dw2[rest.cuda()].any()
    assert nss.mb_sync_status() == 0


def test_very_many_rows_in_one_group(nss):
    """2^29 rows, all of them one expert's of 1024: two contractions of 1.15 s, longer than a wait may take that does not count its
    blocks."""
    rows, t = 1 << 29, torch.bfloat16
    x, dy = (torch.zeros(rows, 8, device="cuda", dtype=t) for _ in range(2))
    dy += 1
    at = torch.tensor([0, 1, rows // 2 - 1, rows // 2, rows - 1], device="cuda")
    x[at] = torch.tensor([1.0, 2.0, 4.0, 8.0, 16.0], device="cuda", dtype=t)[:, None]
    ends = torch.full((1024,), rows, dtype=torch.int32, device="cuda")
    ends[:700] = 0
    w = torch.zeros(1024, 8, 8, device="cuda", dtype=t)
    _, dw, _ = nss.mb_linear_backward(dy, x, w, ends=ends, input_grad=False)
    assert nss.mb_sync_status() == 0
    assert (dw[700] == 31).all() and not dw[:700].any() and not dw[701:].any()


def test_what_small_fp16_gradients_lose(nss):
    """fp16 holds dz below 2^-14 in steps of 2^-24: gradients of 1e-6 keep the bound that counts half a step per term, which is some
    percent of dW here; the same gradients 2^12 larger, as a scaled loss makes them, keep fp16's own half step."""
    g, t, rows, cols, out = _gen(71), torch.float16, 4096, 64, 72
    x, w, z = _rows(rows, cols, t, g), _rows(out, cols, t, g, std=cols ** -0.5), _rows(rows, out, t, g)
    dy = torch.randn(rows, out, generator=g, device="cuda")
    off = {}
    for size in (1e-6, 1e-6 * 2 ** 12):
        d = (size * dy).to(t)
        _, dw, db = _check_backward(nss, d, x, w, z, "silu", None)
        want = (d.double() * _slope(z.double(), "silu")).T @ x.double()
        off[size] = ((dw.double() - want).norm() / want.norm()).item()
        # dbias takes dz as it is
        _near(db, (d.double() * _slope(z.double(), "silu")).sum(0), (_add(rows) + 2.0 ** -18) * d.double().abs().sum(0) * 1.1)
    # an even error within half a step has a deviation of 2^-24 / sqrt(12) a term, beside dz of 1e-6 * 0.61 (silu' of a normal)
    expected = 2.0 ** -24 / math.sqrt(12) / (1e-6 * 0.61)
    assert 0.5 * expected <= off[1e-6] <= 1.5 * expected
    assert off[1e-6 * 2 ** 12] <= 2.0 ** -11


@pytest.mark.parametrize("ends", [None, [6001, 6001, 6100, 19990]])
def test_large_backward_in_graphs_and_at_once(nss, ends):
    """dz formed under the products: two graphs replayed in turn with new inputs, and two calls at once on streams of their own,
    give the bits of a call alone."""
    g, t, rows, cols, out = _gen(73), torch.bfloat16, 20000, 136, 2528
    x, dy, z = _rows(rows, cols, t, g), _rows(rows, out, t, g), _rows(rows, out, t, g)
    n = 1 if ends is None else len(ends)
    w = (torch.randn(n, out, cols, generator=g, device="cuda") * cols ** -0.5).to(t)
    w = w[0] if ends is None else w
    dev = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    call = lambda: nss.mb_linear_backward(dy, x, w, z, "silu", dev, bias=True)               # noqa: E731
    first = call()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    for turn in range(3):
        if turn:
            dy.mul_(-0.5)
            z.neg_()
            torch.cuda.synchronize()
        want = call()
        assert turn or all(torch.equal(a, b) for a, b in zip(first, want))
        for graph, got in zip(graphs, outs):
            for o in got:
                o.fill_(7.0)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([call() for _ in range(3)])
    torch.cuda.synchronize()
    for calls in got:
        for o in calls:
            assert all(torch.equal(a, b) for a, b in zip(o, want))
    assert nss.mb_sync_status() == 0
