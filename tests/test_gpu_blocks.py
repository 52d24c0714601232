"""The block operators on the GPU against their definitions in 64 bits.

Tolerances are bounds on fp32 evaluation, derived here from the operations (U = 2^-24, one
rounding each) before any run, plus one rounding to the result's type.
"""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# one rounding to each 16-bit type: half its epsilon relative to the value, or half its smallest
# subnormal (fp32 results have theirs in the bounds below)
ROUND = {t: (torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2)
         for t in (torch.bfloat16, torch.float16)}
ROUND[torch.float32] = (0.0, 2.0 ** -149)


@pytest.fixture(scope="module")
def nss():
    from newton_schulz_stacked_gb300.build import build_all
    build_all()
    import newton_schulz_stacked_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.load_library()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def rounding(value, dtype):
    rel, tiny = ROUND[dtype]
    return rel * value.abs() + tiny


def within(got, ref, bound, what):
    """Every element of `got` within `bound` of the 64-bit `ref`."""
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    n = int(bad.sum())
    if n:
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(f"{what}: {n} elements outside the bound, first {i}: got {got.reshape(-1)[i].item()!r}, "
                             f"want {ref.reshape(-1)[i].item()!r}, bound {bound.expand_as(ref).reshape(-1)[i].item():.3g}")


def same_bits(a, b, what):
    assert a.dtype == b.dtype and a.shape == b.shape
    view = {4: torch.int32, 2: torch.int16}[a.element_size()]
    assert torch.equal(a.contiguous().view(view), b.contiguous().view(view)), what


class Guarded:
    """A result tensor inside a larger buffer of a known pattern, which must stay untouched."""

    def __init__(self, shape, dtype, before=24, pad=0):
        n = 1
        for s in shape[:-1]:
            n *= s
        ld = shape[-1] + pad
        self.buf = torch.full((before + n * ld + 64,), 7, device="cuda", dtype=torch.float32).to(dtype)
        self.mark = torch.zeros_like(self.buf, dtype=torch.bool)
        at = (torch.arange(n, device="cuda")[:, None] * ld + torch.arange(shape[-1], device="cuda")).reshape(-1) + before
        self.mark[at] = True
        self.t = torch.as_strided(self.buf, (n, shape[-1]), (ld, 1), before)

    def check(self, what):
        assert bool((self.buf[~self.mark] == 7).all()), f"{what}: wrote outside its rows"


# ---------------------------------------------------------------- layer norm

def depth(cols):
    """Sequential additions of one fp32 row sum: a thread's elements, five shuffles, the warps."""
    return min(cols, 32 + cols / 1024) + 5 + 32


def norm_forward_ref(x, w, b, eps):
    xd = x.double()
    n = xd.shape[-1]
    m = xd.mean(-1)
    d = xd - m[:, None]
    r = (d.square().mean(-1) + eps).rsqrt()
    h = d * r[:, None]
    wd = torch.ones(n, device="cuda", dtype=torch.float64) if w is None else w.double()
    bd = torch.zeros(n, device="cuda", dtype=torch.float64) if b is None else b.double()
    y = h * wd + bd
    D = depth(n)
    e_m = (D + 2) * U * xd.abs().mean(-1)                     # the mean's sum, its scale and rounding
    rel_r = (0.5 * (D + 8) + 4) * U + 2 * (e_m * r) ** 2      # sum of squares, their roundings, the root; (x - m)^2 shifts by e_m^2
    e_h = (e_m * r)[:, None] + h.abs() * (rel_r[:, None] + 3 * U)
    bound = 1.01 * (e_h * wd.abs() + 2 * U * ((h * wd).abs() + y.abs()))
    return y, m, r, bound + rounding(y, x.dtype), 1.01 * e_m, 1.01 * (rel_r + U) * r


def check_norm_forward(nss, x, w, b, eps=1e-5, **out):
    y, mean, rstd = nss.mb_layer_norm(x, w, b, eps, **out)
    torch.cuda.synchronize()
    flat = x.reshape(-1, x.shape[-1])
    ref, m, r, by, bm, br = norm_forward_ref(flat, w, b, eps)
    within(y.reshape(ref.shape), ref, by, "y")
    within(mean.reshape(-1), m, bm, "mean")
    within(rstd.reshape(-1), r, br, "rstd")
    return y, mean, rstd


def norm_backward_ref(dy, x, mean, rstd, w):
    dyd, xd = dy.double(), x.double()
    rows, n = xd.shape
    r = rstd.double()[:, None]
    h = (xd - mean.double()[:, None]) * r
    wd = torch.ones(n, device="cuda", dtype=torch.float64) if w is None else w.double()
    g = dyd * wd
    c1, c2 = g.mean(-1, keepdim=True), (g * h).mean(-1, keepdim=True)
    dx = r * (g - c1 - h * c2)
    D = depth(n)
    bound = 1.01 * U * r * (4 * g.abs() + (D + 6) * g.abs().mean(-1, keepdim=True) +
                            h.abs() * (D + 14) * (g * h).abs().mean(-1, keepdim=True)) + 3 * U * dx.abs()
    # a column's sum: a thread's rows (at most rows / SMs + its group's), the CTA's groups, the parts in eight slices
    E = min(rows, rows / 100 + 8) + 64 + 304 / 8 + 8 + 4
    dw, db = (dyd * h).sum(0), dyd.sum(0)
    wtype = x.dtype if w is None else w.dtype
    return (dx, bound + rounding(dx, x.dtype), dw, 1.01 * E * U * (dyd * h).abs().sum(0) + rounding(dw, wtype), db,
            1.01 * E * U * dyd.abs().sum(0) + rounding(db, wtype))


def check_norm_backward(nss, dy, x, mean, rstd, w, **out):
    dx, dw, db = nss.mb_layer_norm_backward(dy, x, mean, rstd, w, **out)
    torch.cuda.synchronize()
    flat = (dy.reshape(-1, dy.shape[-1]), x.reshape(-1, x.shape[-1]), mean.reshape(-1), rstd.reshape(-1))
    rx, bx, rw, bw, rb, bb = norm_backward_ref(*flat, w)
    within(dx.reshape(rx.shape), rx, bx, "dx")
    if w is not None:
        within(dw, rw, bw, "dw")
        within(db, rb, bb, "db")
    return dx, dw, db


def norm_inputs(seed, rows, cols, dtype, wtype, offset=0.3):
    g = gen(seed)
    x = (randn(g, rows, cols) * torch.exp(0.5 * randn(g, 1, cols)) + offset * randn(g, rows, 1)).to(dtype)
    w, b = (1 + 0.3 * randn(g, cols)).to(wtype), (0.2 * randn(g, cols)).to(wtype)
    return x, w, b, (0.1 * randn(g, rows, cols)).to(dtype)


# one element; one thread; sub-warp groups; a warp; warps; the widest kept in registers; re-read rows; odd ones of each
NORM_SHAPES = [(1, 1), (7, 2), (3, 7), (130, 8), (33, 40), (9, 64), (1000, 96), (37, 249), (5, 256), (64, 768), (2053, 768),
               (37, 1001), (6, 1024), (5, 1032), (2, 4096), (11, 4100), (3, 5000), (3, 8192), (3, 8200), (2, 32768),
               (2, 33001), (3, 40000)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_layer_norm(nss, rows, cols, dtype, wtype):
    x, w, b, dy = norm_inputs(cols * 7 + rows, rows, cols, TYPES[dtype], TYPES[wtype])
    _, mean, rstd = check_norm_forward(nss, x, w, b)
    check_norm_backward(nss, dy, x, mean, rstd, w)


@pytest.mark.parametrize("cols", [96, 768, 1001, 8200])
def test_layer_norm_without_parameters(nss, cols):
    x, w, b, dy = norm_inputs(5, 19, cols, torch.bfloat16, torch.float32)
    _, mean, rstd = check_norm_forward(nss, x, None, None)
    check_norm_forward(nss, x, w, None)
    check_norm_forward(nss, x, None, b)
    dx, dw, db = check_norm_backward(nss, dy, x, mean, rstd, None)
    assert dw is None and db is None
    dx2, dw, db = nss.mb_layer_norm_backward(dy, x, mean, rstd, w, bias=False)
    assert db is None
    same_bits(dw, nss.mb_layer_norm_backward(dy, x, mean, rstd, w)[1], "dw with and without db")


@pytest.mark.parametrize("offset,scale", [(1000.0, 1.0), (-3e4, 100.0), (0.0, 1e-6), (1.0, 0.0)])
def test_layer_norm_far_from_zero(nss, offset, scale):
    """The mean far above the deviation, tiny rows, constant rows."""
    g = gen(8)
    x = offset + scale * randn(g, 40, 770)
    w, b, dy = 1 + 0.1 * randn(g, 770), 0.1 * randn(g, 770), randn(g, 40, 770)
    _, mean, rstd = check_norm_forward(nss, x, w, b)
    check_norm_backward(nss, dy, x, mean, rstd, w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,pad,before", [(64, 8, 0), (64, 3, 1), (63, 1, 0), (768, 8, 8), (768, 0, 1), (770, 2, 0),
                                             (4096, 16, 8), (8200, 8, 0), (8200, 1, 1), (33000, 8, 0)])
def test_layer_norm_strided_rows_and_guard_bands(nss, dtype, cols, pad, before):
    dtype = TYPES[dtype]
    rows = 21
    x, w, b, dy = norm_inputs(cols + pad, rows, cols, dtype, torch.float32)
    src, grad, y, dx = (Guarded((rows, cols), dtype, before, pad) for _ in range(4))
    src.t.copy_(x)
    grad.t.copy_(dy)
    got, mean, rstd = check_norm_forward(nss, src.t, w, b, y=y.t)
    assert got is y.t
    y.check("y")
    check_norm_backward(nss, grad.t, src.t, mean, rstd, w, dx=dx.t)
    dx.check("dx")


# every distance of a row from a 16-byte boundary, the same and different ones in a call's tensors, and
# enough rows that every group of threads takes several
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(9001, 17), (3001, 130), (4003, 251), (5001, 263), (4001, 517), (3501, 775), (2501, 1009),
                                       (1203, 1031), (903, 2051), (703, 3999), (403, 5003)])
def test_layer_norm_unaligned_rows(nss, dtype, rows, cols):
    dtype = TYPES[dtype]
    x, w, b, dy = norm_inputs(rows + cols, rows, cols, dtype, torch.float32)
    _, mean, rstd = check_norm_forward(nss, x, w, b)
    check_norm_backward(nss, dy, x, mean, rstd, w)
    for before, pads in ((3, (0, 0, 0, 0)), (5, (7, 7, 7, 7)), (2, (8, 0, 16, 8)), (1, (1, 0, 3, 2))):
        src, grad, y, dx = (Guarded((rows, cols), dtype, before, pad) for pad in pads)
        src.t.copy_(x)
        grad.t.copy_(dy)
        # a neighbour of the row that is not finite must not be taken in
        src.buf[~src.mark], grad.buf[~grad.mark] = float("nan"), float("inf")
        check_norm_forward(nss, src.t, w, b, y=y.t)
        y.check("y")
        check_norm_backward(nss, grad.t, src.t, mean, rstd, w, dx=dx.t)
        dx.check("dx")


@pytest.mark.parametrize("cols", [40, 768, 1001, 4096, 8200, 33001])
def test_layer_norm_in_place_and_broadcast(nss, cols):
    x, w, b, dy = norm_inputs(11, 45, cols, torch.bfloat16, torch.float32)
    y, mean, rstd = nss.mb_layer_norm(x, w, b)
    inplace = x.clone()
    nss.mb_layer_norm(inplace, w, b, y=inplace)
    same_bits(inplace, y, "y over x")
    want = nss.mb_layer_norm_backward(dy, x, mean, rstd, w)
    for over in ("x", "dy"):
        xx, dd = x.clone(), dy.clone()
        got = nss.mb_layer_norm_backward(dd, xx, mean, rstd, w, dx=xx if over == "x" else dd)
        for a, c, what in zip(got, want, ("dx", "dw", "db")):
            same_bits(a, c, f"{what} with dx over {over}")
    # one row for all: rows 0 elements apart
    row = x[:1].expand(45, cols)
    a, b2 = nss.mb_layer_norm(row, w, b), nss.mb_layer_norm(row.contiguous(), w, b)
    same_bits(a[0], b2[0], "broadcast x")
    drow = dy[:1].expand(45, cols)
    a, b2 = nss.mb_layer_norm_backward(drow, x, mean, rstd, w), nss.mb_layer_norm_backward(drow.contiguous(), x, mean, rstd, w)
    for c, d in zip(a, b2):
        same_bits(c, d, "broadcast dy")


# rows enough for several turns of the ring of rows of either pass, and too few for one; every number of groups per CTA
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(0, 2048), (1, 1032), (153, 8192), (3100, 8184), (2300, 4608), (7001, 2568), (9001, 1928),
                                       (12001, 1040), (5003, 4096), (1700, 8192)])
def test_layer_norm_long_rows(nss, dtype, rows, cols):
    dtype = TYPES[dtype]
    for wtype in {dtype, torch.float32}:
        x, w, b, dy = norm_inputs(rows + cols, rows, cols, dtype, wtype)
        _, mean, rstd = check_norm_forward(nss, x, w, b)
        src, grad, dx = (Guarded((rows, cols), dtype, 8, pad) for pad in (0, 16, 8))
        src.t.copy_(x)
        grad.t.copy_(dy)
        src.buf[~src.mark], grad.buf[~grad.mark] = float("nan"), float("inf")
        check_norm_forward(nss, src.t, w, b, y=dx.t)
        dx.check("y")
        got = check_norm_backward(nss, grad.t, src.t, mean, rstd, w, dx=dx.t)
        dx.check("dx")
        y, inplace = nss.mb_layer_norm(x, w, b)[0], x.clone()
        nss.mb_layer_norm(inplace, w, b, y=inplace)
        same_bits(inplace, y, "y over x")
        again = nss.mb_layer_norm_backward(dy, x, mean, rstd, w, dx=x)
        for a, c, what in zip(again, got, ("dx", "dw", "db")):
            same_bits(a, c, f"{what} over x, from another layout")


def test_layer_norm_of_nothing(nss):
    w, b = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    x = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = nss.mb_layer_norm(x, w, b)
    assert y.shape == (0, 64) and mean.shape == (0,)
    for cols in (64, 8200):
        x = torch.empty((0, cols), device="cuda")
        dx, dw, db = nss.mb_layer_norm_backward(x, x, mean, rstd, torch.ones(cols, device="cuda"))
        assert dx.shape == (0, cols) and not dw.any() and not db.any()


@pytest.mark.parametrize("cols", [40, 768, 1001, 8200])
def test_layer_norm_bad_rows_stay_alone(nss, cols):
    x, w, b, dy = norm_inputs(12, 50, cols, torch.float32, torch.float32)
    clean = nss.mb_layer_norm(x, w, b)
    dirty = x.clone()
    dirty[7, 3], dirty[20, 0], dirty[33, cols - 1] = float("nan"), float("inf"), float("-inf")
    y, mean, rstd = nss.mb_layer_norm(dirty, w, b)
    ok = torch.ones(50, dtype=torch.bool, device="cuda")
    ok[[7, 20, 33]] = False
    assert torch.isnan(y[~ok]).all()
    for a, c in zip((y, mean, rstd), clean):
        same_bits(a[ok], c[ok], "rows beside a bad one")
    dx = nss.mb_layer_norm_backward(dy, dirty, mean, rstd, w)[0]
    same_bits(dx[ok], nss.mb_layer_norm_backward(dy, x, clean[1], clean[2], w)[0][ok], "dx beside a bad row")
    assert torch.isnan(dx[~ok]).all()


def test_layer_norm_leading_dimensions(nss):
    x, w, b, dy = norm_inputs(13, 60, 96, torch.bfloat16, torch.bfloat16)
    flat = nss.mb_layer_norm(x, w, b)
    deep = nss.mb_layer_norm(x.view(3, 4, 5, 96), w, b)
    same_bits(deep[0].view(60, 96), flat[0], "y")
    assert deep[1].shape == (3, 4, 5)
    back = nss.mb_layer_norm_backward(dy.view(3, 4, 5, 96), x.view(3, 4, 5, 96), deep[1], deep[2], w)
    check_norm_backward(nss, dy, x, flat[1], flat[2], w)
    same_bits(back[0].view(60, 96), nss.mb_layer_norm_backward(dy, x, flat[1], flat[2], w)[0], "dx")


# ---------------------------------------------------------------- rotary

def rotary_ref(x, positions, inv_freq, sections, interleaved, sign):
    """(result, bound) in 64 bits from the fp32 angle, which is part of the definition."""
    pairs = inv_freq.numel()
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).cuda()
    pos = positions.float() if positions.dim() == 3 else positions.float()[:, None].expand(-1, x.shape[0], -1)
    angle = (pos[axis].permute(1, 2, 0) * inv_freq).double()[:, :, None]
    c, s = angle.cos(), angle.sin() * sign
    y = x.double().clone(memory_format=torch.contiguous_format)
    bound = torch.zeros_like(y)
    i = torch.arange(pairs, device="cuda")
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    # sine and cosine within 2 ulp (4 U), two products, a sum
    for at, p, q in ((a, u * c, v * s), (b, v * c, u * s)):
        bound[..., at] = 8 * U * (p.abs() + q.abs()) + 2.0 ** -120
    turned = torch.zeros_like(y, dtype=torch.bool)
    turned[..., :2 * pairs] = True
    return y, torch.where(turned, bound + rounding(y, x.dtype), 0.0)


def check_rotary(nss, q, k, positions, inv_freq, sections, interleaved, **out):
    for call, sign in ((nss.mb_rotary, 1.0), (nss.mb_rotary_backward, -1.0)):
        got = call(q, k, positions, inv_freq, sections, interleaved, **out)
        torch.cuda.synchronize()
        for x, y, what in zip((q, k), got, "qk"):
            if x is None:
                assert y is None
                continue
            x4, y4 = (x, y) if x.dim() == 4 else (x[None], y[None])
            ref, bound = rotary_ref(x4, positions, inv_freq, sections, interleaved, sign)
            within(y4, ref, bound, f"{what}, sign {sign}")


def rotary_inputs(seed, batch, tokens, heads, kv, dim, sections, dtype, base=1e4, first=0):
    g = gen(seed)
    q, k = randn(g, batch, tokens, heads, dim).to(dtype), randn(g, batch, tokens, kv, dim).to(dtype)
    pos = torch.randint(0, 300, (len(sections), batch, tokens), generator=g, device="cuda") + first
    freq = torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections]).float().cuda()
    return q, k, pos, freq


ROTARY = [  # batch, tokens, heads, kv heads, dim, sections
    (1, 1, 1, 1, 2, (1,)), (2, 5, 3, 1, 16, (8,)), (1, 33, 12, 12, 64, (32,)), (3, 17, 4, 2, 64, (16, 16)),
    (2, 50, 5, 1, 128, (16, 24, 24)), (1, 9, 2, 2, 80, (4, 12, 16)), (2, 7, 3, 3, 77, (17, 18)), (1, 200, 1, 1, 66, (33,)),
    (1, 3, 2, 1, 600, (100, 0, 200)), (1, 2, 1, 1, 8200, (4096,)), (1, 5, 70, 3, 40, (8, 8, 2, 2)), (4, 1, 16, 16, 96, (40,)),
    (1, 4, 2, 1, 3000, (1500,))]


@pytest.mark.parametrize("case", ROTARY)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary(nss, case, dtype, interleaved):
    batch, tokens, heads, kv, dim, sections = case
    q, k, pos, freq = rotary_inputs(sum(case[:5]), batch, tokens, heads, kv, dim, sections, TYPES[dtype])
    check_rotary(nss, q, k, pos.int(), freq, sections, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,sections", [(64, (16, 16)), (72, (16, 16)), (70, (17, 18)), (64, (7, 8))])
def test_rotary_layouts(nss, dim, sections, interleaved):
    """Slices of a fused projection, head-major storage, odd offsets; positions of every type and layout."""
    b, t, h, hk = 2, 37, 6, 2
    q, k, pos, freq = rotary_inputs(3, b, t, h, hk, dim, sections, torch.bfloat16)
    fused = torch.cat((q, k, q[:, :, :hk]), 2)
    views = [(fused[:, :, :h], fused[:, :, h:h + hk]),
             (q.transpose(1, 2).contiguous().transpose(1, 2), k.transpose(1, 2).contiguous().transpose(1, 2)),
             (torch.nn.functional.pad(q, (1, 2))[..., 1:1 + dim], torch.nn.functional.pad(k, (3, 0))[..., 3:])]
    kinds = [pos.int(), pos.long(), pos.float() + 0.25, pos.int().transpose(1, 2).contiguous().transpose(1, 2),
             pos[:, 0].int(), pos[:, :1].expand(-1, b, -1)]
    for (qv, kv), p in zip(itertools.cycle(views), kinds + kinds[:3]):
        check_rotary(nss, qv, kv, p, freq, sections, interleaved)
    check_rotary(nss, q, None, pos, freq, sections, interleaved)
    check_rotary(nss, q[0], k[0], pos[:, :1], freq, sections, interleaved)


@pytest.mark.parametrize("dim,pad", [(64, 0), (64, 8), (70, 3)])
def test_rotary_in_place_and_guard_bands(nss, dim, pad):
    b, t, h = 2, 19, 3
    q, k, pos, freq = rotary_inputs(4, b, t, h, h, dim, (dim // 2 - 2,), torch.bfloat16)
    want = nss.mb_rotary(q, k, pos, freq, (dim // 2 - 2,))
    qi, ki = q.clone(), k.clone()
    got = nss.mb_rotary(qi, ki, pos, freq, (dim // 2 - 2,), q_out=qi, k_out=ki)
    assert got[0] is qi and got[1] is ki
    same_bits(qi, want[0], "q in place")
    same_bits(ki, want[1], "k in place")
    guards = [Guarded((b * t * h, dim), torch.bfloat16, 8, pad) for _ in range(2)]
    outs = [g.t.as_strided((b, t, h, dim), (t * h * (dim + pad), h * (dim + pad), dim + pad, 1), g.t.storage_offset())
            for g in guards]
    nss.mb_rotary(q, k, pos, freq, (dim // 2 - 2,), q_out=outs[0], k_out=outs[1])
    for g, o, w in zip(guards, outs, want):
        same_bits(o, w, "strided result")
        g.check("rotary result")


def test_rotary_far_positions_and_the_way_back(nss):
    """Angles of up to 2^20 radians, negative ones, and the inverse."""
    q, k, pos, freq = rotary_inputs(6, 1, 64, 4, 4, 64, (32,), torch.float32, first=1 << 20)
    pos[:, :, ::2] *= -1
    check_rotary(nss, q, k, pos, freq, (32,), False)
    out = nss.mb_rotary(q, k, pos, freq, (32,))
    back = nss.mb_rotary_backward(*out, pos, freq, (32,))
    for a, c in zip(back, (q, k)):
        # two turns, each within 8 U of |u| + |v|
        assert ((a.double() - c.double()).abs() <= 40 * U * c.double().abs().amax()).all()


def test_rotary_of_nothing(nss):
    freq = torch.ones(4, device="cuda")
    for shape in ((0, 5, 2, 8), (2, 0, 2, 8)):
        q = torch.empty(shape, device="cuda")
        out = nss.mb_rotary(q, q, torch.empty((1,) + shape[:2], device="cuda", dtype=torch.int32), freq, (4,))
        assert out[0].shape == shape
    with pytest.raises(nss.MuonBankError):
        nss.mb_rotary(torch.empty((1, 2, 0, 8), device="cuda"), None, torch.zeros((1, 1, 2), device="cuda"), freq, (4,))


# ---------------------------------------------------------------- router

def router_ref(logits, k, valid, normalize):
    l = logits.double()
    t, e = l.shape
    used = ~(l == float("-inf")).all(1)
    if valid is not None:
        used &= valid.bool()
    p = torch.where(used[:, None], torch.softmax(l, 1), 0.0)
    # the k largest, the lowest index among equals, by a stable sort of the exact values
    top, index = torch.sort(l, dim=1, descending=True, stable=True)
    top, index = top[:, :k], index[:, :k]
    chosen = (top > float("-inf")) & used[:, None]
    gate = torch.where(chosen, p.gather(1, index), 0.0)
    if normalize:
        gate = gate / torch.where(used, gate.sum(1), 1.0)[:, None]
    index = torch.where(chosen, index, -1)
    counts = torch.bincount(index[index >= 0].reshape(-1), minlength=e)
    n = int(used.sum())
    loss = e * (counts.double() * p.sum(0)).sum() / (k * max(n, 1) ** 2)
    return p, index, gate, counts, loss, n


def router_rel(logits):
    """Relative error of a probability: the exponent's argument (its magnitude times U), expf (2 ulp), the sum, a division."""
    l = logits.double()
    span = torch.where(torch.isfinite(l), l, 0.0)
    span = float((span.amax(1) - span.amin(1)).max()) if l.numel() else 0.0
    return (2 * span + 4 + 4 + 37 + 4) * U


def check_router(nss, logits, k, valid=None, normalize=False, seed=0):
    out = nss.mb_router(logits, k, valid, normalize)
    torch.cuda.synchronize()
    t, e = logits.shape
    p, index, gate, counts, loss, n = router_ref(logits, k, valid, normalize)
    assert torch.equal(out.index.long(), index), "index"
    assert torch.equal(out.counts.long(), counts), "counts"
    assert out.used.item() == n
    rel = router_rel(logits)
    # exp(l - max) below the smallest normal loses its relative precision
    within(out.gate, gate, 2.1 * rel * gate + 2.0 ** -125, "gate")
    sums = min(t, t / 100 + 8) + 64 + 304 / 16 + 32 + 40     # tokens of a lane, warps, parts, experts
    within(out.loss, loss.reshape(1), (1.1 * rel + sums * U) * loss.reshape(1) + 2.0 ** -120, "loss")
    g = gen(seed + 1)
    dloss, dgate = randn(g, 1) * max(t, 1), randn(g, t, k)
    for dl, dg in ((dloss, dgate), (dloss, None), (None, dgate), (None, None)):
        got = nss.mb_router_backward(dl, dg, logits, out.index, out.gate, out.counts, out.used, valid, normalize)
        torch.cuda.synchronize()
        d = 0.0 if dl is None else dl.double()
        c = (d * e / (k * max(n, 1) ** 2)) * counts.double().expand_as(p)
        a = torch.zeros_like(p) if dg is None else torch.zeros_like(p).scatter_add(
            1, index.clamp(min=0), torch.where(index >= 0, dg.double(), 0.0))
        if normalize:
            w = torch.zeros_like(p).scatter_add(1, index.clamp(min=0), gate)
            wa = (w * a).sum(1, keepdim=True)
            ref = p * (c - (p * c).sum(1, keepdim=True)) + w * (a - wa)
            size = w * (a.abs() + (w * a).abs().sum(1, keepdim=True)) + p * (c.abs() + (p * c).abs().sum(1, keepdim=True))
        else:
            a = a + c
            ref = p * (a - (p * a).sum(1, keepdim=True))
            size = p * (a.abs() + (p * a).abs().sum(1, keepdim=True))
        within(got, ref, (4 * rel + 60 * U) * size + rounding(ref, logits.dtype) + 2.0 ** -120, "dlogits")
    return out


ROUTER = [(1, 1, 1), (1, 4, 4), (5, 2, 1), (33, 8, 2), (100, 7, 7), (63, 16, 16), (200, 60, 4), (77, 64, 8), (1000, 65, 3),
          (300, 128, 32), (129, 250, 5), (2500, 256, 8), (17, 257, 8), (40, 512, 6), (21, 513, 2), (30, 1000, 7), (19, 1024, 32),
          (4099, 32, 2), (9001, 8, 1)]


@pytest.mark.parametrize("case", ROUTER)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("normalize", [False, True])
def test_router(nss, case, dtype, normalize):
    t, e, k = case
    g = gen(t + e)
    logits = (randn(g, t, e) + randn(g, 1, e)).to(TYPES[dtype])
    check_router(nss, logits, k, None, normalize)
    valid = torch.rand(t, generator=g, device="cuda") < 0.7
    closed = torch.rand((t, e), generator=g, device="cuda") < 0.4
    closed[:: 5] = True
    masked = logits.masked_fill(closed, float("-inf"))
    check_router(nss, masked, k, valid, normalize)
    check_router(nss, masked, k, valid.to(torch.uint8) * 3, normalize)


@pytest.mark.parametrize("experts,k", [(6, 3), (8, 8), (64, 8), (256, 8), (256, 32), (600, 5)])
def test_router_ties_and_extremes(nss, experts, k):
    """Few distinct values, both zeros, the type's lowest value as a mask, and logits far apart."""
    g = gen(2)
    few = torch.randint(-1, 2, (300, experts), generator=g, device="cuda").float() * 0.0
    few[:, ::2] = -0.0
    check_router(nss, few, k)
    few = torch.randint(-2, 3, (300, experts), generator=g, device="cuda").float()
    check_router(nss, few, k)
    check_router(nss, few.bfloat16(), k, normalize=True)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        low = randn(g, 300, experts).to(dtype)
        low[torch.rand((300, experts), generator=g, device="cuda") < 0.5] = torch.finfo(dtype).min
        low[::7] = torch.finfo(dtype).min
        out = nss.mb_router(low, k)
        p, index, gate, counts, loss, n = router_ref(low, k, None, False)
        assert torch.equal(out.index.long(), index) and torch.equal(out.counts.long(), counts) and n == 300
        # the bound of the ordinary span: at the lowest value p is exactly 0, or uniform where all are
        within(out.gate, gate, 2.1 * (2 * 16 + 49) * U * gate + 2.0 ** -125, "gate")
    descending = torch.arange(experts, 0, -1, device="cuda").float().expand(50, experts) * 0.1
    check_router(nss, descending, k)                       # rows 0 elements apart


@pytest.mark.parametrize("experts,k", [(8, 3), (16, 16), (24, 8), (60, 4), (64, 8), (128, 8), (256, 8), (256, 4), (500, 6), (1000, 8)])
def test_router_near_ties(nss, experts, k):
    """Logits that differ in their last bits only, alone and among others, in every order."""
    g = gen(77 + experts)
    t = 700
    near = 2.0 + torch.randint(0, 9, (t, experts), generator=g, device="cuda") * 2.0 ** -22
    few = torch.rand((t, experts), generator=g, device="cuda") < 8.0 / experts
    for scale in (1.0, 1e-3, 300.0):
        check_router(nss, near * scale, k)
        check_router(nss, torch.where(few, near, randn(g, t, experts).clamp(max=1.9)) * scale, k, normalize=True)
        check_router(nss, torch.where(few, near, torch.tensor(float("-inf"), device="cuda")) * scale, k)
    check_router(nss, torch.zeros(t, experts, device="cuda"), k)
    check_router(nss, torch.full((t, experts), -7.25, device="cuda").half(), k, normalize=True)
    # logits near zero under a larger one: distinct bf16 values that one exponent stands for
    tiny = (randn(g, t, experts) * 1e-30).bfloat16()
    tiny[:, 3] = 5.0
    check_router(nss, tiny, k)


@pytest.mark.parametrize("experts,k", [(8, 2), (64, 8), (256, 8), (1000, 3)])
def test_router_huge_logits(nss, experts, k):
    """Finite logits whose exponents overflow fp32: the largest win, and the rest has probability 0."""
    g = gen(5)
    for signs in (1.0, -1.0):
        l = signs * (2.5e38 + 5e37 * torch.rand((90, experts), generator=g, device="cuda"))
        l[::3] = randn(g, 30, experts)                     # ordinary tokens beside them
        l[1::3, ::2] = -3.4e38
        out = nss.mb_router(l, k)
        p, index, gate, counts, loss, n = router_ref(l, k, None, False)
        assert torch.equal(out.index.long(), index) and torch.equal(out.counts.long(), counts) and out.used.item() == 90
        within(out.gate, gate, 2.1 * (2 * 16 + 49) * U * gate + 2.0 ** -120, "gate")
        d = nss.mb_router_backward(torch.ones(1, device="cuda"), torch.ones(90, k, device="cuda"), l, *out[:3], out.used)
        assert torch.isfinite(d).all()


def test_router_without_tokens(nss):
    for t in (0, 5, 1000):
        logits = torch.full((t, 24), float("-inf"), device="cuda")
        out = nss.mb_router(logits, 3)
        assert (out.index == -1).all() and not out.gate.any() and not out.counts.any()
        assert out.loss.item() == 0.0 and out.used.item() == 0
        one = torch.ones(1, device="cuda")
        assert not nss.mb_router_backward(one, torch.ones(t, 3, device="cuda"), logits, *out[:3], out.used).any()
        none = torch.zeros(t, dtype=torch.bool, device="cuda")
        out = nss.mb_router(torch.zeros_like(logits), 3, none)
        assert (out.index == -1).all() and out.loss.item() == 0.0 and out.used.item() == 0


def test_router_nan_and_infinity(nss):
    g = gen(9)
    logits = randn(g, 64, 48)
    logits[3, 40], logits[9, 5], logits[20, :] = float("nan"), float("inf"), float("nan")
    logits[30, :10], logits[30, 11] = float("-inf"), float("nan")
    out = nss.mb_router(logits, 2)
    assert out.index[3, 0] == 40 and out.index[9, 0] == 5 and out.index[20].tolist() == [0, 1] and out.index[30, 0] == 11
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[3, 9, 20, 30]] = True
    assert torch.isnan(out.gate[bad]).all() and torch.isfinite(out.gate[~bad]).all() and torch.isnan(out.loss).all()
    assert out.used.item() == 64 and int(out.counts.sum()) == 128
    d = nss.mb_router_backward(torch.ones(1, device="cuda"), torch.ones(64, 2, device="cuda"), logits, *out[:3], out.used)
    assert torch.isfinite(d[~bad]).all() and torch.isnan(d[bad]).all()


@pytest.mark.parametrize("experts,pad", [(64, 8), (64, 3), (60, 0), (12, 1)])
def test_router_strided_rows_and_guard_bands(nss, experts, pad):
    g = gen(4)
    src, dst = (Guarded((333, experts), torch.bfloat16, 9 if pad == 3 else 8, pad) for _ in range(2))
    src.t.copy_(randn(g, 333, experts))
    out = check_router(nss, src.t, 3)
    dgate = randn(g, 333, 3)
    args = (torch.ones(1, device="cuda"), dgate, src.t, *out[:3], out.used)
    want = nss.mb_router_backward(*args)
    nss.mb_router_backward(*args, dlogits=dst.t)
    same_bits(dst.t, want, "strided dlogits")
    dst.check("dlogits")
    nss.mb_router_backward(*args, dlogits=src.t)
    same_bits(src.t, want, "dlogits over logits")
    src.check("dlogits over logits")


# ---------------------------------------------------------------- what all three share

def _calls(nss):
    g = gen(21)
    x, w, b, dy = norm_inputs(21, 700, 768, torch.bfloat16, torch.float32)
    _, mean, rstd = nss.mb_layer_norm(x, w, b)
    q, k, pos, freq = rotary_inputs(22, 2, 90, 4, 2, 64, (16, 16), torch.bfloat16)
    logits = randn(g, 3000, 64)
    out = nss.mb_router(logits, 4)
    dgate, dloss = randn(g, 3000, 4), torch.ones(1, device="cuda")
    torch.cuda.synchronize()
    return {
        "layer_norm": lambda **s: nss.mb_layer_norm(x, w, b, **s),
        "layer_norm_backward": lambda **s: nss.mb_layer_norm_backward(dy, x, mean, rstd, w, **s),
        "rotary": lambda **s: nss.mb_rotary(q, k, pos, freq, (16, 16), **s),
        "router": lambda **s: nss.mb_router(logits, 4, **s),
        "router_backward": lambda **s: (nss.mb_router_backward(dloss, dgate, logits, *out[:3], out.used, **s),),
    }


def test_identical_runs_and_other_streams(nss):
    for name, call in _calls(nss).items():
        first = call()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        again, there, raw = call(), call(stream=side), call(stream=side.cuda_stream)
        side.synchronize()
        torch.cuda.synchronize()
        for others in (again, there, raw):
            for a, c in zip(first, others):
                same_bits(a, c, name)


def test_graph_capture(nss):
    for name, call in _calls(nss).items():
        want = call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(want, got):
            same_bits(a, c, name)


def test_launch_counts_and_marks(nss):
    for name, call in _calls(nss).items():
        before = nss.mb_launch_count()
        with nss.StageTimer() as timer:
            call()
        assert nss.mb_launch_count() - before == (2 if name in ("layer_norm_backward", "router") else 1), name
        assert [m[0] for m in timer.marks] == [name]


def test_python_refusals(nss):
    x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda")
    stat = torch.zeros(4, device="cuda")
    for call in (lambda: nss.mb_layer_norm(x.double()), lambda: nss.mb_layer_norm(x[:, ::2]),
                 lambda: nss.mb_layer_norm(x, w[:63]), lambda: nss.mb_layer_norm(x, w, w.bfloat16()),
                 lambda: nss.mb_layer_norm(x, w.half()), lambda: nss.mb_layer_norm(x, w, w, y=x[:3]),
                 lambda: nss.mb_layer_norm(x, w.cpu()), lambda: nss.mb_layer_norm(x[:, :0]),
                 lambda: nss.mb_layer_norm(x, w, mean=stat[:3]),
                 lambda: nss.mb_layer_norm_backward(x[:3], x, stat, stat, w),
                 lambda: nss.mb_layer_norm_backward(x.float(), x, stat, stat, w),
                 lambda: nss.mb_layer_norm_backward(x, x, stat.double(), stat, w),
                 lambda: nss.mb_layer_norm_backward(x, x, stat, stat, None, dweight=w),
                 lambda: nss.mb_layer_norm_backward(x, x, stat, stat, w, workspace=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    q, pos, freq = x.view(1, 4, 4, 16), torch.zeros((2, 1, 4), device="cuda", dtype=torch.int32), torch.ones(8, device="cuda")
    for call in (lambda: nss.mb_rotary(q, None, pos, freq, (4, 3)), lambda: nss.mb_rotary(q, None, pos, freq, (8,)),
                 lambda: nss.mb_rotary(q, None, pos[:, :, :3], freq, (4, 4)), lambda: nss.mb_rotary(q, None, pos, freq, ()),
                 lambda: nss.mb_rotary(q, None, pos.short(), freq, (4, 4)), lambda: nss.mb_rotary(x, None, pos, freq, (4, 4)),
                 lambda: nss.mb_rotary(q, q.half(), pos, freq, (4, 4)), lambda: nss.mb_rotary(q, q[:, :3], pos, freq, (4, 4)),
                 lambda: nss.mb_rotary(q, None, pos, freq.half(), (4, 4)),
                 lambda: nss.mb_rotary(q, None, pos, freq, (4, 4), k_out=q),
                 lambda: nss.mb_rotary(q.transpose(2, 3), None, pos, freq, (4, 4))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(nss.MuonBankError):
        nss.mb_rotary(q, None, pos, torch.ones(9, device="cuda"), (5, 4))         # 18 of 16 elements
    with pytest.raises(nss.MuonBankError):
        nss.mb_rotary(q, None, pos, freq, (9, -1))
    l = torch.zeros(4, 16, device="cuda")
    out = nss.mb_router(l, 2)
    for call in (lambda: nss.mb_router(l[0], 2), lambda: nss.mb_router(l.int(), 2), lambda: nss.mb_router(l.t(), 2),
                 lambda: nss.mb_router(l, 2, torch.ones(3, device="cuda", dtype=torch.bool)),
                 lambda: nss.mb_router(l, 2, torch.ones(4, device="cuda")),
                 lambda: nss.mb_router(l, 2, counts=torch.zeros(16, device="cuda")),
                 lambda: nss.mb_router_backward(None, stat, l, *out[:3], out.used),
                 lambda: nss.mb_router_backward(None, None, l, out.index.long(), *out[1:3], out.used),
                 lambda: nss.mb_router_backward(None, None, l, out.index[:3], *out[1:3], out.used)):
        with pytest.raises(ValueError):
            call()
    for k in (0, 17, -1):
        with pytest.raises(nss.MuonBankError):
            nss.mb_router(l, k)
    with pytest.raises(nss.MuonBankError):
        nss.mb_router(torch.zeros(2, 1025, device="cuda"), 2)


# ---------------------------------------------------------------- gradients by differences, autograd, the example

def _difference(f, x, v, eps):
    return (f(x + eps * v) - f(x - eps * v)) / (2 * eps)


def test_gradients_by_differences(nss):
    """Along a random direction, the kernels' forward calls differ as their gradients say: up to
    the difference's own truncation, which the 64-bit formula shows at the same step, and the
    fp32 noise of two forward calls over twice the step."""
    from newton_schulz_stacked_gb300 import autograd as A
    g, eps = gen(31), 2.0 ** -7
    x, w, b, t = randn(g, 40, 96), 1 + 0.2 * randn(g, 96), 0.1 * randn(g, 96), randn(g, 40, 96)
    vx, vw, vb = randn(g, 40, 96), randn(g, 96), randn(g, 96)

    def norm64(x, w, b):
        xd = x.double()
        d = xd - xd.mean(1, keepdim=True)
        return (d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w.double() + b.double())

    def check(ours, ref, point, direction, noise):
        leaf = [p.clone().requires_grad_() for p in point]
        ours(*leaf).backward()
        along = sum((p.grad.double() * v.double()).sum() for p, v in zip(leaf, direction))
        leaf64 = [p.double().requires_grad_() for p in point]
        ref(*leaf64).backward()
        along64 = sum((p.grad * v.double()).sum() for p, v in zip(leaf64, direction))
        at = lambda s, f: f(*[p + s * eps * v for p, v in zip(point, direction)]).double().item()
        ours_diff, ref_diff = ((at(1, f) - at(-1, f)) / (2 * eps) for f in (ours, ref))
        truncation = abs(ref_diff - along64.item())
        assert abs(ours_diff - along.item()) <= 1.5 * truncation + noise, (ours_diff, along.item(), truncation, noise)

    y = norm64(x, w, b)
    # every y within about 60 U of itself, twice, over 2 eps; the step's rounding of x + eps v moves y by U |x| / eps too
    noise = 100 * U * float((t.abs().double() * (y.abs() + 1)).sum()) / eps
    check(lambda a, c, d: (A.layer_norm(a, c, d) * t).double().sum(), lambda a, c, d: (norm64(a, c, d) * t.double()).sum(),
          (x, w, b), (vx, vw, vb), noise)

    q, k, pos, freq = rotary_inputs(32, 2, 9, 4, 2, 24, (4, 6), torch.float32)
    tq, tk = randn(g, *q.shape), randn(g, *k.shape)

    def rot64(a, c):
        out = [rotary_ref_plain(z, pos, freq, (4, 6)) for z in (a, c)]
        return (out[0] * tq.double()).sum() + (out[1] * tk.double()).sum()

    def rotary_ref_plain(z, positions, inv_freq, sections):
        axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).cuda()
        angle = (positions.float()[axis].permute(1, 2, 0) * inv_freq).double()[:, :, None]
        n = inv_freq.numel()
        z = z.double()
        u, v = z[..., :n], z[..., n:2 * n]
        return torch.cat((u * angle.cos() - v * angle.sin(), v * angle.cos() + u * angle.sin(), z[..., 2 * n:]), -1)

    def rot(a, c):
        o = A.rotary(a, c, pos, freq, (4, 6))
        return (o[0] * tq).double().sum() + (o[1] * tk).double().sum()

    noise = 40 * U * float((tq.abs().double() * (q.abs() + 1)).sum() + (tk.abs().double() * (k.abs() + 1)).sum()) / eps
    check(rot, rot64, (q, k), (randn(g, *q.shape), randn(g, *k.shape)), noise)

    # logits whose order no step of the difference changes: at least 0.1 apart, steps of at most 4 eps
    logits = torch.stack([torch.randperm(24, generator=g, device="cuda") for _ in range(50)]).float() * 0.1
    direction = randn(g, 50, 24).clamp(-4, 4)
    tg = randn(g, 50, 3)
    for normalize in (False, True):
        counts = router_ref(logits, 3, None, normalize)[3]

        def ours(l):
            r = A.route(l, 3, normalize=normalize)
            return (r.gate * tg).double().sum() + 5 * r.loss.double()

        def ref(l):
            p = torch.softmax(l.double(), 1)
            gate = p.gather(1, logits.topk(3, 1).indices)
            gate = gate / gate.sum(1, keepdim=True) if normalize else gate
            return (gate * tg.double()).sum() + 5 * 24 / (3 * 50 * 50) * (counts.double() * p.sum(0)).sum()
        noise = 200 * U * (float(tg.abs().sum()) + 50) / eps
        check(ours, ref, (logits,), (direction,), noise)


def test_autograd_of_expanded_and_missing_gradients(nss):
    from newton_schulz_stacked_gb300 import autograd as A
    g = gen(41)
    x, w, b, _ = norm_inputs(41, 30, 72, torch.bfloat16, torch.float32)
    x.requires_grad_(), w.requires_grad_(), b.requires_grad_()
    A.layer_norm(x, w, b).sum().backward()                 # the gradient of a sum is one expanded element
    assert torch.equal(b.grad, torch.full_like(b, 30.0))
    A.layer_norm(x, w).float().square().sum().backward()
    A.layer_norm(x).float().square().sum().backward()
    with pytest.raises(ValueError):
        A.layer_norm(x, None, b)
    q, k, pos, freq = rotary_inputs(42, 1, 6, 2, 1, 16, (8,), torch.float32)
    for use in ((True, True), (True, False), (False, True)):
        leaf = [q.clone().requires_grad_(), k.clone().requires_grad_()]
        out = A.rotary(*leaf, pos, freq, (8,))
        sum(o.sum() for o, u in zip(out, use) if u).backward()
        want = nss.mb_rotary_backward(torch.ones_like(q), torch.ones_like(k), pos, freq, (8,))
        for p, u, r in zip(leaf, use, want):
            assert (p.grad is not None) == u
            if u:
                same_bits(p.grad, r, "expanded gradient")
    A.rotary(leaf[0], None, pos, freq, (8,))[0].sum().backward()
    l = randn(g, 20, 10).requires_grad_()
    A.route(l, 2).loss.backward()
    first = l.grad.clone()
    l.grad = None
    r = A.route(l, 2)
    r.gate.sum().backward()
    l.grad, second = None, l.grad
    r = A.route(l, 2)
    (r.loss + r.gate.sum()).backward()
    assert torch.allclose(l.grad, first + second, rtol=0, atol=8 * U * float(l.grad.abs().max() + 1))


def test_example_trains(nss):
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import moe_block_step
    finally:
        sys.path.pop(0)
    losses = moe_block_step.train(steps=20)
    assert losses[-1][0] < 0.9 * losses[0][0]
    assert all(0.5 < balance < 10 for _, balance in losses)
