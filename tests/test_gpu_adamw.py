"""AdamW over lists of tensors against its formula in 64 bits, and bit for bit against the same fp32 operations."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

LR, WD, BETA1, BETA2, EPS = 1e-2, 0.1, 0.9, 0.95, 1e-8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def nss():
    from newton_schulz_stacked_gb300.build import build_all
    build_all()
    import newton_schulz_stacked_gb300 as nss
    return nss


def _randn(n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda")


def _mix(x):
    low = 0xFFFFFFFF
    x = x * 0x9E3779B1 & low
    x = x ^ x >> 16
    x = x * 0x6A09E667 & low
    x = x ^ x >> 15
    x = x * 0xBB67AE85 & low
    return x ^ x >> 16


def _bits(seed, step, place, n):
    key = _mix((_mix((_mix(seed) + step) & 0xFFFFFFFF) + place) & 0xFFFFFFFF)
    return _mix((torch.arange(n, device="cuda") + key) & 0xFFFFFFFF)


def _weight(state):
    if state.mantissa is None:
        return state.param.float()
    low = state.mantissa.to(torch.int32) & 0xFFFF
    return (state.param.view(torch.int16).to(torch.int32) << 16 | low).view(torch.float32)


def _moments(state):
    """m and r (the root of v) as fp32 holds them."""
    if state.avg_scale is None:
        return state.exp_avg.flatten(), None
    at = torch.arange(state.param.numel(), device="cuda") // 256
    return tuple(c.flatten().float() * s[at] for c, s in ((state.exp_avg, state.avg_scale), (state.exp_avg_sq, state.sq_scale)))


def _codes(values, root, bits):
    """Codes (as float) and scales of a whole tensor's new values, by the header's rules in fp32."""
    n = len(values)
    v = torch.nn.functional.pad(values, (0, -n % 256)).view(-1, 256)
    size = torch.where(v.isfinite(), v.abs(), 0.0).amax(1, keepdim=True)
    some = size >= 2.0 ** -100
    q = v * torch.where(some, size.reciprocal() * 448, 0.0)
    q = torch.where(q.abs() < 480, q, math.nan)
    if bits is not None:
        b = torch.nn.functional.pad(bits, (0, -n % 256)).view(-1, 256).to(torch.int32)
        a = q.abs()
        low = a < 2.0 ** -6
        a = torch.where(low, a + 2.0 ** -6, a)
        a = ((a.view(torch.int32) + (b << 4)) & -(1 << 20)).view(torch.float32)
        a = torch.where(low, a - 2.0 ** -6, a).clamp(max=448)
        q = torch.where(q.isnan(), q, a.copysign(q))
    if root:
        q = torch.where((v > 0) & some, q.clamp(min=2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).flatten()[:n].float(), torch.where(some, size * (1 / 448), 0.0)[:, 0]


def _expect(state, place, step, grad_scale=None, seed=None, lr=LR, wd=WD):
    """The step in fp32, one rounding per operation: (weight, exp_avg, exp_avg_sq, avg_scale, sq_scale)."""
    lr, wd = lr * state.lr_mul, wd * state.wd_mul
    g = state.grad.flatten().float()
    if grad_scale is not None:
        g = g * grad_scale
    m, r = _moments(state)
    v = state.exp_avg_sq.flatten() if r is None else r * r
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * g * (1 - BETA2)
    r = torch.sqrt(v)
    w = _weight(state).flatten() * (1 - lr * wd) - m / (r * (1 / math.sqrt(1 - BETA2 ** step)) + EPS) * (lr / (1 - BETA1 ** step))
    if state.avg_scale is None:
        return w, m, v, None, None
    bits = None if seed is None else _bits(seed, step, place, len(m))
    mc, ms = _codes(m, False, None if bits is None else bits & 0xFFFF)
    vc, vs = _codes(r, True, None if bits is None else bits >> 16)
    return w, mc, vc, ms, vs


def _same(a, b):
    a, b = a.flatten(), b.flatten()
    assert torch.equal(a.isnan(), b.isnan())
    assert torch.equal(a[~a.isnan()], b[~b.isnan()])


def _check(state, want):
    w, m, v, ms, vs = want
    if state.mantissa is None:
        _same(state.param.float(), w.to(state.param.dtype).float())
    else:
        _same(_weight(state), w)
    _same(state.exp_avg.float(), m)
    _same(state.exp_avg_sq.float(), v)
    if ms is not None:
        _same(state.avg_scale, ms)
        _same(state.sq_scale, vs)


def _state(nss, n, param="f32", grad="f32", mantissa=False, bits=32, seed=0, shift=0, lr_mul=1.0, wd_mul=1.0):
    """A tensor some steps into training; shift: elements from a 16-byte boundary to each of its tensors."""
    def place(t):
        whole = torch.empty(n + shift, device="cuda", dtype=t.dtype)
        whole[shift:].copy_(t)
        return whole[shift:]

    w = _randn(n, seed)
    low = None
    if mantissa:
        low, w = place(w.view(torch.int16)[0::2].contiguous()), w.view(torch.int16)[1::2].contiguous().view(torch.bfloat16)
    g = (1e-2 * _randn(n, seed + 1) * torch.exp(_randn(n, seed + 2))).to(TYPES[grad])
    m, r = 1e-3 * _randn(n, seed + 3), 1e-2 * torch.exp(_randn(n, seed + 4))
    scales = (None, None)
    if bits == 8:
        (m, ms), (r, vs) = _codes(m, False, None), _codes(r, True, None)
        scales = (ms, vs)
        m, r = m.to(torch.float8_e4m3fn), r.to(torch.float8_e4m3fn)
    return nss.AdamState(place(w.to(TYPES[param])), place(g), place(m), place(r * r if bits == 32 else r), low, *scales, lr_mul,
                         wd_mul)


FORMS = [("f32", "f32", False), ("f32", "bf16", False), ("f32", "f16", False), ("bf16", "bf16", False), ("bf16", "f32", False),
         ("bf16", "f16", False), ("f16", "f16", False), ("f16", "f32", False), ("f16", "bf16", False), ("bf16", "bf16", True),
         ("bf16", "f32", True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,mantissa", FORMS)
def test_types_and_sizes(nss, bits, param, grad, mantissa):
    sizes = [1, 7, 255, 256, 257, 768, 4096, 4097, 12289]
    states = [_state(nss, n, param, grad, mantissa, bits, seed=10 * n, shift=s) for n in sizes for s in (0, 1)]
    for step in (1, 2, 3):
        want = [_expect(s, i, step) for i, s in enumerate(states)]
        nss.adamw_multi_step(states, LR, WD, BETA1, BETA2, EPS, step)
        for s, w in zip(states, want):
            _check(s, w)


@pytest.mark.parametrize("bits", [32, 8])
def test_against_64_bits(nss, bits):
    """w within the fp32 roundings of the formula: five in the update, two in m, three in v halved by the root, and
    those of the scalars (2^-24 each, of the terms' sizes)."""
    s = _state(nss, 100003, bits=bits)
    m, r = _moments(s)
    v = s.exp_avg_sq.double() if r is None else r.double() ** 2
    m, g, w0 = m.double(), s.grad.double(), s.param.double()
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    size = (BETA1 * (m.abs() + (1 - BETA1) * g.abs()) + (1 - BETA1) * g.abs())       # of the sum's terms
    d = torch.sqrt(v / (1 - BETA2 ** 7)) + EPS
    want = w0 * (1 - LR * WD) - LR / (1 - BETA1 ** 7) * m / d
    nss.adamw_multi_step([s], LR, WD, BETA1, BETA2, EPS, 7)
    bound = 2.0 ** -24 * (3 * w0.abs() + 12 * LR / (1 - BETA1 ** 7) * (2 * size) / d + want.abs())
    assert ((s.param.double() - want).abs() <= bound).all()
    if bits == 32:
        assert ((s.exp_avg.double() - m).abs() <= 2.0 ** -24 * 4 * size).all()
        assert ((s.exp_avg_sq.double() - v).abs() <= 2.0 ** -24 * 6 * v).all()
    else:
        # half a step of a code: 2^-4 of the value, or half of 2^-9 scales where the codes are evenly spaced
        at = torch.arange(len(m), device="cuda") // 256
        got_m, got_r = _moments(s)
        assert ((got_m - m).abs() <= 1.001 * torch.maximum(2.0 ** -4 * m.abs(), 2.0 ** -10 * s.avg_scale[at])).all()
        # (a positive root is held up to a whole 2^-9)
        assert ((got_r - v.sqrt()).abs() <= 1.001 * torch.maximum(2.0 ** -4 * v.sqrt(), 2.0 ** -9 * s.sq_scale[at])).all()


def test_a_mixed_list_with_factors(nss):
    """Types, moments, factors and an empty tensor in one call; two launches."""
    states = [_state(nss, n, *f, bits=b, seed=n, lr_mul=l, wd_mul=d)
              for n, f, b, l, d in ((5000, FORMS[0], 32, 2.0, 0.0), (300, FORMS[9], 8, 0.5, 3.0), (0, FORMS[0], 32, 1.0, 1.0),
                                    (70001, FORMS[3], 32, 1.0, 0.25), (0, FORMS[0], 8, 1.0, 1.0), (4096, FORMS[10], 8, 1.5, 1.0))]
    scale = torch.tensor([0.3], device="cuda")
    want = [_expect(s, i, 5, 0.3, 99) for i, s in enumerate(states)]
    before = nss.mb_launch_count()
    nss.adamw_multi_step(states, LR, WD, BETA1, BETA2, EPS, 5, grad_scale=scale, seed=99)
    assert nss.mb_launch_count() - before == 2
    for s, w in zip(states, want):
        if s.param.numel():
            _check(s, w)


def test_more_tensors_than_a_launch_takes(nss):
    states = [_state(nss, 40 + i % 7, bits=8 if i % 3 == 0 else 32, seed=i) for i in range(1000)]
    want = [_expect(s, i, 2, seed=3) for i, s in enumerate(states)]
    nss.adamw_multi_step(states, LR, WD, BETA1, BETA2, EPS, 2, seed=3)
    for s, w in zip(states, want):
        _check(s, w)


def test_gradient_values_that_are_no_numbers(nss):
    """NaN and infinities stay in their elements, in 8 bits too; gradients whose squares overflow or vanish."""
    for bits in (32, 8):
        s = _state(nss, 1000, bits=bits)
        for i, x in enumerate((math.nan, math.inf, -math.inf, 3e38, 1e-30, 0.0)):
            s.grad[100 + 60 * i] = x
        want = _expect(s, 0, 4)
        nss.adamw_multi_step([s], LR, WD, BETA1, BETA2, EPS, 4)
        _check(s, want)
        bad = (~s.param.isfinite()).nonzero().flatten().tolist()
        assert bad == [100, 160, 220] and s.param.isnan().sum() == 3
        if bits == 8:
            assert s.avg_scale.isfinite().all() and s.sq_scale.isfinite().all()


def test_blocks_of_nothing(nss):
    """Zero moments and gradients stay zero; magnitudes below 2^-100 count as zero; a lone tiny root is kept."""
    s = nss.adamw_state(torch.ones(768, device="cuda"), torch.zeros(768, device="cuda"), bits=8)
    nss.adamw_multi_step([s], LR, WD, BETA1, BETA2, EPS, 1)
    assert not s.exp_avg.float().any() and not s.sq_scale.any() and not s.avg_scale.any()
    assert torch.equal(s.param, torch.full_like(s.param, 1) * (1 - LR * WD))
    s.grad[:256] = 2.0 ** -110
    s.grad[256:512] = 1.0
    s.grad[300] = 1e-12                         # its root would round to code 0 beside 1.0
    want = _expect(s, 0, 2)
    nss.adamw_multi_step([s], LR, WD, BETA1, BETA2, EPS, 2)
    _check(s, want)
    assert s.avg_scale[0] == 0 and not s.exp_avg[:256].float().any()
    assert s.exp_avg_sq[300].float() == 2.0 ** -9 and s.exp_avg[300].float() == 0


def test_random_rounding(nss):
    """Bit for bit by the seed, other seeds and steps other bits; without bias: the mean of the rounded values over
    many seeds comes to the value, within six deviations of a mean of one step's uniform part."""
    n, tries = 4096, 64
    total, exact = torch.zeros(n, device="cuda", dtype=torch.double), None
    for seed in range(tries):
        s = _state(nss, n, bits=8)
        want = _expect(s, 0, 9, seed=seed)
        nss.adamw_multi_step([s], LR, WD, BETA1, BETA2, EPS, 9, seed=seed)
        if seed < 3:
            _check(s, want)
        total += _moments(s)[0].double()
    s = _state(nss, n, bits=8)
    m, _ = _moments(s)
    exact = (BETA1 * m + (1 - BETA1) * s.grad).double()
    at = torch.arange(n, device="cuda") // 256
    nss.adamw_multi_step([s], LR, WD, BETA1, BETA2, EPS, 9, seed=0)
    step = torch.maximum(exact.abs() / 8, 2.0 ** -9 * s.avg_scale[at])             # a step is at most 1/8 of the value
    off = (total / tries - exact).abs()
    assert (off <= 6 * step * 0.5 / math.sqrt(tries)).all()                        # a two-valued mean's deviation: half a step
    assert off.mean() < 0.5 * step.mean() / math.sqrt(tries)
    other = _state(nss, n, bits=8)
    nss.adamw_multi_step([other], LR, WD, BETA1, BETA2, EPS, 9, seed=1)
    assert not torch.equal(other.exp_avg.float(), s.exp_avg.float())


def test_scalars_from_the_device_in_a_graph(nss):
    """The same bits as by value, replayed with new scalars; two graphs with workspaces of their own."""
    def fresh():
        return [_state(nss, n, *f, bits=b, seed=n, lr_mul=2.0) for n, f, b in ((5000, FORMS[9], 32), (4097, FORMS[0], 8))]

    plain, graphed = fresh(), fresh()
    scalars = torch.tensor([LR, WD, BETA1, BETA2, EPS, 1], dtype=torch.float64, device="cuda")
    warm = fresh()
    ws = nss.adamw_multi_step_dev(warm, scalars, seed=5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nss.adamw_multi_step_dev(graphed, scalars, seed=5, workspace=ws)
    for step, lr in ((1, LR), (2, 0.5 * LR), (3, 0.1 * LR)):
        scalars[0], scalars[5] = lr, step
        graph.replay()
        nss.adamw_multi_step(plain, lr, WD, BETA1, BETA2, EPS, step, seed=5)
        for a, b in zip(plain, graphed):
            for x, y in zip(a[:7], b[:7]):
                assert (x is None) == (y is None)
                if x is not None:
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert nss.mb_sync_status() == 0
    scalars[5] = 0
    graph.replay()
    from newton_schulz_stacked_gb300 import _binding as b
    assert nss.mb_sync_status() == b.MB_ERR_ARG
    assert nss.mb_sync_status() == 0


def test_streams(nss):
    a, b = (_state(nss, 1 << 20, "bf16", "bf16", True, 8) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    nss.adamw_multi_step([a], LR, WD, BETA1, BETA2, EPS, 3, stream=side)
    with torch.cuda.stream(side):
        nss.adamw_multi_step([b], LR, WD, BETA1, BETA2, EPS, 3)
    side.synchronize()
    assert torch.equal(a.param, b.param) and torch.equal(a.mantissa, b.mantissa)


def test_versions_and_refusals(nss):
    s = _state(nss, 512, "bf16", "bf16", True, 8)
    version = s.param._version
    nss.adamw_multi_step([s], LR, WD)
    assert s.param._version > version and s.avg_scale._version > 0
    keep = [t.clone() for t in s[:7]]

    def refused(match, tensors=None, error=ValueError, **change):
        with pytest.raises(error, match=match):
            nss.adamw_multi_step(tensors or [s._replace(**change)], LR, WD)

    refused("overlap", [s, s])
    refused("overlap", exp_avg_sq=s.exp_avg)
    refused("elements", exp_avg=s.exp_avg[:511])
    refused("grad", grad=s.grad.view(2, 256))
    refused("grad", grad=s.grad.to(torch.float64))
    refused("contiguous", grad=torch.zeros(1024, device="cuda", dtype=torch.bfloat16)[::2])
    refused("contiguous", grad=torch.zeros(1, device="cuda", dtype=torch.bfloat16).expand(512))
    refused("dtype", exp_avg_sq=torch.zeros(512, device="cuda"))
    refused("missing", avg_scale=None)
    refused("elements", sq_scale=torch.zeros(3, device="cuda"))
    refused("only", exp_avg=torch.zeros(512, device="cuda"), exp_avg_sq=torch.zeros(512, device="cuda"))
    refused("bfloat16", param=torch.zeros(512, device="cuda"), grad=torch.zeros(512, device="cuda"))
    refused("tensor", grad=None)
    refused("cpu", grad=s.grad.cpu())
    with pytest.raises(ValueError, match="seed"):
        nss.adamw_multi_step([s], LR, WD, seed=-1)
    with pytest.raises(ValueError, match="grad_scale"):
        nss.adamw_multi_step([s], LR, WD, grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(nss.MuonBankError):
        nss.adamw_multi_step([s], LR, WD, step=0)
    with pytest.raises(ValueError, match="workspace"):
        nss.adamw_multi_step_dev([s], torch.ones(6, device="cuda", dtype=torch.float64),
                                 workspace=torch.empty(8, device="cuda", dtype=torch.uint8))
    with pytest.raises(ValueError, match="scalars"):
        nss.adamw_multi_step_dev([s], torch.ones(6, device="cuda"))
    torch.cuda.synchronize()
    for t, k in zip(s[:7], keep):
        assert torch.equal(t.view(torch.uint8), k.view(torch.uint8))
