"""The products with a bank's matrices and the step of the tensors that are in no bank, as a training step calls them.

Four operators:

  linear    the product with one matrix or, over groups of rows, with a bank of experts, with bias,
            activation and residual; forward (which may keep what the activation takes) and
            backward (dx, and the gradients of the weights and biases)
  adamw 32  AdamW over many tensors, moments in fp32
  adamw 8   the same, moments in 8 bits with a scale per block of 256 elements

A case is one call.  run() computes it in elementary torch operations in 32 bits, or, where
`own` is true, through this package.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 256                 # elements that share a scale
TOP = 448.0                 # the largest e4m3 number


# ---------------------------------------------------------------- cases

def _linear(name, direction, rows, cols, out, experts, dtype, activation, bias=True, residual=False, keep=False, pad=0):
    """experts = 0: one matrix; else groups of rows, one per expert, uneven, and rows behind the last."""
    return {"name": name, "op": "linear", "direction": direction, "rows": rows, "cols": cols, "out": out, "experts": experts,
            "dtype": dtype, "activation": activation, "bias": bias, "residual": residual, "keep": keep, "pad": pad}


def _adamw(name, bits, count, elements, param, grad, mantissa=False, ragged=False, tight=False, clipped=False, random=False):
    return {"name": name, "op": "adamw", "bits": bits, "count": count, "elements": elements, "param": param, "grad": grad,
            "mantissa": mantissa, "ragged": ragged, "tight": tight, "clipped": clipped, "random": random}


def listed():
    return [
        # one short prompt through a square projection: the call's latency
        _linear("linear fwd 64x768->768 bf16", "forward", 64, 768, 768, 0, "bf16", "none"),
        # the up product of a width-768 block over 64 sequences of 1024 tokens, with z kept for the backward pass
        _linear("linear fwd 65536x768->2816 relu2 bf16", "forward", 65536, 768, 2816, 0, "bf16", "relu2", keep=True),
        # the down product of a width-1024 block onto its residual stream
        _linear("linear fwd 49152x4096->1024 residual bf16", "forward", 49152, 4096, 1024, 0, "bf16", "none", residual=True),
        # 16 experts with uneven numbers of tokens and a width that no vector divides
        _linear("linear fwd 30011x1024->2730 16 experts silu bf16", "forward", 30011, 1024, 2730, 16, "bf16", "silu", keep=True),
        # a small odd micro-batch in fp16: latency and ragged edges
        _linear("linear bwd 777x768->1001 gelu f16", "backward", 777, 768, 1001, 0, "f16", "gelu"),
        # the up product's backward pass
        _linear("linear bwd 65536x768->2816 relu2 bf16", "backward", 65536, 768, 2816, 0, "bf16", "relu2"),
        # the largest: 128 Ki places over 64 experts of width 1024
        _linear("linear bwd 131072x1024->2816 64 experts relu2 bf16", "backward", 131072, 1024, 2816, 64, "bf16", "relu2",
                bias=False),
        # the norms' weights and biases of a 12-layer model: the call's latency
        _adamw("adamw 32 50x768 f32", 32, 50, 768, "f32", "f32"),
        # an embedding and a head of 50304 x 768, bf16 weights with their low halves
        _adamw("adamw 32 2x38633472 bf16+16", 32, 2, 38633472, "bf16", "bf16", mantissa=True),
        # biases, gates and small matrices of all sizes, fp32 weights with bf16 gradients, clipped
        _adamw("adamw 32 120 ragged f32", 32, 120, 400000, "f32", "bf16", ragged=True, clipped=True),
        # the same list with 8-bit moments, rounded at random
        _adamw("adamw 8 120 ragged f32", 8, 120, 400000, "f32", "bf16", ragged=True, clipped=True, random=True),
        # the embedding and the head with 8-bit moments
        _adamw("adamw 8 2x38633472 bf16+16", 8, 2, 38633472, "bf16", "bf16", mantissa=True),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["linear forward", "linear backward", "adamw 32", "adamw 8"])
    if op.startswith("linear"):
        forward = op.endswith("forward")
        cols, out = _log(rng, 64, 4096), _log(rng, 64, 4096)
        if rng.random() < 0.8:              # most widths are multiples of 8
            cols, out = cols // 8 * 8, out // 8 * 8
        experts = rng.choice([0, 0, 2, 8, _log(rng, 1, 64)])
        limit = 500e9 / (cols * out) if forward else 250e9 / (cols * out)
        rows = _log(rng, 1, int(max(1, min(131072, limit))))
        c = _linear("", "forward" if forward else "backward", rows, cols, out, experts, rng.choice(["bf16", "bf16", "f16"]),
                    rng.choice(["none", "relu", "relu2", "silu", "gelu"]), rng.random() < 0.6, rng.random() < 0.3,
                    rng.random() < 0.5, rng.choice([0, 0, 0, 8, 3]))
    else:
        count = _log(rng, 1, 300)
        elements = _log(rng, 1, max(1, (1 << 25) // count))
        param = rng.choice(["f32", "bf16", "bf16", "f16"])
        c = _adamw("", int(op.split()[1]), count, elements, param, rng.choice(["f32", param, param]),
                   param == "bf16" and rng.random() < 0.6, rng.random() < 0.5, rng.random() < 0.2, rng.random() < 0.5,
                   rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _ends(case):
    """Where each expert's rows end: uneven shares, an expert without rows where there are several, and a few rows
    that no expert has (a padded batch's)."""
    r = random.Random(case["rows"] * 31 + case["experts"])
    share = [r.expovariate(1.0) + 0.2 for _ in range(case["experts"])]
    if case["experts"] > 3:
        share[case["experts"] // 2] = 0.0
    used = case["rows"] - case["rows"] // 50
    total, at, ends = sum(share), 0.0, []
    for s in share:
        at += s
        ends.append(min(used, int(round(used * at / total))))
    return ends


def _sizes(case):
    if not case["ragged"]:
        return [case["elements"]] * case["count"]
    r = random.Random(case["count"] * 1000003 + case["elements"])
    return [_log(r, max(1, case["elements"] // 1000), case["elements"]) for _ in range(case["count"])]


def _round_up(n, to):
    return -(-n // to) * to


def _prepare_linear(case, normal):
    rows, cols, out, experts = (case[n] for n in ("rows", "cols", "out", "experts"))
    dtype = _TYPES[case["dtype"]]
    # rows as a norm leaves them, channels of different size; `pad`: the columns of a wider buffer
    x = (normal(rows, cols + case["pad"]) * torch.exp(0.3 * normal(1, cols + case["pad"]))).to(dtype)[:, :cols]
    shape = (experts, out, cols) if experts else (out, cols)
    weight = (normal(*shape) * cols ** -0.5).to(dtype)
    bias = (0.1 * normal(*shape[:-1])).to(dtype) if case["bias"] else None
    s = {"x": x, "weight": weight, "bias": bias, "ends": None, "host_ends": None}
    if experts:
        s["host_ends"] = _ends(case)
        s["ends"] = torch.tensor(s["host_ends"], dtype=torch.int32, device="cuda")
    if case["direction"] == "forward":
        s["residual"] = normal(rows, out).to(dtype) if case["residual"] else None
    else:
        s["dy"] = (normal(rows, out) * 0.02).to(dtype)
        s["z"] = None if case["activation"] == "none" else (1.1 * normal(rows, out)).to(dtype)
    return s


def _prepare_adamw(case, normal):
    sizes, bits = _sizes(case), case["bits"]
    align = 1 if case["tight"] else 64
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += _round_up(n, align)
    blocks, block_at = [], 0
    for n in sizes:
        blocks.append(block_at)
        block_at += -(-n // BLOCK)
    # tensors are views of flat buffers; their gradients differ in size from tensor to tensor and element to element
    weight = 0.02 * normal(at)
    grad = 1e-3 * normal(at) * torch.exp(normal(at))
    avg = 5e-4 * normal(at)
    sq = (1e-3 * torch.exp(normal(at))) ** 2
    flat = {"grad": grad.to(_TYPES[case["grad"]]), "mantissa": None, "avg_scale": None, "sq_scale": None}
    if case["mantissa"]:
        halves = weight.view(torch.int16).view(-1, 2)
        flat["param"] = halves[:, 1].contiguous().view(torch.bfloat16)
        flat["mantissa"] = halves[:, 0].contiguous()
    else:
        flat["param"] = weight.to(_TYPES[case["param"]])
    if bits == 32:
        flat["avg"], flat["sq"] = avg, sq
    else:
        flat["avg"], flat["sq"] = (torch.zeros(at, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
        flat["avg_scale"], flat["sq_scale"] = (torch.zeros(block_at, device="cuda") for _ in range(2))
        for n, a, b in zip(sizes, starts, blocks):
            for name, values in (("avg", avg), ("sq", sq.sqrt())):
                code, scale = _quantize(values[a:a + n], None, name == "sq")
                flat[name][a:a + n] = code
                flat[name + "_scale"][b:b + len(scale)] = scale
    tensors = []
    for n, a, b in zip(sizes, starts, blocks):
        part = {k: None if t is None else t[b:b + -(-n // BLOCK)] if k.endswith("_scale") else t[a:a + n] for k, t in flat.items()}
        tensors.append((part["param"], part["grad"], part["avg"], part["sq"], part["mantissa"], part["avg_scale"],
                        part["sq_scale"]))
    if own:
        import newton_schulz_stacked_gb300 as nss
        tensors = [nss.AdamState(*t) for t in tensors]
    return {"flat": flat, "tensors": tensors, "lr": 1e-3, "wd": 0.1, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "step": 20,
            "seed": 12345 if case["random"] else None,
            "grad_scale": torch.full((1,), 0.7, device="cuda") if case["clipped"] else None}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    state = (_prepare_linear if case["op"] == "linear" else _prepare_adamw)(case, normal)
    state["case"] = case
    return state


# ---------------------------------------------------------------- plain forms

def _groups(s):
    """(first row, last row, weight, bias) of each group."""
    if s["host_ends"] is None:
        return [(0, len(s["x"]), s["weight"], s["bias"])]
    begins = [0] + s["host_ends"][:-1]
    biases = [None] * len(begins) if s["bias"] is None else s["bias"]
    return list(zip(begins, s["host_ends"], s["weight"], biases))


def _activate(z, kind):
    if kind == "none":
        return z
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "relu2":
        return z.clamp(min=0) * z.clamp(min=0)
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _slope(z, kind):
    """The activation's derivative."""
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "relu2":
        return 2 * z.clamp(min=0)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    c = math.sqrt(2 / math.pi)
    p = 1 / (1 + torch.exp(-2 * c * (z + 0.044715 * z * z * z)))
    return p * (1 + 2 * c * z * (1 - p) * (1 + 3 * 0.044715 * z * z))


def _linear_plain(s):
    x, kind = s["x"], s["case"]["activation"]
    out = s["weight"].shape[-2]
    y, z = x.new_zeros(len(x), out), x.new_zeros(len(x), out) if s["case"]["keep"] else None
    for a, b, weight, bias in _groups(s):
        zf = x[a:b].float() @ weight.float().T
        if bias is not None:
            zf = zf + bias.float()
        if z is not None:
            z[a:b] = zf.to(x.dtype)
        yf = _activate(zf, kind)
        if s["residual"] is not None:
            yf = yf + s["residual"][a:b].float()
        y[a:b] = yf.to(x.dtype)
    return y, z


def _linear_backward_plain(s):
    x, dy = s["x"], s["dy"]
    dx, dweight = x.new_zeros(x.shape), torch.zeros_like(s["weight"])
    dbias = None if s["bias"] is None else torch.zeros_like(s["bias"])
    at = [(dweight, dbias)] if s["host_ends"] is None else zip(dweight, [None] * len(dweight) if dbias is None else dbias)
    for (a, b, weight, _), (dw, db) in zip(_groups(s), at):
        dz = dy[a:b].float()
        if s["z"] is not None:
            dz = dz * _slope(s["z"][a:b].float(), s["case"]["activation"])
        dx[a:b] = (dz @ weight.float()).to(x.dtype)
        dw.copy_(dz.T @ x[a:b].float())
        if db is not None:
            db.copy_(dz.sum(0))
    return dx, dweight, dbias


def _mix(x):
    """A hash of 32-bit whole numbers, held in 64."""
    low = 0xFFFFFFFF
    x = x * 0x9E3779B1 & low
    x = x ^ x >> 16
    x = x * 0x6A09E667 & low
    x = x ^ x >> 15
    x = x * 0xBB67AE85 & low
    return x ^ x >> 16


def _blocks_of(t):
    """A tensor's elements as rows of one block each, zeros behind the last."""
    return torch.nn.functional.pad(t, (0, -len(t) % BLOCK)).view(-1, BLOCK)


def _quantize(values, noise, root):
    """(codes, scales): e4m3 numbers and, per block, its largest magnitude over 448.  `noise`: 16 random bits per element
    (rounded at random), or None (to the nearest).  root: a positive value keeps at least the least positive code."""
    blocks = _blocks_of(values)
    size = torch.where(blocks.isfinite(), blocks.abs(), 0.0).amax(1, keepdim=True)
    some = size >= 2.0 ** -100
    q = blocks * torch.where(some, size.reciprocal() * TOP, 0.0)
    q = torch.where(q.abs() < 480, q, float("nan"))
    if noise is not None:
        a = q.abs()
        low = a < 2.0 ** -6                 # where the codes are evenly spaced
        a = torch.where(low, a + 2.0 ** -6, a)
        a = ((a.view(torch.int32) + (_blocks_of(noise).to(torch.int32) << 4)) & -(1 << 20)).view(torch.float32)
        a = torch.where(low, a - 2.0 ** -6, a).clamp(max=TOP)
        q = torch.where(q.isnan(), q, a.copysign(q))
    if root:
        q = torch.where((blocks > 0) & some, q.clamp(min=2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).flatten()[:len(values)], (size * (1 / TOP) * some)[:, 0]


def _wide(code, scale):
    return (_blocks_of(code.float()) * scale[:, None]).flatten()[:len(code)]


def _weight(t):
    """A tensor's weights in fp32: param, or param and its low halves."""
    param, mantissa = t[0], t[4]
    if mantissa is None:
        return param.float()
    return (param.view(torch.int16).to(torch.int32) << 16 | mantissa.to(torch.int32) & 0xFFFF).view(torch.float32)


def _set_weight(t, w):
    param, mantissa = t[0], t[4]
    if mantissa is None:
        param.copy_(w)
        return
    bits = w.view(torch.int32)
    param.view(torch.int16).copy_(bits >> 16)
    low = bits & 0xFFFF
    mantissa.copy_(torch.where(low < 0x8000, low, low - 0x10000))


def _scalars(s):
    """The step's numbers; a product with one of them takes the fp32 value nearest to it."""
    t = s["step"]
    return (s["beta1"], 1 - s["beta1"], s["beta2"], 1 - s["beta2"], 1 / math.sqrt(1 - s["beta2"] ** t), s["eps"],
            1 - s["lr"] * s["wd"], s["lr"] / (1 - s["beta1"] ** t))


def _noise(s, position, n):
    if s["seed"] is None:
        return None, None
    key = _mix(_mix(_mix(s["seed"]) + s["step"] & 0xFFFFFFFF) + position & 0xFFFFFFFF)
    bits = _mix(torch.arange(n, device="cuda") + key & 0xFFFFFFFF)
    return bits & 0xFFFF, bits >> 16


def _adamw_plain(s):
    b1, c1, b2, c2, root, eps, decay, rate = _scalars(s)
    for position, t in enumerate(s["tensors"]):
        _, grad, avg, sq, _, avg_scale, sq_scale = t[:7]
        g = grad.float()
        if s["grad_scale"] is not None:
            g = g * s["grad_scale"]
        if avg_scale is None:
            m, v = avg, sq
        else:
            m, r = _wide(avg, avg_scale), _wide(sq, sq_scale)
            v = r * r
        m = m * b1 + g * c1
        v = v * b2 + g * g * c2
        r = torch.sqrt(v)
        _set_weight(t, _weight(t) * decay - m / (r * root + eps) * rate)
        if avg_scale is None:
            avg.copy_(m)
            sq.copy_(v)
        else:
            low, high = _noise(s, position, len(g))
            for code, scale, values, noise, is_root in ((avg, avg_scale, m, low, False), (sq, sq_scale, r, high, True)):
                q, size = _quantize(values, noise, is_root)
                code.copy_(q)
                scale.copy_(size)


# ---------------------------------------------------------------- one pass

def _flat_outputs(s):
    """All tensors' weights and moments.  The moments' 8-bit codes are e4m3 numbers; times their blocks' scales they are m and
    the root of v."""
    f = s["flat"]
    return f["param"], f["mantissa"], f["avg"], f["sq"], f["avg_scale"], f["sq_scale"]


def run(s):
    case = s["case"]
    if not own:
        if case["op"] == "linear":
            return _linear_plain(s) if case["direction"] == "forward" else _linear_backward_plain(s)
        _adamw_plain(s)
        return _flat_outputs(s)
    import newton_schulz_stacked_gb300 as nss
    if case["op"] == "adamw":
        nss.adamw_multi_step(s["tensors"], s["lr"], s["wd"], s["beta1"], s["beta2"], s["eps"], s["step"],
                             grad_scale=s["grad_scale"], seed=s["seed"])
        return _flat_outputs(s)
    if case["direction"] == "forward":
        return nss.mb_linear(s["x"], s["weight"], s["bias"], s["residual"], case["activation"], s["ends"], keep=case["keep"])
    return nss.mb_linear_backward(s["dy"], s["x"], s["weight"], s["z"], case["activation"], s["ends"], bias=case["bias"])


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        scales = 8 * sum(-(-k // BLOCK) for k in _sizes(case)) if case["bits"] == 8 else 0
        state = 8 if case["bits"] == 32 else 2
        weight = _SIZE[case["param"]] + (2 if case["mantissa"] else 0)
        return {"bytes": (2 * weight + _SIZE[case["grad"]] + 2 * state) * n + 2 * scales, "flops": 18 * n}
    size, rows, cols, out = _SIZE[case["dtype"]], case["rows"], case["cols"], case["out"]
    used = rows if not case["experts"] else _ends(case)[-1]
    weights, biases = max(1, case["experts"]) * out * cols, max(1, case["experts"]) * out * case["bias"]
    if case["direction"] == "forward":
        wide = rows * (1 + case["keep"]) + used * case["residual"]
        return {"bytes": size * (used * cols + weights + biases + wide * out), "flops": 2 * used * cols * out}
    wide = used * (1 + (case["activation"] != "none"))
    return {"bytes": size * ((used + rows) * cols + 2 * weights + biases + wide * out), "flops": 4 * used * cols * out}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_linear(s):
    case, kind = s["case"], s["case"]["activation"]
    x, n = s["x"].double(), len(s["x"])
    many = s["host_ends"] is not None
    weight = s["weight"].double() if many else s["weight"].double()[None]
    bias = None if s["bias"] is None else s["bias"].double() if many else s["bias"].double()[None]
    ends = s["host_ends"] if many else [n]
    out = weight.shape[1]
    forward = case["direction"] == "forward"
    k = 2 * math.sqrt(2 / math.pi)
    gate = {"none": lambda z: torch.ones_like(z), "relu": lambda z: (z > 0).double(), "relu2": torch.relu,
            "silu": torch.sigmoid, "gelu": lambda z: torch.sigmoid(k * (z + 0.044715 * z ** 3))}[kind]     # act(z) = z gate(z)
    y, kept = (torch.zeros(n, out, dtype=torch.float64, device="cuda") for _ in range(2))
    dx, dw, db, start = torch.zeros_like(x), [], [], 0
    for e, end in enumerate(ends):
        at = slice(start, end)
        start = end
        if forward:
            z = torch.einsum("ti,oi->to", x[at], weight[e]) + (0 if bias is None else bias[e])
            kept[at] = z
            y[at] = z * gate(z) + (0 if s["residual"] is None else s["residual"][at].double())
            continue
        d = s["dy"][at].double()
        if s["z"] is not None:
            z = s["z"][at].double()
            p = gate(z)
            inner = {"none": 0, "relu": 0, "relu2": p, "silu": z * p * (1 - p),
                     "gelu": z * p * (1 - p) * k * (1 + 3 * 0.044715 * z ** 2)}[kind]                      # z gate'(z)
            d = d * (p + inner)
        dx[at] = torch.einsum("to,oi->ti", d, weight[e])
        dw.append(torch.einsum("to,ti->oi", d, x[at]))
        db.append(torch.einsum("to->o", d))
    if forward:
        return y, kept if case["keep"] else None
    return dx, torch.stack(dw) if many else dw[0], None if bias is None else torch.stack(db) if many else db[0]


def _exact_adamw(s):
    """The 8-bit codes are rounded from 64-bit moments."""
    f, t = s["flat"], s["step"]
    eight = f["avg_scale"] is not None
    w_out = f["param"].double()
    m_out, v_out = f["avg"].double(), f["sq"].double()
    scales = [torch.zeros(0 if not eight else f["avg_scale"].numel(), dtype=torch.float64, device="cuda") for _ in range(2)]
    for position, tensor in enumerate(s["tensors"]):
        param, grad, avg, sq, mantissa, avg_scale, sq_scale = tensor[:7]
        n, at = len(param), param.storage_offset()
        g = grad.double() * (1 if s["grad_scale"] is None else s["grad_scale"].double())
        block = torch.arange(n, device="cuda") // BLOCK
        m, v = avg.double(), sq.double()
        if eight:
            m, v = m * avg_scale.double()[block], (v * sq_scale.double()[block]) ** 2
        m = s["beta1"] * m + (1 - s["beta1"]) * g
        v = s["beta2"] * v + (1 - s["beta2"]) * g ** 2
        w = _weight(tensor).double()
        w = w - s["lr"] * s["wd"] * w - s["lr"] * (m / (1 - s["beta1"] ** t)) / (torch.sqrt(v / (1 - s["beta2"] ** t)) + s["eps"])
        if mantissa is not None:            # the high half of the fp32 number nearest to it
            w = (w.float().view(torch.int32) & -65536).view(torch.float32).double()
        w_out[at:at + n] = w
        if not eight:
            m_out[at:at + n], v_out[at:at + n] = m, v
            continue
        noise = _noise(s, position, n)
        for out, scale, values, bits, root in ((m_out, scales[0], m, noise[0], False), (v_out, scales[1], v.sqrt(), noise[1], True)):
            top = torch.zeros(len(avg_scale), dtype=torch.float64, device="cuda").scatter_reduce(0, block, values.abs(), "amax")
            scale[avg_scale.storage_offset():avg_scale.storage_offset() + len(top)] = top / TOP
            q = values.abs() * TOP / top.clamp(min=1e-300)[block]
            # e4m3: 8 steps to a power of two, down to 2^-6, evenly spaced below
            step = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
            q = (torch.round(q / step) if bits is None else torch.floor(q / step + bits.double() / 65536)) * step
            q = q.clamp(max=TOP)
            if root:
                q = torch.where(values > 0, q.clamp(min=2.0 ** -9), q)
            out[at:at + n] = torch.where(top[block] > 0, q, 0.0) * values.sign()
    # the low halves are the rest of a rounded fp32 number: 64 bits have no value for them
    return (w_out, None, m_out, v_out) + ((scales[0], scales[1]) if eight else (None, None))


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_linear(s) if case["op"] == "linear" else _exact_adamw(s)
