"""The operators between a block's matrix products, as a training step calls them.

Three operators, each in its two directions:

  layer_norm  the norm before a bank's matrix product; backward returns dx and the reduced
              gradients of the weight and the bias
  rotary      positions with one axis (text) or several (height, width; time, height, width)
              on q and k
  router      top-k selection over a bank of experts, per-expert counts and the balance loss;
              backward returns the gradient of the logits

A case is one call.  run() computes it in elementary torch operations in 32 bits, or, where
`own` is true, through this package.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def _norm(name, direction, rows, cols, dtype, wtype, pad=0):
    return {"name": name, "op": "layer_norm", "direction": direction, "rows": rows, "cols": cols, "dtype": dtype,
            "wtype": wtype, "pad": pad}


def _rotary(name, direction, batch, tokens, heads, kv_heads, dim, sections, dtype, layout, interleaved=False, grid=0):
    return {"name": name, "op": "rotary", "direction": direction, "batch": batch, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "sections": sections, "dtype": dtype, "layout": layout,
            "interleaved": interleaved, "grid": grid}


def _router(name, direction, tokens, experts, top_k, dtype, normalize=False, padded=False, masked=False):
    return {"name": name, "op": "router", "direction": direction, "tokens": tokens, "experts": experts, "top_k": top_k,
            "dtype": dtype, "normalize": normalize, "padded": padded, "masked": masked}


def listed():
    return [
        # one short prompt through a width-768 block: the call's latency
        _norm("norm fwd 64x768 bf16", "forward", 64, 768, "bf16", "f32"),
        # a micro-batch of 48 sequences of 1024 tokens at width 1024
        _norm("norm fwd 49152x1024 bf16", "forward", 49152, 1024, "bf16", "bf16"),
        # a width that no vector divides, in fp32 (a head's input with appended features)
        _norm("norm bwd 5003x1001 f32", "backward", 5003, 1001, "f32", "f32"),
        # the largest micro-batch of the width-768 model: 128 sequences of 1024 tokens
        _norm("norm bwd 131072x768 bf16", "backward", 131072, 768, "bf16", "f32"),
        # an image of 14x14 patches, q and k sliced out of one fused projection
        _rotary("rotary fwd 196 image bf16", "forward", 1, 196, 12, 12, 64, "16,16", "bf16", "qkv", grid=14),
        # text: 64 sequences of 1024 tokens, 12 heads of 64
        _rotary("rotary fwd 64x1024 text bf16", "forward", 64, 1024, 12, 12, 64, "32", "bf16", "qkv"),
        # odd head width and pair counts, shared k heads, adjacent pairs, fp32 (a small vision tower)
        _rotary("rotary bwd 3x785 f32", "backward", 3, 785, 6, 2, 77, "17,18", "f32", "bshd", True, 28),
        # video: 4 clips of 16 frames of 28x28 patches; dq, dk come head-major from attention
        _rotary("rotary bwd 4x12544 video bf16", "backward", 4, 12544, 16, 4, 128, "16,24,24", "bf16", "bhsd", grid=28),
        # a decode-sized batch over 8 experts: the call's latency
        _router("router fwd 32x8 f32", "forward", 32, 8, 2, "f32"),
        # a large micro-batch over 256 experts, 8 of them per token
        _router("router fwd 131072x256 f32", "forward", 131072, 256, 8, "f32", normalize=True),
        # an odd number of experts in bf16, padded sequences and experts that are closed for some tokens
        _router("router bwd 10007x60 bf16", "backward", 10007, 60, 4, "bf16", padded=True, masked=True),
        # the largest: 256 Ki tokens over 256 experts
        _router("router bwd 262144x256 f32", "backward", 262144, 256, 8, "f32", normalize=True),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["layer_norm", "rotary", "router"])
    direction = rng.choice(["forward", "backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
    if op == "layer_norm":
        cols = _log(rng, 48, 8192)
        if rng.random() < 0.7:              # most widths are multiples of 8
            cols = max(8, cols // 8 * 8)
        rows = _log(rng, 1, min(131072, (1 << 26) // cols))
        c = _norm("", direction, rows, cols, dtype, rng.choice(["f32", dtype]), rng.choice([0, 0, 0, 8, 3]))
    elif op == "rotary":
        axes = rng.choice([1, 1, 2, 3])
        interleaved = rng.random() < 0.3
        pairs = rng.choice([16, 24, 32, 32, 48, 64, 64, rng.randint(axes, 64)])
        cut = sorted(rng.sample(range(1, pairs), axes - 1)) if axes > 1 else []
        sections = ",".join(str(b - a) for a, b in zip([0] + cut, cut + [pairs]))
        dim = 2 * pairs + rng.choice([0, 0, 0, 16, rng.randint(1, 20)])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 1, 2, 4])
        batch = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, min(32768, (1 << 26) // (batch * (heads + kv_heads) * dim))))
        c = _rotary("", direction, batch, tokens, heads, kv_heads, dim, sections, dtype,
                    rng.choice(["qkv", "bshd", "bhsd"]), interleaved, max(1, int(math.isqrt(tokens))) if axes > 1 else 0)
    else:
        experts = _log(rng, 4, 512)
        if rng.random() < 0.6:              # most models have a power of two of them
            experts = 1 << int(round(math.log2(experts)))
        tokens = _log(rng, 1, min(262144, (1 << 25) // experts))
        c = _router("", direction, tokens, experts, rng.randint(1, min(8, experts)), rng.choice(["f32", dtype]),
                    rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.3)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    state = {"case": case}
    dtype = _TYPES[case["dtype"]]
    if case["op"] == "layer_norm":
        rows, cols, ld = case["rows"], case["cols"], case["cols"] + case["pad"]
        # a residual stream: rows of different size with an offset, channels of different size
        x = normal(rows, ld) * torch.exp(0.5 * normal(1, ld)) * torch.exp(0.3 * normal(rows, 1)) + 0.2 * normal(rows, 1)
        state["x"] = x.to(dtype)[:, :cols]
        wtype = _TYPES[case["wtype"]]
        state["weight"] = (1 + 0.2 * normal(cols)).to(wtype)
        state["bias"] = (0.1 * normal(cols)).to(wtype)
        state["eps"] = 1e-5
        if case["direction"] == "backward":
            state["dy"] = (normal(rows, cols) * 0.02).to(dtype)
            xf = state["x"].float()
            state["mean"] = xf.mean(1)
            state["rstd"] = torch.rsqrt(xf.var(1, unbiased=False) + state["eps"])
    elif case["op"] == "rotary":
        b, t, h, hk, d = (case[n] for n in ("batch", "tokens", "heads", "kv_heads", "dim"))
        sections = _sections(case)
        if case["layout"] == "qkv":         # slices of the fused projection [batch, tokens, q + k + v heads, dim]
            qkv = normal(b, t, h + 2 * hk, d).to(dtype)
            state["q"], state["k"] = qkv[:, :, :h], qkv[:, :, h:h + hk]
        elif case["layout"] == "bshd":
            state["q"], state["k"] = normal(b, t, h, d).to(dtype), normal(b, t, hk, d).to(dtype)
        else:                               # head-major storage, as attention keeps it
            state["q"] = normal(b, h, t, d).to(dtype).transpose(1, 2)
            state["k"] = normal(b, hk, t, d).to(dtype).transpose(1, 2)
        first = torch.randint(0, 64, (1, b, 1), generator=g, device="cuda")     # each sequence starts somewhere
        at = torch.arange(t, device="cuda").expand(1, b, t)
        if len(sections) == 1:
            positions = at + first
        else:                               # (time,) height, width of patch number `at` in a grid
            w = case["grid"]
            axes = [at // (w * w) + first, at // w % w, at % w][-len(sections):]
            positions = torch.cat(axes) if len(sections) == 3 else torch.cat([axes[0] + first, axes[1]])
        state["positions"] = positions.to(torch.int32).contiguous()
        # every axis has its own geometric series of frequencies, base 10000
        state["inv_freq"] = torch.cat([10000.0 ** (-torch.arange(n, dtype=torch.float64) / n) for n in sections]).float().cuda()
        state["sections"] = sections
        state["axis"] = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).cuda()
    else:
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        # unbalanced experts, as early in training
        logits = (normal(t, e) + 0.7 * normal(1, e)).to(dtype)
        if case["masked"]:                  # experts closed for some tokens; now and then a token has none left
            closed = torch.rand((t, e), generator=g, device="cuda") < 0.15
            closed |= torch.rand((t, 1), generator=g, device="cuda") < 0.01
            logits = logits.masked_fill(closed, float("-inf"))
        state["logits"] = logits
        state["valid"] = torch.rand(t, generator=g, device="cuda") < 0.9 if case["padded"] else None
        if case["direction"] == "backward":
            index, gate, counts, _, used = _router_plain(state)
            state.update(index=index, gate=gate, counts=counts, used=used)
            # the loss is summed over tokens, so that fp16 gradients stay in range
            state["dloss"] = torch.full((1,), 0.01 * t, device="cuda")
            state["dgate"] = 0.01 * normal(t, k)
    return state


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    xf = s["x"].float()
    mean = xf.mean(1, keepdim=True)
    d = xf - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + s["eps"])
    y = d * rstd * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _norm_backward_plain(s):
    xf, dyf, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = (xf - s["mean"][:, None]) * rstd
    g = dyf * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    wtype = s["weight"].dtype
    return dx.to(s["x"].dtype), (dyf * xhat).sum(0).to(wtype), dyf.sum(0).to(wtype)


def _rotate(x, cos, sin, interleaved):
    pairs = cos.shape[-1]
    xf = x.float()
    u, v = (xf[..., 0:2 * pairs:2], xf[..., 1:2 * pairs:2]) if interleaved else (xf[..., :pairs], xf[..., pairs:2 * pairs])
    a, b = u * cos - v * sin, v * cos + u * sin
    turned = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((turned, xf[..., 2 * pairs:]), -1).to(x.dtype)


def _rotary_plain(s):
    angle = s["positions"].float()[s["axis"]].permute(1, 2, 0) * s["inv_freq"]      # [batch, tokens, pairs]
    cos, sin = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
    if s["case"]["direction"] == "backward":
        sin = -sin
    return _rotate(s["q"], cos, sin, s["case"]["interleaved"]), _rotate(s["k"], cos, sin, s["case"]["interleaved"])


def _probabilities(s):
    """The softmax in 32 bits, and which tokens count; the rows of the others are zero."""
    lf = s["logits"].float()
    top = lf.amax(1, keepdim=True)
    used = top[:, 0] > float("-inf")
    if s["valid"] is not None:
        used = used & s["valid"]
    p = torch.exp(lf - top)
    p = p / p.sum(1, keepdim=True)
    return torch.where(used[:, None], p, 0.0), used


def _router_plain(s):
    k, e = s["case"]["top_k"], s["case"]["experts"]
    p, used = _probabilities(s)
    top, index = torch.sort(s["logits"], dim=1, descending=True, stable=True)       # ties: the lowest index first
    top, index = top[:, :k], index[:, :k]
    chosen = (top > float("-inf")) & used[:, None]
    gate = torch.where(chosen, p.gather(1, index), 0.0)
    if s["case"]["normalize"]:
        gate = gate / torch.where(used, gate.sum(1), 1.0)[:, None]
    counts = torch.zeros(e, dtype=torch.int32, device=p.device)
    counts = counts.index_add(0, index.reshape(-1), chosen.reshape(-1).to(torch.int32))
    n = used.sum()
    loss = (counts.float() * p.sum(0)).sum() * e / (k * n.clamp(min=1).float() ** 2)
    return torch.where(chosen, index, -1).to(torch.int32), gate, counts, loss.reshape(1), n.to(torch.int32).reshape(1)


def _router_backward_plain(s):
    k, e = s["case"]["top_k"], s["case"]["experts"]
    p, _ = _probabilities(s)
    c = s["dloss"] * s["counts"].float() * e / (k * s["used"].clamp(min=1).float() ** 2)
    chosen = s["index"] >= 0
    dgate = torch.where(chosen, s["dgate"], 0.0)
    at = s["index"].clamp(min=0).long()
    if s["case"]["normalize"]:
        own_part = s["gate"] * (dgate - (s["gate"] * dgate).sum(1, keepdim=True))
        dl = p * (c - (p * c).sum(1, keepdim=True))
        dl = dl.scatter_add(1, at, own_part)
    else:
        a = c.expand_as(p).scatter_add(1, at, dgate)
        dl = p * (a - (p * a).sum(1, keepdim=True))
    return dl.to(s["logits"].dtype)


# ---------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    forward = case["direction"] == "forward"
    if not own:
        if case["op"] == "layer_norm":
            return _norm_plain(s) if forward else _norm_backward_plain(s)
        if case["op"] == "rotary":
            return _rotary_plain(s)
        return _router_plain(s) if forward else _router_backward_plain(s)
    import newton_schulz_stacked_gb300 as nss
    if case["op"] == "layer_norm":
        if forward:
            return nss.mb_layer_norm(s["x"], s["weight"], s["bias"], s["eps"])
        return nss.mb_layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if case["op"] == "rotary":
        call = nss.mb_rotary if forward else nss.mb_rotary_backward
        return call(s["q"], s["k"], s["positions"], s["inv_freq"], s["sections"], case["interleaved"])
    if forward:
        return nss.mb_router(s["logits"], case["top_k"], s["valid"], case["normalize"])
    return nss.mb_router_backward(s["dloss"], s["dgate"], s["logits"], s["index"], s["gate"], s["counts"], s["used"],
                                  s["valid"], case["normalize"])


def work(case):
    size = _SIZE[case["dtype"]]
    forward = case["direction"] == "forward"
    if case["op"] == "layer_norm":
        n, per_col = case["rows"] * case["cols"], 2 * _SIZE[case["wtype"]]
        if forward:
            return {"bytes": 2 * size * n + 8 * case["rows"] + per_col * case["cols"], "flops": 8 * n}
        return {"bytes": 3 * size * n + 8 * case["rows"] + 1.5 * per_col * case["cols"], "flops": 14 * n}
    if case["op"] == "rotary":
        at = case["batch"] * case["tokens"]
        n = at * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 2 * size * n + 4 * at * len(_sections(case)), "flops": 3 * n}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    valid = t if case["padded"] else 0
    if forward:
        return {"bytes": size * t * e + 8 * t * k + valid + 4 * e, "flops": (5 + k) * t * e}
    return {"bytes": 2 * size * t * e + 12 * t * k + valid + 4 * e, "flops": 9 * t * e}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_norm(s, forward):
    x = s["x"].double()
    n = x.shape[1]
    if forward:
        m = x.sum(1) / n
        r = 1 / torch.sqrt(((x - m[:, None]) ** 2).sum(1) / n + s["eps"])
        return torch.addcmul(s["bias"].double(), (x - m[:, None]) * r[:, None], s["weight"].double()), m, r
    m, r, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
    h = torch.einsum("ij,i->ij", x - m[:, None], r)
    # d sum(dy * y) / dx through the mean and the deviation
    dh = dy * s["weight"].double()
    dx = torch.einsum("ij,i->ij", dh - torch.einsum("ij->i", dh)[:, None] / n - h * (torch.einsum("ij,ij->i", dh, h) / n)[:, None], r)
    return dx, torch.einsum("ij,ij->j", dy, h), torch.einsum("ij->j", dy)


def _exact_rotary(s, forward):
    case, out = s["case"], []
    sign = 1.0 if forward else -1.0
    pairs = s["inv_freq"].numel()
    i = torch.arange(pairs, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
    pos = s["positions"].double()
    angle = torch.stack([pos[a] * f for a, f in zip(s["axis"].tolist(), s["inv_freq"].double())], -1).unsqueeze(2) * sign
    turn = torch.polar(torch.ones_like(angle), angle)
    for x in (s["q"], s["k"]):
        y = x.double().clone(memory_format=torch.contiguous_format)
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_router(s, forward):
    case = s["case"]
    l, k, e = s["logits"].double(), case["top_k"], case["experts"]
    some = (l != float("-inf")).any(1)
    if s["valid"] is not None:
        some &= s["valid"]
    p = torch.zeros_like(l)
    p[some] = torch.softmax(l[some], 1)
    n = max(int(some.sum()), 1)
    if not forward:
        c = s["dloss"].double() * e * s["counts"].double() / k / n / n
        dp = c.repeat(len(l), 1)
        rows, slots = torch.nonzero(s["index"] >= 0, as_tuple=True)
        at = s["index"][rows, slots].long()
        if case["normalize"]:
            w, dw = s["gate"].double(), torch.where(s["index"] >= 0, s["dgate"], 0.0).double()
            dl = p * (dp - torch.einsum("te,te->t", p, dp)[:, None])
            dl.index_put_((rows, at), (w * (dw - torch.einsum("tk,tk->t", w, dw)[:, None]))[rows, slots], accumulate=True)
            return dl
        dp.index_put_((rows, at), s["dgate"].double()[rows, slots], accumulate=True)
        return p * (dp - torch.einsum("te,te->t", p, dp)[:, None])
    left, index, gate = l.clone(), [], []
    for _ in range(k):
        best = left.amax(1)
        j = (left == best[:, None]).int().argmax(1)                 # the first of equals
        ok = some & (best > float("-inf"))
        index.append(torch.where(ok, j, -1))
        gate.append(torch.where(ok, p.gather(1, j[:, None])[:, 0], 0.0))
        left.scatter_(1, j[:, None], float("-inf"))
    index, gate = torch.stack(index, 1), torch.stack(gate, 1)
    if case["normalize"]:
        gate = gate / torch.where(some, gate.sum(1), 1.0)[:, None]
    counts = torch.bincount(index[index >= 0].reshape(-1), minlength=e)
    loss = e * torch.dot(counts.double(), p.sum(0)) / k / n / n
    return index.int(), gate, counts.int(), loss.reshape(1), torch.tensor([int(some.sum())], dtype=torch.int32)


def exact(case, seed):
    s = prepare(case, seed)
    forward = case["direction"] == "forward"
    return {"layer_norm": _exact_norm, "rotary": _exact_rotary, "router": _exact_router}[case["op"]](s, forward)
