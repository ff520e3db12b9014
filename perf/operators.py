"""The operators of a quantization-aware-distillation training step, as they are measured.

Layer norm forward and backward, the global gradient norm with its clip factor, and an AdamW step
over a list of tensors with its states in 32 bits or in 8. ``run`` computes them in elementary
torch operations where ``own`` is false and calls the library where it is true.

The tensors of a list lie in flat buffers, each from a multiple of 128 elements on, as a trainer
that keeps its parameters and gradients contiguous has them; what lies between two tensors is zero
and stays zero.
"""
import math

import torch

own = False

_M32 = 0xFFFFFFFF
_GOLDEN = 0x9E3779B9
_BETA1, _BETA2, _EPS, _LR, _DECAY = 0.9, 0.95, 1e-8, 2e-4, 0.1
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # decoding one token: a single row, where the call's own latency is what counts
        {"name": "norm, one token", "op": "norm", "rows": 1, "cols": 4096, "x": "bf16", "w": "bf16", "amax": True, "stats": False},
        # the activations of a large batch in front of a quantized projection, which wants their amax
        {"name": "norm, 8192x4096 with amax", "op": "norm", "rows": 8192, "cols": 4096, "x": "bf16", "w": "bf16", "amax": True, "stats": False},
        # an odd width in FP32, with the statistics that a backward pass needs
        {"name": "norm, 1237x1003 f32", "op": "norm", "rows": 1237, "cols": 1003, "x": "f32", "w": "f32", "amax": False, "stats": True},
        # the gradient of the same large batch
        {"name": "norm gradient, 8192x4096", "op": "norm_grad", "rows": 8192, "cols": 4096, "x": "bf16", "w": "bf16"},
        # a short sequence of a small model in FP32
        {"name": "norm gradient, 256x1024 f32", "op": "norm_grad", "rows": 256, "cols": 1024, "x": "f32", "w": "f32"},
        # an odd row length: rows begin at every alignment; BF16 activations under FP32 weights
        {"name": "norm gradient, 2049x5001", "op": "norm_grad", "rows": 2049, "cols": 5001, "x": "bf16", "w": "f32"},
        # clipping the gradients of a small model: many short tensors of odd lengths
        {"name": "gradient norm, small", "op": "grad_norm", "layers": 4, "hidden": 331, "ffn": 1001, "grad": "bf16"},
        # clipping the gradients of a large one
        {"name": "gradient norm, large", "op": "grad_norm", "layers": 4, "hidden": 4096, "ffn": 8192, "grad": "bf16"},
        # the step of a large student with FP32 masters, clipped: what a distillation run does
        {"name": "adamw 32, masters, clipped", "op": "adamw", "layers": 4, "hidden": 2048, "ffn": 8192, "param": "bf16", "master": True,
         "grad": "bf16", "bits": 32, "clip": True, "amax": True, "step": 1000},
        # the step of a tiny model in FP32: latency
        {"name": "adamw 32, f32, tiny", "op": "adamw", "layers": 2, "hidden": 64, "ffn": 256, "param": "f32", "master": False,
         "grad": "f32", "bits": 32, "clip": False, "amax": False, "step": 1},
        # a large student whose states are in 8 bits and whose BF16 weights have no master
        {"name": "adamw 8, large", "op": "adamw", "layers": 2, "hidden": 4096, "ffn": 8192, "param": "bf16", "master": False,
         "grad": "bf16", "bits": 8, "clip": False, "amax": True, "step": 1000},
        # odd lengths: blocks of 32 and vectors of 8 end inside every tensor
        {"name": "adamw 8, odd lengths", "op": "adamw", "layers": 6, "hidden": 577, "ffn": 1155, "param": "bf16", "master": False,
         "grad": "f32", "bits": 8, "clip": True, "amax": False, "step": 17},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if n >= 64 and rng.random() < 0.5:
        n -= n % 16  # as widths mostly are; the others stay odd
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "grad_norm", "adamw", "adamw", "adamw"])
    if op in ("norm", "norm_grad"):
        cols = _log_int(rng, 8, 8192)
        rows = _log_int(rng, 1, min(32768, (1 << 25) // cols))
        x = rng.choice(["bf16", "bf16", "f32"])
        case = {"op": op, "rows": rows, "cols": cols, "x": x, "w": rng.choice([x, "f32"])}
        if op == "norm":
            case["amax"], case["stats"] = rng.random() < 0.5, rng.random() < 0.5
        return case
    hidden = _log_int(rng, 16, 2048)
    ffn = _log_int(rng, hidden, 4 * hidden)
    layers = max(1, min(rng.randint(1, 12), 150_000_000 // (2 * hidden * (hidden + ffn))))
    case = {"op": op, "layers": layers, "hidden": hidden, "ffn": ffn, "grad": rng.choice(["bf16", "f32"])}
    if op == "adamw":
        param = rng.choice(["bf16", "bf16", "f32"])
        case.update(param=param, master=param == "bf16" and rng.random() < 0.5, bits=rng.choice([8, 32]), clip=rng.random() < 0.5,
                    amax=rng.random() < 0.5, step=rng.randint(1, 20000))
    return case


# ---- the tensors of a list ----------------------------------------------------------------

def _numels(case):
    """(number of elements, is a matrix) of each tensor: two norms, two square and two wide matrices, a bias a layer."""
    h, f = case["hidden"], case["ffn"]
    return [(h, False), (h * h, True), (h * h, True), (h, False), (h * f, True), (f, False), (f * h, True)] * case["layers"]


def _layout(case):
    """[(offset, number of elements, is a matrix)] and the length of the flat buffers."""
    at, places = 0, []
    for n, matrix in _numels(case):
        places.append((at, n, matrix))
        at += (n + 127) // 128 * 128
    return places, at


def _views(flat, places):
    return [flat[at:at + n] for at, n, _ in places]


def _spread(values, places, total, dtype=torch.float32):
    """A flat buffer that holds values[i] over tensor i and zero between the tensors."""
    out = torch.zeros(total, dtype=dtype, device="cuda")
    for view, value in zip(_views(out, places), values):
        view.fill_(value)
    return out


# ---- inputs -----------------------------------------------------------------------------------

def _prepare_norm(case, gen):
    rows, cols, xt, wt = case["rows"], case["cols"], _TYPES[case["x"]], _TYPES[case["w"]]
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    # activations: a scale of each channel's own with a long tail (a few channels far above the rest), and an offset
    channel = torch.exp(rand(cols))
    state = {"case": case, "eps": 1e-5}
    state["x"] = (rand(rows, cols) * channel + 0.3 * rand(cols)).to(xt)
    state["weight"] = (1 + 0.2 * rand(cols)).to(wt)
    state["bias"] = (0.1 * rand(cols)).to(wt)
    if case["op"] == "norm_grad":
        state["dy"] = (rand(rows, cols) * 1e-3).to(xt)
        x = state["x"].double()  # the statistics that the forward pass left behind
        mean = x.mean(-1)
        var = (x - mean[:, None]).square_().mean(-1)
        state["mean"], state["rstd"] = mean.float(), (var + state["eps"]).rsqrt().float()
    return state


def _prepare_list(case, gen):
    places, total = _layout(case)
    inside = _spread([1.0] * len(places), places, total)
    rand = lambda: torch.randn(total, device="cuda", generator=gen)  # noqa: E731
    # gradients: each tensor at a scale of its own
    scales = torch.exp(1.5 * torch.randn(len(places), device="cuda", generator=gen)).mul_(1e-3).tolist()
    size = _spread(scales, places, total)
    grads = (rand() * size).to(_TYPES[case["grad"]])
    state = {"case": case, "places": places, "total": total, "grads": grads, "max_norm": 1.0}
    if case["op"] == "grad_norm":
        if own:
            import nvfp4_block_scaled_13_b200 as nv
            state["list"] = nv.gradient_list(_views(grads, places))
        return state
    weights = rand().mul_(0.02).mul_(inside)
    state["param"] = weights.to(_TYPES[case["param"]])
    if case["master"]:
        state["master"] = weights
    exp_avg = rand().mul_(size).mul_(0.3)
    root = (rand().abs_().mul_(0.2).add_(0.9)).mul_(size)  # the root of the second moment
    if case["bits"] == 8:
        state["exp_avg"], state["exp_avg_scale"] = _encode_nearest(exp_avg)
        state["exp_avg_sq"], state["exp_avg_sq_scale"] = _encode_nearest(root)
    else:
        state["exp_avg"], state["exp_avg_sq"] = exp_avg, root.square_()
    state["seed"] = case["step"] * 7 + 1
    state["decays"] = [_DECAY if matrix else 0.0 for _, _, matrix in places]
    state["step"] = case["step"] - 1  # steps taken so far
    if own:
        import nvfp4_block_scaled_13_b200 as nv
        plan = nv.adamw_plan(_views(state["param"], places), _views(grads, places), state_bits=case["bits"], masters=case["master"],
                             weight_decay=state["decays"], betas=(_BETA1, _BETA2), eps=_EPS, seed=state["seed"], step=state["step"],
                             with_amax=case["amax"])
        for name in ("master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            if name in state:
                getattr(plan, name).copy_(state[name])
                state[name] = getattr(plan, name)
        state["plan"] = plan
    else:
        state["decay"] = _spread(state["decays"], places, total)
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return _prepare_norm(case, gen) if case["op"] in ("norm", "norm_grad") else _prepare_list(case, gen)


# ---- plain forms --------------------------------------------------------------------------------

def _plain_norm(s):
    case, x = s["case"], s["x"].float()
    mean = x.mean(-1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(-1, keepdim=True) + s["eps"])
    out = {"y": (d * rstd * s["weight"].float() + s["bias"].float()).to(s["x"].dtype)}
    if case["stats"]:
        out["mean"], out["rstd"] = mean.reshape(-1), rstd.reshape(-1)
    if case["amax"]:
        out["amax"] = out["y"].abs().max().float().reshape(1)
    return out


def _plain_norm_grad(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    h = dy * w
    dx = (h - h.mean(-1, keepdim=True) - xh * (h * xh).mean(-1, keepdim=True)) * rstd
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0).to(s["weight"].dtype), "dbias": dy.sum(0).to(s["bias"].dtype)}


def _plain_clip(s):
    norm = torch.sqrt(s["grads"].double().square().sum())  # a long sum
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return norm.float().reshape(1), scale.float().reshape(1)


def _mix(x):
    """A bijection of 32-bit words: multiplications and shifted exclusive ors."""
    x = x ^ (x >> 16)
    x = (x * 0x85EBCA6B) & _M32
    x = x ^ (x >> 13)
    x = (x * 0xC2B2AE35) & _M32
    return x ^ (x >> 16)


def _random_words(total, seed, step):
    """A 32-bit word for each element: a hashed start for each eight, and equal steps of 2^32 / golden ratio from it."""
    key = _mix((seed + _GOLDEN * step) & _M32)
    start = _mix(torch.arange(total // 8, device="cuda") ^ key)
    return ((start[:, None] + torch.arange(8, device="cuda") * _GOLDEN) & _M32).reshape(-1)


def _power(exponent):
    """2 ** (exponent - 127) of an int32 tensor, exactly."""
    return (exponent << 23).view(torch.float32)


def _scale_bytes(x):
    """The exponent byte of each block of 32: the power of two that brings its largest magnitude into (224, 448]."""
    bits = x.view(-1, 32).abs().amax(1).view(torch.int32)
    return ((bits + 0x1FFFFF) >> 23).clamp(min=9) - 8


def _encode_nearest(x):
    s = _scale_bytes(x)
    codes = (x.view(-1, 32) * _power(254 - s)[:, None]).to(torch.float8_e4m3fn).reshape(-1)
    return codes, s.to(torch.uint8).view(torch.float8_e8m0fnu)


def _encode_stochastic(x, words):
    """Non-negative x: the random low bits are added below the three kept bits of the significand; positive x keeps a positive code."""
    s = _scale_bytes(x)
    low = (x.view(-1, 32) * _power(254 - s)[:, None] * 2.0 ** -120).reshape(-1).view(torch.int32).to(torch.int64)
    codes = (low + ((words & 0xFFFF) << 4)) >> 20
    codes = torch.where(x > 0, codes.clamp(min=1), codes)
    return codes.to(torch.uint8).view(torch.float8_e4m3fn), s.to(torch.uint8).view(torch.float8_e8m0fnu)


def _decode(codes, scales):
    return (codes.float().view(-1, 32) * scales.float()[:, None]).reshape(-1)


def _plain_adamw(s):
    case, out = s["case"], {}
    grad = s["grads"].float()
    if case["clip"]:
        out["norm"], scale = _plain_clip(s)
        grad = grad * scale
    eight = case["bits"] == 8
    exp_avg, exp_avg_sq = s["exp_avg"], s["exp_avg_sq"]
    if eight:
        exp_avg = _decode(exp_avg, s["exp_avg_scale"])
        root = _decode(exp_avg_sq, s["exp_avg_sq_scale"])
        exp_avg_sq = root * root
    exp_avg = exp_avg * _BETA1 + grad * (1 - _BETA1)
    exp_avg_sq = exp_avg_sq * _BETA2 + (grad * grad) * (1 - _BETA2)
    root = torch.sqrt(exp_avg_sq)
    step = s["step"] + 1
    denominator = root * (1 / math.sqrt(1 - _BETA2 ** step)) + _EPS
    weights = s["master"] if case["master"] else s["param"].float()
    weights = weights * (1 - s["decay"] * _LR) - (exp_avg / denominator) * (_LR / (1 - _BETA1 ** step))
    words = _random_words(s["total"], s["seed"], s["step"])
    if case["master"]:
        s["master"].copy_(weights)
        s["param"].copy_(weights)
    elif case["param"] == "bf16":
        bits = weights.view(torch.int32).to(torch.int64) & _M32
        s["param"].copy_(((bits + (words >> 16)) >> 16).to(torch.int16).view(torch.bfloat16))
    else:
        s["param"].copy_(weights)
    if eight:
        for name, (codes, scales) in (("exp_avg", _encode_nearest(exp_avg)), ("exp_avg_sq", _encode_stochastic(root, words))):
            s[name].copy_(codes)
            s[name + "_scale"].copy_(scales)
    else:
        s["exp_avg"].copy_(exp_avg)
        s["exp_avg_sq"].copy_(exp_avg_sq)
    s["step"] = step
    if case["amax"]:
        out["amax"] = torch.stack([v.abs().max() for v in _views(s["param"], s["places"])]).float()
    return out


# ---- the passes -----------------------------------------------------------------------------------

def _own(s):
    import nvfp4_block_scaled_13_b200 as nv

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        r = nv.layer_norm_forward(s["x"], s["weight"], s["bias"], s["eps"], with_stats=case["stats"], with_amax=case["amax"])
        out = {"y": r.y}
        if case["stats"]:
            out["mean"], out["rstd"] = r.mean, r.rstd
        if case["amax"]:
            out["amax"] = r.amax
        return out
    if op == "norm_grad":
        dx, dweight, dbias = nv.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "grad_norm":
        norm, scale = nv.grad_norm(s["list"], s["max_norm"])
        return {"norm": norm, "scale": scale}
    out, scale = {}, None
    if case["clip"]:
        out["norm"], scale = nv.grad_norm(s["plan"], s["max_norm"])
    nv.adamw(s["plan"], _LR, scale)
    if case["amax"]:
        out["amax"] = s["plan"].amax
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        out = _own(state)
    elif op == "norm":
        out = _plain_norm(state)
    elif op == "norm_grad":
        out = _plain_norm_grad(state)
    elif op == "grad_norm":
        norm, scale = _plain_clip(state)
        out = {"norm": norm, "scale": scale}
    else:
        out = _plain_adamw(state)
    if op == "adamw":
        for name in ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            if name in state:
                out[name] = state[name]
    return out


def work(case):
    size = lambda t: 2 if t == "bf16" else 4  # noqa: E731
    if case["op"] in ("norm", "norm_grad"):
        n, w, r = case["rows"] * case["cols"], case["cols"] * size(case["w"]), case["rows"]
        if case["op"] == "norm":
            return {"bytes": 2 * n * size(case["x"]) + 2 * w + (8 * r if case["stats"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * size(case["x"]) + 3 * w + 8 * r, "flops": 14 * n}
    n = sum(k for k, _ in _numels(case))
    if case["op"] == "grad_norm":
        return {"bytes": n * size(case["grad"]), "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 + 4 / 32
    param = 8 + size(case["param"]) if case["master"] else 2 * size(case["param"])
    return {"bytes": n * (param + size(case["grad"]) + state), "flops": (16 + 2 * case["clip"]) * n}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _exact_blocks(x):
    """(value / 2^e, 2^e) of each block of 32, not rounded: 2^e is the smallest power that leaves no magnitude over 448."""
    top = x.view(-1, 32).abs().amax(1)
    e = torch.ceil(torch.log2(top / 448)).clamp(min=-126)  # log2(0) is -inf
    scale = torch.pow(torch.full_like(e, 2.0), e)
    return (x.view(-1, 32) / scale[:, None]).reshape(-1), scale


def exact(case, seed):
    global own
    was, own = own, False  # the inputs alone, without a plan
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] in ("norm", "norm_grad"):
        x, w = s["x"].double(), s["weight"].double()
        if case["op"] == "norm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = torch.rsqrt(var + s["eps"])
            y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w)
            out = {"y": y}
            if case["stats"]:
                out["mean"], out["rstd"] = mean, rstd
            if case["amax"]:  # of the stored values
                out["amax"] = y.to(s["x"].dtype).double().abs().amax().reshape(1)
            return out
        dy, r = s["dy"].double(), s["rstd"].double()
        xh = (x - s["mean"].double()[:, None]) * r[:, None]
        h = dy * w
        inner = torch.einsum("rc,rc->r", h, xh) / x.shape[1]
        dx = r[:, None] * (h - (h.sum(1) / x.shape[1])[:, None] - xh * inner[:, None])
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xh), "dbias": dy.sum(0)}
    out, g = {}, s["grads"].double()
    if case["op"] == "grad_norm" or case["clip"]:
        norm = torch.linalg.vector_norm(g)
        scale = torch.minimum(torch.ones_like(norm), s["max_norm"] / (norm + 1e-6))
        out["norm"] = norm.reshape(1)
        if case["op"] == "grad_norm":
            return {**out, "scale": scale.reshape(1)}
        g.mul_(scale)
    m, v = s["exp_avg"].double(), s["exp_avg_sq"].double()
    if case["bits"] == 8:
        m = m * torch.repeat_interleave(s["exp_avg_scale"].double(), 32)
        v = (v * torch.repeat_interleave(s["exp_avg_sq_scale"].double(), 32)).square_()
    m = torch.lerp(g, m, _BETA1)
    v = torch.lerp(g.square(), v, _BETA2)
    t = case["step"]
    update = (m / (1 - _BETA1 ** t)) / ((v / (1 - _BETA2 ** t)).sqrt() + _EPS)
    p = (s["master"] if case["master"] else s["param"]).double()
    p = p - _LR * (update + s["decay"].double() * p)
    out["param"] = p
    if case["master"]:
        out["master"] = p
    if case["bits"] == 8:
        out["exp_avg"], out["exp_avg_scale"] = _exact_blocks(m)
        out["exp_avg_sq"], out["exp_avg_sq_scale"] = _exact_blocks(v.sqrt())
    else:
        out["exp_avg"], out["exp_avg_sq"] = m, v
    if case["amax"]:
        out["amax"] = None  # of values that were rounded by chance
    return out
