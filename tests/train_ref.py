"""Plain references of the training-step operators: the formulas of include/nvfp4_train.h in numpy,
once in binary32 operation by operation (the AdamW step has one right answer, bit for bit) and
once in binary64."""
from __future__ import annotations

import numpy as np

GOLDEN = 0x9E3779B9
M32 = 0xFFFFFFFF


def bf16_round(x):
    """float32 -> nearest BF16, as float32."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16
    return b.astype(np.uint32).view(np.float32)


def bf16_bits(x):
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def from_bf16_bits(b):
    return (b.astype(np.uint32) << 16).view(np.float32)


def bf16_stochastic(x, word):
    b = ((np.asarray(x, np.float32).view(np.uint32).astype(np.uint64) + (word >> np.uint64(16))) >> np.uint64(16)) << np.uint64(16)
    return b.astype(np.uint32).view(np.float32)


def mix(a):
    a = np.asarray(a, np.uint64)
    a = a ^ (a >> np.uint64(16))
    a = (a * np.uint64(0x85EBCA6B)) & np.uint64(M32)
    a = a ^ (a >> np.uint64(13))
    a = (a * np.uint64(0xC2B2AE35)) & np.uint64(M32)
    return a ^ (a >> np.uint64(16))


def words(n, first, seed, steps):
    """The random word of each of n elements whose first has the index `first`."""
    k = np.arange(first, first + n, dtype=np.uint64)
    key = mix((seed + GOLDEN * steps) & M32)
    return (mix((k >> np.uint64(3)) ^ key) + (k & np.uint64(7)) * np.uint64(GOLDEN)) & np.uint64(M32)


def _e4m3_values():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v[c] = (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) * (-1 if c & 128 else 1)
    v[0x7F], v[0xFF] = np.nan, np.nan
    return v


E4M3 = _e4m3_values()


def e4m3_nearest(x):
    """Codes of finite |x| <= 448, ties to the even code."""
    grid = E4M3[:0x7F]
    a = np.abs(x.astype(np.float64))
    hi = np.searchsorted(grid, a).clip(1, 0x7E)
    lo = hi - 1
    up = (a - grid[lo] > grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 7)


def _blocks(x):
    return np.concatenate([x, np.zeros(-len(x) % 32, np.float32)]).reshape(-1, 32)


def scale_bytes(x):
    bits = np.abs(_blocks(x)).max(1).astype(np.float32).view(np.uint32).astype(np.int64)
    return (np.maximum((bits + 0x1FFFFF) >> 23, 9) - 8).astype(np.uint8)


def power(exponent):
    return (exponent.astype(np.uint32) << 23).view(np.float32)


def spread(per_block, n):
    return np.repeat(per_block, 32)[:n]


def decode(codes, scales):
    return (E4M3[codes].astype(np.float32) * spread(power(scales), len(codes))).astype(np.float32)


def encode_nearest(x):
    s = scale_bytes(x)
    return e4m3_nearest(x * spread(power(254 - s.astype(np.int64)), len(x))), s


def encode_stochastic(u, word):
    s = scale_bytes(u)
    y = (u * spread(power(254 - s.astype(np.int64)), len(u))) * np.float32(2.0 ** -120)
    low = y.astype(np.float32).view(np.uint32).astype(np.uint64)
    code = (low + ((word & np.uint64(0xFFFF)) << np.uint64(4))) >> np.uint64(20)
    return np.maximum(code, (u > 0).astype(np.uint64)).astype(np.uint8), s


def fma(a, b, c):
    """a * b + c rounded once to binary32 (the product is exact in 64 bits of significand, and the
    sum's rounding there changes the result for one in 2^40)."""
    wide = np.longdouble
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        return (np.asarray(a, wide) * np.asarray(b, wide) + np.asarray(c, wide)).astype(np.float32)


def adamw_bits(p, g, m, v, *, param_bf16, master, bits, lr, decay, betas, eps, scale, steps, first, seed):
    """One step in binary32, as the header states it. p: float32 values of the master or parameter; m, v:
    float32 arrays, or (codes, scale bytes) of the first moment and of the second one's root."""
    f = np.float32
    n = len(p)
    lr = f(lr)
    b1, r1, b2, r2 = f(betas[0]), f(1.0 - betas[0]), f(betas[1]), f(1.0 - betas[1])
    rate = lr / f(1.0 - np.float64(betas[0]) ** steps * betas[0])
    root_factor = f(1) / np.sqrt(f(1.0 - np.float64(betas[1]) ** steps * betas[1]))
    keep = f(1.0) - f(decay) * lr
    g = g.astype(f) * f(scale)
    if bits == 8:
        m, root = decode(*m), decode(*v)
        v = root * root
    m = fma(m, b1, g * r1)
    v = fma(v, b2, (g * g) * r2)
    root = np.sqrt(v)
    if bits == 8:
        root = np.where(v < f(2.0 ** -126), f(0), root)
    ratio = m / fma(root, root_factor, f(eps))
    q = fma(ratio, -rate, p * keep)
    assert m.dtype == v.dtype == q.dtype == np.float32
    word = words(n, first, seed, steps)
    out = {"_q": q, "_root": root, "_word": word, "_update": np.abs(ratio * rate)}
    if param_bf16 and master:
        out["master"], out["param"] = q, bf16_round(q)
    elif param_bf16:
        out["param"] = bf16_stochastic(q, word)
    else:
        out["param"] = q
    if bits == 8:
        out["exp_avg"], out["exp_avg_scale"] = encode_nearest(m)
        out["exp_avg_sq"], out["exp_avg_sq_scale"] = encode_stochastic(root, word)
    else:
        out["exp_avg"], out["exp_avg_sq"] = m, v
    return out


def assert_step(got, want, bits, what=""):
    """got: what a step left (param, states, master) as arrays; want: adamw_bits'.

    Beside 32-bit states every bit agrees. Beside 8-bit ones the root and the reciprocal under m are
    approximations of 2^-23 each: m's codes and scales agree, u's are those of a root that much
    larger or smaller, and the parameter those of an update within 2^-21 of itself (both errors, the
    rounded product in place of the rounded quotient, and the halves of the rounding) and one more
    rounding of the sum."""
    if bits == 32:
        for k, w in want.items():
            if k[0] != "_":
                np.testing.assert_array_equal(got[k], w, err_msg=f"{what}: {k}")
        return
    for k in ("exp_avg", "exp_avg_scale"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=f"{what}: {k}")
    f = np.float32
    low, high = (encode_stochastic((want["_root"] * f(1 + e)).astype(f), want["_word"]) for e in (-2.0 ** -22, 2.0 ** -22))
    scale = got["exp_avg_sq_scale"]
    assert ((scale == low[1]) | (scale == high[1])).all(), what
    same = spread(low[1] == high[1], len(low[0]))
    code = got["exp_avg_sq"]
    assert ((code >= low[0]) & (code <= high[0]))[same].all(), what
    assert same.mean() > 0.99 or len(same) < 4000
    q = want["_q"].astype(np.float64)
    slack = 2.0 ** -21 * want["_update"] + 2.0 ** -23 * np.abs(q) + 2.0 ** -148
    if "master" in want:
        assert (np.abs(got["master"] - q) <= slack).all(), what
        np.testing.assert_array_equal(got["param"], bf16_round(got["master"]))
    elif (want["param"] == want["_q"]).all():
        assert (np.abs(got["param"] - q) <= slack).all(), what
    else:
        ends = [bf16_stochastic((q + e * slack).astype(f), want["_word"]) for e in (-1.01, 1.01)]
        assert ((got["param"] >= ends[0]) & (got["param"] <= ends[1])).all(), what


def adamw64(p, g, m, v, *, lr, decay, betas, eps, scale, steps):
    """The step in binary64, from the definition. v is the second moment. Returns p', m', v', and
    the magnitudes that rounding errors go by: |b1 m| + |r1 g|, and the update."""
    t = steps + 1
    g = g.astype(np.float64) * float(scale)
    m1 = betas[0] * m.astype(np.float64) + (1 - betas[0]) * g
    v1 = betas[1] * v.astype(np.float64) + (1 - betas[1]) * g * g
    denominator = np.sqrt(v1 / (1 - betas[1] ** t)) + eps
    rate = lr / (1 - betas[0] ** t)
    update = np.zeros_like(m1)
    np.divide(m1, denominator, out=update, where=denominator > 0)
    p1 = p.astype(np.float64) * (1 - lr * decay) - rate * update
    size_m = np.abs(betas[0] * m) + np.abs((1 - betas[0]) * g)
    return p1, m1, v1, size_m, rate * np.abs(update), rate / np.maximum(denominator, 1e-300)


def norm64(x, w, b, eps):
    x = x.astype(np.float64)
    mean = x.mean(1, keepdims=True)
    var = ((x - mean) ** 2).mean(1, keepdims=True)
    rstd = 1 / np.sqrt(var + eps)
    return (x - mean) * rstd * w + b, mean, rstd, var


def norm_grad64(dy, x, w, mean, rstd):
    dy, x = dy.astype(np.float64), x.astype(np.float64)
    xh = (x - mean[:, None].astype(np.float64)) * rstd[:, None].astype(np.float64)
    h = dy * w
    s1, s2 = h.mean(1, keepdims=True), (h * xh).mean(1, keepdims=True)
    return rstd[:, None] * (h - s1 - xh * s2), (dy * xh).sum(0), dy.sum(0), xh, h
