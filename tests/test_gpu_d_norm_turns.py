"""Layer norm over rows that a group of threads takes in many turns, every row compared with binary64 on
the device, within the bounds that test_gpu_a_layer_norm.py derives.

An SM holds at most 2048 threads, a row has at least eight of them, and a thread at most 64 elements
(16 in the backward pass). That bounds the rows in flight of any plan, and with it the turns that a
number of rows takes at least."""
import gc

import pytest
import torch

import nvfp4_block_scaled_13_b200 as nv
from tests.test_gpu_a_layer_norm import HALF, TYPES, U, chain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def leave_no_garbage():
    """Tensors that a failed call's traceback still holds are freed here, not during a later test."""
    yield
    gc.collect()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def make(rows, cols, xt, wt, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    x = rand(rows, cols).mul_(torch.exp(rand(cols))).add_(0.3).to(TYPES[xt])
    return x, (1 + 0.2 * rand(cols)).to(TYPES[wt]), (0.1 * rand(cols)).to(TYPES[wt])


def slices(rows, cols):
    step = max(1, (1 << 24) // cols)
    return [slice(lo, min(rows, lo + step)) for lo in range(0, rows, step)]


def check_forward(r, x, w, b, eps, xt):
    """As in test_gpu_a_layer_norm.py, a part of the rows at a time."""
    D, w, b = chain(x.shape[1]), w.double(), b.double()
    for part in slices(*x.shape):
        X = x[part].double()
        mean = X.mean(1, keepdim=True)
        d = X - mean
        var = (d * d).mean(1, keepdim=True)
        rstd = 1 / (var + eps).sqrt()
        y = d * rstd * w + b
        e = (D + 2) * U * X.abs().mean(1, keepdim=True)
        rel = 0.5 * ((D + 6) * U + e * e / (var + eps)) + 4 * U
        assert ((r.mean[part, None] - mean).abs() <= e + U * mean.abs()).all(), part
        assert ((r.rstd[part, None] / rstd - 1).abs() <= rel + U).all(), part
        tol = w.abs() * rstd * (d.abs() * (rel + 4 * U) + e) + 3 * U * (y.abs() + b.abs())
        tol = tol + HALF[xt] * (y.abs() + tol) + 2.0 ** -134
        assert ((r.y[part].double() - y).abs() <= tol).all(), part
    assert r.amax.item() == r.y.abs().max().item()


@pytest.mark.parametrize("cols", [257, 264, 384, 511, 512])
@pytest.mark.parametrize("turns", [2, 3, 6])
def test_forward_of_short_rows_over_every_stage(gpu, cols, turns):
    """One warp a row, four rows ahead: two CTAs of 16 warps an SM, one turn more than `turns` of them."""
    rows = turns * 2 * 16 * sms() + 77
    x, w, b = make(rows, cols, "bf16", "bf16", seed=cols)
    check_forward(nv.layer_norm_forward(x, w, b, 1e-5, with_amax=True), x, w, b, 1e-5, "bf16")
