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


# ---- every plan ------------------------------------------------------------------------------------

TURNS = 7      # one more than the deepest ring (four stages) and two


def rows_of(cols, most):
    """Rows of which every group takes at least TURNS, whatever the plan, and whose last turn is partly empty."""
    threads = max(8, -(-cols // most))
    return TURNS * (sms() * 2048 // threads) + 1


# Widths within each step of the cut: 8, 16 and 32 lanes a row, each number of units of one to five
# warps, two to eight CTAs, and rows that are read by the element. The odd ones begin at every shift.
GROUPS = [5, 33, 64, 77, 128, 129, 200, 256]
FORWARD = GROUPS + [300, 507, 512, 640, 771, 1024, 1255, 1280, 1400, 1537, 1792, 1801, 2048, 2051, 2560, 2800, 3003, 3080, 3583, 3592,
                    4095, 4096, 4099, 4608, 4611, 5376, 5385, 6144, 6147, 7168, 7173, 8192, 8195, 8960, 8967, 10240, 10243, 16384, 16389,
                    32768, 32771, 65529, 65536]


@pytest.mark.parametrize("cols", FORWARD)
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_forward_of_every_plan_over_many_turns(gpu, cols, xt):
    x, w, b = make(rows_of(cols, 64), cols, xt, xt, seed=cols)
    check_forward(nv.layer_norm_forward(x, w, b, 1e-5, with_amax=True), x, w, b, 1e-5, xt)


def check_backward(got, dy, x, w, mean, rstd, xt, wt):
    """As in test_gpu_a_layer_norm.py, a part of the rows at a time."""
    rows, cols = x.shape
    D, w = chain(cols), w.double()
    sums = torch.zeros(4, cols, dtype=torch.float64, device="cuda")      # dweight, dbias, and their magnitudes
    for part in slices(rows, cols):
        g, r = dy[part].double(), rstd[part, None].double()
        xh = (x[part].double() - mean[part, None].double()) * r
        h = g * w
        s1, s2 = h.mean(1, keepdim=True), (h * xh).mean(1, keepdim=True)
        dx = r * (h - s1 - xh * s2)
        a1, a2 = h.abs().mean(1, keepdim=True), (h * xh).abs().mean(1, keepdim=True)
        tol = r * ((D + 6) * U * (a1 + xh.abs() * a2) + 6 * U * (h.abs() + s1.abs() + (xh * s2).abs()))
        tol = tol + HALF[xt] * (dx.abs() + tol) + 2.0 ** -134
        assert ((got[0][part].double() - dx).abs() <= tol).all(), part
        sums += torch.stack([(g * xh).sum(0), g.sum(0), (g * xh).abs().sum(0), g.abs().sum(0)])
    parts = nv.nvfp4_layer_norm_workspace(rows, cols) // (8 * cols)
    length = (rows / parts + parts / 8 + 24 + 4) * U
    for k in (0, 1):
        tol = length * sums[2 + k]
        tol = tol + HALF[wt] * (sums[k].abs() + tol) + 2.0 ** -134
        assert ((got[1 + k].double() - sums[k]).abs() <= tol).all()


# 8, 16 and 32 lanes of 8 elements, 32 of 16, one to sixteen warps (four groups to one in a CTA), clusters.
BACKWARD = GROUPS + [300, 512, 519, 1000, 1024, 1029, 1536, 1543, 2048, 2055, 4096, 4099, 5001, 8191, 8192, 8200, 10243, 16384, 16389, 32768,
                     32771, 65529, 65536]


@pytest.mark.parametrize("cols", BACKWARD)
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("f32", "f32")])
def test_backward_of_every_plan_over_many_turns(gpu, cols, xt, wt):
    rows = rows_of(cols, 16)
    x, w, _ = make(rows, cols, xt, wt, seed=cols)
    r = nv.layer_norm_forward(x, w)
    dy = (x * 1e-3).roll(1, 0).contiguous()                               # a gradient that does not go with its row
    got = nv.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    check_backward(got, dy, x, w, r.mean, r.rstd, xt, wt)
    again = nv.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, again)), "the same from run to run"


@pytest.mark.parametrize("rows,cols", [(3001, 70001), (5001, 100), (701, 4096)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_rows_by_the_element_over_many_turns(gpu, rows, cols, xt):
    """Over 65536 columns, or x one element past a boundary on which y and dx lie."""
    flat, w, b = make(1, rows * cols + 1, xt, xt, seed=cols)
    x, w, b = flat.view(-1)[1:].view(rows, cols), w[:cols].contiguous(), b[:cols].contiguous()
    r = nv.layer_norm_forward(x, w, b, 1e-5, with_amax=True)
    check_forward(r, x, w, b, 1e-5, xt)
    dy = (x * 1e-3).roll(1, 0).contiguous()
    check_backward(nv.layer_norm_backward(dy, x, w, r.mean, r.rstd), dy, x, w, r.mean, r.rstd, xt, xt)


def test_backward_on_two_streams_is_what_binary64_says(gpu):
    """Two calls that overlap on the GPU, each with a workspace of its own."""
    made = [make(9001, 1029 + k, "bf16", "f32", seed=k) for k in range(2)]
    rs = [nv.layer_norm_forward(x, w) for x, w, _ in made]
    dys = [(x * 1e-3).roll(1, 0).contiguous() for x, _, _ in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        got = [nv.layer_norm_backward(dys[k], made[k][0], made[k][1], rs[k].mean, rs[k].rstd, stream=streams[k]) for k in range(2)]
    torch.cuda.synchronize()
    for k in range(2):
        check_backward(got[k], dys[k], made[k][0], made[k][1], rs[k].mean, rs[k].rstd, "bf16", "f32")
