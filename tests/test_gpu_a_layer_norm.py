"""Layer norm forward and backward on the GPU against binary64, on the values the kernel was given.

Bounds, with u = 2^-24 (half a step of binary32) and D the longest chain of additions of a row
sum: 16 elements of a thread and the trees over warps and CTAs, taken as 48 (rows of over 65000
columns: a thread's share of the row and the tree, cols / 1024 + 16 > 48).
  mean: |e| <= (D + 2) u S|x|/C.  Its effect on the variance is of second order (deviations sum to
  0): var has the relative error (D + 6) u + e^2 / var, rstd half of that plus 4 u.
  y: |w| rstd (|d| (that + 4 u) + e) + 3 u (|y| + |b|), and half a step of the stored type.
  dx: with h = dy w: rstd ((D + 6) u (S|h|/C + |xh| S|h xh|/C) + 6 u (|h| + |s1| + |xh s2|)), and half a step.
  dweight, dbias: a chain of at most rows / parts + parts / 8 + 24 additions with 4 roundings a
  term: that many u times the sum of magnitudes, and half a step."""
import gc

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_13_b200 as nv
from tests import train_ref as R
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def leave_no_garbage():
    """Tensors that a failed call's traceback still holds are freed here, not during a later test."""
    yield
    gc.collect()

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}     # eps / 2 of the type
CODE = {"bf16": nv.TYPE_BF16, "f32": nv.TYPE_F32}


def make(rows, cols, xt, wt, seed=0, shift=0.3):
    rng = np.random.default_rng(seed)
    channel = np.exp(rng.standard_normal(cols))
    x = rng.standard_normal((rows, cols)) * channel + shift
    w, b = 1 + 0.2 * rng.standard_normal(cols), 0.1 * rng.standard_normal(cols)
    dy = rng.standard_normal((rows, cols)) * 1e-3
    to = lambda a, t: torch.from_numpy(a).to(TYPES[t]).cuda()  # noqa: E731
    return to(x, xt), to(w, wt), to(b, wt), to(dy, xt)


def f64(t):
    return t.double().cpu().numpy()


def chain(cols):
    return max(48, cols / 1024 + 16)


def check_forward(r, x, w, b, eps, xt):
    rows, cols = x.shape
    X, W, B = f64(x), 1.0 if w is None else f64(w), 0.0 if b is None else f64(b)
    y, mean, rstd, var = R.norm64(X, W, B, eps)
    D = chain(cols)
    e = (D + 2) * U * np.abs(X).mean(1, keepdims=True)
    rel = 0.5 * ((D + 6) * U + e * e / (var + eps)) + 4 * U
    assert (np.abs(f64(r.mean)[:, None] - mean) <= e + U * np.abs(mean)).all()
    assert (np.abs(f64(r.rstd)[:, None] / rstd - 1) <= rel + U).all()
    tol = np.abs(W) * rstd * (np.abs(X - mean) * (rel + 4 * U) + e) + 3 * U * (np.abs(y) + np.abs(B))
    tol = tol + HALF[xt] * (np.abs(y) + tol) + 2.0 ** -134
    err = np.abs(f64(r.y) - y)
    assert (err <= tol).all(), (err / tol).max()
    assert r.amax.item() == r.y.abs().max().item()


SHAPES = [(1, 1), (3, 1), (1, 5), (4, 8), (33, 16), (9, 256), (65, 264), (7, 512), (5, 1000), (6, 1001), (17, 1024),
          (3, 1032), (1, 4096), (300, 4096), (2, 4100), (5, 8192), (4, 8193), (3, 16384), (2, 16392), (2, 32768), (2, 40000),
          (3, 32771), (2, 65536), (2, 65529), (2, 65530), (300, 16384), (200, 8191), (1500, 72), (700, 129), (3000, 33)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_forward(gpu, rows, cols, xt, wt):
    x, w, b, _ = make(rows, cols, xt, wt, seed=rows * cols)
    check_forward(nv.layer_norm_forward(x, w, b, 1e-5, with_amax=True), x, w, b, 1e-5, xt)


@pytest.mark.parametrize("edge", [256, 512, 768, 1024, 1280, 1536, 1792, 2048, 2560, 3584, 4096, 4608, 5376, 6144, 7168, 8192, 8960, 10240])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_forward_at_the_edges_of_the_row_cuts(gpu, edge, xt):
    """Widths around every number of units a lane: each shift, each last unit whole, partial or missing."""
    for cols in (*range(edge - 8, edge + 9), edge + 31):
        x, w, b, _ = make(9, cols, xt, "f32", seed=cols)
        check_forward(nv.layer_norm_forward(x, w, b, 1e-5, with_amax=True), x, w, b, 1e-5, xt)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("cols", [48, 333, 4096])
def test_forward_without_weight_or_bias(gpu, cols, weight, bias):
    x, w, b, _ = make(10, cols, "bf16", "bf16")
    w, b = w if weight else None, b if bias else None
    r = nv.layer_norm_forward(x, w, b, 1e-6, with_amax=True)
    check_forward(r, x, w, b, 1e-6, "bf16")
    plain = nv.layer_norm_forward(x, w, b, 1e-6, with_stats=False)
    assert plain.mean is None and plain.rstd is None and plain.amax is None and torch.equal(plain.y, r.y)


@pytest.mark.parametrize("rows,cols", [(5, 520), (3, 77), (2, 4096), (2, 33000)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_any_alignment_and_nothing_outside_is_written(gpu, rows, cols, xt, offset):
    """Every operand starts `offset` elements past a 16-byte boundary; canaries around the outputs."""
    x, w, b, dy = make(rows, cols, xt, "f32", seed=3)
    size = 2 if xt == "bf16" else 4
    n = rows * cols

    def shifted(t):
        s = t.element_size()
        buf = torch.empty(t.numel() * s + 64, dtype=torch.uint8, device="cuda")
        view = buf[offset * s:offset * s + t.numel() * s].view(t.dtype)
        view.copy_(t.reshape(-1))
        return view

    xs, ws, bs, ds = (shifted(t) for t in (x, w, b, dy))
    y, mean, rstd, top = Guarded((n + offset) * size), Guarded(4 * rows), Guarded(4 * rows), Guarded(4)
    at = lambda g, s: g.ptr() + offset * s  # noqa: E731
    nv.nvfp4_layer_norm(xs.data_ptr(), CODE[xt], ws.data_ptr(), bs.data_ptr(), nv.TYPE_F32, rows, cols, 1e-5, at(y, size),
                        mean.ptr(), rstd.ptr(), top.ptr())
    dx, dw, db = Guarded((n + offset) * size), Guarded(4 * (cols + offset)), Guarded(4 * (cols + offset))
    need = nv.nvfp4_layer_norm_workspace(rows, cols)
    work = Guarded(need)
    nv.nvfp4_layer_norm_backward(ds.data_ptr(), xs.data_ptr(), CODE[xt], ws.data_ptr(), nv.TYPE_F32, mean.ptr(), rstd.ptr(),
                                 rows, cols, at(dx, size), at(dw, 4), at(db, 4), work.ptr(), need)
    torch.cuda.synchronize()
    for g in (y, mean, rstd, top, dx, dw, db, work):
        assert g.guards_intact()
    for g, s in ((y, size), (dx, size), (dw, 4), (db, 4)):
        assert (g.numpy()[:offset * s] == 0xA5).all()
    take = lambda g, t, s, k: torch.from_numpy(g.numpy()[offset * s:offset * s + k * s].copy()).view(t)  # noqa: E731
    got = nv.Normed(take(y, TYPES[xt], size, n).view(rows, cols).cuda(),
                    *(torch.from_numpy(g.numpy(np.float32).copy()).cuda() for g in (mean, rstd, top)))
    check_forward(got, x, w, b, 1e-5, xt)
    check_backward((take(dx, TYPES[xt], size, n).view(rows, cols), take(dw, torch.float32, 4, cols),
                    take(db, torch.float32, 4, cols)), dy, x, w, got.mean, got.rstd, xt, "f32")


@pytest.mark.parametrize("rows,cols", [(7, 64), (5, 1024), (3, 1003)])
@pytest.mark.parametrize("xt", ["bf16", "f32"])
def test_operands_at_different_places_within_16_bytes(gpu, rows, cols, xt):
    """x on a boundary, y and dx one element past one, dy two: no common shift."""
    x, w, b, dy = make(rows, cols, xt, "f32", seed=6)
    n = rows * cols
    past = lambda k: torch.zeros(n + 8, dtype=TYPES[xt], device="cuda")[k:k + n]  # noqa: E731
    y, dx, g = past(1), past(1), past(2)
    g.copy_(dy.reshape(-1))
    mean, rstd, top = (torch.empty(k, device="cuda") for k in (rows, rows, 1))
    nv.nvfp4_layer_norm(x, CODE[xt], w, b, nv.TYPE_F32, rows, cols, 1e-5, y, mean, rstd, top)
    check_forward(nv.Normed(y.view(rows, cols), mean, rstd, top), x, w, b, 1e-5, xt)
    size = nv.nvfp4_layer_norm_workspace(rows, cols)
    dw, db, work = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda"), torch.empty(size, dtype=torch.uint8, device="cuda")
    nv.nvfp4_layer_norm_backward(g, x, CODE[xt], w, nv.TYPE_F32, mean, rstd, rows, cols, dx, dw, db, work, size)
    # one column a thread and a slab of rows each: the chain is the slab's rows and the slabs
    check_backward((dx.view(rows, cols), dw, db), dy, x, w, mean, rstd, xt, "f32")


def test_two_streams_at_once(gpu):
    """Two calls that overlap on the GPU, each with its own memory, give what they give alone."""
    made = [make(2000, 1024, "bf16", "bf16", seed=k) for k in range(2)]
    alone = []
    for x, w, b, dy in made:
        r = nv.layer_norm_forward(x, w, b, with_amax=True)
        alone.append(tuple(r) + nv.layer_norm_backward(dy, x, w, r.mean, r.rstd))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[], []]
    for turn in range(4):
        for k, (x, w, b, dy) in enumerate(made):
            r = nv.layer_norm_forward(x, w, b, with_amax=True, stream=streams[k])
            got[k] = tuple(r) + nv.layer_norm_backward(dy, x, w, alone[k][1], alone[k][2], stream=streams[k])
    torch.cuda.synchronize()
    for a, g in zip(alone, got):
        assert all(torch.equal(p, q) for p, q in zip(a, g))


def test_a_large_offset_cancels_nothing(gpu):
    """Values of deviation 1 around 4096 in FP32: mean and variance keep their digits."""
    x, w, b, _ = make(6, 4096, "f32", "f32", shift=0.0)
    x = x / x.std() + 4096
    check_forward(nv.layer_norm_forward(x, w, b, 1e-5, with_amax=True), x, w, b, 1e-5, "f32")


def test_constant_rows_and_zero_eps(gpu):
    _, w, b, _ = make(1, 64, "bf16", "bf16")
    x = torch.full((3, 64), 2.5, dtype=torch.bfloat16, device="cuda")
    r = nv.layer_norm_forward(x, w, b, 1e-5)
    assert torch.equal(r.y, b.expand(3, 64)) and (r.mean == 2.5).all()
    assert torch.isnan(nv.layer_norm_forward(x, w, b, 0.0).y).all()      # 0 * infinity, as the formula has it


@pytest.mark.parametrize("cols", [64, 100, 4096])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nan_and_infinity_stay_in_their_row(gpu, cols, bad):
    x, w, b, dy = make(9, cols, "bf16", "bf16")
    clean = nv.layer_norm_forward(x, w, b, with_amax=True)
    x2 = x.clone()
    x2[4, cols // 2] = bad
    r = nv.layer_norm_forward(x2, w, b, with_amax=True)
    assert torch.isnan(r.y[4]).all() and torch.isnan(r.amax).all()
    keep = [i for i in range(9) if i != 4]
    assert torch.equal(r.y[keep], clean.y[keep])
    dx, _, _ = nv.layer_norm_backward(dy, x2, w, r.mean, r.rstd)
    want, _, _ = nv.layer_norm_backward(dy, x, w, clean.mean, clean.rstd)
    assert torch.isnan(dx[4]).all() and torch.equal(dx[keep], want[keep])


def check_backward(got, dy, x, w, mean, rstd, xt, wt):
    rows, cols = x.shape
    W = 1.0 if w is None else f64(w)
    dx, dw, db, xh, h = R.norm_grad64(f64(dy), f64(x), W, f64(mean), f64(rstd))
    D = chain(cols)
    r = f64(rstd)[:, None]
    s1, s2 = h.mean(1, keepdims=True), (h * xh).mean(1, keepdims=True)
    a1, a2 = np.abs(h).mean(1, keepdims=True), np.abs(h * xh).mean(1, keepdims=True)
    tol = r * ((D + 6) * U * (a1 + np.abs(xh) * a2) + 6 * U * (np.abs(h) + np.abs(s1) + np.abs(xh * s2)))
    tol = tol + HALF[xt] * (np.abs(dx) + tol) + 2.0 ** -134
    err = np.abs(f64(got[0]) - dx)
    assert (err <= tol).all(), (err / tol).max()
    parts = nv.nvfp4_layer_norm_workspace(rows, cols) // (8 * cols)
    length = (rows / parts + parts / 8 + 24 + 4) * U
    G = np.abs(f64(dy))
    for g, want, size in ((got[1], dw, (G * np.abs(xh)).sum(0)), (got[2], db, G.sum(0))):
        if g is None:
            continue
        tol = length * size
        tol = tol + HALF[wt] * (np.abs(want) + tol) + 2.0 ** -134
        err = np.abs(f64(g) - want)
        assert (err <= tol).all(), (err / tol).max()


BACK = [(1, 1), (3, 5), (1, 4096), (4, 8), (33, 16), (300, 256), (65, 264), (7, 512), (40, 520), (5, 1000), (300, 1001), (6, 2048),
        (3, 2056), (900, 4096), (2, 4100), (5, 8192), (4, 8193), (300, 9000), (2, 16384), (3, 20001), (2, 65536), (2, 70001), (200, 16384), (300, 8191), (1500, 500), (700, 511), (3000, 72), (2500, 129), (3000, 33)]


@pytest.mark.parametrize("rows,cols", BACK)
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_backward(gpu, rows, cols, xt, wt):
    x, w, b, dy = make(rows, cols, xt, wt, seed=rows + cols)
    r = nv.layer_norm_forward(x, w, b)
    got = nv.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    check_backward(got, dy, x, w, r.mean, r.rstd, xt, wt)
    again = nv.layer_norm_backward(dy, x, w, r.mean, r.rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, again)), "the same from run to run"


@pytest.mark.parametrize("cols", [128, 1003, 4096, 9000])
@pytest.mark.parametrize("dw,db", [(False, False), (True, False), (False, True)])
def test_backward_without_some_gradients(gpu, cols, dw, db):
    x, w, _, dy = make(50, cols, "bf16", "bf16")
    r = nv.layer_norm_forward(x, w)
    got = nv.layer_norm_backward(dy, x, w, r.mean, r.rstd, with_weight=dw, with_bias=db)
    assert (got[1] is not None, got[2] is not None) == (dw, db)
    check_backward(got, dy, x, w, r.mean, r.rstd, "bf16", "bf16")
    check_backward(nv.layer_norm_backward(dy, x, None, r.mean, r.rstd), dy, x, None, r.mean, r.rstd, "bf16", "f32")


@pytest.mark.parametrize("rows,cols", [(3, 24), (4, 37)])
def test_gradient_against_differences(gpu, rows, cols):
    """Central differences of the binary64 formula: step 1e-5, error about 1e-10 of the scale."""
    x, w, b, dy = make(rows, cols, "f32", "f32", seed=5)
    r = nv.layer_norm_forward(x, w, b)
    dx, dw, db = (f64(t) for t in nv.layer_norm_backward(dy, x, w, r.mean, r.rstd))
    X, W, B, G = f64(x), f64(w), f64(b), f64(dy)
    loss = lambda X, W, B: (R.norm64(X, W, B, 1e-5)[0] * G).sum()  # noqa: E731
    step = 1e-5

    def difference(k, at):
        args = [X, W, B]
        up, down = [a.copy() for a in args], [a.copy() for a in args]
        up[k][at] += step
        down[k][at] -= step
        return (loss(*up) - loss(*down)) / (2 * step)

    scale = np.abs(G).max()
    for i in range(rows):
        for j in range(0, cols, 5):
            assert abs(difference(0, (i, j)) - dx[i, j]) < 1e-5 * scale * max(1, f64(r.rstd).max())
    for j in range(cols):
        assert abs(difference(1, j) - dw[j]) < 1e-5 * scale * rows and abs(difference(2, j) - db[j]) < 1e-5 * scale * rows


def test_empty(gpu):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r = nv.layer_norm_forward(x, w, w, with_amax=True)
    assert r.y.shape == (0, 64) and r.amax.item() == 0
    dx, dw, db = nv.layer_norm_backward(x, x, w, r.mean, r.rstd)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_autograd_with_leading_dimensions_and_a_broadcast_gradient(gpu):
    x, w, b, dy = make(12, 96, "bf16", "f32")
    x = x.view(3, 4, 96).requires_grad_()
    w.requires_grad_()
    b.requires_grad_()
    y, top = nv.layer_norm(x, w, b, with_amax=True)
    assert not top.requires_grad and top.item() == y.abs().max().item()
    g = dy[0, 0].expand(3, 4, 96)                                                  # no memory of its own
    y.backward(g)
    r = nv.layer_norm_forward(x.detach(), w.detach())
    want = nv.layer_norm_backward(g.contiguous(), x.detach(), w.detach(), r.mean, r.rstd)
    for got, t in zip((x.grad, w.grad, b.grad), want):
        assert torch.equal(got, t) and got.dtype == t.dtype
    plain = nv.layer_norm(x.detach(), None, b.detach())
    assert not plain.requires_grad
    v = torch.zeros(96, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    nv.layer_norm(x.detach(), None, v).sum().backward()                           # a bias alone
    assert v.grad.dtype == torch.bfloat16 and (v.grad == 12).all()


def test_wrappers_refuse(gpu):
    x, w, b, dy = make(4, 32, "bf16", "bf16")
    r = nv.layer_norm_forward(x, w, b)
    for call in (lambda: nv.layer_norm(x.half(), w, b), lambda: nv.layer_norm(x.t(), None, None), lambda: nv.layer_norm(x, w[:16], b),
                 lambda: nv.layer_norm(x, w, b.float()), lambda: nv.layer_norm(x, w.cpu(), b), lambda: nv.layer_norm(x[:, :16]),
                 lambda: nv.layer_norm(x, w.half(), None), lambda: nv.layer_norm(x[0, 0]),
                 lambda: nv.layer_norm_backward(dy.float(), x, w, r.mean, r.rstd),
                 lambda: nv.layer_norm_backward(dy[:2], x, w, r.mean, r.rstd),
                 lambda: nv.layer_norm_backward(dy, x, w, r.mean[:2], r.rstd),
                 lambda: nv.layer_norm_backward(dy, x, w, r.mean.double(), r.rstd)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(nv.Nvfp4Error):
        nv.layer_norm(x, w, b, eps=-1.0)


def test_side_stream_and_captured_graph(gpu):
    x, w, b, dy = make(300, 1024, "bf16", "bf16")
    want = nv.layer_norm_forward(x, w, b, with_amax=True)
    grads = nv.layer_norm_backward(dy, x, w, want.mean, want.rstd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.layer_norm_forward(x, w, b, with_amax=True, stream=side)
    back = nv.layer_norm_backward(dy, x, w, want.mean, want.rstd, stream=side)
    raw = nv.layer_norm_forward(x, w, b, with_amax=True, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got + back + raw, want + grads + want))
    x2, dy2 = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = nv.layer_norm_forward(x2, w, b, with_amax=True)
        g = nv.layer_norm_backward(dy2, x2, w, r.mean, r.rstd)
    for k in (1, 2):
        x2.copy_(x * k)
        dy2.copy_(dy * k)
        graph.replay()
        want = nv.layer_norm_forward(x2, w, b, with_amax=True)
        grads = nv.layer_norm_backward(dy2, x2, w, want.mean, want.rstd)
        assert all(torch.equal(p, q) for p, q in zip(tuple(r) + g, tuple(want) + grads))


def test_more_than_2_to_the_31_elements(gpu):
    """Offsets past 32 bits: the first and last rows of 2.1e9 BF16 elements."""
    rows, cols = 262144 + 7, 8192
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.normal_()
    r = nv.layer_norm_forward(x, with_amax=True)
    for part in (slice(0, 4), slice(rows - 4, rows)):
        y = R.norm64(f64(x[part]), 1.0, 0.0, 1e-5)[0]
        assert np.abs(f64(r.y[part]) - y).max() <= 2.0 ** -8 * np.abs(y).max() + 1e-5
    dx, _, db = nv.layer_norm_backward(r.y, x, None, r.mean, r.rstd)
    part = slice(rows - 4, rows)
    want = R.norm_grad64(f64(r.y[part]), f64(x[part]), 1.0, f64(r.mean[part]), f64(r.rstd[part]))[0]
    assert np.abs(f64(dx[part]) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-4
    assert db.shape == (cols,)
