"""AdamW over lists of tensors and the gradient norm, on the GPU.

The step's arithmetic is binary32 with every operation rounded, so parameters and states are compared
bit for bit with the same operations in numpy (beside 8-bit states up to two approximations of 2^-23,
as assert_step says); and with the definition in binary64, where u = 2^-24: m within 4 u (|b1 m| + |r1 g|) (three roundings and the rounded
coefficients), v within 8 u v, p within 3 u |p| + 16 u |update| + (the error of m) rate / denominator
(products, the quotient, the root, the factors; 24 u beside 8-bit states, whose root and reciprocal are
off by up to 2 u more and whose quotient has one more rounding), then half a step of a type that is rounded to
nearest, or a whole one of a stochastic rounding. 8-bit values: half an E4M3 step for m (2^-4 of
the value, or 2^-10 of the block's power of two), a whole one for u. Beside 8-bit states a v below
2^-126 counts as 0, which takes at most 2^-63 from the root.
The norm: eights in binary32 (9 roundings) and the rest in binary64: 5 u relative for the root,
u for its rounding."""
import gc

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_13_b200 as nv
from tests import train_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def leave_no_garbage():
    """Tensors that a failed call's traceback still holds are freed here, not during a later test."""
    yield
    gc.collect()

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
LENGTHS = [1, 7, 8, 31, 32, 33, 2047, 2048, 2049, 5000, 100003]


def values(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def raw(t):
    return t.view(torch.uint8).cpu().numpy() if t.element_size() == 1 else values(t)


def make(lengths, param, grad, bits, masters, *, seed=0, offset=0, steps=0, betas=(0.9, 0.95), decay=0.1, with_amax=True, fill=True):
    """Parameters and gradients `offset` elements past the alignment of their allocation."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    params, grads = [], []
    for n in lengths:
        for out, t, size in ((params, param, 0.02), (grads, grad, 1e-3)):
            whole = (torch.randn(n + offset, device="cuda", generator=gen) * size).to(TYPES[t])
            out.append(whole[offset:])
    plan = nv.adamw_plan(params, grads, state_bits=bits, masters=masters, betas=betas, weight_decay=[decay * (i % 2) for i in range(len(lengths))],
                         seed=12345 + seed, step=steps, with_amax=with_amax)
    if fill:
        for i, n in enumerate(lengths):
            state = plan.state(i)
            m = torch.randn(n, device="cuda", generator=gen) * 3e-4
            root = (torch.rand(n, device="cuda", generator=gen) + 0.5) * 1e-3
            if bits == 32:
                state["exp_avg"].copy_(m)
                state["exp_avg_sq"].copy_(root * root)
            else:
                for name, x in (("exp_avg", m), ("exp_avg_sq", root)):
                    codes, scales = R.encode_nearest(values(x))
                    state[name].view(torch.uint8).copy_(torch.from_numpy(codes))
                    state[name + "_scale"].view(torch.uint8).copy_(torch.from_numpy(scales))
    return plan


def before(plan, i):
    state = plan.state(i)
    m, v = raw(state["exp_avg"]), raw(state["exp_avg_sq"])
    if plan.state_bits == 8:
        m, v = (m, raw(state["exp_avg_scale"])), (v, raw(state["exp_avg_sq_scale"]))
    p = state["master"] if "master" in state and plan.params[i].dtype == torch.bfloat16 else plan.params[i]
    return values(p).copy(), values(plan.grads[i]), m, v


def check(plan, olds, lr, scale, steps, decay=0.1):
    for i, (p, g, m, v) in enumerate(olds):
        bf16 = plan.params[i].dtype == torch.bfloat16
        master = plan.master is not None and bf16
        kw = dict(lr=lr, decay=decay * (i % 2), betas=plan.betas, eps=plan.eps, scale=scale, steps=steps)
        want = R.adamw_bits(p, g, m, v, param_bf16=bf16, master=master, bits=plan.state_bits, first=plan.offsets[i], seed=plan.seed, **kw)
        got = {"param": values(plan.params[i]), **{k: raw(t) for k, t in plan.state(i).items()}}
        R.assert_step(got, want, plan.state_bits, f"tensor {i} of {len(p)}")
        if plan.amax is not None:
            assert plan.amax[i].item() == np.abs(got["param"]).max()
        # the definition
        if plan.state_bits == 8:
            m, root = R.decode(*m).astype(np.float64), R.decode(*v).astype(np.float64)
            v = root * root
        p1, m1, v1, size_m, update, per_m = R.adamw64(p, g, m, v, **kw)
        tol_m = 4 * U * size_m + 2.0 ** -147          # and what underflow takes from each of three operations
        tol_p = 3 * U * np.abs(p) + (16 if plan.state_bits == 32 else 24) * U * update + tol_m * per_m
        full = got["master"].astype(np.float64) if master else got["param"].astype(np.float64)
        half = 0.0 if master or not bf16 else 2.0 ** -7
        assert (np.abs(full - p1) <= tol_p + half * (np.abs(p1) + tol_p) + 2.0 ** -133).all()
        if master:
            assert (np.abs(got["param"] - full) <= 2.0 ** -8 * np.abs(full)).all()
        if plan.state_bits == 32:
            assert (np.abs(got["exp_avg"] - m1) <= tol_m).all()
            assert (np.abs(got["exp_avg_sq"] - v1) <= 8 * U * v1 + 2.0 ** -147).all()
        else:
            n = len(p)
            for name, x, tol, step in (("exp_avg", m1, tol_m, 0.5), ("exp_avg_sq", np.sqrt(v1), 7 * U * np.sqrt(v1) + 2.0 ** -62.9, 1.0)):
                unit = R.spread(R.power(got[name + "_scale"]), n).astype(np.float64)
                value = R.decode(got[name], got[name + "_scale"])
                assert (np.abs(value - x) <= tol + step * np.maximum(2.0 ** -3 * np.abs(x), 2.0 ** -9 * unit) * (1 + 4 * U)).all()


@pytest.mark.parametrize("param,masters", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 1])
def test_steps(gpu, param, masters, grad, bits, offset):
    """Three steps over every length, aligned and not, with a clip factor from the second on."""
    plan = make(LENGTHS, param, grad, bits, masters, offset=offset, steps=3)
    for k, (lr, scale) in enumerate(((1e-3, None), (2e-3, 0.25), (0.0, 1.0))):
        olds = [before(plan, i) for i in range(len(LENGTHS))]
        nv.adamw(plan, lr, None if scale is None else torch.tensor([scale], device="cuda"))
        check(plan, olds, lr, 1.0 if scale is None else scale, 3 + k)
    assert plan.steps() == 6


@pytest.mark.parametrize("bits", [32, 8])
def test_long_list_takes_longer_chunks(gpu, bits):
    """Enough elements for chunks of several tiles, with tensors that end inside one."""
    lengths = [9_000_001, 5, 8_388_608, 2048 * 3 + 17]
    plan = make(lengths, "bf16", "bf16", bits, False)
    olds = [before(plan, i) for i in range(len(lengths))]
    nv.adamw(plan, 1e-3)
    check(plan, olds, 1e-3, 1.0, 0)


@pytest.mark.parametrize("param,masters", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_nothing_and_zero_gradients(gpu, param, masters, bits):
    plan = make([64, 100], param, "bf16", bits, masters, fill=False)
    plan.grads[0].zero_()
    olds = [before(plan, i) for i in range(2)]
    nv.adamw(plan, 1e-2)
    check(plan, olds, 1e-2, 1.0, 0)
    assert torch.equal(plan.params[0].float(), torch.from_numpy(olds[0][0]).cuda().to(plan.params[0].dtype).float())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_scale_that_is_not_finite_leaves_everything(gpu, bits, bad):
    plan = make([100, 3000], "bf16", "bf16", bits, True, steps=5)
    nv.adamw(plan, 1e-3)
    keep = [t.clone() for t in (*plan.params, plan.master, plan.exp_avg, plan.exp_avg_sq, plan.control)]
    plan.amax.zero_()
    nv.adamw(plan, 1e-3, torch.tensor([bad], device="cuda"))
    for a, b in zip(keep, (*plan.params, plan.master, plan.exp_avg, plan.exp_avg_sq, plan.control)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert plan.steps() == 6
    assert [v.item() for v in plan.amax] == [p.abs().max().item() for p in plan.params]
    plan.grads[0][3] = float("inf")
    norm, scale = nv.grad_norm(plan, 1.0)
    assert norm.item() == float("inf") and torch.isnan(scale).all()
    nv.adamw(plan, 1e-3, scale)
    assert plan.steps() == 6 and torch.equal(keep[0], plan.params[0])


@pytest.mark.parametrize("param,masters", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("bits", [32, 8])
def test_nan_and_infinity_stay_in_their_element_or_block(gpu, param, masters, bits):
    plan = make([4096], param, "f32", bits, masters)
    clean = make([4096], param, "f32", bits, masters)
    plan.grads[0][100] = float("nan")
    plan.grads[0][1000] = float("inf")
    nv.adamw(plan, 1e-3)
    nv.adamw(clean, 1e-3)
    p, q = values(plan.params[0]), values(clean.params[0])
    assert np.isnan(p[100]) and np.isnan(p[1000])
    at = np.ones(4096, bool)
    at[[100, 1000]] = False
    np.testing.assert_array_equal(p[at], q[at])
    if bits == 8:
        for i in (100, 1000):
            at[i // 32 * 32:i // 32 * 32 + 32] = False
            # NaN's code; an infinite moment saturates at the top of the largest scale, which decodes to infinity
            assert (raw(plan.exp_avg)[i] & 0x7F) == (0x7F if i == 100 else 0x7E) and raw(plan.exp_avg_sq)[i] == 0x7F
    for name in ("exp_avg", "exp_avg_sq"):
        np.testing.assert_array_equal(raw(getattr(plan, name))[at], raw(getattr(clean, name))[at])


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-10, 1e10, 1e17])
def test_8_bit_states_over_the_range_of_gradients(gpu, scale):
    """Blocks whose largest and smallest gradients are 1e9 apart, at the ends of the range."""
    plan = make([4096], "f32", "f32", 8, False, fill=False, betas=(0.9, 0.999))
    gen = torch.Generator(device="cuda").manual_seed(1)
    plan.grads[0].copy_(torch.exp(torch.rand(4096, device="cuda", generator=gen) * 20 - 20) * scale)
    for step in range(2):
        olds = [before(plan, 0)]
        nv.adamw(plan, 1e-3)
        check(plan, olds, 1e-3, 1.0, step)
        root = R.decode(raw(plan.exp_avg_sq), raw(plan.exp_avg_sq_scale))
        positive = np.float32(0.00099) * (values(plan.grads[0]) ** 2) >= np.float32(2.0 ** -126)
        assert (root[positive] > 0).all(), "a positive root keeps a positive code"


def test_stochastic_rounding_is_even(gpu):
    """65536 equal values a quarter of a step above a BF16 (and E4M3) number: the mean of what is
    stored is the value, within 6 standard deviations of independent roundings."""
    n = 1 << 16
    p = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 1.0, dtype=torch.float32, device="cuda")
    plan = nv.adamw_plan([p], [g], state_bits=8, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0, seed=9)
    g.fill_(-(1.0 + 1 / 32))     # u = 1.03125, a quarter of the way from 1 to 1.125 = E4M3's next
    nv.adamw(plan, 2.0 ** -9)    # p' = 1 + 2^-9: a quarter of the way from 1 to BF16's next, 1 + 2^-7
    sigma = (0.25 * 0.75) ** 0.5 / 256
    assert abs((p.double().mean().item() - 1) * 2 ** 7 - 0.25) < 6 * sigma
    root = R.decode(raw(plan.exp_avg_sq), raw(plan.exp_avg_sq_scale)).astype(np.float64)
    assert set(np.unique(root)) == {1.0, 1.125}
    assert abs((root.mean() - 1) * 8 - 0.25) < 6 * sigma


def test_mixed_list_and_learning_rate_on_the_device(gpu):
    """BF16 and FP32 tensors, with masters for the BF16 ones, and an empty tensor among them."""
    a = torch.randn(500, device="cuda").bfloat16()
    b = torch.randn(33, device="cuda")
    c = torch.empty(0, device="cuda")
    grads = [torch.randn_like(t, dtype=torch.float32) for t in (a, c, b)]
    plan = nv.adamw_plan([a, c, b], grads, masters=True, weight_decay=0.0, with_amax=True, betas=(0.9, 0.95))
    lr = torch.tensor([1e-3], device="cuda")
    for step in range(3):
        lr.fill_(1e-3 * (step + 1))
        olds = [before(plan, i) for i in (0, 2)]
        nv.adamw(plan, lr)
        for i, (p, g, m, v) in zip((0, 2), olds):
            want = R.adamw_bits(p, g, m, v, param_bf16=i == 0, master=i == 0, bits=32, first=plan.offsets[i], seed=0, lr=np.float32(1e-3 * (step + 1)),
                                decay=0.0, betas=plan.betas, eps=plan.eps, scale=1.0, steps=step)
            np.testing.assert_array_equal(values(plan.params[i]), want["param"])
        assert plan.amax.tolist() == [a.abs().max().item(), 0.0, b.abs().max().item()]


def test_control_survives_a_long_run_and_a_restart(gpu):
    plan = make([64], "f32", "f32", 32, False, betas=(0.9, 0.999))
    for _ in range(300):
        nv.adamw(plan, 0.0)
    assert plan.steps() == 300
    beta1, beta2 = plan.control[:4].view(torch.float64).tolist()
    assert abs(beta1 / 0.9 ** 300 - 1) < 1e-13 and abs(beta2 / 0.999 ** 300 - 1) < 1e-13
    plan.set_steps(7)
    olds = [before(plan, 0)]
    nv.adamw(plan, 1e-3)
    check(plan, olds, 1e-3, 1.0, 7)
    assert plan.steps() == 8


def test_nothing_between_the_tensors_is_written(gpu):
    """Parameters as slices of one buffer with canaries between; states up to their alignment."""
    flat = torch.full((4000,), 7.0, dtype=torch.bfloat16, device="cuda")
    spans = [(3, 100), (107, 640), (1000, 2049)]
    params = [flat[a:a + n] for a, n in spans]
    grads = [torch.randn(n, device="cuda").bfloat16() for _, n in spans]
    plan = nv.adamw_plan(params, grads, state_bits=8)
    nv.adamw(plan, 1e-3)
    outside = torch.ones(4000, dtype=torch.bool, device="cuda")
    for a, n in spans:
        outside[a:a + n] = False
    assert (flat[outside] == 7).all()
    states = torch.ones(plan.exp_avg.numel(), dtype=torch.bool, device="cuda")
    for a, n in zip(plan.offsets, plan.numels):
        states[a:a + n] = False
    assert (plan.exp_avg.view(torch.uint8)[states] == 0).all() and (plan.exp_avg_sq.view(torch.uint8)[states] == 0).all()


# ---- gradient norm -----------------------------------------------------------------------------

@pytest.mark.parametrize("lengths", [[1], [8], LENGTHS, [20_000_003, 1, 4096], [3] * 3000])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm(gpu, lengths, grad, offset):
    gen = torch.Generator(device="cuda").manual_seed(len(lengths))
    grads = [(torch.randn(n + offset, device="cuda", generator=gen) * 1e-3).to(TYPES[grad])[offset:] for n in lengths]
    handle = nv.gradient_list(grads)
    want = sum(float((g.double() ** 2).sum()) for g in grads) ** 0.5
    for max_norm in (want / 2, want * 2, float("inf"), 0.0):
        norm, scale = nv.grad_norm(handle, max_norm)
        assert abs(norm.item() / want - 1) <= 6 * U
        assert abs(scale.item() - min(1.0, max_norm / (want + 1e-6))) <= 8 * U
    again, _ = nv.grad_norm(handle, 1.0)
    assert again.item() == norm.item()


@pytest.mark.parametrize("size", [0.0, 1e-42, 1e-30, 1e-20, 1e19, 1e30])
def test_norm_over_the_whole_range(gpu, size):
    """Squares that overflow binary32, and squares that vanish in it."""
    g = torch.full((1000,), size, device="cuda")
    g[::3] = 0
    want = float((g.double() ** 2).sum()) ** 0.5
    norm, scale = nv.grad_norm(nv.gradient_list([g]), 1.0)
    assert abs(norm.item() - want) <= 6 * U * want + 2.0 ** -150
    assert abs(scale.item() - min(1.0, 1 / (want + 1e-6))) <= 8 * U * min(1.0, 1 / (want + 1e-6)) + 2.0 ** -150


@pytest.mark.parametrize("bad,want", [(float("nan"), "nan"), (float("inf"), "inf"), (3e38, "inf")])
def test_norm_that_is_not_finite(gpu, bad, want):
    g = torch.ones(5000, device="cuda")
    g[4000:4002] = bad       # two of 3e38 and a norm above binary32's largest number
    norm, scale = nv.grad_norm(nv.gradient_list([g, torch.ones(3, device="cuda")]), 1.0)
    assert str(norm.item()) == want and torch.isnan(scale).all()
    g.fill_(1.0)
    norm, scale = nv.grad_norm(nv.gradient_list([g]), 1.0)
    assert scale.item() < 1


def test_a_plan_of_another_kind_or_length_is_left_alone(gpu):
    """The kernels look at the plan's header: a call that does not belong to it changes nothing."""
    plan = make([100, 3000], "bf16", "bf16", 32, False)
    keep = [t.clone() for t in (*plan.params, plan.exp_avg, plan.exp_avg_sq, plan.control)]
    args = (plan.control, 1e-3, None, 0.9, 0.95, 1e-8, 0)
    nv.nvfp4_adamw(plan.table, plan.chunks, 8, *args)
    nv.nvfp4_adamw(plan.table, plan.chunks, 32, *args, amax=torch.zeros(1, device="cuda"), count=1)
    grads = nv.gradient_list(plan.grads)
    nv.nvfp4_adamw(grads.table, grads.chunks, 32, *args)
    torch.cuda.synchronize()
    for a, b in zip(keep, (*plan.params, plan.exp_avg, plan.exp_avg_sq, plan.control)):
        assert torch.equal(a, b)
    nv.adamw(plan, 1e-3)
    assert plan.steps() == 1 and not torch.equal(keep[1], plan.params[1])


# ---- how it is called ----------------------------------------------------------------------------

def test_refusals(gpu):
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    for call in (lambda: nv.adamw_plan([p], [g, g]), lambda: nv.adamw_plan([p], [g[:32]]), lambda: nv.adamw_plan([p.half()], [g]),
                 lambda: nv.adamw_plan([p], [g.half()]), lambda: nv.adamw_plan([p], [g.cpu()]), lambda: nv.adamw_plan([p[::2]], [g[:32]]),
                 lambda: nv.adamw_plan([p], [g], state_bits=16), lambda: nv.adamw_plan([p], [g], weight_decay=[0.1, 0.1]),
                 lambda: nv.adamw_plan([p], [g], betas=(0.9, 1.0)), lambda: nv.adamw_plan([p], [g], eps=float("nan")),
                 lambda: nv.adamw_plan([p], [g], seed=-1), lambda: nv.adamw_plan([p], [g], step=-1),
                 lambda: nv.adamw_plan([torch.zeros(0, device="cuda")], [torch.zeros(0, device="cuda")]),
                 lambda: nv.gradient_list([]), lambda: nv.adamw(nv.gradient_list([g]), 1e-3),
                 lambda: nv.adamw(nv.adamw_plan([p], [g]), torch.zeros(1)), lambda: nv.adamw(nv.adamw_plan([p], [g]), torch.zeros(2, device="cuda")),
                 lambda: nv.adamw(nv.adamw_plan([p], [g]), 1e-3, torch.zeros((), device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: nv.adamw_plan([p], [p]), lambda: nv.adamw_plan([p, p], [g, g]), lambda: nv.adamw_plan([p[:40], p[32:]], [g[:40], g[32:]]),
                 lambda: nv.adamw_plan([p], [g], weight_decay=float("nan")), lambda: nv.adamw(nv.adamw_plan([p], [g]), float("nan")),
                 lambda: nv.adamw(nv.adamw_plan([p], [g]), -1.0), lambda: nv.grad_norm(nv.gradient_list([g]), -1.0),
                 lambda: nv.grad_norm(nv.gradient_list([g]), float("nan"))):
        with pytest.raises(nv.Nvfp4Error):
            call()


@pytest.mark.parametrize("bits", [32, 8])
def test_side_stream_and_captured_steps(gpu, bits):
    """Three eager steps on a side stream, and one captured step replayed three times with new
    gradients and a new learning rate, give the bits of three plain ones."""
    def gradients(plan, k):
        for g in plan.grads:
            g.copy_(torch.sin(torch.arange(g.numel(), device="cuda") * (k + 1.0)))

    plain, side, captured = (make(LENGTHS, "bf16", "bf16", bits, bits == 32, seed=4) for _ in range(3))
    for k in range(3):
        gradients(plain, k)
        _, scale = nv.grad_norm(plain, 1.0)
        nv.adamw(plain, 1e-3 * (k + 1), scale)
    stream = torch.cuda.Stream()
    for k in range(3):
        gradients(side, k)
        stream.wait_stream(torch.cuda.current_stream())
        _, scale = nv.grad_norm(side, 1.0, stream=stream)
        nv.adamw(side, 1e-3 * (k + 1), scale, stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
    lr = torch.zeros(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, scale = nv.grad_norm(captured, 1.0)
        nv.adamw(captured, lr, scale)
    for k in range(3):
        gradients(captured, k)
        lr.fill_(1e-3 * (k + 1))
        graph.replay()
    for other in (side, captured):
        assert other.steps() == 3
        for a, b in zip((*plain.params, plain.exp_avg, plain.exp_avg_sq, plain.amax), (*other.params, other.exp_avg, other.exp_avg_sq, other.amax)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
