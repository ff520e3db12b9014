"""How the training-step operators are called: derivatives, streams, gradients and versions."""
import gc
import subprocess
import sys
import textwrap

import pytest
import torch

import nvfp4_block_scaled_13_b200 as nv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def leave_no_garbage():
    """Tensors that a failed call's traceback still holds are freed here, not during a later test."""
    yield
    gc.collect()


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_derivatives_are_refused(gpu, which, grad):
    """A dual tensor need not require a gradient; its tangent must not be dropped in silence."""
    args = [torch.randn(3, 64, device="cuda"), torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")]
    want = nv.layer_norm(*args)
    with torch.autograd.forward_ad.dual_level(), torch.set_grad_enabled(grad):
        assert torch.equal(nv.layer_norm(*args), want)                   # inside a level, without a tangent
        dual = list(args)
        dual[which] = torch.autograd.forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        for with_amax in (False, True):
            with pytest.raises(RuntimeError, match="forward|jvp"):
                nv.layer_norm(*dual, with_amax=with_amax)
        with pytest.raises(RuntimeError, match="forward|jvp"):
            nv.fakequant_ste(torch.autograd.forward_ad.make_dual(args[0].bfloat16(), torch.ones_like(args[0].bfloat16())))
    for transform in (lambda f: torch.func.jvp(f, (args[0],), (args[0],)), lambda f: torch.func.vmap(f)(args[0]),
                      lambda f: torch.func.grad(lambda x: f(x).sum())(args[0])):
        with pytest.raises(RuntimeError):
            transform(lambda x: nv.layer_norm(x, *args[1:]))


@pytest.mark.parametrize("as_number", [False, True])
def test_inputs_are_held_for_a_side_stream(gpu, as_number):
    """An input that its caller drops while a side stream still has to read it keeps its memory."""
    n = 1 << 20
    plan = nv.adamw_plan([torch.zeros(64, device="cuda")], [torch.ones(64, device="cuda")])
    nv.adamw(plan, 0.0, torch.full((1,), float("nan"), device="cuda"))    # no step: it loads the kernel, which may outlast the delay below
    x = torch.randn(n // 64, 64, device="cuda")
    w, b = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    r = nv.layer_norm_forward(x, w, b)
    want = (r.y.clone(), *(t.clone() for t in nv.layer_norm_backward(x, x, w, r.mean, r.rstd)))
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_number else side

    def forward(x, w, b):
        return nv.layer_norm_forward(x, w, b, stream=stream).y

    def backward(dy, x, w, mean, rstd):
        return nv.layer_norm_backward(dy, x, w, mean, rstd, stream=stream)

    def step(lr, scale):
        nv.adamw(plan, lr, scale, stream=stream)

    for call, inputs in ((forward, (x, w, b)), (backward, (x, x, w, r.mean, r.rstd)),
                         (step, (torch.full((1,), 1e-3, device="cuda"), torch.ones(1, device="cuda")))):
        given = [t.clone() for t in inputs]
        at = {t.data_ptr() for t in given}
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)                                # about 100 ms in front of the call
        got = call(*given)
        sizes = [t.numel() for t in given]
        given.clear()
        new = [torch.full((k,), 7.0, device="cuda") for k in sizes for _ in range(2)]
        assert not at & {t.data_ptr() for t in new}, call.__name__
        torch.cuda.synchronize()
        del new
        if call is forward:
            assert torch.equal(got, want[0])
        elif call is backward:
            assert all(torch.equal(p, q) for p, q in zip(got, want[1:]))
    assert plan.steps() == 1 and torch.allclose(plan.params[0], torch.full((64,), -1e-3, device="cuda"))


def test_a_replaced_gradient_is_refused(gpu):
    """zero_grad() sets .grad to None and the next backward allocates another: the plan's would be applied again."""
    w = torch.nn.Parameter(torch.randn(64, device="cuda"))
    free = torch.zeros(64, device="cuda")                                # its gradient is nobody's .grad
    loss = lambda: (w * w).sum()  # noqa: E731
    loss().backward()
    plan = nv.adamw_plan([w, free], [w.grad, torch.ones(64, device="cuda")])
    optimizer = torch.optim.SGD([w], lr=0.0)

    def step():
        _, scale = nv.grad_norm(plan, 1.0)
        nv.adamw(plan, 1e-3, scale)

    step()
    optimizer.zero_grad(set_to_none=False)
    loss().backward()                                                     # accumulates in place
    step()
    assert plan.steps() == 2
    kept, before = w.grad, w.detach().clone()
    optimizer.zero_grad()
    for again in (False, True):
        if again:
            loss().backward()
        for call in (lambda: nv.adamw(plan, 1e-3), lambda: nv.grad_norm(plan, 1.0)):
            with pytest.raises(ValueError, match="grad"):
                call()
    assert plan.steps() == 2 and torch.equal(w.detach(), before)
    w.grad = kept
    step()
    assert plan.steps() == 3


@pytest.mark.parametrize("kind", ["plain", "later", "view", "view of a leaf", "inference"])
def test_every_graph_that_saved_a_parameter_notices_the_step(gpu, kind):
    """A parameter that requires no gradient itself, or requires one only after the plan was made."""
    x = torch.randn(64, device="cuda", requires_grad=True)
    if kind == "inference":
        with torch.inference_mode():
            p = torch.randn(64, device="cuda")
        nv.adamw(nv.adamw_plan([p], [torch.ones(64, device="cuda")]), 1e-3)   # has no version to count
        return
    flat = torch.randn(128, device="cuda", requires_grad=kind == "view of a leaf")
    p = flat[64:] if kind.startswith("view") else torch.randn(64, device="cuda")
    other = torch.randn(64, device="cuda")
    plan = nv.adamw_plan([p, other], [torch.ones(64, device="cuda") for _ in range(2)])
    if kind == "later":
        p.requires_grad_()
    y = (p * x).sum() + (other * x).sum()
    nv.adamw(plan, 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    fresh = (p * x).sum() + (other * x).sum()
    fresh.backward()
    assert torch.equal(x.grad, p.detach() + other)


COLD = textwrap.dedent("""
    import torch

    import nvfp4_block_scaled_13_b200 as nv

    x = torch.randn(300, 1029, device="cuda").bfloat16()
    w = torch.ones(1029, device="cuda").bfloat16()
    dy = (x * 1e-3).roll(1, 0).contiguous()
    p, g = torch.ones(5000, device="cuda"), torch.full((5000,), 0.5, device="cuda")
    plan = nv.adamw_plan([p], [g], state_bits=8, with_amax=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = nv.layer_norm_forward(x, w, w, with_amax=True)
        back = nv.layer_norm_backward(dy, x, w, r.mean, r.rstd)
        norm, scale = nv.grad_norm(plan, 1.0)
        nv.adamw(plan, 1e-3, scale)
    for _ in range(3):
        graph.replay()
    want = nv.layer_norm_forward(x, w, w, with_amax=True)
    assert all(torch.equal(a, b) for a, b in zip(r, want))
    assert all(torch.equal(a, b) for a, b in zip(back, nv.layer_norm_backward(dy, x, w, want.mean, want.rstd)))
    assert plan.steps() == 3 and abs(norm.item() - 0.5 * 5000 ** 0.5) < 1e-4 and plan.amax.item() == p.max().item() < 1
    print("done")
""")


def test_first_calls_in_a_process_are_captured(gpu):
    """Nothing has run before the capture: kernels are loaded and their shared memory allowed within it."""
    r = subprocess.run([sys.executable, "-c", COLD], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stderr[-2000:]


def test_two_plans_and_lists_on_two_streams(gpu):
    """Steps and norms that overlap on the GPU, each with a plan of its own, give what they give alone."""
    def made(k):
        gen = torch.Generator(device="cuda").manual_seed(k)
        params = [torch.randn(n, device="cuda", generator=gen).bfloat16() for n in (70001, 4096, 33)]
        grads = [torch.randn(p.numel(), device="cuda", generator=gen) for p in params]
        return nv.adamw_plan(params, grads, state_bits=8, with_amax=True, seed=k)

    def step(plan, stream=None):
        _, scale = nv.grad_norm(plan, 1.0, stream=stream)
        nv.adamw(plan, 1e-3, scale, stream=stream)

    alone, both = [made(k) for k in range(2)], [made(k) for k in range(2)]
    for _ in range(4):
        for plan in alone:
            step(plan)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(4):
        for plan, stream in zip(both, streams):
            step(plan, stream)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for p, q in zip((*a.params, a.exp_avg, a.exp_avg_sq, a.exp_avg_scale, a.exp_avg_sq_scale, a.amax),
                        (*b.params, b.exp_avg, b.exp_avg_sq, b.exp_avg_scale, b.exp_avg_sq_scale, b.amax)):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_another_tensor_over_the_same_gradient_is_accepted(gpu):
    w = torch.nn.Parameter(torch.ones(6, 8, device="cuda"))
    w.grad = torch.ones(6, 8, device="cuda")
    plan = nv.adamw_plan([w], [w.grad])
    w.grad = w.grad.detach()
    nv.adamw(plan, 1e-3)
    assert plan.steps() == 1
    w.grad = plan.grads[0].clone()
    with pytest.raises(ValueError, match="grad"):
        nv.adamw(plan, 1e-3)


@pytest.mark.parametrize("how", ["to", "data"])
def test_a_parameter_with_other_memory_is_refused(gpu, how):
    """The plan's table still points to the old memory, which must not have been given to somebody else."""
    module = torch.nn.Linear(64, 1 << 14, bias=False, device="cuda")
    w = module.weight
    g = torch.ones_like(w)
    plan = nv.adamw_plan([w], [g])
    grads = nv.gradient_list([g])
    nv.adamw(plan, 1e-3)
    at = {w.data_ptr(), g.data_ptr()}
    if how == "to":
        module.to(torch.bfloat16)
    else:
        w.data = w.data.clone()
    g.data = torch.zeros(0, device="cuda")
    assert w is module.weight
    new = [torch.zeros(64 << 14, device="cuda") for _ in range(3)]
    with pytest.raises(ValueError, match="memory"):
        nv.adamw(plan, 1e-3)
    assert not at & {t.data_ptr() for t in new} and grads.held[0].data_ptr() in at
    assert plan.steps() == 1
