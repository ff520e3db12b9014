"""The training-step operators in a run, as a distillation step uses them: layer norm with its
amax, the fake-quantized projection of its result, the KL loss with its gradient, the backward
pass, the clip and the AdamW step, whose new weights' amax feeds the next fake-quantization."""
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

ROWS, HIDDEN, VOCAB = 48, 64, 160


class Student:
    def __init__(self, bits, masters, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.x = rand(ROWS, HIDDEN).bfloat16()
        self.teacher = rand(ROWS, VOCAB).bfloat16()
        self.params = [torch.ones(HIDDEN, device="cuda").bfloat16(), torch.zeros(HIDDEN, device="cuda").bfloat16(),
                       (rand(HIDDEN, HIDDEN) * 0.1).bfloat16(), (rand(VOCAB, HIDDEN) * 0.1).bfloat16()]
        for p in self.params:
            p.requires_grad_()
            p.grad = torch.zeros_like(p)
        self.plan = nv.adamw_plan(self.params, [p.grad for p in self.params], state_bits=bits, masters=masters,
                                  weight_decay=[0.0, 0.0, 0.1, 0.1], with_amax=True)
        for i, p in enumerate(self.params):
            self.plan.amax[i] = p.detach().abs().max()

    def forward_backward(self):
        for p in self.params:
            p.grad.zero_()
        weight, bias, w1, w2 = self.params
        top = self.plan.amax
        h, h_top = nv.layer_norm(self.x, weight, bias, with_amax=True)
        h = nv.fakequant_ste(h, amax_values=h_top) @ nv.fakequant_ste(w1, amax_values=top[2:3]).t()
        h2, h2_top = nv.layer_norm(h, weight, bias, with_amax=True)
        logits = nv.fakequant_ste(h2, amax_values=h2_top) @ nv.fakequant_ste(w2, amax_values=top[3:4]).t()
        kl, grad = nv.qad_kl(self.teacher, logits.detach())
        logits.backward(grad)
        return kl

    def step(self):
        kl = self.forward_backward()
        norm, scale = nv.grad_norm(self.plan, 0.05)
        nv.adamw(self.plan, 1e-3, scale)
        return kl, norm, scale


@pytest.mark.parametrize("bits,masters", [(32, True), (32, False), (8, False)])
def test_steps_in_a_run(gpu, bits, masters):
    s = Student(bits, masters)
    for step in range(3):
        kl = s.forward_backward()
        assert torch.isfinite(kl).all()
        grads = [p.grad.float().cpu().numpy().reshape(-1) for p in s.params]
        assert all(np.abs(g).max() > 0 for g in grads)
        norm, scale = nv.grad_norm(s.plan, 0.05)
        want = np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in grads))
        assert abs(norm.item() / want - 1) <= 6 * 2.0 ** -24
        olds = []
        for i, p in enumerate(s.params):
            st = {k: (t.view(torch.uint8) if t.element_size() == 1 else t).cpu().numpy() for k, t in s.plan.state(i).items()}
            m, v = st["exp_avg"], st["exp_avg_sq"]
            if bits == 8:
                m, v = (m, st["exp_avg_scale"]), (v, st["exp_avg_sq_scale"])
            olds.append((st["master"] if masters else p.detach().float().cpu().numpy().reshape(-1), m, v))
        nv.adamw(s.plan, 1e-3, scale)
        for i, ((old, m, v), g) in enumerate(zip(olds, grads)):
            w = R.adamw_bits(old, g, m, v, param_bf16=True, master=masters, bits=bits, lr=1e-3, decay=(0.0, 0.0, 0.1, 0.1)[i],
                             betas=s.plan.betas, eps=s.plan.eps, scale=scale.item(), steps=step, first=s.plan.offsets[i], seed=0)
            got = {k: (t.view(torch.uint8) if t.element_size() == 1 else t).cpu().numpy() for k, t in s.plan.state(i).items()}
            got["param"] = s.params[i].detach().float().cpu().numpy().reshape(-1)
            R.assert_step(got, w, bits)
            # the amax that the step wrote is the one the quantizer would take
            if s.params[i].dim() == 2:
                assert s.plan.amax[i].item() == nv.amax(s.params[i].detach()).item()


def test_gradient_of_the_norm_inside_the_step(gpu):
    """The first norm's weight gradient against the formula, through the straight-through projection."""
    s = Student(32, True, seed=3)
    weight, bias, w1, _ = s.params
    h, top = nv.layer_norm(s.x, weight, bias, with_amax=True)
    q = nv.fakequant_ste(h, amax_values=top)
    assert torch.equal(q.detach(), nv.fakequant(h.detach()).view_as(q))           # the amax is the quantizer's
    dy = torch.randn(ROWS, HIDDEN, device="cuda").bfloat16()
    q.backward(dy)
    r = nv.layer_norm_forward(s.x, weight.detach(), bias.detach())
    f64 = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    _, dw, db, xh, _ = R.norm_grad64(f64(dy), f64(s.x), f64(weight), f64(r.mean), f64(r.rstd))
    # one rounding to BF16, and a chain of at most ROWS additions
    size = np.abs(f64(dy) * xh).sum(0)
    assert (np.abs(f64(weight.grad) - dw) <= 2.0 ** -8 * np.abs(dw) + 100 * 2.0 ** -24 * size).all()
    assert (np.abs(f64(bias.grad) - db) <= 2.0 ** -8 * np.abs(db) + 100 * 2.0 ** -24 * np.abs(f64(dy)).sum(0)).all()


def test_inference_run_feeds_the_tensor_core_product(gpu):
    """One token and several: norm with amax, one-pass quantization, FP4 product."""
    w = (torch.randn(256, 256, device="cuda") * 0.05).bfloat16()
    wq = nv.quantize_for_gemm(w)
    weight = torch.ones(256, device="cuda").bfloat16()
    for rows in (1, 130):
        x = torch.randn(rows, 256, device="cuda").bfloat16()
        h, top = nv.layer_norm(x, weight, None, with_amax=True)
        a, b = nv.quantize_for_gemm(h, amax_values=top), nv.quantize_for_gemm(h)
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
        assert torch.equal(nv.gemm(a, wq), nv.gemm(b, wq))


def test_a_graph_that_saved_a_parameter_notices_the_step(gpu):
    p = torch.randn(64, device="cuda", requires_grad=True)
    p.grad = torch.zeros_like(p)
    plan = nv.adamw_plan([p], [p.grad])
    y = (p * p).sum()
    y.backward(retain_graph=True)
    nv.adamw(plan, 1e-3)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_a_step_leaves_no_memory_behind(gpu):
    """Without the cycle collector: what the norm, the clip and the step allocate is free after them."""
    s = Student(32, True)

    def step():
        for p in s.params:
            p.grad.zero_()
        y, _ = nv.layer_norm(s.x, s.params[0], s.params[1], with_amax=True)
        y.sum().backward()
        _, scale = nv.grad_norm(s.plan, 0.05)
        nv.adamw(s.plan, 1e-3, scale)

    step()
    gc.collect()
    gc.disable()
    try:
        before = torch.cuda.memory_allocated()
        for _ in range(3):
            step()
        assert torch.cuda.memory_allocated() == before
    finally:
        gc.enable()
