"""AdamW at the ends of its ranges, compared as in test_gpu_b_adamw.py with the same operations in numpy."""
import gc

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_13_b200 as nv
from tests import train_ref as R
from tests.test_gpu_b_adamw import raw, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def leave_no_garbage():
    """Tensors that a failed call's traceback still holds are freed here, not during a later test."""
    yield
    gc.collect()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("first", [0, (1 << 33) - 64, (1 << 34) - 64])
def test_random_words_follow_the_index_past_2_to_the_34(gpu, bits, first):
    """A tensor whose first element has a large index: the words take 32 bits of an index of eights."""
    n, steps = 200, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    p = (torch.randn(n, device="cuda", generator=gen) * 0.02).bfloat16()
    g = torch.randn(n, device="cuda", generator=gen) * 1e-3
    old = values(p).copy()
    dtype = torch.float32 if bits == 32 else torch.uint8
    m, v = torch.zeros(n, dtype=dtype, device="cuda"), torch.zeros(n, dtype=dtype, device="cuda")
    scales = [torch.ones(-(-n // 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
    record = nv.OptTensor(param=p.data_ptr(), grad=g.data_ptr(), exp_avg=m.data_ptr(), exp_avg_sq=v.data_ptr(), numel=n, first=first,
                          weight_decay=0.1, param_type=nv.TYPE_BF16, grad_type=nv.TYPE_F32, state_bits=bits)
    if bits == 8:
        record.exp_avg_scale, record.exp_avg_sq_scale = (s.data_ptr() for s in scales)
    array = (nv.OptTensor * 1)(record)
    size = nv.nvfp4_tensor_plan_bytes(array, 1)
    image = torch.empty(size, dtype=torch.uint8)
    chunks = nv.nvfp4_tensor_plan(array, 1, image.data_ptr(), size)
    control = torch.cat([torch.tensor([0.9 ** steps, 0.95 ** steps], dtype=torch.float64).view(torch.int32),
                         torch.tensor([steps, 0, 0, 0], dtype=torch.int32)]).cuda()
    nv.nvfp4_adamw(image.cuda(), chunks, bits, control, 1e-3, None, 0.9, 0.95, 1e-8, 7)
    zero = np.zeros(n, np.float32 if bits == 32 else np.uint8)
    state = (zero, np.ones(-(-n // 32), np.uint8)) if bits == 8 else zero
    want = R.adamw_bits(old, values(g), state, state, param_bf16=True, master=False, bits=bits, lr=1e-3, decay=0.1, betas=(0.9, 0.95),
                        eps=1e-8, scale=1.0, steps=steps, first=first, seed=7)
    got = {"param": values(p), "exp_avg": raw(m), "exp_avg_sq": raw(v)}
    if bits == 8:
        got["exp_avg_scale"], got["exp_avg_sq_scale"] = (raw(s) for s in scales)
    R.assert_step(got, want, bits)


@pytest.mark.parametrize("param,masters", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-30, 1e-12, 1e31])
def test_8_bit_states_with_an_eps_that_hides_nothing(gpu, param, masters, eps):
    """Gradients whose squares are at and below the smallest normal number, and an eps that a root
    flushed to zero would leave alone in the denominator: every bit is that of the rounded formula."""
    n = 4096 + 50
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = torch.exp2(torch.rand(n, device="cuda", generator=gen) * 20 - 70) * torch.sign(torch.randn(n, device="cuda", generator=gen))
    p = torch.randn(n, device="cuda", generator=gen).to(torch.bfloat16 if param == "bf16" else torch.float32)
    plan = nv.adamw_plan([p], [g], state_bits=8, masters=masters, eps=eps, betas=(0.9, 0.95), weight_decay=0.1, seed=5)
    for step in range(2):
        state = {k: raw(t) for k, t in plan.state(0).items()}
        old = values(plan.state(0)["master"] if masters else p).copy()
        m = R.decode(state["exp_avg"], state["exp_avg_scale"])
        root = R.decode(state["exp_avg_sq"], state["exp_avg_sq_scale"])
        # the step of 32-bit states, whose root and quotient are rounded, from the decoded ones
        want = R.adamw_bits(old, values(g), m, root * root, param_bf16=param == "bf16", master=masters, bits=32, lr=1e-3, decay=0.1,
                            betas=(0.9, 0.95), eps=eps, scale=1.0, steps=step, first=0, seed=5)
        nv.adamw(plan, 1e-3)
        got = {k: raw(t) for k, t in plan.state(0).items()}
        assert np.isfinite(values(p)).all() and (want["_root"] < 2.0 ** -63).any() and (want["_root"] > 0).all()
        np.testing.assert_array_equal(values(p), want["param"])
        if masters:
            np.testing.assert_array_equal(got["master"], want["master"])
        for name, (codes, scales) in (("exp_avg", R.encode_nearest(want["exp_avg"])),
                                      ("exp_avg_sq", R.encode_stochastic(want["_root"], want["_word"]))):
            np.testing.assert_array_equal(got[name], codes)
            np.testing.assert_array_equal(got[name + "_scale"], scales)
        assert (got["exp_avg_sq"] > 0).all(), "a positive root keeps a positive code"


@pytest.mark.parametrize("bits", [32, 8])
def test_a_list_of_empty_tensors_counts_its_steps(gpu, bits):
    """Through the C entry points (the wrapper refuses such a list)."""
    memory = torch.full((64,), 3.0, device="cuda")
    at = memory.data_ptr()
    array = (nv.OptTensor * 1)(nv.OptTensor(param=at, grad=at, exp_avg=at, exp_avg_sq=at, exp_avg_scale=at, exp_avg_sq_scale=at, numel=0,
                                            param_type=nv.TYPE_F32, grad_type=nv.TYPE_F32, state_bits=bits))
    size = nv.nvfp4_tensor_plan_bytes(array, 1)
    image = torch.empty(size, dtype=torch.uint8)
    chunks = nv.nvfp4_tensor_plan(array, 1, image.data_ptr(), size)
    control = torch.cat([torch.ones(2, dtype=torch.float64).view(torch.int32), torch.zeros(4, dtype=torch.int32)]).cuda()
    table = image.cuda()
    for _ in range(2):
        nv.nvfp4_adamw(table, chunks, bits, control, 1e-3, None, 0.5, 0.25, 1e-8, 0)
    assert control[4:].tolist() == [2, 0, 0, 0] and control[:4].view(torch.float64).tolist() == [0.25, 0.0625]
    assert (memory == 3).all()
