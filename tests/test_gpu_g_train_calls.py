"""How the training-step operators are called: derivatives, streams, gradients and versions."""
import gc

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
