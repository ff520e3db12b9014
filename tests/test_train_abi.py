"""The training-step operators without a GPU: the library exports what their header declares and
refuses invalid arguments on the host; the plan of a list of tensors is a host function and is
checked whole; the references that the GPU tests use hold against independent statements."""
import ctypes
import os
import re
import struct

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_13_b200 as nv
from tests import train_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20
NAN, INF = float("nan"), float("inf")


def test_library_exports_the_header_and_the_binding_mirrors_it():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "nvfp4_train.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"NVFP4_API\s+[\w\s\*]+?\b(nvfp4_\w+)\s*\(", text)))
    assert names == ["nvfp4_adamw", "nvfp4_grad_norm", "nvfp4_layer_norm", "nvfp4_layer_norm_backward",
                     "nvfp4_layer_norm_workspace", "nvfp4_tensor_plan", "nvfp4_tensor_plan_bytes"]
    for n in names:
        assert hasattr(nv.load(), n) and hasattr(nv, n) and n in nv.__all__


@pytest.mark.parametrize("call,expected", [
    # nvfp4_layer_norm(x, x_type, weight, bias, w_type, rows, cols, eps, y, mean, rstd, amax, stream)
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 0, 1e-5, A, None, None, None, None), 2),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, -1, 8, 1e-5, A, None, None, None, None), 2),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 1, (1 << 30) + 1, 1e-5, A, None, None, None, None), 2),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 1 << 40, 1 << 30, 1e-5, A, None, None, None, None), 2),
    (lambda L: L.nvfp4_layer_norm(A, 2, A, A, 0, 4, 8, 1e-5, A, None, None, None, None), 7),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, -1, 4, 8, 1e-5, A, None, None, None, None), 7),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 8, -1e-5, A, None, None, None, None), 7),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 8, NAN, A, None, None, None, None), 7),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 8, INF, A, None, None, None, None), 7),
    (lambda L: L.nvfp4_layer_norm(None, 0, A, A, 0, 4, 8, 1e-5, A, None, None, None, None), 1),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 8, 1e-5, None, None, None, None, None), 1),
    (lambda L: L.nvfp4_layer_norm(A + 1, 0, A, A, 0, 4, 8, 1e-5, A, None, None, None, None), 3),
    (lambda L: L.nvfp4_layer_norm(A + 2, 1, A, A, 0, 4, 8, 1e-5, A, None, None, None, None), 3),
    (lambda L: L.nvfp4_layer_norm(A, 0, A + 2, A, 1, 4, 8, 1e-5, A, None, None, None, None), 3),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A + 1, 0, 4, 8, 1e-5, A, None, None, None, None), 3),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 8, 1e-5, A, A + 2, None, None, None), 3),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 8, 1e-5, A, None, A + 2, None, None), 3),
    (lambda L: L.nvfp4_layer_norm(A, 0, A, A, 0, 4, 8, 1e-5, A, None, None, A + 2, None), 3),
    (lambda L: L.nvfp4_layer_norm(None, 0, None, None, 0, 0, 8, 1e-5, None, None, None, None, None), 0),
    # nvfp4_layer_norm_backward(dy, x, x_type, weight, w_type, mean, rstd, rows, cols, dx, dw, db, work, bytes, stream)
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, A, 4, 0, A, A, A, A, 1 << 30, None), 2),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, A, -4, 8, A, A, A, A, 1 << 30, None), 2),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 3, A, 0, A, A, 4, 8, A, A, A, A, 1 << 30, None), 7),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 2, A, A, 4, 8, A, A, A, A, 1 << 30, None), 7),
    (lambda L: L.nvfp4_layer_norm_backward(None, A, 0, A, 0, A, A, 4, 8, A, A, A, A, 1 << 30, None), 1),
    (lambda L: L.nvfp4_layer_norm_backward(A, None, 0, A, 0, A, A, 4, 8, A, A, A, A, 1 << 30, None), 1),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, None, A, 4, 8, A, A, A, A, 1 << 30, None), 1),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, None, 4, 8, A, A, A, A, 1 << 30, None), 1),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, A, 4, 8, None, A, A, A, 1 << 30, None), 1),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, A, 4, 8, A, A, A, None, 1 << 30, None), 1),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, A, 4, 8, A, A, A, A, 16, None), 2),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, A, 4, 8, A, A, A, A + 4, 1 << 30, None), 3),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A, A, 4, 8, A + 1, A, A, A, 1 << 30, None), 3),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 1, A, A, 4, 8, A, A + 2, A, A, 1 << 30, None), 3),
    (lambda L: L.nvfp4_layer_norm_backward(A, A, 0, A, 0, A + 2, A, 4, 8, A, A, A, A, 1 << 30, None), 3),
    (lambda L: L.nvfp4_layer_norm_backward(None, None, 0, None, 0, None, None, 0, 8, None, None, None, None, 0, None), 0),
    # nvfp4_grad_norm(plan, chunks, max_norm, norm, scale, workspace, stream)
    (lambda L: L.nvfp4_grad_norm(None, 1, 1.0, A, A, A, None), 1),
    (lambda L: L.nvfp4_grad_norm(A, 1, 1.0, None, A, A, None), 1),
    (lambda L: L.nvfp4_grad_norm(A, 1, 1.0, A, None, A, None), 1),
    (lambda L: L.nvfp4_grad_norm(A, 1, 1.0, A, A, None, None), 1),
    (lambda L: L.nvfp4_grad_norm(A, -1, 1.0, A, A, A, None), 2),
    (lambda L: L.nvfp4_grad_norm(A, 1, -1.0, A, A, A, None), 7),
    (lambda L: L.nvfp4_grad_norm(A, 1, NAN, A, A, A, None), 7),
    (lambda L: L.nvfp4_grad_norm(A + 8, 1, 1.0, A, A, A, None), 3),
    (lambda L: L.nvfp4_grad_norm(A, 1, 1.0, A + 2, A, A, None), 3),
    (lambda L: L.nvfp4_grad_norm(A, 1, 1.0, A, A, A + 8, None), 3),
    # nvfp4_adamw(plan, chunks, state_bits, control, lr, lr_device, beta1, beta2, eps, seed, scale, amax, count, stream)
    (lambda L: L.nvfp4_adamw(A, 1, 16, A, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 7),
    (lambda L: L.nvfp4_adamw(None, 1, 32, A, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 1),
    (lambda L: L.nvfp4_adamw(A, 1, 32, None, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 1),
    (lambda L: L.nvfp4_adamw(A, -1, 32, A, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 2),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, A, -1, None), 2),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, -1e-3, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 7),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, INF, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 7),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, None, 1.0, 0.99, 1e-8, 0, None, None, 0, None), 7),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, None, 0.9, -0.1, 1e-8, 0, None, None, 0, None), 7),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, None, 0.9, NAN, 1e-8, 0, None, None, 0, None), 7),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, None, 0.9, 0.99, -1.0, 0, None, None, 0, None), 7),
    (lambda L: L.nvfp4_adamw(A + 8, 1, 32, A, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 3),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A + 4, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 3),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, A + 2, 0.9, 0.99, 1e-8, 0, None, None, 0, None), 3),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, None, 0.9, 0.99, 1e-8, 0, A + 1, None, 0, None), 3),
    (lambda L: L.nvfp4_adamw(A, 1, 32, A, 1e-3, None, 0.9, 0.99, 1e-8, 0, None, A + 2, 1, None), 3),
])
def test_invalid_arguments_rejected_on_host(call, expected):
    assert call(nv.load()) == expected


def test_workspace_of_an_empty_and_of_an_invalid_shape():
    assert nv.nvfp4_layer_norm_workspace(0, 8) == 0
    assert nv.nvfp4_layer_norm_workspace(4, 0) == -1 and nv.nvfp4_layer_norm_workspace(-1, 8) == -1
    for rows, cols in ((1, 1), (5, 1000), (100000, 64), (3, 8192), (7, 40000)):
        size = nv.nvfp4_layer_norm_workspace(rows, cols)
        parts = size // (8 * cols)
        assert size == parts * 8 * cols and 1 <= parts <= rows


# ---- the plan of a list -------------------------------------------------------------------------

def tensor(n=64, at=A, **kw):
    d = dict(param=at, grad=at + (1 << 24), exp_avg=at + (2 << 24), exp_avg_sq=at + (3 << 24), numel=n, first=0,
             weight_decay=0.1, param_type=0, grad_type=0, state_bits=32)
    d.update(kw)
    return nv.OptTensor(**d)


def plan(records):
    array = (nv.OptTensor * max(1, len(records)))(*records)
    size = nv.nvfp4_tensor_plan_bytes(array, len(records))
    if size < 0:
        return 2, None, 0
    image = ctypes.create_string_buffer(size + 64)
    image[size:] = b"\xa5" * 64
    chunks = ctypes.c_int64()
    status = nv.load().nvfp4_tensor_plan(array, len(records), image, size, ctypes.byref(chunks))
    assert image.raw[size:] == b"\xa5" * 64, "written past the image"
    return status, image.raw[:size], chunks.value


@pytest.mark.parametrize("lengths", [[1], [0, 5, 0], [2048, 2049, 4096, 7], [3_000_001, 64], [150_000_000, 33_554_432, 17]])
def test_plan_covers_every_element_once(lengths):
    records = []
    for i, n in enumerate(lengths):
        at = (1 + i) << 40
        records.append(tensor(n, at, grad=at + (1 << 36), exp_avg=at + (2 << 36), exp_avg_sq=at + (3 << 36)))
    status, image, chunks = plan(records)
    assert status == 0
    magic, kind, count, n_chunks, length = struct.unpack_from("<5I", image)
    assert kind == 2 and count == len(lengths) and n_chunks == chunks and length % 2048 == 0
    covered = [0] * count
    at = 32
    assert len(image) == 32 + (8 * chunks + 15) // 16 * 16 + count * 104
    for c in range(chunks):
        t, index = struct.unpack_from("<2I", image, at + 8 * c)
        assert index * length == covered[t], "a tensor's chunks come in order"
        covered[t] = min(lengths[t], covered[t] + length)
    assert covered == lengths


def test_plan_of_gradients_alone():
    status, image, chunks = plan([nv.OptTensor(grad=A, numel=100, grad_type=1), nv.OptTensor(grad=A, numel=100, grad_type=1)])
    assert status == 0 and chunks == 2 and struct.unpack_from("<2I", image)[1] == 1   # reads may share memory


@pytest.mark.parametrize("records,expected", [
    ([tensor(grad=None)], 1),
    ([tensor(exp_avg=None)], 1),
    ([tensor(exp_avg_sq=None)], 1),
    ([tensor(state_bits=8, exp_avg_scale=1 << 30)], 1),
    ([tensor(-1)], 2),
    ([tensor(1 << 34)], 2),
    ([tensor(1 << 33, A), tensor(1 << 33, 1 << 45)], 2),
    ([tensor(first=4)], 2),
    ([tensor(first=-8)], 2),
    ([tensor(param=A + 1)], 3),
    ([tensor(param_type=1, param=A + 2)], 3),
    ([tensor(grad=A + (1 << 24) + 1)], 3),
    ([tensor(exp_avg=A + (2 << 24) + 2)], 3),
    ([tensor(master=(9 << 24) + 2)], 3),
    ([tensor(param_type=2)], 7),
    ([tensor(grad_type=-1)], 7),
    ([tensor(state_bits=16)], 7),
    ([tensor(weight_decay=NAN)], 7),
    ([tensor(param_type=1, master=9 << 24)], 7),
    ([tensor(), nv.OptTensor(grad=1 << 40, numel=8)], 7),            # both kinds in one list
    ([tensor(), tensor(at=1 << 40, state_bits=8, exp_avg_scale=1 << 30, exp_avg_sq_scale=1 << 31)], 7),   # both kinds of state
    ([tensor(), tensor()], 7),                                         # the same tensor twice
    ([tensor(), tensor(at=A + 64)], 7),                               # overlapping parameters
    ([tensor(grad=A)], 7),                                             # a gradient over its parameter
    ([tensor(exp_avg_sq=A + (2 << 24) + 128)], 7),                    # states over one another
    ([tensor(state_bits=8, exp_avg_scale=1 << 30, exp_avg_sq_scale=(1 << 30) + 1)], 7),
])
def test_plan_refuses(records, expected):
    assert plan(records)[0] == expected


def test_plan_refuses_a_short_image_and_null():
    array = (nv.OptTensor * 1)(tensor())
    size = nv.nvfp4_tensor_plan_bytes(array, 1)
    image, chunks = ctypes.create_string_buffer(size), ctypes.c_int64()
    L = nv.load()
    assert L.nvfp4_tensor_plan(array, 1, image, size - 1, ctypes.byref(chunks)) == 2
    assert L.nvfp4_tensor_plan(array, 1, None, size, ctypes.byref(chunks)) == 1
    assert L.nvfp4_tensor_plan(array, 1, image, size, None) == 1
    assert L.nvfp4_tensor_plan(None, 1, image, size, ctypes.byref(chunks)) == 2
    assert L.nvfp4_tensor_plan_bytes(array, -1) == -1 and L.nvfp4_tensor_plan_bytes(array, 1 << 24) == -1
    # neighbours that touch do not overlap
    assert plan([tensor(64), tensor(64, A + 256)])[0] == 0


@pytest.mark.parametrize("call", [
    lambda: nv.layer_norm(torch.zeros(4, 8)),
    lambda: nv.layer_norm_forward(torch.zeros(4, 8, dtype=torch.bfloat16)),
    lambda: nv.layer_norm_backward(torch.zeros(4, 8), torch.zeros(4, 8), None, torch.zeros(4), torch.zeros(4)),
    lambda: nv.gradient_list([torch.zeros(4)]),
    lambda: nv.gradient_list([]),
    lambda: nv.adamw_plan([torch.zeros(4)], [torch.zeros(4)]),
    lambda: nv.adamw_plan([], []),
    lambda: nv.adamw(None, 1e-3),
])
def test_wrappers_refuse_what_is_not_on_a_gpu(call):
    with pytest.raises(ValueError):
        call()


# ---- the references ------------------------------------------------------------------------------

def test_reference_e4m3_matches_torch():
    x = torch.cat([torch.randn(20000) * s for s in (0.01, 1.0, 60.0)]).clamp(-448, 448)
    x = torch.cat([x, torch.tensor([0.0, -0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10, 2.0 ** -10 * 1.0001, 1.0625, 1.1875])])
    np.testing.assert_array_equal(R.e4m3_nearest(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    codes = np.arange(256, dtype=np.uint8)
    np.testing.assert_array_equal(R.E4M3, torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy())


def test_reference_blocks_fill_the_grid():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(4096) * np.exp(rng.uniform(-60, 60, 4096))).astype(np.float32)
    top = np.abs(x.reshape(-1, 32)).max(1).astype(np.float64) / 2.0 ** (R.scale_bytes(x).astype(np.float64) - 127)
    assert (top > 224).all() and (top <= 448).all()


def test_reference_random_words_are_even():
    w = R.words(1 << 16, 0, 7, 3)
    for half in (w >> np.uint64(16), w & np.uint64(0xFFFF)):
        # mean of 65536 uniform values: 6 standard deviations of an independent sample
        assert abs(half.mean() / 65536 - 0.5) < 6 * (1 / 12) ** 0.5 / 256
    assert len(np.unique(R.words(1 << 12, 0, 7, 3))) > 4090 and (R.words(64, 0, 7, 3) != R.words(64, 0, 7, 4)).any()


def test_reference_step_in_32_bits_follows_the_definition():
    rng = np.random.default_rng(2)
    n = 1000
    p, g, m = (rng.standard_normal(n).astype(np.float32) * s for s in (0.02, 1e-3, 3e-4))
    v = (rng.uniform(0.5, 2, n) * 1e-6).astype(np.float32)
    kw = dict(lr=1e-3, decay=0.1, betas=(0.9, 0.99), eps=1e-8, scale=0.7, steps=4)
    got = R.adamw_bits(p, g, m, v, param_bf16=False, master=False, bits=32, first=0, seed=0, **kw)
    want = R.adamw64(p, g, m, v, **kw)
    # a dozen roundings of 2^-24 each
    assert np.abs(got["param"] - want[0]).max() < 12 * 2.0 ** -24 * np.abs(p).max()
    assert (np.abs(got["exp_avg_sq"] - want[2]) <= 12 * 2.0 ** -24 * want[2]).all()
