"""What a plan says of its list, without a GPU: its kind, where tensors have no element."""
import struct

import pytest

from tests.test_train_abi import plan, tensor

KINDS = {32: 2, 8: 3}
SCALES = dict(exp_avg_scale=1 << 30, exp_avg_sq_scale=1 << 31)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lengths", [[0], [0, 0], [0, 64], [64, 0]])
def test_kind_of_a_list_with_empty_tensors(bits, lengths):
    records = [tensor(n, (1 + i) << 40, grad=(1 + i) << 40 | 1 << 36, exp_avg=(1 + i) << 40 | 2 << 36, exp_avg_sq=(1 + i) << 40 | 3 << 36,
                      state_bits=bits, **SCALES) for i, n in enumerate(lengths)]
    status, image, _ = plan(records)
    assert status == 0
    _, kind, count, _ = struct.unpack_from("<4I", image)
    assert (kind, count) == (KINDS[bits], len(lengths))


@pytest.mark.parametrize("lengths", [[0, 0], [0, 64], [64, 0]])
def test_an_empty_tensor_with_other_states_is_refused(lengths):
    records = [tensor(n, (1 + i) << 40, state_bits=b, **SCALES) for i, (n, b) in enumerate(zip(lengths, (32, 8)))]
    assert plan(records)[0] == 7
