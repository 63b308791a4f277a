"""A rotation handle used at once, on a stream that does not wait for the
default one."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("T", [3, 100])
def test_a_new_handle_on_another_stream(cuda_lib, T, group):
    from rotated_w4_linear_b200 import binding as B
    n_in = 4096
    x = torch.from_numpy(synth.activations(T, n_in, 1)).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for seed in range(4):
        rot = B.paro_rot_create(*synth.rotation_params(n_in, 8, seed, pairs_per_group=group // 2, group=group), group=group)
        first = B.paro_rotate(rot, x, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(first, B.paro_rotate(rot, x))
    assert B.paro_fault_status() == 0
