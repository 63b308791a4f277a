"""Layer calls with weights of another shape or group size than the call says:
refused by the binding, with the weights as they are packed on a GPU."""
import pytest
import torch

from test_gpu_linear_act import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    yield binding
    assert binding.paro_fault_status() == 0


def test_weights_of_another_shape_or_group(B):
    L = Layer(B, 4, 512, 64, rotated=False)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    other = Layer(B, 4, 256, 64, rotated=False)
    for call in (lambda: B.paro_linear_gated(None, L.x, *G, 64),              # 2 inter for inter
                 lambda: B.paro_linear_gated(None, L.x, *G, 32, group=64),
                 lambda: B.paro_linear_act(None, L.x, *L.packed, 64, group=64),
                 lambda: B.paro_linear_act(None, L.x, *L.packed, 80),
                 lambda: B.paro_linear_act(None, L.x, L.packed[0], *other.packed[1:], 64),
                 lambda: B.paro_linear_ex(None, L.x, *L.packed, 64, group=64),
                 lambda: B.ParoLinear(None, *L.packed, 512, 64, group=64),
                 lambda: B.ParoLinear(None, *L.packed, 512, 64, bias=torch.zeros(64, dtype=torch.float16)),
                 lambda: B.ParoLinear(None, *L.packed, 512, 64, device="cpu"),
                 lambda: B.paro_pack_weights(L.q, other.s, L.z)):
        with pytest.raises((ValueError, TypeError)):
            call()
    layer = B.ParoLinear(None, *L.packed, 512, 64, device="cuda")
    assert torch.equal(layer(L.x), B.paro_linear_act(None, L.x, *L.packed, 64))
