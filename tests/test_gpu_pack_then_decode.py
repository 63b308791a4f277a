"""A decode call right behind the call that packs its weights, on the same
buffers as the weights before them."""
import pytest
import torch

from test_gpu_linear_act import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    yield binding
    assert binding.paro_fault_status() == 0


@pytest.mark.parametrize("T", [1, 16, 40])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_the_weights_just_packed(B, T, rotated, gated):
    n_in, n_out = 2048, 4096
    sets = [Layer(B, T, n_in, n_out, rotated=rotated, gated=gated, bias=False, seed=s) for s in (1, 2)]
    rot, x = sets[0].rot, sets[0].x
    L, f = B.lib(), B.paro_linear_gated if gated else B.paro_linear_act
    width = n_out // 2 if gated else n_out
    want = [f(rot, x, *s.packed, width, act="silu") for s in sets]
    buf = [torch.empty_like(t) for t in sets[0].packed]
    ys = [torch.empty_like(want[0]) for _ in range(40)]
    ws = B.workspace(T, n_in, n_out)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    for k, y in enumerate(ys):
        s = sets[k & 1]
        args = (s.q.data_ptr(), s.s.data_ptr(), s.z.data_ptr(), n_in)
        out = tuple(t.data_ptr() for t in buf)
        if gated:
            assert L.paro_pack_gated(*args, n_out // 2, 128, *out, stream) == 0
            f(rot, x, *buf, width, act="silu", H=y, ws=ws)
        else:
            assert L.paro_pack_weights_ex(*args, n_out, 128, *out, stream) == 0
            f(rot, x, *buf, width, act="silu", Y=y, ws=ws)
    torch.cuda.synchronize()
    for k, y in enumerate(ys):
        assert torch.equal(y, want[k & 1]), k
