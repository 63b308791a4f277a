"""Both forms of the CTA-pair GEMM, each at sizes that reach it (which
test_pair_plan_host.py checks): group sizes, biases, every activation, the
residual in place, and the rows behind the batch, against the 64-bit forms of
layer64 at its bars."""
import pytest
import torch

import layer64 as R
from pair_forms import SPLIT, WHOLE
from test_gpu_linear_act import ACTS, Layer, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    yield binding
    assert binding.paro_fault_status() == 0


def guarded(T, width, fill=7.0, behind=300):
    """[T + behind][width], of which a call gets the first T rows."""
    return torch.full((T + behind, width), fill, dtype=torch.float16, device="cuda")


@pytest.mark.parametrize("T,n_in,n_out,group", [(*size, group) for size in SPLIT + WHOLE for group in (64, 128, 256)
                                               if size[1] % group == 0])
def test_epilogues(B, T, n_in, n_out, group):
    L = Layer(B, T, n_in, n_out, group=group, rotated=T % 2 == 1, seed=T)
    G = B.paro_pack_gated(L.q, L.s, L.z, group=group)
    xr = L.xr()
    for k, act in enumerate(ACTS):
        bias, res = (L.bias if k != 3 else None), (L.residual if k != 1 else None)
        want, bound = R.linear_act(xr, L.w, act, bias, res)
        y = guarded(T, n_out)
        B.paro_linear_act(L.rot, L.x, *L.packed, n_out, act=act, group=group, bias=bias, residual=res, Y=y[:T])
        close(y[:T], want, bound)
        assert bool((y[T:] == 7).all()), "rows behind the batch"
        if res is not None:                                 # the residual in place: the same bits
            h = guarded(T, n_out)
            h[:T] = res
            B.paro_linear_act(L.rot, L.x, *L.packed, n_out, act=act, group=group, bias=bias, residual=h[:T], Y=h[:T])
            assert torch.equal(h, y)
        h = guarded(T, n_out // 2)
        B.paro_linear_gated(L.rot, L.x, *G, n_out // 2, act=act, group=group, bias=bias, H=h[:T])
        close(h[:T], *R.gated(xr, L.w, act, bias))
        assert bool((h[T:] == 7).all()), "rows behind the batch"


@pytest.mark.parametrize("T,n_in,n_out", SPLIT + WHOLE)
def test_a_channels_bias_is_its_own(B, T, n_in, n_out):
    """Zero weights: Y is the bias and the residual exactly, in every tile that a cluster walks."""
    L = Layer(B, T, n_in, n_out, rotated=False, seed=1)
    L.s.zero_()
    packed, G = B.paro_pack_weights(L.q, L.s, L.z), B.paro_pack_gated(L.q, L.s, L.z)
    y = B.paro_linear_act(None, L.x, *packed, n_out, bias=L.bias, residual=L.residual)
    assert torch.equal(y, (L.bias.float() + L.residual.float()).half())
    h = B.paro_linear_gated(None, L.x, *G, n_out // 2, act="none", bias=L.bias)
    gate, up = L.bias.float()[:n_out // 2], L.bias.float()[n_out // 2:]
    assert torch.equal(h, (gate * up).half().expand(T, -1))


@pytest.mark.parametrize("T,n_in,n_out", SPLIT + WHOLE)
def test_a_token_alone_and_in_its_batch(B, T, n_in, n_out):
    """Tokens in another order give the same rows, bit by bit."""
    L = Layer(B, T, n_in, n_out, rotated=False, seed=2)
    y = B.paro_linear_act(None, L.x, *L.packed, n_out, act="silu", bias=L.bias)
    order = torch.randperm(T, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))
    assert torch.equal(y[order], B.paro_linear_act(None, L.x[order].contiguous(), *L.packed, n_out, act="silu", bias=L.bias))
