"""The contraction on CTA pairs (paro_linear_act and paro_linear_gated above 16
tokens): what its two CTAs exchange, and what shares an SM with it."""
import pytest
import torch

import layer64 as R
from test_gpu_linear_act import Layer, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    yield binding
    assert binding.paro_fault_status() == 0


@pytest.mark.parametrize("T,n_in,n_out", [
    (17, 1024, 4096), (64, 2048, 528), (128, 14336, 512), (200, 4096, 1040),   # one tile per cluster
    (256, 128, 28672), (2000, 384, 8192), (600, 2048, 17408),                  # many tiles per cluster
])
def test_each_call_multiplies_its_own_tokens(B, T, n_in, n_out):
    """Calls in a row on inputs that differ in the tokens of one CTA of a pair
    (the first or the second half of each tile) or in all of them: every call
    gives the bits that its input gives alone, so the MMAs read what both CTAs
    loaded for this stage and nothing older. The input's own result is held to
    the 64-bit bars."""
    L = Layer(B, T, n_in, n_out, rotated=False, bias=True, seed=T)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    gen = torch.Generator(device="cuda").manual_seed(T)
    other = torch.randn(T, n_in, device="cuda", generator=gen).half()
    half = (torch.arange(T, device="cuda") // 16 % 2).bool()[:, None]
    inputs = [L.x, torch.where(half, other, L.x), torch.where(half, L.x, other), other]
    want = []
    for x in inputs:
        torch.cuda.synchronize()
        y = B.paro_linear_act(None, x, *L.packed, n_out, act="silu", bias=L.bias, residual=L.residual)
        h = B.paro_linear_gated(None, x, *G, n_out // 2, bias=L.bias)
        close(y, *R.linear_act(x, L.w, "silu", L.bias, L.residual))
        close(h, *R.gated(x, L.w, "silu", L.bias))
        want.append((y, h))
    y, h = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    ws = B.workspace(T, n_in, n_out)
    for k in range(60):
        i = (k * 7 + k // 4) % 4
        B.paro_linear_act(None, inputs[i], *L.packed, n_out, act="silu", bias=L.bias, residual=L.residual, Y=y, ws=ws)
        B.paro_linear_gated(None, inputs[i], *G, n_out // 2, bias=L.bias, H=h, ws=ws)
        assert torch.equal(y, want[i][0]) and torch.equal(h, want[i][1]), k


@pytest.mark.parametrize("T", [17, 40, 64])
def test_layers_with_tensor_memory_one_after_another(B, T):
    """Launches in a row that each allocate tensor memory, the second one before
    the first is done (programmatic dependents): the pair kernel and the
    single-CTA kernel's smallest form, unrotated, on one stream and on two."""
    n_in, n_out = 1024, 37888                               # 148 row tiles of 256: two rounds of pairs
    L = Layer(B, T, n_in, n_out, rotated=False, bias=False, seed=T)
    want, bound = R.linear_act(L.x, L.w, "none")
    one = B.paro_linear_act(None, L.x, *L.packed, n_out)
    two = B.paro_linear_ex(None, L.x, *L.packed, n_out)
    close(one, want, bound)
    close(two, want, bound)
    ys = [torch.empty_like(one) for _ in range(4)]
    side = torch.cuda.Stream()
    ws = [B.workspace(T, n_in, n_out) for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(100):
        B.paro_linear_act(None, L.x, *L.packed, n_out, Y=ys[0], ws=ws[0])
        B.paro_linear_ex(None, L.x, *L.packed, n_out, Y=ys[1], ws=ws[0])
        if k >= 50:
            B.paro_linear_ex(None, L.x, *L.packed, n_out, Y=ys[2], ws=ws[1], stream=side)
            B.paro_linear_act(None, L.x, *L.packed, n_out, Y=ys[3], ws=ws[1], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(ys[0], one) and torch.equal(ys[3], one)
    assert torch.equal(ys[1], two) and torch.equal(ys[2], two)
