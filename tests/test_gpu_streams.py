"""Calls on another stream than the current one that allocate their outputs
and scratch themselves."""
import pytest
import torch

import synth
from test_gpu_linear_act import Layer

pytestmark = pytest.mark.gpu
T, N_IN, N_OUT = 300, 1024, 512


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    yield binding
    assert binding.paro_fault_status() == 0


@pytest.fixture(scope="module")
def L(B):
    return Layer(B, T, N_IN, N_OUT, seed=8)


def calls(B, L):
    """name -> (call(stream), bytes of what it allocates)."""
    ws = B.paro_linear_workspace_size(T, N_IN, N_OUT)
    packed = tuple(t.numel() for t in L.packed)
    w = (0.02 * torch.randn(N_OUT, N_IN, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))).half()
    sums = torch.randn(T, N_OUT, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    rotation = synth.rotation_params(N_IN, 3, 13, pairs_per_group=64, group=128)
    few, y = L.x[:9], 2 * T * N_OUT
    return {
        "linear": (lambda st: B.paro_linear(L.rot, L.x, *L.packed, N_OUT, stream=st), (y, ws)),
        "bias": (lambda st: B.paro_linear_bias(L.rot, L.x, *L.packed, L.bias, N_OUT, stream=st), (y, ws)),
        "ex": (lambda st: B.paro_linear_ex(L.rot, L.x, *L.packed, N_OUT, bias=L.bias, stream=st), (y, ws)),
        "partial": (lambda st: B.paro_linear_partial(L.rot, L.x, *L.packed, N_OUT, stream=st), (2 * y, ws)),
        "decode": (lambda st: B.paro_linear(L.rot, few, *L.packed, N_OUT, stream=st), (2 * 9 * N_OUT, 2 * 9 * N_IN)),
        "noalloc": (lambda st: B.paro_linear_noalloc(L.rot, few, *L.packed, N_OUT, stream=st), (2 * 9 * N_OUT,)),
        "finalize": (lambda st: B.paro_finalize(sums, L.bias, stream=st), (y,)),
        "rotate": (lambda st: B.paro_rotate(L.rot, L.x, stream=st), (2 * T * N_IN,)),
        "pack": (lambda st: B.paro_pack_weights(L.q, L.s, L.z, stream=st), packed),
        "pack_gated": (lambda st: B.paro_pack_gated(L.q, L.s, L.z, stream=st), packed),
        "dequant": (lambda st: B.paro_dequant(*L.packed, N_IN, N_OUT, stream=st), (2 * N_IN * N_OUT,)),
        "quantize": (lambda st: B.paro_quantize_weights(L.rot, w, stream=st),
                     (N_IN * N_OUT, 2 * N_OUT * N_IN // 128, N_OUT * N_IN // 128)),
        "rotate_once": (lambda st: B.paro_rotate_once(L.x, *rotation, stream=st), (2 * T * N_IN,)),
        "linear_once": (lambda st: B.paro_linear_once(L.x, *rotation, *L.packed, N_OUT, stream=st), (y,)),
    }


def each(v):
    return v if isinstance(v, tuple) else (v,)


def test_outputs_and_scratch_do_not_take_memory_still_in_use(B, L):
    """Tensors freed while the current stream still has work on them do not
    become the outputs or the workspace of a call on another stream, and no
    workspace is filled on the current stream after the call has started."""
    st = torch.cuda.Stream()
    for name, (call, sizes) in calls(B, L).items():
        want = call(None)
        torch.cuda.synchronize()
        for stream in (st, st.cuda_stream):
            held = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in sizes]
            st.synchronize()
            torch.cuda._sleep(20_000_000)                   # about 10 ms: the copies below come after the call
            copies = [h.clone() for h in held]
            del held
            got = call(stream)
            torch.cuda.synchronize()
            assert all(bool((c == 77).all()) for c in copies), name
            for g, e in zip(each(got), each(want)):
                assert torch.equal(g.view(torch.uint8), e.view(torch.uint8)), name


def test_scratch_is_not_handed_out_while_its_stream_uses_it(B, L):
    """Memory asked for on the current stream right after the call is not the
    call's scratch: bytes of 255, which are NaN in fp16, would show in Y."""
    st = torch.cuda.Stream()
    n = B.paro_linear_workspace_size(T, N_IN, N_OUT)
    for name, (call, _) in calls(B, L).items():
        if name not in ("linear", "bias", "ex", "partial", "decode"):
            continue
        want = call(None)
        torch.cuda.synchronize()
        got = []
        for _ in range(30):
            got.append(call(st))
            torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got), name
