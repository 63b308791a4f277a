"""A call on another stream allocates its outputs and scratch as that stream's
memory: every allocation of the binding goes through one function, with the
call's stream. The library is replaced by a stand-in that launches nothing, so
no GPU is needed."""
import contextlib

import pytest
import torch

T, N_IN, N_OUT, GROUP = 5, 256, 64, 128


@pytest.fixture
def B(monkeypatch):
    from rotated_w4_linear_b200 import binding, build
    build.build()
    real = binding.lib()
    made = []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size") or name.endswith("_size_ex"):
                return getattr(real, name)
            return lambda *args: 0

    empty = torch.empty

    def recorded(shape, dtype, device, stream):
        made.append(stream)
        return empty(shape, dtype=dtype, device=device)

    def refuse(*args, **kwargs):
        raise AssertionError("allocated as the current stream's memory")

    monkeypatch.setattr(binding, "lib", Library)
    monkeypatch.setattr(binding, "_empty", recorded)
    monkeypatch.setattr(binding, "_dev", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(binding, "_stream", lambda stream, device=None: 0)
    monkeypatch.setattr(binding, "_on", lambda device: contextlib.nullcontext())
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, refuse)
    binding.made = made
    return binding


class Rot:                                                  # a handle-shaped stand-in
    handle, in_features, group = None, N_IN, GROUP


X = torch.ones(T, N_IN, dtype=torch.float16)
W = torch.ones(N_OUT, N_IN, dtype=torch.float16)
LOGICAL = (torch.ones(N_OUT, N_IN, dtype=torch.uint8), torch.ones(N_OUT, N_IN // GROUP, dtype=torch.float16),
           torch.ones(N_OUT, N_IN // GROUP, dtype=torch.uint8))
PACKED = tuple(torch.ones(n, dtype=torch.uint8) for n in (N_IN * N_OUT // 2, N_OUT * 2 * 2, N_OUT // 16 * 2 * 8))
SUMS, NORM = torch.ones(T, N_OUT), torch.ones(N_IN, dtype=torch.float16)
PAIRS = torch.zeros(0, 2, 64, 2, dtype=torch.int16).numpy()
THETA, ALPHA = torch.zeros(0, 2, 64).numpy(), torch.ones(N_IN).numpy()
CPU = torch.device("cpu")

CALLS = {                                                   # call, tensors it allocates
    "rotate": (lambda B, s: B.paro_rotate(Rot, X, stream=s), 1),
    "pack": (lambda B, s: B.paro_pack_weights(*LOGICAL, stream=s, device=CPU), 3),
    "pack_gated": (lambda B, s: B.paro_pack_gated(*LOGICAL, stream=s, device=CPU), 3),
    "dequant": (lambda B, s: B.paro_dequant(*PACKED, N_IN, N_OUT, stream=s), 1),
    "quantize": (lambda B, s: B.paro_quantize_weights(Rot, W, stream=s), 3),
    "linear": (lambda B, s: B.paro_linear(None, X, *PACKED, N_OUT, stream=s), 2),
    "bias": (lambda B, s: B.paro_linear_bias(None, X, *PACKED, None, N_OUT, stream=s), 2),
    "ex": (lambda B, s: B.paro_linear_ex(None, X, *PACKED, N_OUT, stream=s), 2),
    "partial": (lambda B, s: B.paro_linear_partial(None, X, *PACKED, N_OUT, stream=s), 2),
    "finalize": (lambda B, s: B.paro_finalize(SUMS, stream=s), 1),
    "noalloc": (lambda B, s: B.paro_linear_noalloc(None, X, *PACKED, N_OUT, stream=s), 1),
    "act": (lambda B, s: B.paro_linear_act(None, X, *PACKED, N_OUT, stream=s), 2),
    "gated": (lambda B, s: B.paro_linear_gated(None, X, *PACKED, N_OUT // 2, stream=s), 2),
    "rotate_once": (lambda B, s: B.paro_rotate_once(X, PAIRS, THETA, ALPHA, stream=s), 1),
    "linear_once": (lambda B, s: B.paro_linear_once(X, PAIRS, THETA, ALPHA, *PACKED, N_OUT, stream=s), 1),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocations_are_the_calls_stream(B, name):
    call, tensors = CALLS[name]
    for stream in (None, object()):
        B.made.clear()
        call(B, stream)
        assert len(B.made) == tensors and all(s is stream for s in B.made)
