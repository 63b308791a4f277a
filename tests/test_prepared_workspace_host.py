"""The workspace of a prepared layer: as large as the largest batch and no
larger, an outgrown one kept only while a captured graph or another stream may
use it. The library and the tensors on a GPU are stand-ins."""
import pytest
import torch

N_IN, N_OUT = 256, 64


class Gpu:
    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, *shape, dtype=torch.float16):
        self.shape, self.dtype = shape, dtype

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return id(self)


class Machine:
    """The current stream, whether it is being captured, and the workspace of each call."""

    def __init__(self):
        self.stream, self.capturing, self.used = 7, False, []


@pytest.fixture
def machine(monkeypatch):
    from rotated_w4_linear_b200 import binding, build
    build.build()
    real, m = binding.lib(), Machine()

    class Library:
        def __getattr__(self, name):
            if name.endswith(("_size", "_size_ex")):
                return getattr(real, name)

            def call(*args):
                m.used.append(args[-3])                     # workspace, its size, stream
                assert args[-2] >= real_size(args[-6])
                return 0
            return call

    def real_size(tokens):
        return binding.paro_linear_workspace_size(tokens, N_IN, N_OUT)

    monkeypatch.setattr(binding, "lib", Library)
    monkeypatch.setattr(binding, "_empty", lambda shape, dtype, device, stream: Gpu(shape, dtype=dtype)
                        if isinstance(shape, int) else Gpu(*shape, dtype=dtype))
    monkeypatch.setattr(binding, "_dev", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(binding, "_raw_stream", lambda device: m.stream)
    monkeypatch.setattr(binding, "_stream", lambda stream, device=None: m.stream if stream is None else stream)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_is_capturing", lambda: m.capturing)
    m.binding = binding
    return m


def layer(m, gated=False):
    B = m.binding
    w = [Gpu(n, dtype=torch.uint8) for n in B.paro_pack_size(N_IN, 2 * N_OUT, 128)]
    return (B.ParoGated if gated else B.ParoLinear)(None, *w, N_IN, N_OUT)


def held(lay):
    return ([lay._ws] if lay._ws is not None else []) + lay._kept


@pytest.mark.parametrize("gated", [False, True])
def test_grows_to_the_batch_and_no_further(machine, gated):
    lay = layer(machine, gated)
    size = machine.binding.paro_linear_workspace_size
    for T in (8191, 8192, 17, 9000, 1):
        lay(Gpu(T, N_IN))
    assert [w.numel() for w in held(lay)] == [size(9000, N_IN, N_OUT)]


def test_a_captured_workspace_is_kept(machine):
    lay = layer(machine)
    lay(Gpu(20, N_IN))
    machine.capturing = True
    lay(Gpu(20, N_IN))
    captured = machine.used[-1]
    machine.capturing = False
    for T in (20, 100, 101, 300):
        lay(Gpu(T, N_IN))
    size = machine.binding.paro_linear_workspace_size
    assert captured in [w.data_ptr() for w in held(lay)]
    assert sorted(w.numel() for w in held(lay)) == [size(T, N_IN, N_OUT) for T in (20, 300)]
    machine.capturing = True                                # first use and growth inside a capture
    lay(Gpu(400, N_IN))
    machine.capturing = False
    lay(Gpu(500, N_IN))
    assert sorted(w.numel() for w in held(lay)) == [size(T, N_IN, N_OUT) for T in (20, 400, 500)]


def test_a_workspace_used_on_another_stream_is_kept(machine):
    lay = layer(machine)
    lay(Gpu(20, N_IN))
    machine.stream = 9
    lay(Gpu(10, N_IN))                                      # stream 9 on stream 7's memory
    machine.stream = 7
    lay(Gpu(30, N_IN))
    lay(Gpu(40, N_IN))                                      # the workspace for 30 was stream 7's alone
    size = machine.binding.paro_linear_workspace_size
    assert sorted(w.numel() for w in held(lay)) == [size(T, N_IN, N_OUT) for T in (20, 40)]
