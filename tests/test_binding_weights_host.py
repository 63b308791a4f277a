"""Packed weights that a layer call is given must hold what its shape and group
size make the kernels read, on the device of X, and the logical ones of a pack
what it packs: a mistake is a ValueError, not a read past a buffer. The checks
are the binding's own, so stand-ins for the tensors on a GPU do."""
import pytest
import torch

N_IN, N_OUT = 512, 64


class Gpu:
    """What the checks look at of a contiguous tensor on CUDA device `index`."""

    is_cuda = True

    def __init__(self, n, dtype=torch.uint8, index=0, shape=None):
        self.n, self.dtype, self.index, self.shape = n, dtype, index, shape or (n,)
        self.device = torch.device("cuda", index)

    def numel(self):
        return self.n

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


@pytest.fixture
def B(monkeypatch):
    from rotated_w4_linear_b200 import binding, build
    build.build()
    real = binding.lib()

    class Library:                                          # nothing is launched
        def __getattr__(self, name):
            if name.endswith(("_size", "_size_ex", "_last_error")):
                return getattr(real, name)
            return lambda *args: pytest.fail(f"{name} was reached")

    monkeypatch.setattr(binding, "lib", Library)
    monkeypatch.setattr(binding, "_dev", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(binding, "_any", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(binding, "_empty", lambda shape, dtype, device, stream: Gpu(1, dtype))
    return binding


def packed(B, rows=N_OUT, n_in=N_IN, group=128, index=0):
    return [Gpu(n, index=index) for n in B.paro_pack_size(n_in, rows, group)]


X = Gpu(4 * N_IN, torch.float16, shape=(4, N_IN))
LAYERS = {                                                  # call(weights, group) of 64 output rows
    "act": lambda B, w, group: B.paro_linear_act(None, X, *w, N_OUT, group=group),
    "gated": lambda B, w, group: B.paro_linear_gated(None, X, *w, N_OUT // 2, group=group),
    "ex": lambda B, w, group: B.paro_linear_ex(None, X, *w, N_OUT, group=group),
    "partial": lambda B, w, group: B.paro_linear_partial(None, X, *w, N_OUT, group=group),
    "dequant": lambda B, w, group: B.paro_dequant(*w, N_IN, N_OUT, group=group),
    "ParoLinear": lambda B, w, group: B.ParoLinear(None, *w, N_IN, N_OUT, group=group),
    "ParoGated": lambda B, w, group: B.ParoGated(None, *w, N_IN, N_OUT // 2, group=group),
    "linear": lambda B, w, group: B.paro_linear(None, X, *w, N_OUT),
    "bias": lambda B, w, group: B.paro_linear_bias(None, X, *w, None, N_OUT),
    "noalloc": lambda B, w, group: B.paro_linear_noalloc(None, X, *w, N_OUT),
}


@pytest.mark.parametrize("name", LAYERS)
def test_weights_too_small_for_the_call(B, name):
    call = LAYERS[name]
    for k, part in enumerate(("qweight", "scales", "zeros")):
        w = packed(B)
        w[k] = Gpu(w[k].n - 1)
        with pytest.raises(ValueError, match=part):
            call(B, w, 128)
    with pytest.raises(ValueError, match="qweight"):        # half the rows, as 2 inter given for inter
        call(B, packed(B, N_OUT // 2), 128)
    with pytest.raises(ValueError, match="scales"):         # another layer's scales
        call(B, packed(B)[:1] + packed(B, N_OUT // 2)[1:], 128)
    if name not in ("linear", "bias", "noalloc"):
        with pytest.raises(ValueError, match="scales"):     # packed in groups of 128, read in groups of 64
            call(B, packed(B), 64)


@pytest.mark.parametrize("name", LAYERS)
def test_weights_on_another_device(B, name):
    for k, part in enumerate(("qweight", "scales", "zeros")):
        if name in ("dequant", "ParoLinear", "ParoGated") and k == 0:
            continue                                        # their device is qweight's
        w = packed(B)
        w[k] = Gpu(w[k].n, index=1)
        with pytest.raises(ValueError, match=f"{part} is on cuda:1"):
            LAYERS[name](B, w, 128)


def test_prepared_layers_keep_to_one_device(B):
    bias = Gpu(N_OUT, torch.float16, index=1)
    with pytest.raises(ValueError, match="bias is on cuda:1"):
        B.ParoLinear(None, *packed(B), N_IN, N_OUT, bias=bias)
    with pytest.raises(ValueError, match="bias is on cuda:1"):
        B.ParoGated(None, *packed(B), N_IN, N_OUT // 2, bias=bias)
    with pytest.raises(ValueError, match="where its weights are"):
        B.ParoLinear(None, *packed(B), N_IN, N_OUT, device="cpu")


@pytest.mark.parametrize("pack", ["paro_pack_weights", "paro_pack_gated"])
def test_packs(B, pack):
    call = getattr(B, pack)

    def logical(**other):
        t = {"q": Gpu(N_OUT * N_IN, shape=(N_OUT, N_IN)),
             "s": Gpu(N_OUT * N_IN // 128, torch.float16, shape=(N_OUT, N_IN // 128)),
             "z": Gpu(N_OUT * N_IN // 128, shape=(N_OUT, N_IN // 128))}
        t.update(other)
        return t["q"], t["s"], t["z"]

    for name in ("s", "z"):
        with pytest.raises(ValueError):
            call(*logical(**{name: Gpu(N_OUT * N_IN // 256, shape=(N_OUT, N_IN // 256))}))
    for name, t in zip("qsz", logical()):
        away = Gpu(t.n, t.dtype, 1, t.shape)
        with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
            call(*logical(**{name: away}), device=torch.device("cuda", 0))
    with pytest.raises(B.ParoError):
        call(*logical(), group=0)


def test_host_weights_never_reach_the_library(monkeypatch):
    """The same calls on host tensors, with the real type checks."""
    from rotated_w4_linear_b200 import binding
    w = [torch.zeros(n, dtype=torch.uint8) for n in binding.paro_pack_size(N_IN, N_OUT, 128)]
    monkeypatch.setattr(binding, "_check", lambda *args: pytest.fail("the library was reached"))
    x = torch.zeros(4, N_IN, dtype=torch.float16)
    for call in (lambda: binding.paro_dequant(*w, N_IN, N_OUT), lambda: binding.paro_linear_act(None, x, *w, N_OUT),
                 lambda: binding.paro_linear_ex(None, x, *w, N_OUT), lambda: binding.ParoLinear(None, *w, N_IN, N_OUT),
                 lambda: binding.paro_dequant(None, *w[1:], N_IN, N_OUT)):
        with pytest.raises((TypeError, AttributeError)):
            call()
