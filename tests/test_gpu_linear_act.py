"""paro_linear_act and paro_linear_gated against the 64-bit forms of layer64
(bars derived there), over token counts of every kernel (decode tiles of 8 and
16 tokens, prefill tiles of 64, 128 and, on CTA pairs, 256), odd widths, group
sizes, activations, biases and residuals."""
import numpy as np
import pytest
import torch

import layer64 as R
import synth
from oracle import paro_oracle as O

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    yield binding
    assert binding.paro_fault_status() == 0


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    """Inputs of one layer on the device, its packed weights and rotation."""

    def __init__(self, B, T, n_in, n_out, group=128, rotated=True, bias=True, gated=False, seed=0, K=3):
        rng = np.random.default_rng([T, n_in, n_out, seed])
        self.x = dev(synth.activations(T, n_in, seed + 1))
        q, s, z = synth.w4_codes(n_out, n_in, seed + n_out, group)
        self.q, self.s, self.z = dev(q), dev(s), dev(z)
        self.bias = dev((0.5 * rng.standard_normal(n_out)).astype(np.float16)) if bias else None
        self.rot = B.paro_rot_create(*synth.rotation_params(n_in, K, seed + 5, pairs_per_group=group // 2, group=group),
                                     group=group) if rotated else None
        pack = B.paro_pack_gated if gated else B.paro_pack_weights
        self.packed = pack(self.q, self.s, self.z, group=group)
        self.w = R.w_hat(self.q, self.s, self.z, group)
        self.B, self.group, self.n_out, self.n_in = B, group, n_out, n_in
        self.residual = dev((3 * rng.standard_normal((T, n_out))).astype(np.float16))

    def xr(self, x=None):
        x = self.x if x is None else x
        return self.B.paro_rotate(self.rot, x) if self.rot is not None else x


def close(got, want, bound):
    err = (got.double() - want).abs()
    worst = (err - bound).max().item()
    assert bool((err <= bound).all()), f"worst excess {worst:.3e}, largest error {err.max().item():.3e}"


TOKENS = [1, 2, 7, 8, 9, 13, 16, 17, 40, 64, 65, 100, 128, 129, 200, 256, 257, 385, 513]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("n_in,n_out", [(384, 272), (128, 16), (1024, 1040)])
def test_linear_act(B, T, n_in, n_out):
    L = Layer(B, T, n_in, n_out, seed=T)
    xr = L.xr()
    for k, act in enumerate(ACTS):
        bias = L.bias if k % 2 == 0 else None
        res = L.residual if k != 1 else None
        y = B.paro_linear_act(L.rot, L.x, *L.packed, n_out, act=act, bias=bias, residual=res)
        close(y, *R.linear_act(xr, L.w, act, bias, res))


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("n_in,inter", [(384, 136), (128, 8), (1024, 520)])
def test_gated(B, T, n_in, inter):
    L = Layer(B, T, n_in, 2 * inter, gated=True, seed=T)
    xr = L.xr()
    for k, act in enumerate(ACTS):
        bias = L.bias if k % 2 == 0 else None
        h = B.paro_linear_gated(L.rot, L.x, *L.packed, inter, act=act, bias=bias)
        close(h, *R.gated(xr, L.w, act, bias))


@pytest.mark.parametrize("group", [64, 256])
@pytest.mark.parametrize("rotated", [False, True])
@pytest.mark.parametrize("T", [1, 11, 33, 128, 130, 300])
def test_group_sizes(B, T, group, rotated):
    L = Layer(B, T, 768, 400, group=group, rotated=rotated, seed=T)
    y = B.paro_linear_act(L.rot, L.x, *L.packed, 400, act="silu", group=group, bias=L.bias, residual=L.residual)
    close(y, *R.linear_act(L.xr(), L.w, "silu", L.bias, L.residual))
    G = Layer(B, T, 768, 400, group=group, rotated=rotated, gated=True, seed=T)
    h = B.paro_linear_gated(G.rot, G.x, *G.packed, 200, act="gelu", group=group, bias=G.bias)
    close(h, *R.gated(G.xr(), G.w, "gelu", G.bias))


@pytest.mark.parametrize("T,n_in,n_out", [
    (1, 14336, 4096), (16, 4096, 4096), (5, 17408, 5120),     # decode: split k, deep chunks
    (3, 256, 17408), (16, 2560, 19456),                       # wide: one k chunk, several row blocks per warp
    (40, 14336, 4096), (100, 4096, 6144), (77, 2560, 9744),   # prefill, split channels
    (200, 4096, 28672), (256, 4096, 4096), (500, 9728, 2560),
    (2048, 4096, 4096), (1000, 14336, 2576), (300, 5120, 34832),
    (2000, 384, 8192), (3000, 128, 4096), (1500, 640, 9728),  # an odd number of stages in each of a cluster's tiles
])
def test_layer_sizes(B, T, n_in, n_out):
    L = Layer(B, T, n_in, n_out, seed=3, bias=False)
    close(B.paro_linear_act(L.rot, L.x, *L.packed, n_out, residual=L.residual), *R.linear_act(L.xr(), L.w, "none", None, L.residual))
    G = B.paro_pack_gated(L.q, L.s, L.z)
    close(B.paro_linear_gated(L.rot, L.x, *G, n_out // 2), *R.gated(L.xr(), L.w, "silu"))


def test_gated_pack_is_the_interleaved_pack(B):
    """paro_pack_gated of (gate, up) is paro_pack_weights_ex of the rows in
    blocks of eight and eight, bit by bit, from device and from host memory."""
    for n_in, inter, group in ((256, 40, 128), (384, 8, 64), (512, 24, 256)):
        q, s, z = synth.w4_codes(2 * inter, n_in, 9, group)
        rows = np.arange(inter).reshape(-1, 8)
        order = np.concatenate([rows, rows + inter], axis=1).reshape(-1)
        want = B.paro_pack_weights(dev(q[order]), dev(s[order]), dev(z[order]), group=group)
        for got in (B.paro_pack_gated(dev(q), dev(s), dev(z), group=group),
                    B.paro_pack_gated(torch.from_numpy(q), torch.from_numpy(s), torch.from_numpy(z), group=group)):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [3, 16, 90, 400])
def test_plain_epilogue_agrees_with_the_layer(B, T):
    """act none without a residual is paro_linear_ex; H with act none is the product of its halves."""
    L = Layer(B, T, 640, 352, seed=T)
    y = B.paro_linear_act(L.rot, L.x, *L.packed, 352, bias=L.bias)
    want, bound = R.linear_act(L.xr(), L.w, "none", L.bias)
    close(y, want, bound)
    close(B.paro_linear_ex(L.rot, L.x, *L.packed, 352, bias=L.bias), want, bound)


@pytest.mark.parametrize("T", [1, 9, 16, 100, 129, 700])
def test_residual_in_place(B, T):
    L = Layer(B, T, 512, 656, seed=T)
    y = B.paro_linear_act(L.rot, L.x, *L.packed, 656, act="gelu_tanh", bias=L.bias, residual=L.residual)
    h = L.residual.clone()
    assert B.paro_linear_act(L.rot, L.x, *L.packed, 656, act="gelu_tanh", bias=L.bias, residual=h, Y=h) is h
    assert torch.equal(y, h)


@pytest.mark.parametrize("T,n_in,n_out", [(1, 4096, 4096), (16, 4096, 1024), (7, 14336, 4096), (12, 640, 6144),
                                          (100, 2048, 512), (600, 2048, 512)])
def test_the_same_bits_in_every_call(B, T, n_in, n_out):
    """Decode joins its warps' sums in a fixed order, and so does every prefill tile."""
    L = Layer(B, T, n_in, n_out, seed=8)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    y = B.paro_linear_act(L.rot, L.x, *L.packed, n_out, act="silu", residual=L.residual)
    h = B.paro_linear_gated(L.rot, L.x, *G, n_out // 2)
    p = B.paro_linear(L.rot, L.x, *L.packed, n_out)
    for _ in range(30):
        assert torch.equal(y, B.paro_linear_act(L.rot, L.x, *L.packed, n_out, act="silu", residual=L.residual))
        assert torch.equal(h, B.paro_linear_gated(L.rot, L.x, *G, n_out // 2))
        assert torch.equal(p, B.paro_linear(L.rot, L.x, *L.packed, n_out))


@pytest.mark.parametrize("T,inter", [(40, 264), (100, 264), (300, 264), (700, 9728)])
def test_a_token_does_not_depend_on_its_place_in_the_batch(B, T, inter):
    L = Layer(B, T, 1024, 2 * inter, gated=True, seed=2)
    h = B.paro_linear_gated(L.rot, L.x, *L.packed, inter, bias=L.bias)
    order = torch.randperm(T, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))
    assert torch.equal(h[order], B.paro_linear_gated(L.rot, L.x[order].contiguous(), *L.packed, inter, bias=L.bias))


@pytest.mark.parametrize("T", [4, 16, 70, 300])
def test_bad_values_stay_in_their_rows(B, T):
    L = Layer(B, T, 512, 272, seed=T)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    y = B.paro_linear_act(L.rot, L.x, *L.packed, 272, act="silu", residual=L.residual)
    h = B.paro_linear_gated(L.rot, L.x, *G, 136)
    x, res = L.x.clone(), L.residual.clone()
    x[1, 77] = float("nan")
    x[3, 5] = float("inf")
    res[2, 9] = float("inf")
    y2 = B.paro_linear_act(L.rot, x, *L.packed, 272, act="silu", residual=res)
    h2 = B.paro_linear_gated(L.rot, x, *G, 136)
    keep = [t for t in range(T) if t not in (1, 2, 3)]
    assert torch.equal(y2[keep], y[keep]) and torch.equal(h2[keep + [2]], h[keep + [2]])
    assert torch.isinf(y2[2, 9]) and torch.equal(y2[2, :9], y[2, :9])
    assert bool(torch.isnan(y2[1]).all()) and bool(torch.isnan(h2[1]).all())


def test_large_arguments_of_the_activations(B):
    """Sums far out on both sides: saturated sigmoids, vanishing tails, fp16 overflow of the result."""
    n = 256
    q = torch.full((n, n), 8, dtype=torch.uint8, device="cuda")
    q[torch.arange(n), torch.arange(n)] = 9                 # w_hat = 4 on the diagonal
    s = torch.full((n, 2), 4.0, dtype=torch.float16, device="cuda")
    z = torch.full((n, 2), 8, dtype=torch.uint8, device="cuda")
    v = torch.tensor([0, 1e-4, -1e-4, 1, -1, 3, -3, 6, -6, 12, -12, 22, -22, 25, -25, 100, -100, 3e4, -3e4], device="cuda")
    for T in (16, 129):
        x = v.half().repeat(n)[:n].repeat(T, 1).contiguous()
        w = R.w_hat(q, s, z, 128)
        packed, gp = B.paro_pack_weights(q, s, z), B.paro_pack_gated(q, s, z)
        for act in ACTS:
            want, bound = R.linear_act(x, w, act)
            got = B.paro_linear_act(None, x, *packed, n, act=act)
            over = want.abs() > 65520                       # rounds to infinity
            assert torch.equal(torch.isinf(got), over) and not bool(torch.isnan(got).any())
            close(got[~over], want[~over], bound[~over])
            want, bound = R.gated(x, w, act)
            got = B.paro_linear_gated(None, x, *gp, n // 2, act=act)
            sure, over = want.abs() < 65400, want.abs() > 65600
            close(got[sure], want[sure], bound[sure])
            assert bool(torch.isinf(got[over]).all()) and not bool(torch.isnan(got).any())


def block(B, T, hidden, inter, seed, group=128):
    """One feed-forward block's parameters: norm weight, gated and down layers."""
    g = Layer(B, T, hidden, 2 * inter, group=group, bias=False, gated=True, seed=seed)
    d = Layer(B, T, inter, hidden, group=group, bias=False, seed=seed + 1)
    g.s.mul_(0.25)
    d.s.mul_(0.25)
    g.packed = B.paro_pack_gated(g.q, g.s, g.z, group=group)
    d.packed = B.paro_pack_weights(d.q, d.s, d.z, group=group)
    g.w, d.w = R.w_hat(g.q, g.s, g.z, group), R.w_hat(d.q, d.s, d.z, group)
    weight = (1 + 0.2 * torch.randn(hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))).half()
    return g, d, weight


@pytest.mark.parametrize("T", [1, 12, 48, 333])
def test_a_feed_forward_block(B, T):
    """norm -> gated -> down with the residual in place, each step against its
    64-bit form on the step's own input."""
    hidden, inter = 512, 896
    g, d, weight = block(B, T, hidden, inter, 40)
    stream = (2 * torch.randn(T, hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))).half()
    delta = g.x * 0.1
    v64, x64 = O.rmsnorm(delta.cpu().numpy(), weight.cpu().numpy(), 1e-5, residual=stream.cpu().numpy())
    x, h = B.paro_rmsnorm(delta, weight, 1e-5, residual=stream, H=stream)
    assert h is stream
    x64 = torch.from_numpy(x64).cuda()
    close(x, x64, 2.0 ** -11 * x64.abs() + 2.0 ** -17 * (1 + x64.abs()))
    a = B.paro_linear_gated(g.rot, x, *g.packed, inter)
    close(a, *R.gated(g.xr(x), g.w, "silu"))
    before = stream.clone()
    y = B.paro_linear_act(d.rot, a, *d.packed, hidden, residual=stream, Y=stream)
    assert y is stream
    close(stream, *R.linear_act(d.xr(a), d.w, "none", None, before))


def test_blocks_replayed_from_two_graphs_with_shared_workspaces(B):
    """Two captured blocks on one stream that share the prepared layers'
    workspaces, replayed in turn with new inputs: the bits of eager calls."""
    T, hidden, inter = 9, 512, 896
    g, d, weight = block(B, T, hidden, inter, 60)
    gated = B.ParoGated(g.rot, *g.packed, hidden, inter)
    down = B.ParoLinear(d.rot, *d.packed, inter, hidden)

    def step(delta, stream, x, a):
        B.paro_rmsnorm(delta, weight, 1e-5, residual=stream, H=stream, Y=x)
        gated(x, a)
        down(a, stream, residual=stream)

    def state(seed, n):
        r = torch.Generator(device="cuda").manual_seed(seed)
        return [torch.randn(n, k, device="cuda", generator=r).half() for k in (hidden, hidden, hidden, inter)]

    bufs = [state(1, T), state(2, 200)]                     # a decode batch and a prompt
    for b in bufs[::-1]:
        step(*b)                                            # the largest batch sizes the workspaces
    graphs = []
    for b in bufs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(3):
                step(*b)
        graphs.append(graph)
    for k in range(4):
        want = []
        for b, n in zip(bufs, (T, 200)):
            for dst, src in zip(b, state(10 * k + n, n)):
                dst.copy_(src)
            e = [t.clone() for t in b]
            for _ in range(3):
                step(*e)
            want.append(e[1])
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for b, w in zip(bufs, want):
            assert torch.equal(b[1], w)
    assert B.paro_fault_status() == 0


def test_prepared_layers_and_side_stream(B):
    L = Layer(B, 20, 512, 272, seed=1)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    lin = B.ParoLinear(L.rot, *L.packed, 512, 272, bias=L.bias, act="gelu")
    gat = B.ParoGated(L.rot, *G, 512, 136, bias=L.bias, act="relu")
    want_y = B.paro_linear_act(L.rot, L.x, *L.packed, 272, act="gelu", bias=L.bias, residual=L.residual)
    want_h = B.paro_linear_gated(L.rot, L.x, *G, 136, act="relu", bias=L.bias)
    assert torch.equal(lin(L.x, residual=L.residual), want_y) and torch.equal(gat(L.x), want_h)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y, h = lin(L.x, residual=L.residual), gat(L.x)
    st.synchronize()
    assert torch.equal(y, want_y) and torch.equal(h, want_h)
    y, h = torch.empty_like(want_y), torch.empty_like(want_h)
    lin(L.x, y, stream=st, residual=L.residual)
    gat(L.x, h, stream=st)
    st.synchronize()
    assert torch.equal(y, want_y) and torch.equal(h, want_h)


@pytest.mark.parametrize("T", [3, 16, 50, 128, 300])
def test_rows_behind_the_batch_stay(B, T):
    L = Layer(B, T, 512, 272, seed=T)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    y = torch.full((T + 40, 272), 7.0, dtype=torch.float16, device="cuda")
    h = torch.full((T + 40, 136), 7.0, dtype=torch.float16, device="cuda")
    B.paro_linear_act(L.rot, L.x, *L.packed, 272, act="silu", residual=L.residual, Y=y[:T])
    B.paro_linear_gated(L.rot, L.x, *G, 136, H=h[:T])
    assert bool((y[T:] == 7).all()) and bool((h[T:] == 7).all())
    close(y[:T], *R.linear_act(L.xr(), L.w, "silu", None, L.residual))


@pytest.mark.parametrize("T", [4, 30, 140])
def test_bias_at_any_two_byte_address(B, T):
    L = Layer(B, T, 384, 80, seed=T)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    moved = torch.empty(81, dtype=torch.float16, device="cuda")
    moved[1:] = L.bias
    assert torch.equal(B.paro_linear_act(L.rot, L.x, *L.packed, 80, act="gelu", bias=moved[1:]),
                       B.paro_linear_act(L.rot, L.x, *L.packed, 80, act="gelu", bias=L.bias))
    assert torch.equal(B.paro_linear_gated(L.rot, L.x, *G, 40, bias=moved[1:]),
                       B.paro_linear_gated(L.rot, L.x, *G, 40, bias=L.bias))


@pytest.mark.parametrize("T,n_in", [(9, 41088), (8, 82048), (40, 82048)])
def test_layers_wider_than_the_decode_kernel_splits(B, T, n_in):
    """Above 16 k-chunks of 20 (40) groups a decode batch takes the prefill kernels."""
    L = Layer(B, T, n_in, 48, seed=T, K=1)
    L.s.mul_(0.1)
    L.packed, L.w = B.paro_pack_weights(L.q, L.s, L.z), R.w_hat(L.q, L.s, L.z, 128)
    close(B.paro_linear_act(L.rot, L.x, *L.packed, 48, bias=L.bias, residual=L.residual),
          *R.linear_act(L.xr(), L.w, "none", L.bias, L.residual))
    close(B.paro_linear_gated(L.rot, L.x, *B.paro_pack_gated(L.q, L.s, L.z), 24), *R.gated(L.xr(), L.w, "silu"))
    close(B.paro_linear(L.rot, L.x, *L.packed, 48), *R.linear_act(L.xr(), L.w, "none"))


def test_outputs_beyond_32_bits(B):
    T, n_in, n_out = 66000, 128, 32768                      # 2.16e9 outputs
    L = Layer(B, 64, n_in, n_out, rotated=False, bias=False)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, n_in, device="cuda", generator=gen).half()
    y = torch.empty(T, n_out, dtype=torch.float16, device="cuda").normal_(generator=gen)
    rows = [0, 32767, 65535, 65536, T - 1]
    before = y[rows].clone()
    B.paro_linear_act(None, x, *L.packed, n_out, act="relu", residual=y, Y=y)
    close(y[rows], *R.linear_act(x[rows], L.w, "relu", None, before))


def test_blocks_on_two_streams_at_once(B):
    """Calls in flight together, each with its own workspace and outputs."""
    L = Layer(B, 200, 1024, 2048, seed=4)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    want_y = B.paro_linear_act(L.rot, L.x, *L.packed, 2048, residual=L.residual)
    want_h = B.paro_linear_gated(L.rot, L.x[:50], *G, 1024)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [B.workspace(200, 1024, 2048) for _ in streams]
    ys, hs = [torch.empty_like(want_y) for _ in range(20)], [torch.empty_like(want_h) for _ in range(20)]
    torch.cuda.synchronize()
    for k in range(20):
        B.paro_linear_act(L.rot, L.x, *L.packed, 2048, residual=L.residual, Y=ys[k], ws=ws[0], stream=streams[0])
        B.paro_linear_gated(L.rot, L.x[:50], *G, 1024, H=hs[k], ws=ws[1], stream=streams[1])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want_y) for y in ys) and all(torch.equal(h, want_h) for h in hs)


def test_side_stream_calls_without_a_workspace(B):
    """Scratch that a call allocates itself is neither filled on another stream
    nor handed out again while the call's stream still uses it."""
    L = Layer(B, 300, 1024, 512, seed=6)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    want_y = B.paro_linear_act(L.rot, L.x, *L.packed, 512, residual=L.residual)
    want_h = B.paro_linear_gated(L.rot, L.x, *G, 256)
    st = torch.cuda.Stream()
    ys, hs = [torch.empty_like(want_y) for _ in range(30)], [torch.empty_like(want_h) for _ in range(30)]
    torch.cuda.synchronize()
    n = B.paro_linear_workspace_size(300, 1024, 512)
    for k in range(30):
        B.paro_linear_act(L.rot, L.x, *L.packed, 512, residual=L.residual, Y=ys[k], stream=st)
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")     # would land in freed scratch: NaN in X'
        B.paro_linear_gated(L.rot, L.x, *G, 256, H=hs[k], stream=st.cuda_stream)
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(y, want_y) for y in ys) and all(torch.equal(h, want_h) for h in hs)


def test_side_stream_outputs_do_not_take_memory_still_in_use(B):
    """Tensors freed while the current stream still has work on them do not
    become the outputs or the workspace of a call on another stream."""
    T, in_f, out_f = 300, 1024, 512
    L = Layer(B, T, in_f, out_f, seed=8)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    w = torch.ones(in_f, dtype=torch.float16, device="cuda")
    layer = B.ParoLinear(L.rot, *L.packed, in_f, out_f, act="silu")
    calls = {
        "act": (lambda st: B.paro_linear_act(L.rot, L.x, *L.packed, out_f, stream=st), (2 * T * out_f,)),
        "gated": (lambda st: B.paro_linear_gated(L.rot, L.x, *G, out_f // 2, stream=st), (T * out_f,)),
        "norm": (lambda st: B.paro_rmsnorm(L.x, w, 1e-6, residual=L.x, stream=st), (2 * T * in_f,) * 2),
        "q8": (lambda st: B.paro_rmsnorm_q8(L.x, w, 1e-6, residual=L.x, stream=st), (T * in_f, 2 * T * in_f, 4 * T * in_f // 128)),
        "layer": (lambda st: layer(L.x, stream=st), (2 * T * out_f,)),
    }
    st = torch.cuda.Stream()
    ws = B.paro_linear_workspace_size(T, in_f, out_f)
    for name, (call, sizes) in calls.items():
        want = call(None)
        torch.cuda.synchronize()
        for stream in (st, st.cuda_stream):
            held = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in (*sizes, ws)]
            torch.cuda._sleep(20_000_000)                   # about 10 ms: the copies below come after the call
            copies = [h.clone() for h in held]
            del held
            got = call(stream)
            torch.cuda.synchronize()
            assert all(bool((c == 77).all()) for c in copies), name
            for g, e in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
                assert torch.equal(g.view(torch.uint8), e.view(torch.uint8)), name
    y = B.paro_linear_act(L.rot, L.x, *L.packed, out_f, stream=0)       # the default stream by its raw handle
    torch.cuda.synchronize()
    assert torch.equal(y, calls["act"][0](None))


def test_a_captured_call_survives_a_larger_batch(B):
    """A graph goes on using the workspace it was captured with after the
    prepared layer has grown another."""
    L = Layer(B, 300, 1024, 512, seed=7)
    layer = B.ParoLinear(L.rot, *L.packed, 1024, 512, act="silu")
    x = L.x[:40].clone()
    want = layer(x)
    y = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, y)
    big = layer(L.x)                                        # outgrows the captured workspace
    junk = [torch.full((x.numel() * 2,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(5):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert torch.equal(big, layer(L.x)) and all(bool((j == 255).all()) for j in junk)


def test_empty_batches_and_binding_refusals(B):
    L = Layer(B, 4, 256, 64, seed=1)
    G = B.paro_pack_gated(L.q, L.s, L.z)
    empty = L.x[:0]
    assert B.paro_linear_act(L.rot, empty, *L.packed, 64, act="silu").shape == (0, 64)
    assert B.paro_linear_gated(L.rot, empty, *G, 32).shape == (0, 32)
    lin, gat = B.ParoLinear(L.rot, *L.packed, 256, 64, act="silu"), B.ParoGated(L.rot, *G, 256, 32)
    assert lin(empty).shape == (0, 64) and gat(empty).shape == (0, 32)
    with pytest.raises(ValueError):
        B.paro_linear_act(L.rot, L.x, *L.packed, 64, act="swish")
    with pytest.raises(ValueError):
        B.paro_linear_act(L.rot, L.x, *L.packed, 64, residual=L.residual[:2])
    with pytest.raises(TypeError):
        B.paro_linear_act(L.rot, L.x, *L.packed, 64, residual=L.residual.float())
    with pytest.raises(ValueError):
        B.paro_linear_act(L.rot, L.x, *L.packed, 64, residual=L.residual.t().contiguous().t())
    with pytest.raises(ValueError):
        B.paro_linear_gated(L.rot, L.x, *G, 32, bias=L.bias[:32])
    with pytest.raises(ValueError):
        B.paro_pack_gated(L.q, L.s[:32], L.z)
    with pytest.raises(ValueError):
        B.ParoGated(L.rot, *G, 256, 64)                     # twice the rows the weights hold
    with pytest.raises(ValueError):
        lin(L.x, residual=L.residual[:3])
    both = torch.zeros(8, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(B.ParoError):
        B.paro_linear_act(L.rot, L.x, *L.packed, 64, residual=both[1:5], Y=both[:4])
