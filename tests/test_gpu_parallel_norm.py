"""The norm beside the parallel layers on a one-rank NCCL group: a row-parallel
layer whose summed shares go straight into the residual norm, and a
column-parallel layer fed with 8-bit token shards."""
import socket

import numpy as np
import pytest
import torch

import layer64 as R
import synth
from oracle import paro_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    return binding


@pytest.fixture()
def group():
    import torch.distributed as dist
    with socket.socket() as sk:
        sk.bind(("127.0.0.1", 0))
        port = sk.getsockname()[1]
    dist.init_process_group("nccl", init_method=f"tcp://127.0.0.1:{port}", rank=0, world_size=1)
    yield dist
    dist.destroy_process_group()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("T", [5, 40])
def test_row_parallel_into_the_norm(B, group, T):
    from rotated_w4_linear_b200.row_parallel import RowParallelLinear
    in_f, out_f, eps = 1024, 640, 1e-5
    pairs, theta, alpha = synth.rotation_params(in_f, 8, 3)
    q, s, z = synth.w4_codes(out_f, in_f, 3)
    rng = np.random.default_rng(T)
    bias = rng.standard_normal(out_f).astype(np.float16)
    weight = (1 + 0.2 * rng.standard_normal(out_f)).astype(np.float16)
    x, r = dev(synth.activations(T, in_f, 3)), dev((2 * rng.standard_normal((T, out_f))).astype(np.float16))
    layer = RowParallelLinear(pairs, theta, alpha, q, s, z, rank=0, world=1, bias=bias)
    sums, es = R.sums(B.paro_rotate(layer.rot, x), R.w_hat(dev(q), dev(s), dev(z), 128), dev(bias))
    want_h = sums + r.double()
    stream = r.clone()
    y, h = layer.forward_norm(x, dev(weight), eps, residual=stream, H=stream)
    assert h is stream
    eh = es + 2.0 ** -23 * want_h.abs()
    assert bool(((h.double() - want_h).abs() <= R.rounding(want_h, eh)).all())
    # the norm of h to its own error: h's, scaled, plus the change of the root (at most h's largest relative to the rms)
    rms = 1 / torch.sqrt((want_h ** 2).mean(1, keepdim=True) + eps)
    want_y = want_h * rms * dev(weight).double()
    ey = (eh * rms + want_h.abs() * rms ** 2 * eh.amax(1, keepdim=True)) * dev(weight).double().abs() + 2.0 ** -18 * want_y.abs()
    assert bool(((y.double() - want_y).abs() <= R.rounding(want_y, ey)).all())
    layer.close()


@pytest.mark.parametrize("scale_group", [128, 0])
def test_column_parallel_from_token_shards(B, group, scale_group):
    from rotated_w4_linear_b200.column_parallel import ColumnParallelLinear
    T, in_f, out_f = 21, 1024, 512
    pairs, theta, alpha = synth.rotation_params(in_f, 8, 4)
    q, s, z = synth.w4_codes(out_f, in_f, 4)
    x = dev(synth.activations(T, in_f, 4))
    Q, S, _ = B.paro_rmsnorm_q8(x, torch.ones(in_f, dtype=torch.float16, device="cuda"), 1e-5, scale_group=scale_group)
    layer = ColumnParallelLinear(pairs, theta, alpha, q, s, z, rank=0, world=1)
    y = layer.forward_q8(Q, S, counts=[T], scale_group=scale_group, gather=True)
    assert torch.equal(y, layer.forward(B.paro_q8_expand(Q, S, scale_group)))
    assert torch.equal(y, layer.forward_q8(Q, S, scale_group=scale_group))
    # against the layer on the unquantised norm: an e4m3 code is off by at most
    # 2^-4 of its value, so a row of codes by at most 2^-4 of the row (2^-5.3
    # typically), and the random layer keeps that ratio to a few per cent
    _, n = O.rmsnorm(x.cpu().numpy(), np.ones(in_f), 1e-5)
    full = O.linear(n, pairs, theta, alpha, q, s, z)
    err = np.linalg.norm(y.double().cpu().numpy() - full, axis=1) / np.linalg.norm(full, axis=1)
    assert err.max() <= 2.0 ** -4
    layer.close()
