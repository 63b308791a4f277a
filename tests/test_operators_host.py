"""Argument checks of the block's operators: every refusal comes from the
host, before anything is enqueued, so no GPU is needed (the pointers are
numbers that nothing reads)."""
import pytest

P = [0x1000000 * (i + 1) for i in range(12)]               # far apart and 16-byte aligned
ARG, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    from rotated_w4_linear_b200 import binding, build
    build.build()
    return binding.lib()


def refused(L, status, expected, text):
    assert status == expected, L.paro_last_error()
    assert text in L.paro_last_error().decode()


def norm(L, X=P[0], x32=0, R=P[1], b=P[2], w=P[3], eps=1e-5, H=P[4], Y=P[5], T=4, F=256):
    return L.paro_rmsnorm(X, x32, R, b, w, eps, H, Y, T, F, None)


def norm8(L, X=P[0], x32=0, R=P[1], b=P[2], w=P[3], eps=1e-5, group=128, H=P[4], Q=P[5], S=P[6], T=4, F=256):
    return L.paro_rmsnorm_q8(X, x32, R, b, w, eps, group, H, Q, S, T, F, None)


@pytest.mark.parametrize("call", [norm, norm8])
def test_norm_refusals(L, call):
    for F in (0, -16, 8, 250, 4095):
        refused(L, call(L, F=F), ARG, "multiple of 16")
    refused(L, call(L, F=32784), UNSUPPORTED, "features")
    for eps in (0.0, -1.0, float("inf"), float("nan"), 1e-60):
        refused(L, call(L, eps=eps), ARG, "eps")
    refused(L, call(L, x32=2), ARG, "x_fp32")
    refused(L, call(L, T=-1), ARG, "tokens")
    refused(L, call(L, T=1 << 40), UNSUPPORTED, "tokens")
    refused(L, call(L, X=None), ARG, "null")
    refused(L, call(L, w=None), ARG, "null")
    for name in ("X", "R", "b", "w", "H"):
        refused(L, call(L, **{name: P[7] + 8}), ARG, "aligned")
    assert call(L, T=0, X=None, w=None) == 0               # nothing to do


def test_norm_overlaps(L):
    n = 4 * 256 * 2
    refused(L, norm(L, Y=None), ARG, "null")
    refused(L, norm(L, H=P[0] + 16), ARG, "H overlaps")                 # shifted into X
    refused(L, norm(L, Y=P[1] + n - 16), ARG, "Y overlaps")             # tail of the residual
    refused(L, norm(L, Y=P[3]), ARG, "Y overlaps")                      # the weights
    refused(L, norm(L, H=P[2]), ARG, "H overlaps")                      # the bias
    refused(L, norm(L, H=P[5]), ARG, "overlap")                         # H and Y the same
    refused(L, norm(L, x32=1, H=P[0]), ARG, "H overlaps")               # fp16 rows over fp32 rows
    refused(L, norm(L, x32=1, Y=P[0] + 2 * n - 16), ARG, "Y overlaps")  # X is twice as long in fp32
    refused(L, norm8(L, Q=P[1]), ARG, "Y overlaps")                     # codes are never in place
    refused(L, norm8(L, S=P[1]), ARG, "scales overlaps")
    refused(L, norm8(L, S=P[4] + 16), ARG, "overlap")                   # scales inside H
    refused(L, norm8(L, S=None), ARG, "null")
    refused(L, norm8(L, group=64), UNSUPPORTED, "scale_group")


def test_expand_refusals(L):
    def call(Q=P[0], S=P[1], group=128, Y=P[2], T=4, F=256):
        return L.paro_q8_expand(Q, S, group, Y, T, F, None)
    refused(L, call(F=100), ARG, "multiple of 16")
    refused(L, call(F=40000), UNSUPPORTED, "features")
    refused(L, call(group=32), UNSUPPORTED, "scale_group")
    refused(L, call(T=-2), ARG, "tokens")
    refused(L, call(T=1 << 45), UNSUPPORTED, "tokens")
    refused(L, call(Y=P[0]), ARG, "overlaps")
    refused(L, call(Y=P[1] - 16), ARG, "overlaps")
    refused(L, call(S=None), ARG, "null")
    refused(L, call(Q=P[0] + 4), ARG, "aligned")
    assert call(T=0, Q=None) == 0


def act(L, rot=None, X=P[0], qw=P[1], s=P[2], z=P[3], b=P[4], R=P[5], act=2, group=128, Y=P[6], T=4, n_in=256, n_out=64,
        ws=P[7], wsb=1 << 20):
    return L.paro_linear_act(rot, X, qw, s, z, b, R, act, group, Y, T, n_in, n_out, ws, wsb, None)


def gated(L, rot=None, X=P[0], qw=P[1], s=P[2], z=P[3], b=P[4], act=2, group=128, H=P[6], T=4, n_in=256, inter=32,
          ws=P[7], wsb=1 << 20):
    return L.paro_linear_gated(rot, X, qw, s, z, b, act, group, H, T, n_in, inter, ws, wsb, None)


@pytest.mark.parametrize("call", [act, gated])
def test_layer_refusals(L, call):
    for a in (-1, 5, 99):
        refused(L, call(L, act=a), ARG, "act")
    refused(L, call(L, n_in=200), ARG, "in_features")
    refused(L, call(L, group=32), UNSUPPORTED, "group")
    refused(L, call(L, group=256, n_in=384), ARG, "multiple of 256")
    refused(L, call(L, T=-1), ARG, "tokens")
    refused(L, call(L, T=1 << 30), UNSUPPORTED, "tokens")
    refused(L, call(L, wsb=16), ARG, "workspace_bytes")
    for name in ("X", "qw", "s", "z", "ws"):
        refused(L, call(L, **{name: None}), ARG, "null")
        refused(L, call(L, **{name: P[8] + 8}), ARG, "aligned")
    refused(L, call(L, b=P[4] + 1), ARG, "bias")
    assert call(L, T=0, X=None) == 0


def test_layer_overlaps(L):
    n = 4 * 64 * 2
    refused(L, act(L, R=P[5] + 4), ARG, "aligned")
    refused(L, act(L, Y=P[0] + 16), ARG, "overlaps an input")
    refused(L, act(L, Y=P[7]), ARG, "workspace")
    refused(L, act(L, Y=P[4]), ARG, "overlaps an input")
    refused(L, act(L, Y=P[1] + 32), ARG, "overlaps an input")
    refused(L, act(L, R=P[6] + n - 16), ARG, "residual")
    refused(L, act(L, R=P[6] - 16), ARG, "residual")
    refused(L, act(L, ws=P[0]), ARG, "workspace")
    refused(L, act(L, ws=P[5]), ARG, "workspace")
    refused(L, gated(L, H=P[0]), ARG, "overlaps an input")
    refused(L, gated(L, H=P[7] + 64), ARG, "workspace")


def test_gated_widths(L):
    for inter in (0, -8, 4, 12, 33):
        refused(L, gated(L, inter=inter), ARG, "inter_features")
        refused(L, L.paro_pack_gated(P[0], P[1], P[2], 256, inter, 128, P[3], P[4], P[5], None), ARG, "inter_features")
    refused(L, gated(L, inter=1 << 22), UNSUPPORTED, "large")
    refused(L, L.paro_pack_gated(None, P[1], P[2], 256, 32, 128, P[3], P[4], P[5], None), ARG, "null")
    refused(L, L.paro_pack_gated(P[0], P[1], P[2], 250, 32, 128, P[3], P[4], P[5], None), ARG, "in_features")
    refused(L, L.paro_pack_gated(P[0], P[1], P[2], 256, 32, 32, P[3], P[4], P[5], None), UNSUPPORTED, "group")
    refused(L, L.paro_pack_gated(P[0], P[1], P[2], 256, 32, 128, P[3] + 8, P[4], P[5], None), ARG, "aligned")


def test_static_scratch_refuses_what_the_decode_kernel_has_no_plan_for(L):
    """41088 channels at 12 tokens fit the scratch but not sixteen k-chunks of
    20 groups: refused, where the planner once divided by its empty plan."""
    assert L.paro_linear_noalloc(None, P[0], P[1], P[2], P[3], P[4], 12, 41088, 64, None) == UNSUPPORTED
    assert b"too wide" in L.paro_last_error()
