"""The layer's output and workspace share no memory with the packed scales and
zeros (nor the workspace with the codes): refused on the host, by the byte,
before anything is enqueued (the pointers are numbers that nothing reads)."""
import pytest

P = [0x1000000 * (i + 1) for i in range(12)]               # far apart and 16-byte aligned
ARG = 1


@pytest.fixture(scope="module")
def L():
    from rotated_w4_linear_b200 import binding, build
    build.build()
    return binding.lib()


def act(L, T=4, n_in=768, n_out=64, group=128, qw=P[1], s=P[2], z=P[3], Y=P[6], ws=P[7]):
    return L.paro_linear_act(None, P[0], qw, s, z, P[4], P[5], 2, group, Y, T, n_in, n_out, ws, 1 << 20, None)


def gated(L, T=4, n_in=768, n_out=64, group=128, qw=P[1], s=P[2], z=P[3], Y=P[6], ws=P[7]):
    return L.paro_linear_gated(None, P[0], qw, s, z, P[4], 2, group, Y, T, n_in, n_out // 2, ws, 1 << 20, None)


@pytest.mark.parametrize("call,width", [(act, 64), (gated, 32)])
@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("T", [4, 200])
def test_weights_share_no_memory_with_what_is_written(L, call, width, group, T):
    from rotated_w4_linear_b200 import binding
    n_in, n_out = 768, 64
    sizes = binding.paro_pack_size(n_in, n_out, group)
    ny, ws = T * width * 2, binding.paro_linear_workspace_size(T, n_in, n_out)
    for name, at, n in zip(("qw", "s", "z"), P[1:4], sizes):
        for Y in (at, at + n - 16, at - ny + 16):           # the start, the last 16 bytes, the output's own end
            assert call(L, T, group=group, Y=Y) == ARG, name
            assert b"the output overlaps" in L.paro_last_error()
        for w in (at, at + n - 16, at - ws + 16):
            assert call(L, T, group=group, ws=w) == ARG, name
            assert b"the workspace overlaps" in L.paro_last_error()


@pytest.mark.parametrize("call,width", [(act, 64), (gated, 32)])
def test_neighbours_are_not_overlaps(L, call, width):
    """Buffers that only touch pass these checks: the next one, a workspace
    over X, is what is refused."""
    from rotated_w4_linear_b200 import binding
    T, n_in, n_out = 4, 768, 64
    ny = T * width * 2
    for at, n in zip(P[1:4], binding.paro_pack_size(n_in, n_out, 128)):
        for Y in (at + n, at - ny):
            assert call(L, T, Y=Y, ws=P[0]) == ARG
            assert b"the workspace overlaps" in L.paro_last_error()
