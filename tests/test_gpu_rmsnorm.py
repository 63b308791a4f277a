"""The residual RMS norm (fp16 and 8-bit output) against the fp64 oracle.

Bars, derived before the first run (u = 2^-24, the relative half step of an
fp32 operation; 2^-11 that of fp16, 2^-25 half its smallest step):
  * v = x + b + r takes at most two rounded sums: its error is at most
    2 u (|x| + |b| + |r|) =: ev;
  * H rounds v once: |H - v| <= 2^-11 |v| + 2^-25 + 2 ev;
  * y = (v w) r: the mean of squares is a sum of at most 32768 positive terms
    added in a tree (16 terms in sequence per thread at most, then 10
    shuffle steps, one division-free scaling), under 64 u relative, halved by
    the square root; the products and the reciprocal root add under 8 u; so y
    is off by at most 2^-18 |y| + ev |w| r, and its fp16 rounding adds
    2^-11 |y| + 2^-25. (The change of r by ev is inside 2^-18: ev / |v| enters
    the mean of squares at its average, below 4 u sqrt(F) for the inputs here.)
  * a scale is max|y| / 448: 2^-17 relative, plus the worst ev |w| r / 448;
  * a code rounds y / s to e4m3: |Q s - y| <= 2^-4 |y| + 2^-10 s plus y's own
    error and 2^-17 |y| for s.
"""
import numpy as np
import pytest
import torch

import synth
from oracle import paro_oracle as O

pytestmark = pytest.mark.gpu
EPS = 1e-5
U = 2.0 ** -24


@pytest.fixture(scope="module")
def B(cuda_lib):
    from rotated_w4_linear_b200 import binding
    return binding


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(T, F, x32=False, residual=True, bias=True, seed=0):
    rng = np.random.default_rng([T, F, seed])
    x = synth.activations(T, F, seed + 7)
    x = (x.astype(np.float32) + rng.standard_normal((T, F), dtype=np.float32) * 1e-4) if x32 else x
    r = (2 * rng.standard_normal((T, F))).astype(np.float16) if residual else None
    b = (0.1 * rng.standard_normal(F)).astype(np.float16) if bias else None
    w = (1 + 0.2 * rng.standard_normal(F)).astype(np.float16)
    return x, r, b, w


def reference(x, r, b, w, eps=EPS):
    v, y = O.rmsnorm(x, w, eps, r, b)
    mag = np.abs(x.astype(np.float64)) + (0 if b is None else np.abs(b.astype(np.float64))) \
        + (0 if r is None else np.abs(r.astype(np.float64)))
    ev = 2 * U * mag
    rms = 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    ey = 2.0 ** -18 * np.abs(y) + ev * np.abs(w.astype(np.float64)) * rms
    return v, y, ev, ey


def check_h(H, v, ev):
    assert np.all(np.abs(host(H) - v) <= 2.0 ** -11 * np.abs(v) + 2.0 ** -25 + 2 * ev)


def check_y(Y, y, ey):
    assert np.all(np.abs(host(Y) - y) <= 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + ey)


def check_q8(Q, S, y, ey, group):
    F = y.shape[1]
    want, s = O.q8_scales(y, group), host(S)
    assert s.shape == want.shape
    c = 128 if group else F
    idx = np.arange(F) // c
    es = np.zeros_like(want)
    np.maximum.at(es.T, idx, ey.T)
    assert np.all(np.abs(s - want) <= 2.0 ** -17 * want + es / 448)
    each = s[:, idx]
    assert np.all(np.abs(host(Q) * each - y) <= 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * each + ey + 2.0 ** -17 * np.abs(y))
    assert np.all(np.abs(host(Q)) <= 448)


SHAPES = [(1, 16), (3, 48), (2, 128), (5, 144), (1, 4096), (16, 4096), (17, 2560), (300, 272), (301, 1040),
          (1023, 2576), (7, 8192), (5, 8208), (3, 10768), (2, 14336), (3, 14352),
          (3, 16384), (2, 16400), (3, 17408), (2, 28688), (2, 32768)]


@pytest.mark.parametrize("T,F", SHAPES)
@pytest.mark.parametrize("x32", [False, True])
def test_norm(B, T, F, x32):
    x, r, b, w = inputs(T, F, x32)
    v, y, ev, ey = reference(x, r, b, w)
    Y, H = B.paro_rmsnorm(dev(x), dev(w), EPS, residual=dev(r), bias=dev(b))
    check_h(H, v, ev)
    check_y(Y, y, ey)
    for group in (128, 0):
        Q, S, H2 = B.paro_rmsnorm_q8(dev(x), dev(w), EPS, residual=dev(r), bias=dev(b), scale_group=group)
        check_q8(Q, S, y, ey, group)
        assert torch.equal(H2, H)
        E = B.paro_q8_expand(Q, S, group)
        each = host(S)[:, np.arange(F) // (128 if group else F)]
        want = host(Q) * each
        assert np.all(np.abs(host(E) - want) <= (2.0 ** -11 + U) * np.abs(want) + 2.0 ** -25)


@pytest.mark.parametrize("residual,bias", [(False, False), (True, False), (False, True)])
def test_optional_inputs(B, residual, bias):
    x, r, b, w = inputs(9, 656, residual=residual, bias=bias)
    v, y, ev, ey = reference(x, r, b, w)
    Y, H = B.paro_rmsnorm(dev(x), dev(w), EPS, residual=dev(r), bias=dev(b))
    check_y(Y, y, ey)
    if residual or bias:
        check_h(H, v, ev)
    else:
        assert H is None                                    # nothing was added: H would be X
        H = torch.empty_like(Y)
        B.paro_rmsnorm(dev(x), dev(w), EPS, H=H)
        assert np.array_equal(host(H), x.astype(np.float64))


def test_a_row_does_not_depend_on_the_batch(B):
    x, r, b, w = inputs(700, 4096)
    X, R, W = dev(x), dev(r), dev(w)
    Y, H = B.paro_rmsnorm(X, W, EPS, residual=R)
    for lo, hi in ((699, 700), (3, 20), (0, 310)):
        y, h = B.paro_rmsnorm(X[lo:hi], W, EPS, residual=R[lo:hi])
        assert torch.equal(y, Y[lo:hi]) and torch.equal(h, H[lo:hi])


@pytest.mark.parametrize("T,F", [(5, 400), (400, 4096)])
def test_in_place(B, T, F):
    x, r, b, w = inputs(T, F)
    X, R, W = dev(x), dev(r), dev(w)
    Y, H = B.paro_rmsnorm(X, W, EPS, residual=R)
    r2, x2 = R.clone(), X.clone()
    y, h = B.paro_rmsnorm(x2, W, EPS, residual=r2, H=r2, Y=x2)     # residual stream and norm both in place
    assert h is r2 and y is x2 and torch.equal(r2, H) and torch.equal(x2, Y)


def test_rows_that_are_zero_nan_or_infinite(B):
    T, F = 8, 272
    x, _, _, w = inputs(T, F)
    x[1] = 0
    x[3, 200] = np.nan
    x[5, 17] = np.inf
    x[6] = 65504                                            # the largest fp16 in every channel: finite norms
    X, W = dev(x), dev(w)
    Y, _ = B.paro_rmsnorm(X, W, EPS)
    got = host(Y)
    fine = [0, 2, 4, 6, 7]
    v, y, ev, ey = reference(x[fine], None, None, w)
    check_y(Y[fine], y, ey)
    assert np.all(got[1] == 0) and np.all(np.isnan(got[3]))
    assert np.isnan(got[5, 17]) and np.all(np.delete(got[5], 17) == 0)
    for group in (128, 0):
        Q, S, _ = B.paro_rmsnorm_q8(X, W, EPS, scale_group=group)
        check_q8(Q[fine], S[fine], y, ey, group)
        q, s = host(Q), host(S)
        assert np.all(q[1] == 0) and np.all(s[1] == 2.0 ** -100)
        assert np.all(np.isnan(q[3]))
        assert np.isnan(q[5, 17]) and np.all(np.delete(q[5], 17) == 0)
        assert np.all(np.isfinite(s)) and np.all(s > 0)


def test_small_values_and_a_large_eps(B):
    """The smallest fp16 magnitudes, where eps decides the norm."""
    T, F = 4, 512
    rng = np.random.default_rng(3)
    x = (rng.integers(-3, 4, (T, F)) * 2.0 ** -24).astype(np.float16)
    w = np.ones(F, np.float16)
    for eps in (1e-6, 1.0, 1e-30):
        _, y, _, ey = reference(x, None, None, w, eps)
        check_y(B.paro_rmsnorm(dev(x), dev(w), eps)[0], y, ey)
        Q, S, _ = B.paro_rmsnorm_q8(dev(x), dev(w), eps)
        check_q8(Q, S, y, ey, 128)


def test_channels_below_the_scale_floor(B):
    """Zeros, and values whose scale is the floor, under an eps so small that
    the norm's factor over the scale exceeds fp32."""
    T, F, eps = 3, 256, 2.0 ** -60
    rng = np.random.default_rng(4)
    x = np.zeros((T, F), np.float32)
    x[1, :128] = rng.standard_normal(128).astype(np.float32) * 1e-15     # the row's second group is zero
    x[2] = rng.standard_normal(F).astype(np.float32) * np.float32(2.0 ** -123)    # y about 2^-93: codes above the floor
    x[2, :128] *= np.float32(2.0 ** -5)                     # and below it
    w = np.full(F, 1.5, np.float16)
    ey = 2.0 ** -18
    _, y = O.rmsnorm(x, w, eps)
    for group in (128, 0):
        Q, S, _ = B.paro_rmsnorm_q8(dev(x), dev(w), eps, scale_group=group)
        q, s = host(Q), host(S)
        assert np.all(q[0] == 0) and np.all(q[1, 128:] == 0) and np.all(np.isfinite(q)) and np.all(s >= 2.0 ** -100)
        check_q8(Q[:2], S[:2], y[:2], ey * np.abs(y[:2]), group)
        each = s[2, np.arange(F) // (128 if group else F)]
        assert np.all(np.abs(q[2] * each - y[2]) <= 2.0 ** -4 * np.abs(y[2]) + 2.0 ** -10 * each + ey * np.abs(y[2]))


def test_on_a_side_stream_and_in_a_graph(B):
    x, r, b, w = inputs(33, 4096, x32=True)
    X, R, W, b_ = dev(x), dev(r), dev(w), dev(b)
    Y0, H0 = B.paro_rmsnorm(X, W, EPS, residual=R, bias=b_)
    Q0, S0, _ = B.paro_rmsnorm_q8(X, W, EPS, residual=R, bias=b_)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    Y, H = torch.empty_like(Y0), torch.empty_like(H0)
    Q, S = torch.empty_like(Q0), torch.empty_like(S0)
    E = torch.empty_like(Y0)
    with torch.cuda.stream(st):
        B.paro_rmsnorm(X, W, EPS, residual=R, bias=b_, H=H, Y=Y)
    st.synchronize()
    assert torch.equal(Y, Y0) and torch.equal(H, H0)
    Y.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.paro_rmsnorm(X, W, EPS, residual=R, bias=b_, H=H, Y=Y)
        B.paro_rmsnorm_q8(X, W, EPS, residual=R, bias=b_, H=H, Y=Q, S=S)
        B.paro_q8_expand(Q, S, 128, Y=E)
    for k in range(3):                                      # new inputs in the captured buffers
        x2, r2, _, _ = inputs(33, 4096, x32=True, seed=10 + k)
        X.copy_(dev(x2))
        R.copy_(dev(r2))
        g.replay()
        torch.cuda.synchronize()
        v, y, ev, ey = reference(x2, r2, b, w)
        check_h(H, v, ev)
        check_y(Y, y, ey)
        check_q8(Q, S, y, ey, 128)
        assert torch.equal(E, B.paro_q8_expand(Q, S, 128))


def test_chained_norms_see_each_other(B):
    """A run of dependent launches (each starts before the last has ended):
    every norm reads what the one before it wrote."""
    T, F = 64, 2560
    x, r, _, w = inputs(T, F)
    X, R, W = dev(x), dev(r), dev(w)
    want_y, want_h = X, R
    for _ in range(8):
        want_y, want_h = B.paro_rmsnorm(want_y, W, EPS, residual=want_h)
        torch.cuda.synchronize()
    for _ in range(20):
        y, h = X.clone(), R.clone()
        for _ in range(8):
            B.paro_rmsnorm(y, W, EPS, residual=h, H=h, Y=y)
        assert torch.equal(y, want_y) and torch.equal(h, want_h)


def test_offsets_beyond_32_bits(B):
    T, F = 65600, 32768                                     # 2.15e9 channels
    X = torch.empty((T, F), dtype=torch.float16, device="cuda")
    X.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    W = torch.ones(F, dtype=torch.float16, device="cuda")
    rows = [0, 32767, 65535, 65536, T - 1]
    Y, _ = B.paro_rmsnorm(X, W, EPS)
    Q, S, _ = B.paro_rmsnorm_q8(X, W, EPS)
    x = X[rows].cpu().numpy()
    _, y, _, ey = reference(x, None, None, np.ones(F, np.float16))
    check_y(Y[rows], y, ey)
    check_q8(Q.view(torch.uint8)[rows].view(torch.float8_e4m3fn), S[rows], y, ey, 128)
    E = B.paro_q8_expand(Q, S, Y=Y)
    assert torch.equal(E[-1], B.paro_q8_expand(Q[-1:].contiguous(), S[-1:].contiguous())[0])


def test_empty_batch_and_binding_refusals(B):
    W = torch.ones(256, dtype=torch.float16, device="cuda")
    X = torch.zeros((0, 256), dtype=torch.float16, device="cuda")
    assert B.paro_rmsnorm(X, W, EPS)[0].shape == (0, 256)
    assert B.paro_rmsnorm_q8(X, W, EPS)[1].shape == (0, 2)
    X = torch.zeros((4, 256), dtype=torch.float16, device="cuda")
    for bad in (X[:, :128], X.t(), X[0]):
        with pytest.raises((TypeError, ValueError, B.ParoError)):
            B.paro_rmsnorm(bad, W, EPS)
    with pytest.raises(TypeError):
        B.paro_rmsnorm(X.bfloat16(), W, EPS)
    with pytest.raises(TypeError):
        B.paro_rmsnorm(X, W.float(), EPS)
    with pytest.raises(ValueError):
        B.paro_rmsnorm(X, W, EPS, residual=X[:3])
    with pytest.raises(ValueError):
        B.paro_rmsnorm(X, W, EPS, Y=torch.empty((4, 128), dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError):
        B.paro_rmsnorm(X.cpu(), W, EPS)
    with pytest.raises(B.ParoError):
        B.paro_rmsnorm(X, W, 0.0)
    Q, S, _ = B.paro_rmsnorm_q8(X, W, EPS)
    with pytest.raises(ValueError):
        B.paro_q8_expand(Q, S, 0)
