"""Gradients through frozen NVFP4 weights on the GPU against 64-bit computations.

dx on whole numbers: products and sums exact in FP32 and the result exact in fp16, compared bit for bit. Random values:
one fp16 rounding (2^-11 relative, 2^-25 for subnormals), the global scale's product (2^-24), and the sum, whose every
addition is off by at most 2^-23 of the sum of magnitudes: (terms) * 2^-23 of it bounds any order of adding.

The gated gradient: g and u are off by dg, du <= (K + 2) 2^-23 of their sums of magnitudes. With sig = sigma(g),
|d/dg sig (1 + g (1 - sig))| <= 1/2 and |sig (1 + g (1 - sig))| <= 1.1, |d/dg g sig| <= 1.1; the functions themselves
are off by (|g| + 8) 2^-22 relative of their terms (the exponential's argument, the exponential, the reciprocal and
the products), whose magnitudes sum to sig (1 + |g|).
"""
import numpy as np
import pytest
import torch

import gemm_nvfp4_amd as G
from synth import inputs as S

pytestmark = pytest.mark.gpu

HALF, TINY, ADD = 2.0 ** -11, 2.0 ** -25, 2.0 ** -23
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])

# batch sizes on both sides of every change of kernel: sixteens of rows pass by the stream, always up to 64; with more rows
# large weights stream too, small ones are decoded for tiles
BATCHES = [1, 2, 15, 16, 17, 33, 48, 49, 64, 65, 127, 130, 300]


def _weight(seed, n, k, whole):
    rng = np.random.default_rng(seed)
    if whole:  # every code; scales 1, 2 and 4
        codes = rng.integers(0, 256, (1, n, k // 2)).astype(np.uint8)
        scales = np.array([0x38, 0x40, 0x48], np.uint8)[rng.integers(0, 3, (1, n, k // 16))]
        return codes, scales, np.array([0.5], np.float32)
    codes, scales, _ = S.nvfp4_weights(rng, 1, n, k)
    return codes, scales, np.array([0.37], np.float32)


def _dense(w):
    codes, scales, gs = w
    v = np.stack((E2M1[codes[0] & 15], E2M1[codes[0] >> 4]), axis=-1).reshape(codes.shape[1], -1)
    sc = torch.from_numpy(scales[0]).view(torch.float8_e4m3fn).double().numpy()
    return v * np.repeat(sc, 16, axis=1) * np.float64(gs[0])


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _mm(a, b):
    return (torch.from_numpy(a).cuda() @ torch.from_numpy(b).cuda()).cpu().numpy()


def _guarded(m, n):
    buf = torch.full((m * n + 256,), float("nan"), dtype=torch.float16, device="cuda")
    return buf[128:128 + m * n].view(m, n), lambda: bool(buf[:128].isnan().all() and buf[128 + m * n:].isnan().all())


def _work(need):
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    return ws[:need], lambda: bool((ws[need:] == 0xFF).all())


@pytest.mark.parametrize("n,k", [(16, 128), (48, 384), (528, 256), (1072, 640), (4352, 128)])
@pytest.mark.parametrize("m", BATCHES)
def test_grad_whole_numbers(m, n, k):
    w = _weight(n + k, n, k, True)
    rng = np.random.default_rng(m)
    dy = rng.integers(-2, 3, (m, n)).astype(np.float64)
    dy *= rng.random((m, n)) < min(1.0, 12 / n)  # few terms: the result fits fp16's 11 bits
    ref = _mm(dy, _dense(w))
    assert np.array_equal(ref, ref.astype(np.float16).astype(np.float64))
    dx, ok = _guarded(m, k)
    ws, ws_ok = _work(G.nvfp4_linear_grad_ws_bytes(m, n, k))
    G.nvfp4_linear_grad(_cuda(dy.astype(np.float16)), G.NVFP4Tensor.from_numpy(w), dx=dx, ws=ws)
    torch.cuda.synchronize()
    assert ok() and ws_ok()
    assert np.array_equal(dx.double().cpu().numpy(), ref)


def _check_grad(dx, dy, w):
    d = dy.astype(np.float64)
    ref, size = _mm(d, w), _mm(np.abs(d), np.abs(w))
    err = np.abs(dx.double().cpu().numpy() - ref)
    assert np.all(err <= (HALF + 2.0 ** -20) * np.abs(ref) + TINY + (dy.shape[1] + 2) * ADD * size)


@pytest.mark.parametrize("m,n,k", [(1, 4352, 5120), (24, 4352, 5120), (64, 80, 5120), (100, 1040, 1152), (150, 4352, 5120),
                                   (250, 4368, 4992), (333, 2064, 2176), (1000, 4352, 896), (4096, 1040, 5120),
                                   # a size for each shape of the tiles; a short last stage, and runs of stages
                                   (500, 1040, 2048), (532, 32, 6656), (907, 1040, 4352), (388, 32, 7040), (1030, 96, 7296),
                                   (1159, 32, 7040), (1055, 1040, 8192), (1580, 32, 7296), (2061, 32, 7808),
                                   (3201, 1040, 5120), (289, 6464, 8064), (588, 6368, 6784)])
def test_grad_random(m, n, k):
    w = _weight(m, n, k, False)
    dy = np.random.default_rng(m).standard_normal((m, n)).astype(np.float16)
    _check_grad(G.nvfp4_linear_grad(_cuda(dy), G.NVFP4Tensor.from_numpy(w)), dy, _dense(w))


@pytest.mark.parametrize("m,n,k", [(17, 32, 32768), (70, 48, 32768)])
def test_grad_widest(m, n, k):
    w = _weight(m, n, k, False)
    dy = np.random.default_rng(m).standard_normal((m, n)).astype(np.float16)
    _check_grad(G.nvfp4_linear_grad(_cuda(dy), G.NVFP4Tensor.from_numpy(w)), dy, _dense(w))


@pytest.mark.parametrize("m", [5, 40, 100])
def test_grad_of_a_tall_weight(m):
    """As many rows as a vocabulary has, ragged against every step."""
    n, k = 151664 + 16, 128
    w = _weight(m, n, k, False)
    dy = np.random.default_rng(m).standard_normal((m, n)).astype(np.float16)
    _check_grad(G.nvfp4_linear_grad(_cuda(dy), G.NVFP4Tensor.from_numpy(w)), dy, _dense(w))


def test_grad_is_the_linear_map_of_the_projection():
    """<dy, linear(x)> = <linear_grad(dy), x>: the gradient by its definition, against differences of the projection (which
    is linear, so one difference of any length is exact) on whole numbers."""
    n, k = 96, 256
    w = G.NVFP4Tensor.from_numpy(_weight(1, n, k, True))
    rng = np.random.default_rng(2)
    dy = np.zeros((3, n))
    dy[:, rng.integers(0, n, 6)] = 1
    dx = G.nvfp4_linear_grad(_cuda(dy.astype(np.float16)), w).double().cpu().numpy()
    for j in rng.integers(0, k, 12):
        e = np.zeros((1, k), np.float16)
        e[0, j] = 1
        y = G.nvfp4_linear(_cuda(e), w).double().cpu().numpy()[0]
        assert np.array_equal(dy @ y, dx[:, j])


def _swiglu(x, dh, w, layout):
    """dz, and the bound of the module's docstring for every element."""
    m, half = dh.shape
    x, dh = x.astype(np.float64), dh.astype(np.float64)
    z, size = _mm(x, w.T.copy()), _mm(np.abs(x), np.abs(w.T))
    at = (slice(0, None, 2), slice(1, None, 2)) if layout else (slice(0, half), slice(half, None))
    g, u = z[:, at[0]], z[:, at[1]]
    eg, eu = ((x.shape[1] + 2) * ADD * size[:, a] for a in at)
    sig = 1 / (1 + np.exp(-g))
    own = (np.abs(g) + 8) * 2.0 ** -22 * sig * (1 + np.abs(g))
    dz, bound = np.empty_like(z), np.empty_like(z)
    dz[:, at[0]], dz[:, at[1]] = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig
    bound[:, at[0]] = np.abs(dh) * (1.1 * eu + np.abs(u) * (0.5 * eg + own) + eu * (eg + own))
    bound[:, at[1]] = np.abs(dh) * (1.1 * eg + own)
    return dz, bound + (HALF + 2.0 ** -20) * np.abs(dz) + TINY


@pytest.mark.parametrize("n,k", [(32, 128), (96, 640), (544, 256), (1056, 1536)])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("m", [1, 16, 17, 64, 65, 127, 300])
def test_swiglu_grad(m, n, k, layout):
    w = _weight(n + k, n, k, False)
    rng = np.random.default_rng(m)
    x, dh = (rng.standard_normal((m, c)).astype(np.float16) for c in (k, n // 2))
    dz, ok = _guarded(m, n)
    ws, ws_ok = _work(G.nvfp4_linear_swiglu_grad_ws_bytes(m, n, k))
    G.nvfp4_linear_swiglu_grad(_cuda(x), _cuda(dh), G.NVFP4Tensor.from_numpy(w), layout, dz=dz, ws=ws)
    torch.cuda.synchronize()
    assert ok() and ws_ok()
    ref, bound = _swiglu(x, dh, _dense(w), layout)
    assert np.all(np.abs(dz.double().cpu().numpy() - ref) <= bound)


# packed tiles of 64 x 64 with two groups and with one and of 128 x 128, each in both layouts with ragged rows and columns
# and an odd number of stages; then decoded weights and chunk products
@pytest.mark.parametrize("m,n,k,layout", [(333, 4352, 5120, 1), (397, 4384, 1152, 0), (500, 4352, 896, 1), (1500, 4384, 640, 0),
                                          (1000, 4384, 5120, 0), (1100, 4352, 4992, 1), (2100, 4352, 1152, 0),
                                          (4100, 2080, 896, 1), (2500, 4352, 5120, 0), (2017, 2080, 1152, 0),
                                          (1055, 8192, 1152, 1), (5384, 2080, 1152, 1), (7715, 2080, 128, 0),
                                          (71, 32, 1664, 1), (3474, 864, 128, 0), (770, 1280, 6912, 1), (988, 2144, 7424, 0),
                                          (1155, 7136, 128, 1), (1428, 5504, 128, 0), (2060, 7712, 256, 1),
                                          (20, 2048, 16384, 0)])
def test_swiglu_grad_large(m, n, k, layout):
    w = _weight(m, n, k, False)
    rng = np.random.default_rng(m)
    x, dh = (rng.standard_normal((m, c)).astype(np.float16) * 0.5 for c in (k, n // 2))
    dz = G.nvfp4_linear_swiglu_grad(_cuda(x), _cuda(dh), G.NVFP4Tensor.from_numpy(w), layout)
    ref, bound = _swiglu(x, dh, _dense(w), layout)
    assert np.all(np.abs(dz.double().cpu().numpy() - ref) <= bound)


def test_swiglu_grad_against_differences():
    """d sum(dh * h) / dx through dz and nvfp4_linear_grad, against central differences of the gated projection in 64
    bits; the bound is the two fp16 roundings (of dz, then of dx) and the differences' own error."""
    m, n, k = 3, 64, 128
    w = _weight(9, n, k, False)
    rng = np.random.default_rng(4)
    x, dh = (rng.standard_normal((m, c)).astype(np.float16) for c in (k, n // 2))
    wt = G.NVFP4Tensor.from_numpy(w)
    dz = G.nvfp4_linear_swiglu_grad(_cuda(x), _cuda(dh), wt, 1)
    dx = G.nvfp4_linear_grad(dz, wt).double().cpu().numpy()
    d = _dense(w)

    def loss(v):
        z = v @ d.T
        g, u = z[:, 0::2], z[:, 1::2]
        return float(np.sum(dh.astype(np.float64) * g / (1 + np.exp(-g)) * u))

    ref_dz, bound = _swiglu(x, dh, d, 1)
    for i, j in ((0, 0), (1, 77), (2, 127)):
        e = np.zeros((m, k))
        e[i, j] = 1e-6
        ref = (loss(x + e) - loss(x - e)) / 2e-6
        assert abs(dx[i, j] - ref) <= bound[i] @ np.abs(d[:, j]) + (HALF + n * ADD) * abs(ref) + 1e-6


@pytest.mark.parametrize("m", [30, 100, 700])
def test_rows_stay_apart(m):
    """A row that holds an infinity or a NaN leaves the others' bits as they are, and a repeated call gives the same."""
    n, k = 1056, 640
    w = G.NVFP4Tensor.from_numpy(_weight(3, n, k, False))
    dy = torch.randn(m, n, device="cuda").half()
    x, dh = torch.randn(m, k, device="cuda").half(), torch.randn(m, n // 2, device="cuda").half()
    dx, dz = G.nvfp4_linear_grad(dy, w), G.nvfp4_linear_swiglu_grad(x, dh, w)
    dy2, x2, dh2 = dy.clone(), x.clone(), dh.clone()
    dy2[7, n - 1], x2[9, k - 1], dh2[11, 5], dy2[m - 1, 0] = float("inf"), float("nan"), float("inf"), float("nan")
    dx2, dz2 = G.nvfp4_linear_grad(dy2, w), G.nvfp4_linear_swiglu_grad(x2, dh2, w)
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[[7, m - 1]] = False
    assert torch.equal(dx2[keep].view(torch.int16), dx[keep].view(torch.int16))
    assert dx2[m - 1].isnan().all() and (~dx2[7].isfinite()).any()
    keep[:] = True
    keep[[9, 11]] = False
    assert torch.equal(dz2[keep].view(torch.int16), dz[keep].view(torch.int16))
    assert dz2[9].isnan().all() and (~dz2[11].isfinite()).sum() == 2


def test_no_rows():
    w = G.NVFP4Tensor.from_numpy(_weight(3, 64, 128, False))
    empty = lambda c: torch.empty((0, c), dtype=torch.float16, device="cuda")  # noqa: E731
    assert G.nvfp4_linear_grad(empty(64), w).shape == (0, 128)
    assert G.nvfp4_linear_swiglu_grad(empty(128), empty(32), w).shape == (0, 64)


@pytest.mark.parametrize("m", [12, 200])
def test_backward_of_the_gated_mlp_in_a_graph(m):
    """The backward pass of s = x + r, y = norm(s), out = linear(swiglu(y)), as a training step runs it: every gradient by
    the library, captured and replayed on other inputs with eager work between, against the 64-bit chain. Each of the
    four fp16 roundings on the way (dh, dz, dy, dx) is at most 2^-11 of its row's values, and passes on with the size of
    the next map: an error of 2e-3 of a row's norm is four of them and FP32's sums, with a factor of two."""
    k, half = 640, 512
    w13, w2 = _weight(1, 2 * half, k, False), _weight(2, k, half, False)
    a, b = G.NVFP4Tensor.from_numpy(w13), G.NVFP4Tensor.from_numpy(w2)
    g = (1 + 0.1 * torch.randn(k, device="cuda")).half()
    x, r, dout = (torch.randn(m, k, device="cuda").half() for _ in range(3))
    out = {}

    def step():
        s, y, _, _ = G.nvfp4_add_rms_norm(x, g, residual=r)
        dh = G.nvfp4_linear_grad(dout, b)
        dz = G.nvfp4_linear_swiglu_grad(y, dh, a)
        dy = G.nvfp4_linear_grad(dz, a)
        out["dx"], out["dw"] = G.nvfp4_add_rms_norm_grad(s, dy, g, ds=dout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kept = dict(out)
    d13, d2 = (torch.from_numpy(_dense(w)).cuda() for w in (w13, w2))
    for _ in range(3):
        x.normal_(), r.normal_(), dout.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in kept.items()}
        step()
        torch.cuda.synchronize()
        for n in got:
            assert torch.equal(got[n].view(torch.uint8), out[n].view(torch.uint8)), n
        s = x.double() + r.double()
        rstd = 1 / torch.sqrt(s.square().mean(dim=1, keepdim=True) + 1e-6)
        y = s * rstd * g.double()
        z = y @ d13.t()
        gate, up = z[:, :half], z[:, half:]
        sig = torch.sigmoid(gate)
        dh = dout.double() @ d2
        dz = torch.cat((dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig), dim=1)
        dy = dz @ d13
        wdy = dy * g.double()
        dx = dout.double() + rstd * (wdy - s * rstd ** 2 * (wdy * s).mean(dim=1, keepdim=True))
        dw = (dy * s * rstd).sum(dim=0)
        err = (got["dx"].double() - dx).norm(dim=1) / dx.norm(dim=1)
        assert float(err.max()) <= 2e-3
        assert float((got["dw"].double() - dw).norm() / dw.norm()) <= 2e-3


def test_two_streams_at_once():
    """The same calls on two streams, each with a workspace of its own, give the bits of one alone."""
    m, n, k = 96, 1056, 640
    w = G.NVFP4Tensor.from_numpy(_weight(3, n, k, False))
    dys = [torch.randn(m, n, device="cuda").half() for _ in range(2)]
    ref = [G.nvfp4_linear_grad(d, w) for d in dys]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[G.nvfp4_linear_grad(d, w, stream=s) for _ in range(4)] for d, s in zip(dys, streams)]
    torch.cuda.synchronize()
    for r, g in zip(ref, got):
        for t in g:
            assert torch.equal(t.view(torch.int16), r.view(torch.int16))


def test_two_streams_at_once_gated():
    """Packed tiles of both kinds and decoded ones on two streams, each with a workspace of its own."""
    n, k = 1056, 640
    w = G.NVFP4Tensor.from_numpy(_weight(3, n, k, False))
    ins = [(torch.randn(m, k, device="cuda").half(), torch.randn(m, n // 2, device="cuda").half()) for m in (300, 1500, 3000)]
    ref = [G.nvfp4_linear_swiglu_grad(x, dh, w) for x, dh in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[G.nvfp4_linear_swiglu_grad(x, dh, w, stream=s) for x, dh in ins] for s in streams]
    torch.cuda.synchronize()
    for one in got:
        for t, r in zip(one, ref):
            assert torch.equal(t.view(torch.int16), r.view(torch.int16))


@pytest.mark.parametrize("m", [5, 40, 100, 600])
def test_grad_of_a_tall_weight_whole_numbers(m):
    """297 planes of 512 weight rows, the last one of 128, bit for bit: a row of dy has twenty terms (|dx| <= 20 * 2 * 12 in
    steps of 1/4 fits fp16's 11 bits), among them one of the last 16 weight rows, one of the last plane and one of the first;
    the others pass through all planes. 600 rows take decoded weights."""
    n, k = 151664 + 16, 128
    w = _weight(m, n, k, True)
    rng = np.random.default_rng(m)
    at = np.empty((m, 20), np.int64)
    at[:, 0], at[:, 1], at[:, 2] = n - 1 - np.arange(m) % 16, n - 17 - np.arange(m) % 112, np.arange(m) % 512
    at[:, 3:] = (512 * (1 + np.arange(17 * m) % 295) + rng.integers(0, 512, 17 * m)).reshape(m, 17)
    dy = np.zeros((m, n), np.float16)
    np.put_along_axis(dy, at, rng.choice(np.array([-2, -1, 1, 2], np.float16), at.shape), axis=1)
    d = _dense(w)
    ref = np.stack([dy[i, at[i]].astype(np.float64) @ d[at[i]] for i in range(m)])
    assert len(set(map(len, map(set, at.tolist())))) == 1 and np.array_equal(ref, ref.astype(np.float16).astype(np.float64))
    ws, ws_ok = _work(G.nvfp4_linear_grad_ws_bytes(m, n, k))
    dx, ok = _guarded(m, k)
    G.nvfp4_linear_grad(_cuda(dy), G.NVFP4Tensor.from_numpy(w), dx=dx, ws=ws)
    torch.cuda.synchronize()
    assert ok() and ws_ok()
    assert np.array_equal(dx.double().cpu().numpy(), ref)
