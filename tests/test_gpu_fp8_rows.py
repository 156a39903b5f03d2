"""The channel-FP8 projection of 8-bit rows on the GPU against 64-bit computations.

Whole numbers: products and sums exact in FP32, results below 2^11, compared bit for bit. Random bytes: one fp16
rounding (2^-11 relative, 2^-25 for subnormals), two FP32 products (2^-22 relative together) and the sum, whose every
addition is off by at most 2^-23 of the sum of magnitudes so far: K * 2^-23 of that sum bounds any order of adding.
"""
import numpy as np
import pytest
import torch

import gemm_nvfp4_amd as G

pytestmark = pytest.mark.gpu

# batch sizes on both sides of every change of kernel: few rows of few columns stream, up to 16 or 32, more take tiles
BATCHES = [1, 2, 15, 16, 17, 32, 33, 64, 65, 130, 333]


def _values(b):
    return torch.from_numpy(b).view(torch.float8_e4m3fn).double()


def _case(seed, m, n, k, whole):
    rng = np.random.default_rng(seed)
    if whole:  # bytes of -2 .. 2, scales that are powers of two
        ints = np.array([0xC0, 0xB8, 0x00, 0x38, 0x40], np.uint8)
        xq, wq = ints[rng.integers(0, 5, (m, k))], ints[rng.integers(0, 5, (n, k))]
        keep = rng.random((m, k)) < min(1.0, 200 / k)  # few enough terms to stay below 2^11
        xq = np.where(keep, xq, 0).astype(np.uint8)
        xs, ws = 2.0 ** rng.integers(-2, 1, m), 2.0 ** rng.integers(-2, 1, n)
    else:
        xq, wq = rng.integers(0, 256, (m, k)).astype(np.uint8), rng.integers(0, 256, (n, k)).astype(np.uint8)
        xq[(xq & 0x7F) == 0x7F] = 0x01  # no NaN
        wq[(wq & 0x7F) == 0x7F] = 0x81
        xs, ws = rng.uniform(1e-4, 1e-3, m), rng.uniform(1e-4, 1e-3, n)
    return xq, xs.astype(np.float32), wq, ws.astype(np.float32)


def _run(xq, xs, wq, ws, y=None):
    w = G.FP8ChannelTensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    return G.nvfp4_linear_fp8_rows(torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda(), w, y=y)


@pytest.mark.parametrize("n,k", [(16, 128), (48, 640), (272, 1536), (64, 16384)])
@pytest.mark.parametrize("m", BATCHES)
def test_whole_numbers(m, n, k):
    case = _case(m + n + k, m, n, k, True)
    xq, xs, wq, ws = case
    ref = (_values(xq) @ _values(wq).t()) * torch.from_numpy(xs).double()[:, None] * torch.from_numpy(ws).double()
    assert ref.abs().max() < 2048
    buf = torch.full((m * n + 256,), float("nan"), dtype=torch.float16, device="cuda")
    y = _run(*case, y=buf[128:128 + m * n].view(m, n))
    assert torch.equal(y.double().cpu(), ref.half().double())
    assert buf[:128].isnan().all() and buf[128 + m * n:].isnan().all()


@pytest.mark.parametrize("m,n,k", [(1, 64, 5120), (13, 4352, 5120), (33, 80, 384), (333, 1040, 2048), (1030, 2064, 896)])
def test_random_bytes(m, n, k):
    xq, xs, wq, ws = case = _case(m, m, n, k, False)
    a, b = _values(xq), _values(wq)
    scale = torch.from_numpy(xs).double()[:, None] * torch.from_numpy(ws).double()
    ref, size = (a @ b.t()) * scale, (a.abs() @ b.abs().t()) * scale
    err = (_run(*case).double().cpu() - ref).abs()
    assert bool((err <= (2.0 ** -11 + 2.0 ** -21) * ref.abs() + 2.0 ** -25 + k * 2.0 ** -23 * size).all())


@pytest.mark.parametrize("n,k", [(4352, 5120), (208, 1664)])
def test_rows_do_not_depend_on_the_batch(n, k):
    """One result for a row at every batch size: streams, small, medium and large tiles."""
    m = 4000
    xq, xs, wq, ws = _case(n, m, n, k, False)
    w = G.FP8ChannelTensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    x, s = torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda()
    y = G.nvfp4_linear_fp8_rows(x, s, w)
    # streams of 1, 17 and 30 rows, then tiles: of 4352 x 5120 one size for each shape
    for lo, hi in ((0, 1), (3999, 4000), (77, 94), (100, 130), (1000, 1080), (300, 556), (300, 700), (200, 1050),
                   (3, 1299), (1, 2051), (0, 2400), (7, 3207)):
        part = G.nvfp4_linear_fp8_rows(x[lo:hi].contiguous(), s[lo:hi].contiguous(), w)
        assert torch.equal(part.view(torch.int16), y[lo:hi].view(torch.int16)), (lo, hi)


@pytest.mark.parametrize("m", [5, 100, 700])
def test_values_that_are_not_numbers_stay_in_their_row_or_column(m):
    n, k = 4352, 1024
    xq, xs, wq, ws = _case(m, m, n, k, False)
    plain = _run(xq, xs, wq, ws)
    xq[3, 1000], wq[17, 5], xs[1], ws[4000] = 0x7F, 0xFF, np.inf, np.nan
    y = _run(xq, xs, wq, ws)
    bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
    bad[3], bad[1], bad[:, 17], bad[:, 4000] = True, True, True, True
    assert torch.equal(y[~bad].view(torch.int16), plain[~bad].view(torch.int16))
    assert y[3].isnan().all() and y[:, 17].isnan().all() and y[:, 4000].isnan().all()
    assert (~y[1].isfinite()).all()


def test_two_streams_at_once():
    """Batches of several kernels on two streams at once, again and again, give the bits of one call alone."""
    n, k = 4352, 5120
    xq, xs, wq, ws = _case(5, 1000, n, k, False)
    w = G.FP8ChannelTensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    ins = [(torch.from_numpy(xq[:m]).cuda(), torch.from_numpy(xs[:m]).cuda()) for m in (1, 20, 120, 333, 640, 1000)]
    ref = [G.nvfp4_linear_fp8_rows(x, s, w) for x, s in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[G.nvfp4_linear_fp8_rows(x, s, w, stream=t) for t in streams for _ in range(3)] for x, s in ins]
    torch.cuda.synchronize()
    for r, many in zip(ref, got):
        for y in many:
            assert torch.equal(y.view(torch.int16), r.view(torch.int16))


def test_no_rows():
    _, _, wq, ws = _case(0, 1, 64, 256, True)
    y = _run(np.zeros((0, 256), np.uint8), np.zeros(0, np.float32), wq, ws)
    assert y.shape == (0, 64)


def test_behind_the_norm_in_a_graph():
    """norm -> 8-bit rows -> projection, as a decode step runs them, captured and replayed with other inputs; against
    the 64-bit chain within the rows' own 8-bit rounding (2^-4 relative of a value at most, 2^-10 of the scale for the
    smallest): |dy| <= sum over k of the row's rounding times |w|."""
    m, n, k = 9, 512, 2048
    _, _, wq, ws = _case(1, 1, n, k, False)
    ws *= 1e-2
    w = G.FP8ChannelTensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    x, r = torch.randn(m, k, device="cuda").half(), torch.randn(m, k, device="cuda").half()
    g = (1 + 0.1 * torch.randn(k, device="cuda")).half()
    s, y = torch.empty_like(x), torch.empty((m, n), dtype=torch.float16, device="cuda")
    q, qs = torch.empty((m, k), dtype=torch.uint8, device="cuda"), torch.empty(m, device="cuda")

    def step():
        G.nvfp4_add_rms_norm(x, g, residual=r, s=s, q=q, q_scale=qs, want_y=False, want_q=True)
        G.nvfp4_linear_fp8_rows(q, qs, w, y=y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    wd = _values(wq).cuda() * w.channel_scale.double()[:, None]
    for _ in range(3):
        x.normal_(), r.normal_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(replayed.view(torch.int16), y.view(torch.int16))
        t = x.double() + r.double()
        v = t / torch.sqrt(t.square().mean(dim=1, keepdim=True) + 1e-6) * g.double()
        ref = v @ wd.t()
        step8 = (2.0 ** -4 + 2.0 ** -14) * v.abs() + 2.0 ** -10 * 1.001 * qs.double()[:, None]
        bound = step8 @ wd.abs().t() + 2.0 ** -11 * ref.abs() + 2.0 ** -25 + (k + 64) * 2.0 ** -23 * (v.abs() @ wd.abs().t())
        assert bool(((y.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("n,k", [(64, 5120), (512, 8192), (80, 16384), (4096, 4096)])
def test_wide_streams_give_the_bits_of_tiles(n, k):
    """Up to 4096 columns stream up to 16 rows with one row tile, and 17 to 32 with two where K is at least 4096; the
    larger batches take tiles. On random bytes, whose sums depend on the order of adding."""
    m = 400
    xq, xs, wq, ws = _case(n + k, m, n, k, False)
    w = G.FP8ChannelTensor(torch.from_numpy(wq).cuda(), torch.from_numpy(ws).cuda())
    x, s = torch.from_numpy(xq).cuda(), torch.from_numpy(xs).cuda()
    y = G.nvfp4_linear_fp8_rows(x, s, w)
    for lo, hi in ((0, 1), (399, 400), (7, 23), (77, 94), (100, 130), (368, 400), (200, 233), (0, 64), (50, 200)):
        part = G.nvfp4_linear_fp8_rows(x[lo:hi].contiguous(), s[lo:hi].contiguous(), w)
        assert torch.equal(part.view(torch.int16), y[lo:hi].view(torch.int16)), (lo, hi)
