"""The root-mean-square norm with the residual's sum, its 8-bit rows and its gradient on the GPU, against plain
computations in 64 bits.

Tolerances. A row's sum of squares (or of products) passes at most 32 (one thread's elements) + 6 (lanes) + 16 (waves)
additions and a few more operations, each off by 2^-24 relative of the sum of magnitudes: 64 * 2^-24 = 2^-18 with room.
rstd halves it and adds three roundings. So FP32 values are off by at most EPS32 = 2^-18 relative (to the terms that
they are sums of), and fp16 outputs by 2^-11 relative + 2^-25 (half a step, subnormals included) on top.
"""
import numpy as np
import pytest
import torch

import gemm_nvfp4_amd as G

pytestmark = pytest.mark.gpu

EPS32, HALF, TINY = 2.0 ** -18, 2.0 ** -11, 2.0 ** -25
GUARD = 64  # poisoned elements around every output


def _guarded(shape, dtype):
    """An output of this shape inside a poisoned buffer, and a check that its surroundings kept the poison."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), 0x7F if dtype == torch.uint8 else float("nan"), dtype=dtype, device="cuda")
    if dtype == torch.uint8:
        check = lambda: bool((buf[:GUARD] == 0x7F).all() and (buf[n + GUARD:] == 0x7F).all())  # noqa: E731
    else:
        check = lambda: bool(buf[:GUARD].isnan().all() and buf[n + GUARD:].isnan().all())  # noqa: E731
    return buf[GUARD:n + GUARD].view(shape), check


def _e4m3(q):
    return q.view(torch.float8_e4m3fn).float().double().cpu().numpy()


def _inputs(seed, m, k, residual=True, weight=True):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((m, k)) * np.exp(0.7 * rng.standard_normal(k))).astype(np.float16)
    r = rng.standard_normal((m, k)).astype(np.float16) if residual else None
    w = (1 + 0.3 * rng.standard_normal(k)).astype(np.float16) if weight else None
    return x, r, w


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _forward(x, r, w, eps):
    t = x.astype(np.float64) + (0 if r is None else r.astype(np.float64))
    rstd = 1 / np.sqrt(np.mean(t * t, axis=1, keepdims=True) + eps)
    return t, rstd, t * rstd * (1 if w is None else w.astype(np.float64))


def _close16(got, ref, scale=None, what=""):
    """|got - ref| <= (2^-11 + 2^-18) |ref| + 2^-25 (+ `scale`: what FP32 may add)."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bound = (HALF + EPS32) * np.abs(ref) + TINY + (0 if scale is None else scale)
    worst = np.max(np.abs(got - ref) / bound)
    assert worst <= 1, f"{what}: {worst} times the bound"


SHAPES = [(1, 8), (3, 64), (5, 520), (2, 1024), (7, 1536), (4, 2048), (3, 2056), (2, 4104), (333, 5120), (3, 6152), (2, 8192),
          (2, 8200), (1, 16392), (2, 24584), (2, 32768), (4099, 128)]


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(m, k, residual):
    x, r, w = _inputs(m + k, m, k, residual, weight=k % 16 == 0)
    t, rstd, v = _forward(x, r, w, 1e-6)
    y, y_ok = _guarded((m, k), torch.float16)
    s, s_ok = _guarded((m, k), torch.float16)
    q, q_ok = _guarded((m, k), torch.uint8)
    qs, qs_ok = _guarded((m,), torch.float32)
    out = G.nvfp4_add_rms_norm(_cuda(x), _cuda(w), residual=_cuda(r), s=s if residual else None, y=y, q=q, q_scale=qs,
                               want_q=True)
    torch.cuda.synchronize()
    assert y_ok() and s_ok() and q_ok() and qs_ok()
    assert (out[0] is s) == residual and out[1] is y and out[2] is q and out[3] is qs
    _close16(y, v, what="y")
    if residual:
        _close16(s, t, what="s")
    most = np.abs(v).max(axis=1) / 448
    scale = qs.double().cpu().numpy()
    assert np.all(np.abs(scale - most) <= 2 * EPS32 * most)
    # half a step of a value with three bits behind the point, or of the smallest steps (2^-9 of the scale)
    err = np.abs(_e4m3(q) * scale[:, None] - v)
    assert np.all(err <= (2.0 ** -4 + 4 * EPS32) * np.abs(v) + (2.0 ** -10 * (1 + 4 * EPS32)) * scale[:, None])
    # the outputs one at a time are the same bits
    only_y = G.nvfp4_add_rms_norm(_cuda(x), _cuda(w), residual=_cuda(r))[1]
    _, none, q2, qs2 = G.nvfp4_add_rms_norm(_cuda(x), _cuda(w), residual=_cuda(r), want_y=False, want_q=True)
    assert none is None and torch.equal(only_y.view(torch.int16), y.view(torch.int16))
    assert torch.equal(q2, q) and torch.equal(qs2, qs)


@pytest.mark.parametrize("k", [64, 2048, 5120, 16384])
def test_rows_do_not_depend_on_the_batch(k):
    x, r, w = (_cuda(a) for a in _inputs(k, 37, k))
    s, y, q, qs = G.nvfp4_add_rms_norm(x, w, residual=r, want_q=True)
    for lo, hi in ((0, 1), (36, 37), (5, 18)):
        s1, y1, q1, qs1 = G.nvfp4_add_rms_norm(x[lo:hi].contiguous(), w, residual=r[lo:hi].contiguous(), want_q=True)
        assert torch.equal(s1.view(torch.int16), s[lo:hi].view(torch.int16))
        assert torch.equal(y1.view(torch.int16), y[lo:hi].view(torch.int16))
        assert torch.equal(q1, q[lo:hi]) and torch.equal(qs1, qs[lo:hi])


@pytest.mark.parametrize("k", [128, 5120, 9216])
def test_in_place(k):
    x, r, w = (_cuda(a) for a in _inputs(k + 1, 9, k))
    s, y, _, _ = G.nvfp4_add_rms_norm(x, w, residual=r)
    x1, r1 = x.clone(), r.clone()
    s1, y1, _, _ = G.nvfp4_add_rms_norm(x1, w, residual=r1, s=r1, y=x1)
    assert torch.equal(r1.view(torch.int16), s.view(torch.int16)) and torch.equal(x1.view(torch.int16), y.view(torch.int16))
    dy, ds = torch.randn_like(y), torch.randn_like(y)
    dx, dw = G.nvfp4_add_rms_norm_grad(s, dy, w, ds=ds)
    for other in (dy.clone(), ds.clone()):
        over = other.clone()
        a, b = (over, ds) if torch.equal(other, dy) else (dy, over)
        dx1, dw1 = G.nvfp4_add_rms_norm_grad(s, a, w, ds=b, dx=over)
        assert torch.equal(dx1.view(torch.int16), dx.view(torch.int16)) and torch.equal(dw1, dw)


def test_special_rows():
    k = 2056
    x = np.random.default_rng(3).standard_normal((6, k)).astype(np.float16)
    x[0] = 0
    x[1, 7] = np.inf
    x[2, 9] = np.nan
    x[3] = 65504  # squares far above fp16, fine in FP32
    x[4] = 6e-8   # the smallest fp16: its mean square is below eps
    _, y, q, qs = G.nvfp4_add_rms_norm(_cuda(x), want_q=True)
    y, qs, v = y.double().cpu().numpy(), qs.cpu().numpy(), _e4m3(q)
    assert np.all(y[0] == 0) and np.all(v[0] == 0) and qs[0] == np.float32(2.0 ** -100)
    assert np.isnan(y[1, 7]) and np.all(np.delete(y[1], 7) == 0) and np.isnan(qs[1]) and np.isnan(v[1]).all()
    assert np.isnan(y[2]).all() and np.isnan(qs[2]) and np.isnan(v[2]).all()
    for row in (3, 4, 5):
        _close16(torch.from_numpy(y[row:row + 1]), _forward(x[row:row + 1], None, None, 1e-6)[2])
    assert np.all(np.isfinite(v[3:])) and np.all(v[3] == 448)
    zero = G.nvfp4_add_rms_norm(torch.zeros((1, 64), dtype=torch.float16, device="cuda"), eps=0.0)[1]
    assert zero.isnan().all()


def _grad(t, dy, ds, w, eps):
    """dx, dweight and the magnitudes that FP32 roundings are relative to."""
    t, dy = t.astype(np.float64), dy.astype(np.float64)
    g = dy * (1 if w is None else w.astype(np.float64))
    rstd = 1 / np.sqrt(np.mean(t * t, axis=1, keepdims=True) + eps)
    dx = rstd * (g - t * rstd ** 2 * np.mean(g * t, axis=1, keepdims=True))
    size = rstd * (np.abs(g) + np.abs(t) * rstd ** 2 * np.mean(np.abs(g * t), axis=1, keepdims=True))
    if ds is not None:
        dx, size = dx + ds, size + np.abs(ds.astype(np.float64))
    return dx, size, np.sum(dy * t * rstd, axis=0), np.sum(np.abs(dy * t * rstd), axis=0)


@pytest.mark.parametrize("m,k", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_gradient(m, k, residual):
    x, _, w = _inputs(2 * m + k, m, k, False, weight=k % 16 == 0)
    rng = np.random.default_rng(k)
    dy = rng.standard_normal((m, k)).astype(np.float16)
    ds = rng.standard_normal((m, k)).astype(np.float16) if residual else None
    dx, dx_ok = _guarded((m, k), torch.float16)
    dw, dw_ok = _guarded((k,), torch.float32)
    need = G.nvfp4_add_rms_norm_grad_ws_bytes(m, k)
    ws, ws_ok = _guarded((need,), torch.uint8)
    G.nvfp4_add_rms_norm_grad(_cuda(x), _cuda(dy), _cuda(w), ds=_cuda(ds), dx=dx, dweight=dw, ws=ws)
    torch.cuda.synchronize()
    assert dx_ok() and dw_ok() and ws_ok()
    ref, size, ref_w, size_w = _grad(x, dy, ds, w, 1e-6)
    _close16(dx, ref, scale=2 * EPS32 * size, what="dx")
    # a column's sum passes m / 512 rows of a block, its groups, and the blocks: far fewer than 2^6 + m / 256 additions
    bound = (2 * EPS32 + m / 256 * 2.0 ** -24) * size_w
    assert np.all(np.abs(dw.double().cpu().numpy() - ref_w) <= bound)
    # each output alone: the same bits
    dx1, none = G.nvfp4_add_rms_norm_grad(_cuda(x), _cuda(dy), _cuda(w), ds=_cuda(ds), want_dweight=False)
    assert none is None and torch.equal(dx1.view(torch.int16), dx.view(torch.int16))
    none, dw1 = G.nvfp4_add_rms_norm_grad(_cuda(x), _cuda(dy), _cuda(w), want_dx=False)
    assert none is None and torch.equal(dw1, dw)


def test_gradient_against_differences():
    """d loss / dt and d loss / dweight of loss = sum(dy * y) by central differences of the forward formula in 64 bits."""
    m, k, h = 3, 64, 1e-6
    x, _, w = _inputs(5, m, k, False)
    dy = np.random.default_rng(6).standard_normal((m, k)).astype(np.float16)
    dx, dw = G.nvfp4_add_rms_norm_grad(_cuda(x), _cuda(dy), _cuda(w))
    loss = lambda t, ww: float(np.sum(dy.astype(np.float64) * (t / np.sqrt(np.mean(t * t, axis=1, keepdims=True) + 1e-6) * ww)))  # noqa: E731,E501
    t0, w0 = x.astype(np.float64), w.astype(np.float64)
    _, size, _, size_w = _grad(x, dy, None, w, 1e-6)
    for i, j in ((0, 0), (1, 17), (2, 63)):
        d = np.zeros_like(t0)
        d[i, j] = h
        ref = (loss(t0 + d, w0) - loss(t0 - d, w0)) / (2 * h)
        assert abs(float(dx[i, j]) - ref) <= (HALF + EPS32) * abs(ref) + 2 * EPS32 * size[i, j] + TINY + 1e-7
        e = np.zeros_like(w0)
        e[j] = h
        ref = (loss(t0, w0 + e) - loss(t0, w0 - e)) / (2 * h)
        assert abs(float(dw[j]) - ref) <= 2 * EPS32 * size_w[j] + 1e-7


def test_gradient_of_an_empty_batch():
    t = torch.empty((0, 128), dtype=torch.float16, device="cuda")
    dw = torch.full((128,), float("nan"), device="cuda")
    dx, got = G.nvfp4_add_rms_norm_grad(t, t, dweight=dw)
    assert dx.shape == (0, 128) and got is dw and torch.equal(dw, torch.zeros_like(dw))
    assert G.nvfp4_add_rms_norm(t)[1].shape == (0, 128)


def test_graph_replays_on_another_stream():
    m, k = 70, 5120
    x, r, w = (_cuda(a) for a in _inputs(1, m, k))
    dy = torch.randn(m, k, device="cuda").half()
    s, y = torch.empty_like(x), torch.empty_like(x)
    q, qs = torch.empty((m, k), dtype=torch.uint8, device="cuda"), torch.empty(m, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(k, device="cuda")
    ws = torch.empty(G.nvfp4_add_rms_norm_grad_ws_bytes(m, k), dtype=torch.uint8, device="cuda")

    def step():
        G.nvfp4_add_rms_norm(x, w, residual=r, s=s, y=y, q=q, q_scale=qs, want_q=True)
        G.nvfp4_add_rms_norm_grad(s, dy, w, ds=y, dx=dx, dweight=dw, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        a, b, _ = _inputs(seed + 10, m, k)
        x.copy_(_cuda(a)), r.copy_(_cuda(b)), dy.normal_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in (s, y, q, qs, dx, dw)]
        for o in (s, y, q, qs, dx, dw, ws):
            o.zero_()
        step()
        torch.cuda.synchronize()
        for u, v in zip(got, (s, y, q, qs, dx, dw)):
            assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))


def test_offsets_past_2_31_elements():
    """More than 2^32 bytes a matrix: the last rows against the same rows alone."""
    m, k = 65600, 32768
    x = torch.empty((m, k), dtype=torch.float16, device="cuda")
    x[:1024].normal_()
    for lo in range(1024, m, 1024):
        hi = min(m, lo + 1024)
        x[lo:hi] = x[:hi - lo]
    y = G.nvfp4_add_rms_norm(x)[1]
    ref = G.nvfp4_add_rms_norm(x[-3:].contiguous())[1]
    assert torch.equal(y[-3:].view(torch.int16), ref.view(torch.int16))
    dx, _ = G.nvfp4_add_rms_norm_grad(x, x, want_dweight=False, dx=y)
    ref, _ = G.nvfp4_add_rms_norm_grad(x[-3:].contiguous(), x[-3:].contiguous(), want_dweight=False)
    assert torch.equal(dx[-3:].view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("m,k", [(2 ** 26, 8), (2 ** 24 + 1, 2056), (2 ** 22 + 1, 8200)])
def test_more_rows_than_one_grid_axis_holds(m, k):
    """A launch holds fewer than 2^32 threads along one axis; a row has 64, 256 and 1024 of them here. In place; the first,
    the last and the rows around 2^20 blocks against the same rows alone."""
    x = torch.empty((m, k), dtype=torch.float16, device="cuda")
    pattern = torch.randn((4093, k), device="cuda").half()  # a prime number of rows: blocks apart hold other rows
    for lo in range(0, m, 4093 * 64):
        part = x[lo:lo + 4093 * 64]
        part.copy_(pattern.repeat(-(-len(part) // 4093), 1)[:len(part)])
    at = [0, 1, 2 ** 20 - 1, 2 ** 20, 2 ** 22 - 1, 2 ** 22, m // 2, m - 5, m - 2, m - 1]
    rows = x[at].contiguous()
    G.nvfp4_add_rms_norm(x, y=x)
    ref = G.nvfp4_add_rms_norm(rows)[1]
    assert torch.equal(x[at].view(torch.int16), ref.view(torch.int16))
    del x
    torch.cuda.empty_cache()


def test_given_8_bit_outputs_are_written():
    """q or q_scale alone, or both, without want_q: written as with it."""
    x = torch.randn(5, 520, device="cuda").half()
    _, y, q, qs = G.nvfp4_add_rms_norm(x, want_q=True)
    for give in ("q", "q_scale", "both"):
        mine = torch.full_like(q, 0x7F) if give != "q_scale" else None
        scale = torch.full_like(qs, float("nan")) if give != "q" else None
        _, y1, q1, qs1 = G.nvfp4_add_rms_norm(x, q=mine, q_scale=scale)
        assert (mine is None or q1 is mine) and (scale is None or qs1 is scale)
        assert torch.equal(q1, q) and torch.equal(qs1, qs) and torch.equal(y1, y)


# a turn of the gradient's row loop is 2048, 512 and 256 rows at 64, 256 and 1024 threads a row: several turns, the last ragged
@pytest.mark.parametrize("m,k", [(5000, 2048), (1301, 2056), (1301, 5120), (1030, 8192), (701, 8200), (520, 16392), (600, 32768)])
@pytest.mark.parametrize("residual", [False, True])
def test_gradient_of_several_turns(m, k, residual):
    x, _, w = _inputs(m + k, m, k, False)
    rng = np.random.default_rng(m)
    dy = rng.standard_normal((m, k)).astype(np.float16)
    ds = rng.standard_normal((m, k)).astype(np.float16) if residual else None
    dx, dx_ok = _guarded((m, k), torch.float16)
    dw, dw_ok = _guarded((k,), torch.float32)
    ws, ws_ok = _guarded((G.nvfp4_add_rms_norm_grad_ws_bytes(m, k),), torch.uint8)
    cx, cdy, cds, cw = _cuda(x), _cuda(dy), _cuda(ds), _cuda(w)
    G.nvfp4_add_rms_norm_grad(cx, cdy, cw, ds=cds, dx=dx, dweight=dw, ws=ws)
    torch.cuda.synchronize()
    assert dx_ok() and dw_ok() and ws_ok()
    ref, size, ref_w, size_w = _grad(x, dy, ds, w, 1e-6)
    _close16(dx, ref, scale=2 * EPS32 * size, what="dx")
    assert np.all(np.abs(dw.double().cpu().numpy() - ref_w) <= (2 * EPS32 + m / 256 * 2.0 ** -24) * size_w)
    # a row's dx has one order of adding: the same bits from calls of one turn
    for lo in range(0, m, 255):
        part = slice(lo, min(m, lo + 255))
        one, _ = G.nvfp4_add_rms_norm_grad(cx[part], cdy[part], cw, ds=None if ds is None else cds[part], want_dweight=False)
        assert torch.equal(one.view(torch.int16), dx[part].view(torch.int16)), lo
    # dweight again: its order is fixed
    _, again = G.nvfp4_add_rms_norm_grad(cx, cdy, cw, ds=cds)
    assert torch.equal(again, dw)
