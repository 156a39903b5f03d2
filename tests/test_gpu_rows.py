"""Rows moved by the routing plan on the GPU (nvfp4_moe_permute, nvfp4_moe_unpermute,
nvfp4_moe_unpermute_grad) against plain 64-bit computations on the host.

Tolerances, from the definition (u16 = 2^-11 and u32 = 2^-24 are half a step of fp16 and FP32; fp16 has a
fixed step of 2^-24 below 2^-14, so half a step there is 2^-25):
  permute      without weights the bits of x. With weights fp16_rne(fl32(w * x)): numpy's own FP32 product
               and conversion, compared bit for bit.
  unpermute    topk fmaf steps, each off by at most u32 of a partial sum, whose magnitude is at most
               S = sum |w y| (1 + topk u32); then one rounding to fp16:
               |out - ref| <= u16 |ref| + 1.01 topk u32 S + 2^-25.
  grad         dys as the weighted permute, bit for bit. dw: a fixed tree whose longest path is n =
               8 ceil(pieces / threads) fmaf steps in a lane, 6 over the wave and up to 3 over the waves:
               |dw - ref| <= 1.01 (n + 9) u32 sum |d y|.
"""
import itertools

import numpy as np
import pytest
import torch

import gemm_nvfp4_amd as G
from oracle import oracle as O

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -11, 2.0 ** -24
POISON = 0x7E00


def _case(m, topk, e, k, seed, bad="some"):
    rng = np.random.default_rng([seed, m, topk, e, k])
    ids = rng.integers(0, e, size=(m, topk)).astype(np.int32)  # repeated ids within a token occur
    if bad == "some":
        ids[rng.random((m, topk)) < 0.2] = -1
        ids[rng.random((m, topk)) < 0.05] = e + 3
    elif bad == "all":
        ids[:] = -1
    if bad == "some" and m >= 2:
        ids[m // 2] = -1  # a token with no valid slot
    x = rng.standard_normal((m, k)).astype(np.float16)
    ys = rng.standard_normal((m * topk, k)).astype(np.float16)
    w = rng.standard_normal((m, topk)).astype(np.float32)
    pos = O.plan(ids, e)["pos_of_pair"].reshape(m, topk)
    return ids, x, ys, w, pos


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _poisoned(*shape):
    return torch.full(shape, POISON, dtype=torch.int16, device="cuda").view(torch.float16)


def _bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _expect_sorted(rows, w, pos, total, topk):
    """Bits of the sorted rows: fp16_rne(fl32(w * row)), or the row, over poison."""
    out = np.full((total, rows.shape[1]), POISON, np.uint16)
    for t, k in zip(*np.nonzero(pos >= 0)):
        r = rows[t] if w is None else (w[t, k] * rows[t].astype(np.float32)).astype(np.float16)
        out[pos[t, k]] = r.view(np.uint16)
    return out


def _check_unpermute(got, ys, w, pos, what):
    m, topk = pos.shape
    there = pos >= 0
    rows = np.where(there[:, :, None], ys.astype(np.float64)[np.maximum(pos, 0)], 0.0)
    terms = rows if w is None else np.where(there, w.astype(np.float64), 0.0)[:, :, None] * rows
    ref, s = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    tol = U16 * np.abs(ref) + 1.01 * topk * U32 * s + 2.0 ** -25
    err = np.abs(got.cpu().double().numpy() - ref)
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol)}"
    none = ~there.any(axis=1)
    assert not _bits(got)[none].any(), f"{what}: a token without slots is not +0"


def _check_grad(dys, dw, dout, ys, w, pos, what):
    m, topk = pos.shape
    k = dout.shape[1]
    if dys is not None:
        assert np.array_equal(_bits(dys), _expect_sorted(dout, w, pos, ys.shape[0], topk)), f"{what}: dys"
    there = pos >= 0
    prod = dout.astype(np.float64)[:, None, :] * ys.astype(np.float64)[np.maximum(pos, 0)]
    ref = np.where(there, prod.sum(axis=2), 0.0)
    pieces = k // 8
    threads = min(256, -(-pieces // 64) * 64)
    n = 8 * -(-pieces // threads) + 9
    tol = np.where(there, 1.01 * n * U32 * np.abs(prod).sum(axis=2), 0.0)
    got = dw.cpu().double().numpy()
    assert (np.abs(got - ref) <= tol).all(), f"{what}: dw off by {np.abs(got - ref).max()}"
    assert not np.signbit(got[~there]).any()


# one token and many, odd sizes, one slot and 32, rows of one piece and of many, plans of both builders
SHAPES = [(1, 1, 1, 8), (1, 10, 512, 2048), (3, 2, 8, 264), (16, 10, 512, 2048), (7, 32, 40, 136), (33, 17, 5, 5120),
          (129, 3, 64, 520), (1100, 2, 16, 72), (2, 1, 4096, 65536), (257, 8, 128, 1032)]


@pytest.mark.parametrize("bad", ["none", "some", "all"])
@pytest.mark.parametrize("m,topk,e,k", SHAPES)
def test_rows(m, topk, e, k, bad):
    ids, x, ys, w, pos = _case(m, topk, e, k, 1, bad)
    plan = G.nvfp4_moe_plan(_dev(ids), e)
    dx, dys, dw = _dev(x), _dev(ys), _dev(w)
    for weights in (None, w):
        xs = G.nvfp4_moe_permute(plan, m, topk, e, dx, None if weights is None else dw, xs=_poisoned(m * topk, k))
        torch.cuda.synchronize()
        assert np.array_equal(_bits(xs), _expect_sorted(x, weights, pos, m * topk, topk))
        out = G.nvfp4_moe_unpermute(plan, m, topk, e, dys, None if weights is None else dw, out=_poisoned(m, k))
        torch.cuda.synchronize()
        _check_unpermute(out, ys, weights, pos, f"weights {weights is not None}")
    g, gw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, dx, dys, dw, dys=_poisoned(m * topk, k),
                                       dweights=torch.full((m, topk), float("nan"), device="cuda"))
    torch.cuda.synchronize()
    _check_grad(g, gw, x, ys, w, pos, "grad")
    none, gw2 = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, dx, dys, None, want_dys=False)
    assert none is None and torch.equal(gw2.view(torch.int32), gw.view(torch.int32))


def test_longer_row_buffers_and_empty_batch():
    """Bucket-order buffers may hold more than M*topk rows; M = 0 touches nothing."""
    m, topk, e, k = 5, 3, 7, 48
    ids, x, ys, w, pos = _case(m, topk, e, k, 3)
    plan = G.nvfp4_moe_plan(_dev(ids), e)
    xs = G.nvfp4_moe_permute(plan, m, topk, e, _dev(x), xs=_poisoned(m * topk + 4, k))
    torch.cuda.synchronize()
    assert np.array_equal(_bits(xs), _expect_sorted(x, None, pos, m * topk + 4, topk))
    empty = torch.empty((0, k), dtype=torch.float16, device="cuda")
    p0 = torch.zeros(4096, dtype=torch.int32, device="cuda")
    keep = _poisoned(4, k)
    G.nvfp4_moe_permute(p0, 0, topk, e, empty, xs=keep)
    assert G.nvfp4_moe_unpermute(p0, 0, topk, e, keep).shape == (0, k)
    g, gw = G.nvfp4_moe_unpermute_grad(p0, 0, topk, e, empty, keep, torch.empty((0, topk), device="cuda"), dys=keep)
    torch.cuda.synchronize()
    assert gw.shape == (0, topk) and (_bits(keep) == POISON).all()


def test_values_that_are_not_finite():
    """NaN and infinities stay in their token's rows; what skipped pairs hold is not read."""
    m, topk, e, k = 6, 3, 8, 64
    ids, x, ys, w, pos = _case(m, topk, e, k, 5)
    ids[:, 0] = np.arange(m) % e  # every token keeps a slot
    pos = O.plan(ids, e)["pos_of_pair"].reshape(m, topk)
    n_valid = int((pos >= 0).sum())
    ys[n_valid:] = np.nan
    w[pos < 0] = np.nan
    plan = G.nvfp4_moe_plan(_dev(ids), e)
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, _dev(ys), _dev(w))
    _check_unpermute(out, np.where(np.isnan(ys), 0, ys).astype(np.float16), np.nan_to_num(w), pos, "NaN in skipped places")
    _, gw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, _dev(x), _dev(ys), _dev(w))
    assert np.array_equal(gw.cpu().numpy() == 0, pos < 0)
    clean = ys.copy()
    ys[pos[2, 0], 5], ys[pos[4, 0], 6] = np.nan, np.inf
    w[4, 0] = -2.0
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, _dev(clean), _dev(w))
    big = G.nvfp4_moe_unpermute(plan, m, topk, e, _dev(ys), _dev(w)).cpu().numpy()
    assert np.isnan(big[2, 5]) and big[4, 6] == -np.inf
    rest = np.ones_like(big, bool)
    rest[2, 5] = rest[4, 6] = False
    assert np.array_equal(big.view(np.uint16)[rest], _bits(out)[rest])
    x[3, 7] = 60000.0
    w[3, :] = 2.0  # overflows to +inf, as fp16 rounding says
    xs = G.nvfp4_moe_permute(plan, m, topk, e, _dev(x), _dev(w)).cpu().numpy()
    assert (xs[pos[3][pos[3] >= 0], 7] == np.inf).all()


def test_skipped_pairs_beside_a_row_of_nan():
    """Bucket row 0 holds NaN and infinities; tokens that do not own it are untouched by it, skipped slots too."""
    m, topk, e, k = 9, 10, 16, 136
    ids, x, ys, w, pos = _case(m, topk, e, k, 6)
    ys[0, ::2], ys[0, 1::2] = np.nan, np.inf
    owner = int(np.argwhere(pos == 0)[0][0])
    plan = G.nvfp4_moe_plan(_dev(ids), e)
    g, gw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, _dev(x), _dev(ys), _dev(w), dys=_poisoned(m * topk, k))
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, _dev(ys), _dev(w)).cpu().numpy()
    rest = np.arange(m) != owner
    assert np.isfinite(out[rest]).all() and not np.isfinite(out[owner]).all()
    gw = gw.cpu().numpy()
    assert np.isfinite(gw[pos != 0]).all() and np.isnan(gw[pos == 0]).all() and (gw[pos < 0] == 0).all()
    assert np.array_equal(_bits(g), _expect_sorted(x, w, pos, m * topk, topk))


def test_offsets_past_32_bits():
    """Bucket rows of 5.2 GB: rows on both sides of the 2^32-byte line, against the rows they come from."""
    m, topk, e, k = 40000, 8, 64, 8192
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, e, (m, topk), generator=gen, device="cuda", dtype=torch.int32)
    ids[5] = -1
    x = torch.randn((m, k), generator=gen, device="cuda").half()
    w = torch.rand((m, topk), generator=gen, device="cuda")
    plan = G.nvfp4_moe_plan(ids, e)
    pos = G.plan_fields(plan, m, topk, e)["pos_of_pair"].reshape(m, topk)
    xs = G.nvfp4_moe_permute(plan, m, topk, e, x)
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, xs, w)
    dys, dw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, x, xs, w)
    torch.cuda.synchronize()
    rng = np.random.default_rng(4)
    line = 2 ** 32 // (2 * k)
    for t in np.unique(np.concatenate([rng.integers(0, m, 20), [0, 5, m - 1], np.argwhere(abs(pos - line) < 2)[:, 0]])):
        row = x[t].cpu().numpy()
        for s in range(topk):
            if pos[t, s] < 0:
                continue
            j = int(pos[t, s])
            assert torch.equal(xs[j], x[t])
            want = (w[t, s].cpu().numpy() * row.astype(np.float32)).astype(np.float16)
            assert np.array_equal(_bits(dys[j]), want.view(np.uint16))
        terms = np.where(pos[t] >= 0, w[t].cpu().double().numpy(), 0.0)
        ref = terms.sum() * row.astype(np.float64)
        err = np.abs(out[t].cpu().double().numpy() - ref)
        assert (err <= U16 * np.abs(ref) + 1.01 * topk * U32 * np.abs(terms).sum() * np.abs(row.astype(np.float64)) + 2.0 ** -25).all()
        dot = (row.astype(np.float64) ** 2).sum()
        n = 8 * -(-(k // 8) // 256) + 9
        assert (np.abs(dw[t].cpu().double().numpy() - np.where(pos[t] >= 0, dot, 0.0)) <= 1.01 * n * U32 * dot).all()


def test_results_do_not_depend_on_the_batch():
    m, topk, e, k = 70, 4, 16, 1032
    ids, x, ys, w, pos = _case(m, topk, e, k, 7)
    plan = G.nvfp4_moe_plan(_dev(ids), e)
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, _dev(ys), _dev(w))
    _, gw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, _dev(x), _dev(ys), _dev(w))
    for t in (0, 1, 33, m - 1):
        one = np.zeros((topk, k), np.float16)
        p1 = O.plan(ids[t:t + 1], e)["pos_of_pair"]
        for s in range(topk):
            if p1[s] >= 0:
                one[p1[s]] = ys[pos[t, s]]
        plan1 = G.nvfp4_moe_plan(_dev(ids[t:t + 1]), e)
        o1 = G.nvfp4_moe_unpermute(plan1, 1, topk, e, _dev(one), _dev(w[t:t + 1]))
        _, g1 = G.nvfp4_moe_unpermute_grad(plan1, 1, topk, e, _dev(x[t:t + 1]), _dev(one), _dev(w[t:t + 1]))
        assert torch.equal(o1[0].view(torch.int16), out[t].view(torch.int16))
        assert torch.equal(g1[0].view(torch.int32), gw[t].view(torch.int32))


def test_gradients_against_differences():
    """d loss / d input of unpermute and permute against central differences of the 64-bit formula, for loss =
    <out, c>: the maps are linear, so a difference of step 1 is exact but for 64-bit rounding."""
    m, topk, e, k = 5, 3, 6, 40
    ids, x, ys, w, pos = _case(m, topk, e, k, 9)
    plan = G.nvfp4_moe_plan(_dev(ids), e)
    c = x  # the gradient that comes from above
    there = pos >= 0

    def loss(ys64, w64):
        rows = np.where(there[:, :, None], ys64[np.maximum(pos, 0)], 0.0)
        return float(((w64[:, :, None] * rows).sum(axis=1) * c.astype(np.float64)).sum())

    g, gw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, _dev(c), _dev(ys), _dev(w))
    g, gw = g.cpu().double().numpy(), gw.cpu().double().numpy()
    ys64, w64 = ys.astype(np.float64), w.astype(np.float64)
    s = np.abs(c.astype(np.float64)[:, None, :] * ys64[np.maximum(pos, 0)]).sum(axis=2)
    for t, i in itertools.product(range(m), range(topk)):
        up, down = w64.copy(), w64.copy()
        up[t, i] += 1.0
        down[t, i] -= 1.0
        diff = (loss(ys64, up) - loss(ys64, down)) / 2
        assert abs(gw[t, i] - diff) <= 1.01 * 17 * U32 * s[t, i] + 1e-10
    for t, i in itertools.product(range(m), range(topk)):
        if not there[t, i]:
            continue
        n = (7 * t + i) % k
        up, down = ys64.copy(), ys64.copy()
        up[pos[t, i], n] += 1.0
        down[pos[t, i], n] -= 1.0
        diff = (loss(up, w64) - loss(down, w64)) / 2
        assert abs(g[pos[t, i], n] - diff) <= (U16 + U32) * abs(diff) + 2.0 ** -25 + 1e-10
    # the gradient of permute (weights and none): unpermute of the sorted rows' gradient
    for weights in (None, w):
        dx = G.nvfp4_moe_unpermute(plan, m, topk, e, _dev(ys), None if weights is None else _dev(w))
        _check_unpermute(dx, ys, weights, pos, "dx of permute")


def test_graph_replays_and_streams():
    """Captured calls replayed between eager calls on other data equal the eager results; a call on a stream
    that is not the current one, with its outputs allocated there, equals them too."""
    m, topk, e, k = 40, 6, 32, 2048
    ids, x, ys, w, pos = _case(m, topk, e, k, 11)
    ids2, x2, ys2, w2, _ = _case(m, topk, e, k, 12)
    di, dx, dy, dw = _dev(ids), _dev(x), _dev(ys), _dev(w)
    plan = torch.empty(G.nvfp4_moe_plan_bytes(m, topk, e) // 4, dtype=torch.int32, device="cuda")

    def calls(i, a, b, c, xs, out, g, gw):
        G.nvfp4_moe_plan(i, e, plan=plan)
        G.nvfp4_moe_permute(plan, m, topk, e, a, c, xs=xs)
        G.nvfp4_moe_unpermute(plan, m, topk, e, b, c, out=out)
        G.nvfp4_moe_unpermute_grad(plan, m, topk, e, a, b, c, dys=g, dweights=gw)

    bufs = [torch.zeros((m * topk, k), dtype=torch.float16, device="cuda"), torch.zeros((m, k), dtype=torch.float16, device="cuda"),
            torch.zeros((m * topk, k), dtype=torch.float16, device="cuda"), torch.zeros((m, topk), device="cuda")]
    calls(di, dx, dy, dw, *bufs)
    torch.cuda.synchronize()
    want = [b.clone() for b in bufs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(di, dx, dy, dw, *bufs)
    other = (_dev(ids2), _dev(x2), _dev(ys2), _dev(w2))
    for _ in range(3):
        for b in bufs:
            b.zero_()
        calls(*other, *[torch.empty_like(b) for b in bufs])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for b, v in zip(bufs, want):
            assert torch.equal(b.view(torch.uint8), v.view(torch.uint8))
    # a second graph on the same plan buffer, replayed in turn with the first
    bufs2 = [torch.empty_like(b) for b in bufs]
    calls(*other, *bufs2)
    torch.cuda.synchronize()
    want2 = [b.clone() for b in bufs2]
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        calls(*other, *bufs2)
    for _ in range(2):
        for b in bufs + bufs2:
            b.zero_()
        graph2.replay()
        graph.replay()
        torch.cuda.synchronize()
        for b, v in zip(bufs, want):
            assert torch.equal(b.view(torch.uint8), v.view(torch.uint8))
        assert torch.equal(bufs2[1].view(torch.uint8), want2[1].view(torch.uint8))
        assert torch.equal(bufs2[3].view(torch.uint8), want2[3].view(torch.uint8))
    G.nvfp4_moe_plan(di, e, plan=plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, dy, dw, stream=side)
    g, gw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, dx, dy, dw, dys=torch.zeros_like(bufs[2]), stream=side)
    side.synchronize()
    assert torch.equal(out, want[1]) and torch.equal(g, want[2]) and torch.equal(gw, want[3])


def test_sort_and_combine_around_experts():
    """The operators as a program uses them: route, sort the tokens, run each expert on its rows, combine with
    the routing weights; and the layer's own W13 in the same bucket order, on the plan of nvfp4_moe_route."""
    from synth import inputs as S
    m, e, topk, k, i = 24, 8, 2, 256, 128
    rng = np.random.default_rng(21)
    case = S.moe_case(S.MoEShape(m=m, e=e, topk=topk, k=k, i=i), workload="tiny")
    w13, w2 = G.NVFP4Tensor.from_numpy(case["w13"]), G.NVFP4Tensor.from_numpy(case["w2"])
    x = _dev(case["x"])
    ids, tw, plan = G.nvfp4_moe_route(_dev(rng.standard_normal((m, e)).astype(np.float32)), topk)
    f = G.plan_fields(plan, m, topk, e)
    xs = G.nvfp4_moe_permute(plan, m, topk, e, x)
    h = G.nvfp4_moe_w13_swiglu(plan, m, topk, e, x, w13)
    ys = torch.empty((m * topk, k), dtype=torch.float16, device="cuda")
    for ex in range(e):  # the expert's dense gated MLP on its sorted rows
        a, b = int(f["offsets"][ex]), int(f["offsets"][ex + 1])
        if a == b:
            continue
        one13 = G.NVFP4Tensor(w13.codes[ex:ex + 1], w13.scales[ex:ex + 1], w13.global_scale[ex:ex + 1])
        one2 = G.NVFP4Tensor(w2.codes[ex:ex + 1], w2.scales[ex:ex + 1], w2.global_scale[ex:ex + 1])
        he = G.nvfp4_linear_swiglu(xs[a:b], one13)
        assert torch.equal(he.view(torch.int16), h[a:b].view(torch.int16))
        ys[a:b] = G.nvfp4_linear(he, one2)
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, ys, tw)
    layer = G.nvfp4_moe_layer(ids, e, x, w13, w2, tw)
    # the layer sums FP32 expert results; here each was rounded to fp16 first (u16 sum |w y|, the weights summing
    # to 1), and each side rounds its result
    pos = f["pos_of_pair"].reshape(m, topk)
    s = np.abs(tw.cpu().double().numpy()[:, :, None] * ys.cpu().double().numpy()[pos]).sum(axis=1)
    diff = np.abs(out.double().cpu().numpy() - layer.double().cpu().numpy())
    tol = 1.01 * U16 * s + 2.02 * U16 * np.abs(layer.double().cpu().numpy()) + 3 * 2.0 ** -25
    assert (diff <= tol).all(), float((diff / tol).max())
    dys, dw = G.nvfp4_moe_unpermute_grad(plan, m, topk, e, x, ys, tw)
    _check_grad(dys, dw, case["x"], ys.cpu().numpy(), tw.cpu().numpy(), pos, "combine")


# bucket rows past the L2s in whole lines, one to eight slots at once and two rounds of six; rows shorter than a wave
LARGE = [(8200, 1, 16, 2048), (4100, 2, 16, 2048), (2740, 3, 16, 2048), (2060, 4, 16, 2048), (1640, 5, 16, 2048),
         (1370, 6, 16, 2048), (1175, 7, 16, 2048), (1030, 8, 16, 2048), (6000, 12, 40, 256), (140000, 2, 8, 64)]


@pytest.mark.parametrize("m,topk,e,k", LARGE)
def test_rows_past_the_caches(m, topk, e, k):
    test_rows(m, topk, e, k, "some")
