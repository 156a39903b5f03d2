"""Low-rank adapters on the GPU (nvfp4_lora_add, nvfp4_linear_lora, nvfp4_linear_swiglu_lora) against plain
64-bit computations on the host.

Two kinds of inputs:
  whole numbers  small integers (and power-of-two scales) for which every product and every sum on the
                 way is exact in FP32, and v exact in the 22 bits that the expand product keeps: the result
                 is then the exact value rounded to FP32 (the last fmaf) and to fp16, compared bit for bit.
                 A v rounded to fp16, a wrong rank, row or column, or a rounding more would show.
  random         the library's acceptance rule (parity.py: relative L2 <= 1e-3 per row, max <= 1e-2 RMS).
                 One fp16 rounding is at most 2^-11 relative, about 2.8e-4 RMS; FP32 sums add about
                 sqrt(K) 2^-24.
SwiGLU on whole numbers: g and u are exact in FP32; e^-g is off by at most (|g| + 2) 2^-23 relative (the
rounding of -g log2 e, the base-2 exponential and its conversion), the reciprocal and the two products by 2^-23
each; then one fp16 rounding: |h - ref| <= (2^-11 + (|g| + 8) 2^-22) |ref| + 2^-25.
"""
import numpy as np
import pytest
import torch

import gemm_nvfp4_amd as G
from oracle import oracle as O
from synth import inputs as S
from tests.parity import assert_rows_close_all

pytestmark = pytest.mark.gpu

POISON = 0x7E00


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bits(t):
    return t.cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def _rounded(exact):
    """Bits of the exact result after the last fmaf (FP32) and the rounding to fp16; no negative zeros."""
    with np.errstate(over="ignore"):
        return (exact + 0.0).astype(np.float32).astype(np.float16).view(np.uint16)


def _poisoned(*shape):
    return torch.full(shape, POISON, dtype=torch.int16, device="cuda").view(torch.float16)


def _ids(rng, rows, adapters, how):
    """Adapter ids of `rows` rows: mixed (some -1, some out of range), one for all, runs, each row its own, none."""
    if how == "mixed":
        ids = rng.integers(0, adapters, rows)
        ids[rng.random(rows) < 0.25] = -1
        ids[rng.random(rows) < 0.05] = adapters + 1
    elif how == "one":
        ids = np.full(rows, adapters - 1)
    elif how == "runs":
        ids = np.arange(rows) * adapters // rows
    elif how == "own":
        ids = rng.permutation(rows) % adapters
    else:
        ids = np.full(rows, -1)
    return ids.astype(np.int32)


def _adapters(rng, adapters, n, k, rank, whole):
    if whole:
        a = rng.integers(-2, 3, (adapters, rank, k)).astype(np.float16)
        b = rng.integers(-2, 3, (adapters, n, rank)).astype(np.float16)
        scale = (2.0 ** rng.integers(-3, 2, adapters)).astype(np.float32)
    else:
        a = (rng.standard_normal((adapters, rank, k)) * k ** -0.5).astype(np.float16)
        b = (rng.standard_normal((adapters, n, rank)) * 0.1).astype(np.float16)
        scale = rng.uniform(0.5, 2.0, adapters).astype(np.float32)
    return a, b, scale


def _x(rng, rows, k, whole):
    return (rng.integers(-3, 4, (rows, k)) if whole else rng.standard_normal((rows, k))).astype(np.float16)


def _low_rank(x, ids, a, b, scale):
    """s_a (x A_a^T) B_a^T in 64 bits; zero rows without an adapter."""
    d = np.zeros((x.shape[0], b.shape[1]))
    x64 = x.astype(np.float64)
    for e in range(a.shape[0]):
        m = ids == e
        if m.any():
            d[m] = float(scale[e]) * ((x64[m] @ a[e].astype(np.float64).T) @ b[e].astype(np.float64).T)
    return d


def _tensor(a, b, scale):
    return G.LoRATensor(_dev(a), _dev(b), _dev(scale))


# ---- adapters added to a finished result ----------------------------------------------------------------

# rows, N, K, rank, adapters: one row; odd counts; every rank step; K of one short chunk, of several, with a
# short last one; N below, at and past a 64-column group
ADD = [(1, 16, 128, 8, 1, "one"), (1, 4352, 5120, 16, 4, "one"), (5, 80, 640, 24, 3, "mixed"), (16, 64, 512, 16, 16, "own"),
       (17, 272, 1152, 40, 5, "mixed"), (40, 128, 2176, 64, 2, "mixed"), (100, 1040, 256, 72, 64, "mixed"),
       (260, 96, 384, 128, 7, "runs"), (33, 48, 896, 256, 3, "mixed"), (700, 512, 1024, 16, 9, "mixed"),
       (2100, 208, 640, 32, 4, "runs"), (50, 64, 128, 8, 4096, "own"), (21, 112, 512, 200, 4, "none")]

# batches whose work takes the kernels for many rows per adapter (rows * rank * (K + N) >= 2.5e8), every rank
# step; a single adapter, several in one group of 64 rows, adapters without rows, rows without an adapter
ADD += [(6100, 1040, 1664, 16, 7, "mixed"), (9001, 1648, 2176, 8, 180, "mixed"), (3500, 1056, 2048, 24, 3, "runs"),
        (2050, 1104, 2176, 40, 60, "own"), (1200, 2000, 1408, 64, 1, "one"), (1030, 912, 1152, 120, 5, "mixed"),
        (515, 1232, 1280, 200, 16, "mixed"), (700, 1424, 128, 256, 2, "runs"), (2100, 1040, 1152, 64, 4, "none")]

# rows past the caches: y and out together more than 64 MiB, then each of them (the call in place too)
ADD += [(4100, 4160, 128, 64, 5, "mixed"), (8330, 4160, 256, 8, 2, "mixed")]


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("rows,n,k,rank,adapters,how", ADD)
def test_add(rows, n, k, rank, adapters, how, whole):
    rng = np.random.default_rng([1, rows, n, k, rank, whole])
    a, b, scale = _adapters(rng, adapters, n, k, rank, whole)
    x, y = _x(rng, rows, k, whole), _x(rng, rows, n, whole)
    ids = _ids(rng, rows, adapters, how)
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), adapters)
    lora, dx, dy = _tensor(a, b, scale), _dev(x), _dev(y)
    out = G.nvfp4_lora_add(plan, rows, 1, dx, lora, dy, out=_poisoned(rows, n))
    torch.cuda.synchronize()
    ref = y.astype(np.float64) + _low_rank(x, ids, a, b, scale)
    if whole:
        assert np.array_equal(_bits(out), _rounded(ref))
    else:
        assert_rows_close_all(out.cpu().double().numpy(), ref, "add")
    none = (ids < 0) | (ids >= adapters)
    assert np.array_equal(_bits(out)[none], y.view(np.uint16)[none])
    G.nvfp4_lora_add(plan, rows, 1, dx, lora, dy, out=dy)  # in place
    assert torch.equal(dy.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("m,topk,n,k,rank,experts", [(1, 1, 64, 128, 8, 4), (9, 3, 144, 640, 16, 8), (200, 4, 256, 512, 48, 32),
                                                     (300, 8, 1024, 2048, 16, 64), (750, 8, 1040, 1664, 16, 64),
                                                     (421, 5, 592, 896, 88, 50)])
def test_add_in_bucket_order(m, topk, n, k, rank, experts):
    """The experts' adapters on rows that the plan sorted; rows behind the last valid one stay as they were."""
    rng = np.random.default_rng([2, m, n, k])
    a, b, scale = _adapters(rng, experts, n, k, rank, True)
    x, y = _x(rng, m * topk, k, True), _x(rng, m * topk, n, True)
    ids = _ids(rng, m * topk, experts, "mixed" if m > 1 else "one").reshape(m, topk)
    plan = G.nvfp4_moe_plan(_dev(ids), experts)
    flat = ids.reshape(-1)
    sorted_ids = np.sort(flat[(flat >= 0) & (flat < experts)], kind="stable")
    nv = sorted_ids.size
    out = G.nvfp4_lora_add(plan, m, topk, _dev(x), _tensor(a, b, scale), _dev(y), order=1, out=_poisoned(m * topk, n))
    torch.cuda.synchronize()
    ref = y[:nv].astype(np.float64) + _low_rank(x[:nv], sorted_ids, a, b, scale)
    assert np.array_equal(_bits(out)[:nv], _rounded(ref))
    assert (_bits(out)[nv:] == POISON).all()
    # pair order with the same plan: the same rows in the pairs' own places
    pos = O.plan(ids, experts)["pos_of_pair"]
    xp, yp = np.zeros_like(x), np.ones_like(y)
    xp[pos >= 0], yp[pos >= 0] = x[pos[pos >= 0]], y[pos[pos >= 0]]
    outp = G.nvfp4_lora_add(plan, m, topk, _dev(xp), _tensor(a, b, scale), _dev(yp))
    assert np.array_equal(_bits(outp)[pos >= 0], _bits(out)[pos[pos >= 0]])
    assert (outp.cpu().numpy()[pos < 0] == 1).all()


def test_large_and_small_values():
    """v far beyond fp16's range and far below it keeps its bits; a rank whose v cancels another's is not lost."""
    rows, n, k, rank = 20, 64, 640, 16
    rng = np.random.default_rng(4)
    a, b, scale = _adapters(rng, 2, n, k, rank, True)
    x = _x(rng, rows, k, True)
    ids = _ids(rng, rows, 2, "own")
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), 2)
    y = np.zeros((rows, n), np.float16)
    base = _low_rank(x, ids, a, b, scale)
    for xs, as_ in ((2.0 ** 12, 2.0 ** 10), (2.0 ** -12, 2.0 ** -9)):
        sc = (scale.astype(np.float64) / (xs * as_)).astype(np.float32)
        out = G.nvfp4_lora_add(plan, rows, 1, _dev((x * np.float16(xs)).astype(np.float16)),
                               _tensor((a.astype(np.float64) * as_).astype(np.float16), b, sc), _dev(y))
        assert np.array_equal(_bits(out), _rounded(base)), (xs, as_)
    # v[1] = -(v[0] + 1): the sum over ranks is -1 for every row, where each v has up to 17 bits
    x = rng.integers(-1000, 1001, (rows, k)).astype(np.float16)
    a[:, 1:] = 0
    a[:, 1] = -a[:, 0]
    x[:, 0], a[:, 0, 0], a[:, 1, 0] = 1.0, 1.0, -2.0
    b[:] = 1
    out = G.nvfp4_lora_add(plan, rows, 1, _dev(x), _tensor(a, b, np.ones(2, np.float32)), _dev(y))
    assert (out.cpu().numpy() == -1).all()


def test_values_that_are_not_finite_stay_in_their_rows():
    rows, n, k, rank, adapters = 24, 80, 256, 16, 3
    rng = np.random.default_rng(5)
    a, b, scale = _adapters(rng, adapters, n, k, rank, False)
    x, y = _x(rng, rows, k, False), _x(rng, rows, n, False)
    ids = _ids(rng, rows, 2, "own")  # adapter 2 is used by no row
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), adapters)
    want = G.nvfp4_lora_add(plan, rows, 1, _dev(x), _tensor(a, b, scale), _dev(y))
    a[2], b[2], scale[2] = np.nan, np.inf, np.nan
    x[3, 10], x[7, 200], y[9, 4], y[11, 5] = np.nan, np.inf, np.nan, np.inf
    out = G.nvfp4_lora_add(plan, rows, 1, _dev(x), _tensor(a, b, scale), _dev(y)).cpu().numpy()
    assert np.isnan(out[3]).all() and not np.isfinite(out[7]).any()
    assert np.isnan(out[9, 4]) and out[11, 5] == np.inf
    rest = np.ones(out.shape, bool)
    rest[3] = rest[7] = rest[9, 4] = rest[11, 5] = False
    assert np.array_equal(out.view(np.uint16)[rest], _bits(want)[rest])


def test_infinite_adapter_values_stay_in_their_column_and_adapter():
    """An infinity in B: that output column of that adapter's rows is NaN or infinite, everything else is bitwise as
    without it, and a row alone agrees with the row in a batch (an odd number of 8-rank pieces, so that the staged
    matrix has places behind the rank)."""
    rows, n, k, rank, adapters = 2100, 1040, 1152, 56, 3
    rng = np.random.default_rng(12)
    a, b, scale = _adapters(rng, adapters, n, k, rank, False)
    x, y, ids = _x(rng, rows, k, False), _x(rng, rows, n, False), _ids(rng, rows, adapters, "mixed")
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), adapters)
    want = _bits(G.nvfp4_lora_add(plan, rows, 1, _dev(x), _tensor(a, b, scale), _dev(y)))
    b[1, 70, 0], b[1, 71, 55] = np.inf, -np.inf
    lora = _tensor(a, b, scale)
    out = G.nvfp4_lora_add(plan, rows, 1, _dev(x), lora, _dev(y))
    got, bits = out.cpu().numpy(), _bits(out)
    hit = np.zeros((rows, n), bool)
    hit[np.ix_(ids == 1, [70, 71])] = True
    assert not np.isfinite(got[hit]).any() and np.array_equal(bits[~hit], want[~hit])
    for t in np.nonzero(ids == 1)[0][:8]:
        p1 = G.nvfp4_moe_plan(_dev(ids[t:t + 1].reshape(1, 1)), adapters)
        one = G.nvfp4_lora_add(p1, 1, 1, _dev(x[t:t + 1]), lora, _dev(y[t:t + 1])).cpu().numpy()[0]
        assert np.array_equal(one, got[t], equal_nan=True)


def test_adapters_that_get_new_memory():
    """One LoRATensor through a training loop that puts its tensors' data elsewhere, then overwrites what was there."""
    rng = np.random.default_rng(61)
    rows, n, k, rank = 20, 48, 256, 8
    x, y = _x(rng, rows, k, True), _x(rng, rows, n, True)
    ids = _ids(rng, rows, 2, "mixed")
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), 2)
    lora = _tensor(*_adapters(rng, 2, n, k, rank, True))
    dx, dy = _dev(x), _dev(y)
    for _ in range(3):
        a, b, scale = _adapters(rng, 2, n, k, rank, True)
        for name, new in (("a", a), ("b", b), ("scale", scale)):
            old = getattr(lora, name).data
            getattr(lora, name).data = _dev(new)
            old.fill_(7.0)
            cur = [getattr(lora, t).cpu().numpy() for t in ("a", "b", "scale")]
            out = G.nvfp4_lora_add(plan, rows, 1, dx, lora, dy)
            assert np.array_equal(_bits(out), _rounded(y.astype(np.float64) + _low_rank(x, ids, *cur))), name


def test_add_offsets_past_32_bits():
    """y of 4.6 GB, rows on both sides of its 2^32-byte line; whole numbers, compared bit for bit."""
    rows, n, k, rank, adapters = 140000, 16384, 128, 8, 3
    rng = np.random.default_rng(13)
    a, b, scale = _adapters(rng, adapters, n, k, rank, True)
    x, ids = _x(rng, rows, k, True), _ids(rng, rows, adapters, "mixed")
    y = torch.randint(-3, 4, (rows, n), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").half()
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), adapters)
    out = G.nvfp4_lora_add(plan, rows, 1, _dev(x), _tensor(a, b, scale), y)
    torch.cuda.synchronize()
    line = 2 ** 32 // (2 * n)
    for t in np.concatenate([rng.integers(0, rows, 12), np.arange(line - 2, line + 3), [0, rows - 1]]):
        ref = y[t].cpu().double().numpy() + _low_rank(x[t:t + 1], ids[t:t + 1], a, b, scale)[0]
        assert np.array_equal(_bits(out[t]), _rounded(ref)), t


# ---- adapters beside the projections --------------------------------------------------------------------

# M, N, K, rank, adapters: the dense workload, its gated MLP's down projection, short and long reductions, batches
# on both sides of every path change
LINEAR = [(1, 4352, 5120, 16, 4, "one"), (1, 64, 128, 8, 1, "none"), (4, 256, 640, 32, 3, "mixed"), (13, 5120, 2176, 16, 13, "own"),
          (32, 544, 1024, 64, 8, "mixed"), (33, 96, 1536, 16, 5, "mixed"), (64, 1088, 2176, 24, 6, "runs"),
          (65, 64, 512, 128, 2, "mixed"), (50, 128, 640, 16, 2, "mixed"), (200, 4352, 1664, 16, 3, "mixed"), (130, 288, 896, 16, 40, "mixed"), (3, 32, 16512, 8, 2, "mixed"),
          (9, 96, 256, 256, 3, "mixed")]


def _weight(rng, n, k, whole):
    gs = 0.5 if whole else 0.37
    return S.nvfp4_weights(rng, 1, n, k, gscale=gs)


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("m,n,k,rank,adapters,how", LINEAR)
def test_linear(m, n, k, rank, adapters, how, whole):
    rng = np.random.default_rng([6, m, n, k, rank, whole])
    w = _weight(rng, n, k, whole)
    a, b, scale = _adapters(rng, adapters, n, k, rank, whole)
    x, ids = _x(rng, m, k, whole), _ids(rng, m, adapters, how)
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(m, 1)), adapters)
    wt, lora, dx = G.NVFP4Tensor.from_numpy(w), _tensor(a, b, scale), _dev(x)
    ws = torch.full((G.nvfp4_linear_lora_ws_bytes(m, n, k, rank),), 0xFF, dtype=torch.uint8, device="cuda")
    y = G.nvfp4_linear_lora(plan, dx, wt, lora, y=_poisoned(m, n), ws=ws)
    torch.cuda.synchronize()
    ref = x.astype(np.float64) @ O.dequant(*w)[0].T + _low_rank(x, ids, a, b, scale)
    if whole:
        assert np.array_equal(_bits(y), _rounded(ref))
    else:
        assert_rows_close_all(y.cpu().double().numpy(), ref, "linear")
    none = (ids < 0) | (ids >= adapters)
    plain = G.nvfp4_linear(dx, wt)
    assert np.array_equal(_bits(y)[none], _bits(plain)[none])
    for t in {0, m // 2, m - 1}:  # the same row alone
        p1 = G.nvfp4_moe_plan(_dev(ids[t:t + 1].reshape(1, 1)), adapters)
        y1 = G.nvfp4_linear_lora(p1, dx[t:t + 1].contiguous(), wt, lora)
        assert torch.equal(y1[0].view(torch.int16), y[t].view(torch.int16)), f"row {t} alone differs"


SWIGLU = [(1, 32, 128, 8, 1, "one"), (1, 4352, 5120, 16, 3, "one"), (13, 4352, 5120, 32, 3, "mixed"), (5, 160, 640, 24, 5, "own"),
          (33, 224, 1536, 64, 4, "mixed"), (70, 96, 896, 16, 9, "mixed"), (8, 64, 512, 256, 2, "none")]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("m,rows,k,rank,adapters,how", SWIGLU)
def test_swiglu(m, rows, k, rank, adapters, how, layout):
    rng = np.random.default_rng([7, m, rows, k, rank])
    w = _weight(rng, rows, k, True)
    a, b, scale = _adapters(rng, adapters, rows, k, rank, True)
    scale /= 64.0  # gates of the size that SiLU bends
    x, ids = _x(rng, m, k, True), _ids(rng, m, adapters, how)
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(m, 1)), adapters)
    wt, lora, dx = G.NVFP4Tensor.from_numpy(w), _tensor(a, b, scale), _dev(x)
    h = G.nvfp4_linear_swiglu_lora(plan, dx, wt, lora, layout, h=_poisoned(m, rows // 2))
    torch.cuda.synchronize()
    y = x.astype(np.float64) @ O.dequant(*w)[0].T + _low_rank(x, ids, a, b, scale)
    g, u = (y[:, 0::2], y[:, 1::2]) if layout else (y[:, :rows // 2], y[:, rows // 2:])
    with np.errstate(over="ignore"):
        ref = g / (1.0 + np.exp(-g)) * u
    big = np.abs(ref) >= 65504
    tol = (2.0 ** -11 + (np.abs(g) + 8) * 2.0 ** -22) * np.abs(ref) + 2.0 ** -25
    got = h.cpu().double().numpy()
    assert (np.abs(got - ref)[~big] <= tol[~big]).all()
    assert (np.abs(got[big]) >= 65472).all()
    none = (ids < 0) | (ids >= adapters)
    assert np.array_equal(_bits(h)[none], _bits(G.nvfp4_linear_swiglu(dx, wt, layout))[none])
    t = m // 2
    p1 = G.nvfp4_moe_plan(_dev(ids[t:t + 1].reshape(1, 1)), adapters)
    h1 = G.nvfp4_linear_swiglu_lora(p1, dx[t:t + 1].contiguous(), wt, lora, layout)
    assert torch.equal(h1[0].view(torch.int16), h[t].view(torch.int16))


def test_a_rows_result_does_not_depend_on_the_batch():
    """lora_add of 2100 rows (in groups of 64) against single rows and against the same rows in another order."""
    rows, n, k, rank, adapters = 2100, 1104, 1152, 56, 5
    rng = np.random.default_rng(8)
    a, b, scale = _adapters(rng, adapters, n, k, rank, False)
    x, y, ids = _x(rng, rows, k, False), _x(rng, rows, n, False), _ids(rng, rows, adapters, "mixed")
    lora = _tensor(a, b, scale)

    def call(sel):
        plan = G.nvfp4_moe_plan(_dev(ids[sel].reshape(-1, 1)), adapters)
        return _bits(G.nvfp4_lora_add(plan, len(sel), 1, _dev(x[sel]), lora, _dev(y[sel])))

    full = call(np.arange(rows))
    perm = rng.permutation(rows)
    assert np.array_equal(call(perm), full[perm])
    for t in (0, 17, 1044, rows - 1):
        assert np.array_equal(call(np.array([t])), full[t:t + 1])


def test_graph_replays_and_two_streams():
    """Captured calls with changed ids and rows equal eager calls on every replay; two streams with a
    workspace each, run at once, do not disturb one another."""
    m, rows, k, rank, adapters = 24, 544, 1024, 16, 6
    rng = np.random.default_rng(9)
    w13, w2 = _weight(rng, rows, k, False), _weight(rng, k, rows // 2 // 128 * 128, False)
    i = w2[0].shape[2] * 2
    w13 = tuple(np.ascontiguousarray(v[:, :2 * i]) if v.ndim == 3 else v for v in w13)
    t13, t2 = G.NVFP4Tensor.from_numpy(w13), G.NVFP4Tensor.from_numpy(w2)
    l13, l2 = _tensor(*_adapters(rng, adapters, 2 * i, k, rank, False)), _tensor(*_adapters(rng, adapters, k, i, rank, False))
    sets = [(_dev(_x(rng, m, k, False)), _dev(_ids(rng, m, adapters, "mixed").reshape(m, 1))) for _ in range(3)]
    x, ids = sets[0][0].clone(), sets[0][1].clone()

    def buffers():
        need = max(G.nvfp4_linear_lora_ws_bytes(m, 2 * i, k, rank), G.nvfp4_linear_lora_ws_bytes(m, k, i, rank),
                   G.nvfp4_lora_add_ws_bytes(m, k, rank))
        return (torch.empty(G.nvfp4_moe_plan_bytes(m, 1, adapters) // 4, dtype=torch.int32, device="cuda"),
                torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty((m, i), dtype=torch.float16, device="cuda"),
                torch.empty((m, k), dtype=torch.float16, device="cuda"))

    def mlp(x, ids, bufs, stream=None):
        plan, ws, h, y = bufs
        G.nvfp4_moe_plan(ids, adapters, plan=plan, stream=stream)
        G.nvfp4_linear_swiglu_lora(plan, x, t13, l13, 1, h=h, ws=ws, stream=stream)
        G.nvfp4_linear_lora(plan, h, t2, l2, y=y, ws=ws, stream=stream)
        return y

    want = [mlp(*s, buffers()).clone() for s in sets]
    held = buffers()
    mlp(x, ids, held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp(x, ids, held)
    for turn in (1, 2, 0, 1):
        x.copy_(sets[turn][0])
        ids.copy_(sets[turn][1])
        held[1].fill_(0xFF)
        mlp(*sets[(turn + 1) % 3], buffers())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[3].view(torch.int16), want[turn].view(torch.int16)), turn
    # a second graph on the same plan, workspace and outputs, replayed in turn with the first
    x2, ids2 = sets[2][0].clone(), sets[2][1].clone()
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):
        mlp(x2, ids2, held)
    x.copy_(sets[1][0])
    ids.copy_(sets[1][1])
    for _ in range(3):
        for g, w in ((second, want[2]), (graph, want[1])):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(held[3].view(torch.int16), w.view(torch.int16))
    streams, bufs = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for j in range(2):
            mlp(*sets[j + 1], bufs[j], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert torch.equal(bufs[j][3].view(torch.int16), want[j + 1].view(torch.int16))
    # outputs and workspace allocated by the call, on its stream
    add = _tensor(*_adapters(rng, adapters, k, k, rank, False))
    here = G.nvfp4_lora_add(bufs[0][0], m, 1, want[1], add, want[2])
    torch.cuda.synchronize()
    there = G.nvfp4_lora_add(bufs[0][0], m, 1, want[1], add, want[2], stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(here.view(torch.int16), there.view(torch.int16))


def test_expert_adapters_between_sort_and_combine():
    """The operators together: tokens sorted by expert, the experts' projection (the layer's W13 h), adapters
    of the experts on the sorted rows, rows combined with the routing weights; against the same in 64 bits from
    the library's own h."""
    m, e, topk, k, i, rank = 40, 8, 2, 256, 128, 16
    rng = np.random.default_rng(10)
    case = S.moe_case(S.MoEShape(m=m, e=e, topk=topk, k=k, i=i), workload="tiny")
    x = _dev(case["x"])
    w13 = G.NVFP4Tensor.from_numpy(case["w13"])
    ids, tw, plan = G.nvfp4_moe_route(_dev(rng.standard_normal((m, e)).astype(np.float32)), topk)
    a, b, scale = _adapters(rng, e, i, k, rank, False)
    xs = G.nvfp4_moe_permute(plan, m, topk, e, x)
    h = G.nvfp4_moe_w13_swiglu(plan, m, topk, e, x, w13)
    h0 = h.cpu().numpy().astype(np.float64)
    G.nvfp4_lora_add(plan, m, topk, xs, _tensor(a, b, scale), h, order=1, out=h)
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, h, tw)
    f = G.plan_fields(plan, m, topk, e)
    pos, nid = f["pos_of_pair"].reshape(m, topk), ids.cpu().numpy()
    ref = np.zeros((m, i))
    for t in range(m):
        for s in range(topk):
            d = _low_rank(case["x"][t:t + 1], nid[t, s:s + 1], a, b, scale)[0]
            ref[t] += float(tw[t, s]) * (h0[pos[t, s]] + d)
    assert_rows_close_all(out.cpu().double().numpy(), ref, "experts with adapters")


# below and above the work at which lora_add goes by groups of 64 rows
@pytest.mark.parametrize("rows,n,k,rank,adapters", [(37, 80, 640, 24, 3), (2100, 1040, 1152, 64, 4)])
def test_rows_without_an_adapter_keep_every_bit(rows, n, k, rank, adapters):
    """y's rows without an adapter hold every fp16 bit pattern (quiet and signalling NaN, infinities, zeros of both
    signs, subnormals); out holds the same, into another buffer and in place."""
    rng = np.random.default_rng([14, rows])
    ids = _ids(rng, rows, adapters, "mixed")
    none = (ids < 0) | (ids >= adapters)
    bits = rng.integers(0, 1 << 16, (rows, n)).astype(np.uint16)
    at = np.nonzero(none)[0]
    special = np.array([0x7C01, 0xFC01, 0x7DFF, 0xFDFF, 0x7E00, 0xFFFF, 0x7C00, 0xFC00, 0x8000, 0x0001, 0x83FF], np.uint16)
    bits[at[0], :special.size], bits[at[-1], -special.size:] = special, special
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), adapters)
    lora = _tensor(*_adapters(rng, adapters, n, k, rank, True))
    x, y = _dev(_x(rng, rows, k, True)), _dev(bits.view(np.int16)).view(torch.float16)
    out = G.nvfp4_lora_add(plan, rows, 1, x, lora, y, out=_poisoned(rows, n))
    assert np.array_equal(_bits(out)[none], bits[none])
    G.nvfp4_lora_add(plan, rows, 1, x, lora, y, out=y)
    assert np.array_equal(_bits(y)[none], bits[none])


def test_linear_of_the_largest_batch():
    """2^26 rows, the most that a plan holds, at the largest rank: a grid of more than 2^32 threads, base partials and
    outputs past 2^32 bytes. Whole numbers: some rows bit for bit against the exact value, and slices of the batch from
    both ends and the middle against calls of their own."""
    m, n, k, rank, adapters, part = 1 << 26, 16, 128, 256, 2, 1 << 16
    need = 2 * m * (k + n) + G.nvfp4_linear_lora_ws_bytes(m, n, k, rank) + G.nvfp4_moe_plan_bytes(m, 1, adapters)
    if torch.cuda.mem_get_info()[1] < need + (8 << 30):
        pytest.skip("needs about 100 GB of device memory")
    torch.cuda.empty_cache()
    rng = np.random.default_rng(15)
    w = _weight(rng, n, k, True)
    a, b, scale = _adapters(rng, adapters, n, k, rank, True)
    a[:, 16:] = 0  # sums over the ranks stay exact in FP32
    a[:, rank - 1] = a[:, 0]
    x = torch.empty((m // part, part, k), dtype=torch.float16, device="cuda")
    x.copy_(_dev(_x(rng, part, k, True)))
    for digit in range(4):  # the number of the part, in digits from -3 to 3: no two parts are alike
        x[:, :, digit] = ((torch.arange(m // part, device="cuda") // 7 ** digit) % 7 - 3).half()[:, None]
    x = x.view(m, k)
    ids = torch.randint(-1, adapters, (m, 1), dtype=torch.int32, device="cuda",
                        generator=torch.Generator(device="cuda").manual_seed(15))
    wt, lora = G.NVFP4Tensor.from_numpy(w), _tensor(a, b, scale)
    plan = G.nvfp4_moe_plan(ids, adapters)
    y = G.nvfp4_linear_lora(plan, x, wt, lora)
    torch.cuda.synchronize()
    line = 1 << 25  # row n * 2 bytes * line = 2^30; base partials there start at 2^31 bytes
    sel = np.concatenate([[0, 1, m - 1, line - 1, line, 2 * line - 1], rng.integers(0, m, 40)])
    for t in sel:
        xt, it = x[t:t + 1].cpu().numpy(), ids[t].cpu().numpy()
        ref = xt.astype(np.float64) @ O.dequant(*w)[0].T + _low_rank(xt, it, a, b, scale)
        assert np.array_equal(_bits(y[t]), _rounded(ref)[0]), t
    for first in (0, m // 2 - part // 2, m - part, 12345 * 4096 + 7):
        cut = slice(first, first + part)
        p1 = G.nvfp4_moe_plan(ids[cut].contiguous(), adapters)
        y1 = G.nvfp4_linear_lora(p1, x[cut].contiguous(), wt, lora)
        assert torch.equal(y1.view(torch.int16), y[cut].view(torch.int16)), first
    del x, y, plan, ids
    torch.cuda.empty_cache()


# gated forms of 65 to 128 ranks; rank 16 in more than three expand blocks per CU (B asked for behind v); more than ten
# chunks of base partials in the interleaved form, the longest reduction; batches with the weights kept
SWIGLU_MORE = [(9, 96, 384, 72, 3, "mixed"), (40, 160, 640, 128, 4, "mixed"), (96, 8192, 256, 16, 20, "own"),
               (96, 8192, 384, 8, 30, "mixed"), (7, 64, 5248, 16, 2, "mixed"), (33, 96, 10752, 40, 3, "mixed"),
               (5, 32, 16384, 8, 2, "mixed"), (300, 224, 1152, 24, 5, "mixed"), (1111, 96, 640, 16, 3, "runs")]


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("m,rows,k,rank,adapters,how", SWIGLU_MORE)
def test_swiglu_in_every_form(m, rows, k, rank, adapters, how, layout):
    test_swiglu(m, rows, k, rank, adapters, how, layout)


@pytest.mark.parametrize("m,n,k,rank,adapters,how", [(1111, 96, 1664, 16, 3, "runs"), (2050, 272, 640, 40, 70, "mixed"),
                                                     (96, 8192, 256, 16, 20, "own"), (300, 64, 5632, 128, 4, "mixed")])
def test_linear_of_many_rows(m, n, k, rank, adapters, how):
    test_linear(m, n, k, rank, adapters, how, True)


# the groups of 64 rows with more than ten and more than twenty chunks of v
@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("rows,n,k,rank,adapters,how", [(700, 1040, 5632, 64, 3, "mixed"), (1500, 160, 10752, 16, 4, "mixed"),
                                                        (600, 64, 32768, 16, 2, "runs")])
def test_add_of_long_rows(rows, n, k, rank, adapters, how, whole):
    test_add(rows, n, k, rank, adapters, how, whole)


def test_long_rows_do_not_depend_on_the_batch():
    """lora_add in groups of 64 rows, eleven chunks, against single rows and against the rows in another order."""
    rows, n, k, rank, adapters = 700, 1040, 5632, 64, 3
    rng = np.random.default_rng(16)
    lora = _tensor(*_adapters(rng, adapters, n, k, rank, False))
    x, y, ids = _x(rng, rows, k, False), _x(rng, rows, n, False), _ids(rng, rows, adapters, "mixed")

    def call(sel):
        plan = G.nvfp4_moe_plan(_dev(ids[sel].reshape(-1, 1)), adapters)
        return _bits(G.nvfp4_lora_add(plan, len(sel), 1, _dev(x[sel]), lora, _dev(y[sel])))

    full, perm = call(np.arange(rows)), rng.permutation(rows)
    assert np.array_equal(call(perm), full[perm])
    for t in (0, 15, 16, 333, rows - 1):
        assert np.array_equal(call(np.array([t])), full[t:t + 1])


def test_graph_replays_and_two_streams_of_many_rows():
    """lora_add in groups of 64 rows (three launches that hand on partials, split terms and shifts in the workspace):
    two graphs on one plan, workspace and output in turn, and two streams with a workspace each."""
    rows, n, k, rank, adapters = 1500, 1040, 1152, 80, 5
    rng = np.random.default_rng(17)
    lora = _tensor(*_adapters(rng, adapters, n, k, rank, False))
    sets = [(_dev(_ids(rng, rows, adapters, how).reshape(rows, 1)), _dev(_x(rng, rows, k, False)), _dev(_x(rng, rows, n, False)))
            for how in ("mixed", "runs", "own")]

    def buffers():
        return (torch.empty(G.nvfp4_moe_plan_bytes(rows, 1, adapters) // 4, dtype=torch.int32, device="cuda"),
                torch.empty(G.nvfp4_lora_add_ws_bytes(rows, k, rank), dtype=torch.uint8, device="cuda"),
                torch.empty((rows, n), dtype=torch.float16, device="cuda"))

    def call(ids, x, y, bufs, stream=None):
        plan, ws, out = bufs
        G.nvfp4_moe_plan(ids, adapters, plan=plan, stream=stream)
        return G.nvfp4_lora_add(plan, rows, 1, x, lora, y, out=out, ws=ws, stream=stream)

    want = [call(*s, buffers()).clone() for s in sets]
    held = buffers()
    call(*sets[0], held)
    torch.cuda.synchronize()
    graphs = []
    for s in sets[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(*s, held)
    for turn in (0, 1, 1, 0, 1, 0):
        held[1].fill_(0xFF)
        held[2].zero_()
        call(*sets[2], buffers())
        torch.cuda.synchronize()
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert torch.equal(held[2].view(torch.int16), want[turn].view(torch.int16)), turn
    streams, bufs = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for j in range(2):
            call(*sets[j + 1], bufs[j], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert torch.equal(bufs[j][2].view(torch.int16), want[j + 1].view(torch.int16))


def test_projection_offsets_past_32_bits():
    """26000 rows of 4352 x 5120: ten planes of base partials, 4.5 GB. Whole numbers: rows on both sides of the
    2^32-byte line of the planes bit for bit against the exact value, slices against calls of their own, the gated
    forms too."""
    m, n, k, rank, adapters, part = 26000, 4352, 5120, 16, 3, 100
    rng = np.random.default_rng(18)
    w = _weight(rng, n, k, True)
    a, b, scale = _adapters(rng, adapters, n, k, rank, True)
    ids = _ids(rng, m, adapters, "mixed")
    x = torch.randint(-3, 4, (m, k), generator=torch.Generator(device="cuda").manual_seed(18), device="cuda").half()
    wt, lora = G.NVFP4Tensor.from_numpy(w), _tensor(a, b, scale)
    plan = G.nvfp4_moe_plan(_dev(ids.reshape(m, 1)), adapters)
    ws = torch.empty(G.nvfp4_linear_lora_ws_bytes(m, n, k, rank), dtype=torch.uint8, device="cuda")
    line = 2 ** 30 // n - 9 * m  # the row whose partial in the last plane crosses the line
    assert 2 < line < m - 2
    y = G.nvfp4_linear_lora(plan, x, wt, lora, ws=ws)
    full = O.dequant(*w)[0]
    for t in np.concatenate([[0, 1, m - 1], np.arange(line - 2, line + 3), rng.integers(0, m, 12)]):
        xt = x[t:t + 1].cpu().numpy()
        ref = xt.astype(np.float64) @ full.T + _low_rank(xt, ids[t:t + 1], a, b, scale)
        assert np.array_equal(_bits(y[t]), _rounded(ref)[0]), t
    h = [G.nvfp4_linear_swiglu_lora(plan, x, wt, lora, layout, ws=ws) for layout in (0, 1)]
    for first in (0, line - part // 2, m - part):
        cut = slice(first, first + part)
        p1, x1 = G.nvfp4_moe_plan(_dev(ids[cut].reshape(part, 1)), adapters), x[cut].contiguous()
        assert torch.equal(G.nvfp4_linear_lora(p1, x1, wt, lora).view(torch.int16), y[cut].view(torch.int16))
        for layout in (0, 1):
            h1 = G.nvfp4_linear_swiglu_lora(p1, x1, wt, lora, layout)
            assert torch.equal(h1.view(torch.int16), h[layout][cut].view(torch.int16)), layout


def test_expert_down_projections_with_adapters():
    """Adapters of a MoE's experts where a model has them: tokens sorted by expert, each expert's gated projection and
    down projection with nvfp4_linear on its rows, the down projection's adapters on all sorted rows at once, rows
    combined with the routing weights; against the same in 64 bits from the library's own h."""
    m, e, topk, k, i, rank = 40, 8, 2, 256, 128, 16
    rng = np.random.default_rng(19)
    case = S.moe_case(S.MoEShape(m=m, e=e, topk=topk, k=k, i=i), workload="tiny")
    w13, w2 = G.NVFP4Tensor.from_numpy(case["w13"]), G.NVFP4Tensor.from_numpy(case["w2"])
    ids, tw, plan = G.nvfp4_moe_route(_dev(rng.standard_normal((m, e)).astype(np.float32)), topk)
    f = G.plan_fields(plan, m, topk, e)
    a, b, scale = _adapters(rng, e, k, i, rank, False)
    h = G.nvfp4_moe_w13_swiglu(plan, m, topk, e, _dev(case["x"]), w13)  # in bucket order
    ys = torch.empty((m * topk, k), dtype=torch.float16, device="cuda")
    for ex in range(e):
        first, last = int(f["offsets"][ex]), int(f["offsets"][ex + 1])
        if first < last:
            one = G.NVFP4Tensor(w2.codes[ex:ex + 1], w2.scales[ex:ex + 1], w2.global_scale[ex:ex + 1])
            ys[first:last] = G.nvfp4_linear(h[first:last], one)
    G.nvfp4_lora_add(plan, m, topk, h, _tensor(a, b, scale), ys, order=1, out=ys)
    out = G.nvfp4_moe_unpermute(plan, m, topk, e, ys, tw)
    h64, w64 = h.cpu().numpy(), O.dequant(*case["w2"])
    pos, nid, ref = f["pos_of_pair"].reshape(m, topk), ids.cpu().numpy(), np.zeros((m, k))
    for t in range(m):
        for s in range(topk):
            row = h64[pos[t, s]:pos[t, s] + 1]
            ref[t] += float(tw[t, s]) * (row.astype(np.float64) @ w64[nid[t, s]].T + _low_rank(row, nid[t, s:s + 1], a, b, scale))[0]
    assert_rows_close_all(out.cpu().double().numpy(), ref, "down projections with adapters")


@pytest.mark.parametrize("rows,n,k", [(21, 80, 640), (1300, 2000, 1152)])
def test_a_part_of_a_larger_table(rows, n, k):
    """Adapters 3 to 5 of a table of nine as a descriptor of their own, the ids counted from there."""
    rng = np.random.default_rng([20, rows])
    a, b, scale = _adapters(rng, 9, n, k, 64, True)
    table = _tensor(a, b, scale)
    part = G.LoRATensor(table.a[3:6], table.b[3:6], table.scale[3:6])
    x, y, ids = _dev(_x(rng, rows, k, True)), _dev(_x(rng, rows, n, True)), _ids(rng, rows, 3, "mixed")
    ids[ids >= 3] = -1
    want = np.where(ids >= 0, ids + 3, -1).astype(np.int32)
    out = G.nvfp4_lora_add(G.nvfp4_moe_plan(_dev(ids.reshape(rows, 1)), 3), rows, 1, x, part, y)
    ref = G.nvfp4_lora_add(G.nvfp4_moe_plan(_dev(want.reshape(rows, 1)), 9), rows, 1, x, table, y)
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    assert np.array_equal(_bits(out), _rounded(y.cpu().double().numpy() + _low_rank(x.cpu().numpy(), want, a, b, scale)))
