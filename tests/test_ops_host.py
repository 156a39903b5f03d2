"""Host-side checks of the further operators (include/nvfp4moe_ops.h), without a GPU: the header's
functions are exported and bound, workspace sizes are as documented, every argument check refuses
before anything is enqueued (fake device pointers are never read), and the Python wrappers compare the
tensors that they are given with the sizes that the library will read and write."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import gemm_nvfp4_amd as G
from gemm_nvfp4_amd import _lib
from gemm_nvfp4_amd._lib import nvfp4_lora, nvfp4_weights

OK, NULL, SHAPE, ALIGN, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3, 4, 5
fake, odd, null = C.c_void_p(0x1000), C.c_void_p(0x1002), None


@pytest.fixture(scope="module")
def L():
    path = os.environ.get("NVFP4_TEST_LIB")
    if not path:
        return _lib.lib()
    lib = C.CDLL(path)
    for name, (res, args) in _lib._SIGS.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


def test_header_functions_are_exported_and_bound(L):
    names = _lib.header_functions(_lib.OPS_HEADER)
    assert names == sorted([
        "nvfp4_moe_permute", "nvfp4_moe_unpermute", "nvfp4_moe_unpermute_grad", "nvfp4_lora_add_ws_bytes",
        "nvfp4_lora_add", "nvfp4_linear_lora_ws_bytes", "nvfp4_linear_lora", "nvfp4_linear_swiglu_lora"])
    for name in names:
        assert hasattr(L, name) and name in _lib._SIGS and callable(getattr(G, name))


@pytest.mark.parametrize("fn", ["nvfp4_moe_permute", "nvfp4_moe_unpermute"])
def test_row_moves_refuse(L, fn):
    f = getattr(L, fn)
    call = lambda plan=fake, M=4, topk=2, E=8, a=fake, w=fake, K=64, b=fake: f(plan, M, topk, E, a, w, K, b, null)  # noqa: E731
    assert call(M=-1) == SHAPE and call(topk=0) == SHAPE and call(topk=33) == SHAPE and call(E=0) == SHAPE
    assert call(K=0) == SHAPE and call(M=1 << 26) == SHAPE
    assert call(E=4097) == UNSUPPORTED and call(K=60) == UNSUPPORTED and call(K=65544) == UNSUPPORTED
    assert call(M=0, plan=null, a=null, w=null, b=null) == OK
    assert call(plan=null) == NULL and call(a=null) == NULL and call(b=null) == NULL
    assert call(plan=odd) == ALIGN and call(a=odd) == ALIGN and call(b=odd) == ALIGN
    assert call(w=odd) == ALIGN


def test_row_gradient_refuses(L):
    f = L.nvfp4_moe_unpermute_grad
    call = lambda plan=fake, M=4, E=8, d=fake, y=fake, w=fake, K=64, dy=fake, dw=fake: f(plan, M, 2, E, d, y, w, K, dy, dw, null)  # noqa: E731
    assert call(M=-1) == SHAPE and call(K=-8) == SHAPE and call(K=12) == UNSUPPORTED and call(E=5000) == UNSUPPORTED
    assert call(M=0, plan=null, d=null, y=null, w=null, dy=null, dw=null) == OK
    for k in ("plan", "d", "y", "dw"):
        assert call(**{k: null}) == NULL
    assert call(w=null) == NULL  # dys needs the weights
    for k in ("plan", "d", "y", "dy", "w", "dw"):
        assert call(**{k: odd}) == ALIGN


def test_header_is_plain_c(tmp_path):
    """The header compiles by itself as C, and its descriptor has the size that the binding gives it."""
    src = tmp_path / "h.c"
    src.write_text('#include "nvfp4moe_ops.h"\n_Static_assert(sizeof(nvfp4_lora) == %d, "size");\n'
                   'int (*f)(const void *, int32_t, int32_t, int32_t, const uint16_t *, const float *, int32_t, uint16_t *, void *)'
                   ' = nvfp4_moe_permute;\n' % C.sizeof(nvfp4_lora))
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", include, "-c", str(src), "-o",
                        str(tmp_path / "h.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _lora(a=fake, b=fake, s=fake, adapters=8, rows=64, k=256, rank=16):
    return C.byref(nvfp4_lora(a, b, s, adapters, rows, k, rank))


BAD_LORA = [(dict(a=null), NULL), (dict(b=null), NULL), (dict(s=null), NULL), (dict(adapters=0), SHAPE),
            (dict(rank=0), SHAPE), (dict(a=odd), ALIGN), (dict(b=odd), ALIGN), (dict(s=odd), ALIGN),
            (dict(rank=12), UNSUPPORTED), (dict(rank=264), UNSUPPORTED), (dict(adapters=4097), UNSUPPORTED)]


def test_lora_add_refuses(L):
    need = L.nvfp4_lora_add_ws_bytes(8, 256, 16)
    assert need >= 8 * 16 * 4 and need % 256 == 0
    # FP32 chunk partials of v at least, and no more than those, v once more and a word per row
    assert 10 * 4096 * 64 * 4 <= L.nvfp4_lora_add_ws_bytes(4096, 5120, 64) <= 11 * 4096 * 64 * 4 + 4096 * 4
    assert L.nvfp4_lora_add_ws_bytes(-1, 256, 16) == 0 and L.nvfp4_lora_add_ws_bytes(4, 0, 16) == 0
    assert L.nvfp4_lora_add_ws_bytes(4, 256, 0) == 0 and L.nvfp4_lora_add_ws_bytes(0, 256, 16) == 0
    call = lambda plan=fake, M=4, topk=2, order=0, x=fake, lora=_lora(), y=fake, out=fake, ws=fake, n=need: L.nvfp4_lora_add(plan, M, topk, order, x, lora, y, out, ws, n, null)  # noqa: E731,E501
    assert call(M=-1) == SHAPE and call(topk=33) == SHAPE and call(order=2) == SHAPE and call(order=-1) == SHAPE
    assert call(lora=None) == NULL
    for bad, want in BAD_LORA + [(dict(k=192), UNSUPPORTED), (dict(k=32896), UNSUPPORTED), (dict(rows=72), UNSUPPORTED),
                            (dict(rows=(1 << 22) + 16), UNSUPPORTED)]:
        assert call(lora=_lora(**bad)) == want, bad
        assert call(M=0, lora=_lora(**bad)) == want, bad
    assert call(M=0, plan=null, x=null, y=null, out=null, ws=null, n=0) == OK
    for k in ("plan", "x", "y", "out", "ws"):
        assert call(**{k: null}) == NULL and call(**{k: odd}) == ALIGN
    assert call(n=need - 1) == WORKSPACE


@pytest.mark.parametrize("gated", [False, True])
def test_linear_lora_refuses(L, gated):
    rows, k, rank, m = 64, 256, 16, 4
    w0 = lambda codes=fake, groups=1, rows=rows, k=k: C.byref(nvfp4_weights(codes, fake, fake, groups, rows, k))  # noqa: E731
    need = L.nvfp4_linear_lora_ws_bytes(m, rows, k, rank)
    assert need >= m * rows * 4 + m * rank * 4 and need % 256 == 0
    assert L.nvfp4_linear_lora_ws_bytes(-1, rows, k, rank) == 0 and L.nvfp4_linear_lora_ws_bytes(m, 0, k, rank) == 0

    def call(plan=fake, x=fake, M=m, w=w0(), layout=0, lora=_lora(), y=fake, ws=fake, n=need):
        if gated:
            return L.nvfp4_linear_swiglu_lora(plan, x, M, w, layout, lora, y, ws, n, null)
        return L.nvfp4_linear_lora(plan, x, M, w, lora, y, ws, n, null)

    assert call(M=-1) == SHAPE and call(M=(1 << 26) + 1) == SHAPE
    assert call(w=w0(codes=None)) == NULL and call(w=w0(groups=2)) == SHAPE
    assert call(lora=_lora(rows=80)) == SHAPE and call(lora=_lora(k=128)) == SHAPE  # not the weight's shape
    for bad, want in BAD_LORA:
        assert call(lora=_lora(**bad)) == want, bad
    assert call(w=w0(k=192), lora=_lora(k=192)) == UNSUPPORTED
    assert call(w=w0(rows=72), lora=_lora(rows=72)) == UNSUPPORTED
    if gated:
        assert call(layout=2) == SHAPE
        assert call(w=w0(rows=48), lora=_lora(rows=48)) == UNSUPPORTED  # I = 24
        assert call(w=w0(k=16512), lora=_lora(k=16512)) == UNSUPPORTED
    assert call(M=0, plan=null, x=null, y=null, ws=null, n=0) == OK
    for key in ("plan", "x", "y", "ws"):
        assert call(**{key: null}) == NULL and call(**{key: odd}) == ALIGN
    assert call(n=need - 1) == WORKSPACE


# ---- the Python wrappers (CPU tensors: shapes are compared before devices) ----------------------------

M, TOPK, E, K, N, R = 4, 2, 8, 256, 64, 16


def _f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _plan(m=M, topk=TOPK, e=E):
    return torch.zeros(G.nvfp4_moe_plan_bytes(m, topk, e) // 4, dtype=torch.int32)


def _t(e=E, n=N, k=K, r=R):
    return G.LoRATensor(_f16(e, r, k), _f16(e, n, r), torch.ones(e))


def _w(rows=N, k=K):
    return G.NVFP4Tensor(torch.zeros((1, rows, k // 2), dtype=torch.uint8), torch.zeros((1, rows, k // 16), dtype=torch.uint8),
                         torch.ones(1))


def test_wrappers_check_shapes():
    tw = torch.zeros(M, TOPK)
    rows = [
        (lambda: G.nvfp4_moe_permute(_plan(), M, TOPK, E, _f16(M + 1, K)), "x must have shape"),
        (lambda: G.nvfp4_moe_permute(_plan()[:-64], M, TOPK, E, _f16(M, K)), "plan holds"),
        (lambda: G.nvfp4_moe_permute(_plan(), M, TOPK, E, _f16(M, K), tw[:, :1]), "topk_weights must have shape"),
        (lambda: G.nvfp4_moe_permute(_plan(), M, TOPK, E, _f16(M, K), xs=_f16(M * TOPK - 1, K)), "xs must have shape"),
        (lambda: G.nvfp4_moe_unpermute(_plan(), M, TOPK, E, _f16(M * TOPK - 1, K)), "ys must have shape"),
        (lambda: G.nvfp4_moe_unpermute(_plan(), M, TOPK, E, _f16(M * TOPK, K), out=_f16(M, K + 8)), "out must have shape"),
        (lambda: G.nvfp4_moe_unpermute_grad(_plan(), M, TOPK, E, _f16(M, K), _f16(M * TOPK, K + 8), tw), "ys must have shape"),
        (lambda: G.nvfp4_moe_unpermute_grad(_plan(), M, TOPK, E, _f16(M, K), _f16(M * TOPK, K), tw,
                                            dweights=tw[:3]), "dweights must have shape"),
        (lambda: G.nvfp4_lora_add(_plan(), M, TOPK, _f16(M, K), _t(), _f16(M * TOPK, N)), "x must have shape"),
        (lambda: G.nvfp4_lora_add(_plan(), M, TOPK, _f16(M * TOPK, K), _t(), _f16(M * TOPK, N + 16)), "y must have shape"),
        (lambda: G.nvfp4_lora_add(_plan(M, 1), M, TOPK, _f16(M * TOPK, K), _t(), _f16(M * TOPK, N),
                                  ws=torch.zeros(16, dtype=torch.uint8)), "plan holds|ws holds"),
        (lambda: G.nvfp4_lora_add(_plan(), M, TOPK, _f16(M * TOPK, K), _t(), _f16(M * TOPK, N),
                                  ws=torch.zeros(16, dtype=torch.uint8)), "ws holds"),
        (lambda: G.nvfp4_linear_lora(_plan(M, 1), _f16(M, K + 128), _w(), _t()), "x must have shape"),
        (lambda: G.nvfp4_linear_lora(_plan(M, 1), _f16(M, K), _w(), _t(n=80)), "the adapters are for"),
        (lambda: G.nvfp4_linear_lora(_plan(M, 1)[:8], _f16(M, K), _w(), _t()), "plan holds"),
        (lambda: G.nvfp4_linear_lora(_plan(M, 1), _f16(M, K), _w(), _t(), y=_f16(M, N // 2)), "y must have shape"),
        (lambda: G.nvfp4_linear_lora(_plan(M, 1), _f16(M, K), _w(), _t(), ws=torch.zeros(64, dtype=torch.uint8)), "ws holds"),
        (lambda: G.nvfp4_linear_swiglu_lora(_plan(M, 1), _f16(M, K), _w(), _t(), h=_f16(M, N)), "h must have shape"),
        (lambda: G.LoRATensor(_f16(2, 8, 128), _f16(2, 64, 16), torch.ones(2)), "inconsistent"),
        (lambda: G.LoRATensor(_f16(8, 128), _f16(2, 64, 8), torch.ones(2)), "must be"),
    ]
    for fn, what in rows:
        with pytest.raises(ValueError, match=what):
            fn()
    swapped = _t()
    swapped.b = _f16(E, N + 16, R)
    with pytest.raises(ValueError, match="must keep the shapes"):
        swapped.desc()


def test_wrappers_refuse_cpu_tensors():
    with pytest.raises(ValueError, match="GPU tensor"):
        G.nvfp4_moe_permute(_plan(), M, TOPK, E, _f16(M, K))
    with pytest.raises(ValueError, match="GPU tensor"):
        G.nvfp4_lora_add(_plan(), M, TOPK, _f16(M * TOPK, K), _t(), _f16(M * TOPK, N))
    with pytest.raises(ValueError, match="GPU tensor"):
        G.nvfp4_linear_lora(_plan(M, 1), _f16(M, K), _w(), _t())


def test_adapters_changed_in_place_are_checked_again(monkeypatch):
    """Data put in place of an adapter's at the same address: another shape, type or order raises, as it does at another
    address, and what fits is taken. The library and the device checks are replaced, so that CPU tensors do."""
    def ptr(t, name, dtype, dev):
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    class Library:
        def nvfp4_lora_add(self, plan, m, topk, order, x, lora, *rest):
            self.seen = lora._obj
            return OK

        def nvfp4_linear_lora(self, plan, x, m, w, lora, *rest):
            self.seen = lora._obj
            return OK

    need, stub = G.nvfp4_lora_add_ws_bytes(M * TOPK, K, R), Library()
    plans, ws = (_plan(), _plan(M, 1)), torch.zeros(need + G.nvfp4_linear_lora_ws_bytes(M, N, K, R), dtype=torch.uint8)
    _lib._plan_bytes(M, TOPK, E), _lib._plan_bytes(M, 1, E), _lib._add_ws_bytes(M * TOPK, K, R), _lib._linear_ws_bytes(M, N, K, R)
    monkeypatch.setattr(_lib, "lib", lambda: stub)
    monkeypatch.setattr(_lib, "_ptr", ptr)
    monkeypatch.setattr(_lib, "_current_device", lambda t: -1)
    monkeypatch.setattr(_lib, "_raw_stream", lambda stream, dev: 0)
    monkeypatch.setattr(_lib, "_dev", lambda t, name, dtype: t.data_ptr())
    calls = [lambda t: G.nvfp4_lora_add(plans[0], M, TOPK, _f16(M * TOPK, K), t, _f16(M * TOPK, N), ws=ws),
             lambda t: G.nvfp4_linear_lora(plans[1], _f16(M, K), _w(), t, ws=ws)]
    changes = [  # tensor, its new data at the same address
        ("a", lambda d: d[:, :8]), ("a", lambda d: d[:4]), ("a", lambda d: d.view(2 * E, R // 2, K)), ("a", lambda d: d.view(torch.bfloat16)),
        ("a", lambda d: d.as_strided((E, R, K), (R * K, 1, R))), ("b", lambda d: d[:, :, :8]), ("b", lambda d: d.view(E, R, N)),
        ("b", lambda d: d.as_strided((E, N, R), (N * R, 1, N))), ("b", lambda d: d.view(torch.int16)), ("scale", lambda d: d[:2]),
        ("scale", lambda d: d.view(torch.int32)), ("scale", lambda d: d.as_strided((E,), (0,)))]
    for call in calls:
        for name, change in changes:
            lora = _t()
            call(lora)
            t = getattr(lora, name)
            old, before = t.data, (t.data_ptr(), stub.seen.a, stub.seen.b, stub.seen.scale)
            t.data = change(old)
            assert t.data_ptr() == before[0]
            with pytest.raises((ValueError, TypeError), match="must"):
                call(lora)
            t.data = old  # as it was: taken again
            call(lora)
            assert (t.data_ptr(), stub.seen.a, stub.seen.b, stub.seen.scale) == before
            t.data = old.clone()  # other memory that fits
            call(lora)
            assert getattr(stub.seen, name) == t.data_ptr() != before[0]
            assert (stub.seen.adapters, stub.seen.rows, stub.seen.k, stub.seen.rank) == (E, N, K, R)
