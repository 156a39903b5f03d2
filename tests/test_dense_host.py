"""Host-side checks of the calls around the dense projections (include/nvfp4moe_dense.h), without a GPU: exports and
bindings, workspace sizes, every refusal before anything is enqueued (fake device pointers are never read), and the
Python wrappers' checks."""
import ctypes as C
import os
import subprocess

import pytest
import torch

import gemm_nvfp4_amd as G
from gemm_nvfp4_amd import _lib
from gemm_nvfp4_amd._lib import fp8_channel_weights, nvfp4_weights

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
    names = _lib.header_functions(_lib.DENSE_HEADER)
    assert names == sorted([
        "nvfp4_add_rms_norm", "nvfp4_add_rms_norm_grad_ws_bytes", "nvfp4_add_rms_norm_grad", "nvfp4_linear_fp8_rows",
        "nvfp4_linear_grad_ws_bytes", "nvfp4_linear_grad", "nvfp4_linear_swiglu_grad_ws_bytes",
        "nvfp4_linear_swiglu_grad"])
    for name in names:
        assert hasattr(L, name) and name in _lib._SIGS and callable(getattr(G, name))


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "nvfp4moe_dense.h"\nint (*f)(const uint16_t *, int32_t, const nvfp4_weights *, uint16_t *, void *, '
                   'size_t, void *) = nvfp4_linear_grad;\n')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", include, "-c", str(src), "-o",
                        str(tmp_path / "h.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_norm_refuses(L):
    def call(x=fake, r=fake, w=fake, M=4, K=64, eps=1e-6, s=fake, y=fake, q=fake, qs=fake):
        return L.nvfp4_add_rms_norm(x, r, w, M, K, eps, s, y, q, qs, null)

    assert call(M=-1) == SHAPE and call(M=(1 << 26) + 1) == SHAPE and call(K=0) == SHAPE and call(K=-8) == SHAPE
    assert call(eps=-1e-6) == SHAPE and call(eps=float("nan")) == SHAPE
    assert call(K=60) == UNSUPPORTED and call(K=32776) == UNSUPPORTED
    assert call(M=0, x=null, r=null, w=null, s=null, y=null, q=null, qs=null) == OK
    assert call(x=null) == NULL and call(y=null, q=null, qs=null) == NULL
    assert call(q=null) == NULL and call(qs=null) == NULL  # only both or neither
    for k in ("x", "r", "w", "s", "y", "q"):
        assert call(**{k: odd}) == ALIGN
    assert call(qs=C.c_void_p(0x1001)) == ALIGN


def test_norm_gradient_refuses(L):
    need = L.nvfp4_add_rms_norm_grad_ws_bytes(333, 5120)
    assert need >= 5120 * 4
    assert L.nvfp4_add_rms_norm_grad_ws_bytes(1, 64) == 256 and L.nvfp4_add_rms_norm_grad_ws_bytes(0, 64) == 0
    for bad in ((-1, 64), (4, 0), (4, 60), (4, 32776), ((1 << 26) + 1, 64)):
        assert L.nvfp4_add_rms_norm_grad_ws_bytes(*bad) == 0, bad

    def call(t=fake, dy=fake, ds=fake, w=fake, M=333, K=5120, eps=1e-6, dx=fake, dw=fake, ws=fake, n=need):
        return L.nvfp4_add_rms_norm_grad(t, dy, ds, w, M, K, eps, dx, dw, ws, n, null)

    assert call(M=-1) == SHAPE and call(K=0) == SHAPE and call(eps=-1.0) == SHAPE and call(K=5124) == UNSUPPORTED
    assert call(M=0, t=null, dy=null, ds=null, w=null, dx=null, dw=null, ws=null, n=0) == OK
    assert call(t=null) == NULL and call(dy=null) == NULL and call(ws=null) == NULL and call(dx=null, dw=null) == NULL
    for k in ("t", "dy", "ds", "w", "dx", "ws"):
        assert call(**{k: odd}) == ALIGN
    assert call(dw=C.c_void_p(0x1001)) == ALIGN and call(M=0, dw=C.c_void_p(0x1001)) == ALIGN
    assert call(n=need - 1) == WORKSPACE


def test_rows_refuse(L):
    w0 = lambda codes=fake, scale=fake, rows=64, k=256: C.byref(fp8_channel_weights(codes, scale, rows, k))  # noqa: E731
    call = lambda x=fake, xs=fake, M=4, w=w0(), y=fake: L.nvfp4_linear_fp8_rows(x, xs, M, w, y, null)  # noqa: E731
    assert call(M=-1) == SHAPE and call(M=(1 << 26) + 1) == SHAPE and call(w=None) == NULL
    assert call(w=w0(codes=null)) == NULL and call(w=w0(scale=null)) == NULL and call(w=w0(rows=0)) == SHAPE
    assert call(w=w0(k=8)) == SHAPE and call(w=w0(k=192)) == UNSUPPORTED and call(w=w0(k=16512)) == UNSUPPORTED
    assert call(w=w0(rows=72)) == UNSUPPORTED and call(w=w0(codes=odd)) == ALIGN and call(w=w0(scale=odd)) == ALIGN
    assert call(M=0, x=null, xs=null, y=null) == OK
    for k in ("x", "xs", "y"):
        assert call(**{k: null}) == NULL and call(**{k: odd}) == ALIGN


@pytest.mark.parametrize("gated", [False, True])
def test_gradients_refuse(L, gated):
    size = L.nvfp4_linear_swiglu_grad_ws_bytes if gated else L.nvfp4_linear_grad_ws_bytes
    rows, k, top = 64, 256, 16384 if gated else 32768
    w0 = lambda codes=fake, scales=fake, gs=fake, groups=1, rows=rows, k=k: C.byref(nvfp4_weights(codes, scales, gs, groups, rows, k))  # noqa: E731,E501

    for m in (1, 64, 65, 333, 8192):
        assert size(m, rows, k) > 0 and size(m, rows, k) % 256 == 0
    for bad in ((-1, rows, k), ((1 << 26) + 1, rows, k), (4, 0, k), (4, rows, 0), (4, 72, k), (4, rows, 192),
                (4, rows, top + 128), (4, (1 << 20) + 32, k)):
        assert size(*bad) == 0, bad
    assert size(0, rows, k) == 0 and size(4, rows, top) > 0

    for m in (4, 333):  # packed weights; decoded ones
        need = size(m, rows, k)

        def call(x=fake, dh=fake, M=m, w=w0(), layout=0, out=fake, ws=fake, n=need):
            if gated:
                return L.nvfp4_linear_swiglu_grad(x, dh, M, w, layout, out, ws, n, null)
            return L.nvfp4_linear_grad(x, M, w, out, ws, n, null)

        assert call(M=-1) == SHAPE and call(M=(1 << 26) + 1) == SHAPE and call(w=None) == NULL
        for key in ("codes", "scales", "gs"):
            assert call(w=w0(**{key: null})) == NULL
        assert call(w=w0(codes=odd)) == ALIGN and call(w=w0(scales=odd)) == ALIGN
        assert call(w=w0(groups=2)) == SHAPE and call(w=w0(rows=0)) == SHAPE and call(w=w0(k=24)) == SHAPE
        assert call(w=w0(k=192)) == UNSUPPORTED and call(w=w0(k=top + 128)) == UNSUPPORTED
        assert call(w=w0(rows=72)) == UNSUPPORTED and call(w=w0(rows=(1 << 20) + 32)) == UNSUPPORTED
        if gated:
            assert call(layout=2) == SHAPE and call(layout=-1) == SHAPE
            assert call(w=w0(rows=63)) == SHAPE and call(w=w0(rows=48)) == UNSUPPORTED  # I = 24
        assert call(M=0, x=null, dh=null, out=null, ws=null, n=0) == OK
        for key in ("x", "out", "ws") + (("dh",) if gated else ()):
            assert call(**{key: null}) == NULL and call(**{key: odd}) == ALIGN
        assert call(n=need - 1) == WORKSPACE


# ---- the Python wrappers (CPU tensors: shapes are compared before devices) ----------------------------

M, K, N = 4, 256, 64


def _f16(*shape):
    return torch.zeros(shape, dtype=torch.float16)


def _u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def _w(rows=N, k=K):
    return G.NVFP4Tensor(_u8(1, rows, k // 2), _u8(1, rows, k // 16), torch.ones(1))


def _w8(rows=N, k=K):
    return G.FP8ChannelTensor(_u8(rows, k), torch.ones(rows))


def test_wrappers_check_shapes():
    x = _f16(M, K)
    rows = [
        (lambda: G.nvfp4_add_rms_norm(_f16(M, K, 1)), "x must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, _f16(K + 8)), "weight must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, residual=_f16(M - 1, K)), "residual must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, residual=x, s=_f16(M + 1, K)), "s must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, y=_f16(M, K - 8)), "y must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, want_q=True, q=_u8(M, K + 8)), "q must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, want_q=True, q_scale=torch.zeros(M + 1)), "q_scale must have shape"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, _f16(M, K + 8)), "dy must have shape"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, x, ds=_f16(M + 1, K)), "ds must have shape"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, x, _f16(K - 8)), "weight must have shape"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, x, dx=_f16(M, 8)), "dx must have shape"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, x, dweight=torch.zeros(K + 1)), "dweight must have shape"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, x, ws=_u8(16)), "ws holds"),
        (lambda: G.nvfp4_linear_fp8_rows(_u8(M, K + 128), torch.ones(M), _w8()), "xq must have shape"),
        (lambda: G.nvfp4_linear_fp8_rows(_u8(M, K), torch.ones(M + 1), _w8()), "x_scale must have shape"),
        (lambda: G.nvfp4_linear_fp8_rows(_u8(M, K), torch.ones(M), _w8(), y=_f16(M, N + 16)), "y must have shape"),
        (lambda: G.nvfp4_linear_grad(_f16(M, N + 16), _w()), "dy must have shape"),
        (lambda: G.nvfp4_linear_grad(_f16(M, N), _w(), dx=_f16(M, N)), "dx must have shape"),
        (lambda: G.nvfp4_linear_grad(_f16(M, N), _w(), ws=_u8(16)), "ws holds"),
        (lambda: G.nvfp4_linear_swiglu_grad(_f16(M, K + 128), _f16(M, N // 2), _w()), "x must have shape"),
        (lambda: G.nvfp4_linear_swiglu_grad(x, _f16(M, N), _w()), "dh must have shape"),
        (lambda: G.nvfp4_linear_swiglu_grad(x, _f16(M, N // 2), _w(), dz=_f16(M, N // 2)), "dz must have shape"),
        (lambda: G.nvfp4_linear_swiglu_grad(x, _f16(M, N // 2), _w(), ws=_u8(16)), "ws holds"),
    ]
    for fn, what in rows:
        with pytest.raises(ValueError, match=what):
            fn()
    for swap in ("codes", "scales", "global_scale"):
        w = _w()
        setattr(w, swap, getattr(_w(N + 16), swap) if swap != "global_scale" else torch.ones(2))
        with pytest.raises(ValueError, match="must keep the shapes"):
            _lib._frozen(w, -1)


def test_wrappers_refuse_cpu_tensors():
    for fn in (lambda: G.nvfp4_add_rms_norm(_f16(M, K)), lambda: G.nvfp4_add_rms_norm_grad(_f16(M, K), _f16(M, K)),
               lambda: G.nvfp4_linear_fp8_rows(_u8(M, K), torch.ones(M), _w8()),
               lambda: G.nvfp4_linear_grad(_f16(M, N), _w()),
               lambda: G.nvfp4_linear_swiglu_grad(_f16(M, K), _f16(M, N // 2), _w())):
        with pytest.raises(ValueError, match="GPU tensor"):
            fn()


def test_given_outputs_are_never_dropped():
    """A buffer that is given is written, so its shape is checked, or it is refused."""
    x = _f16(M, K)
    rows = [
        (lambda: G.nvfp4_add_rms_norm(x, q=_u8(M, K + 8)), "q must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, q_scale=torch.zeros(M + 1)), "q_scale must have shape"),
        (lambda: G.nvfp4_add_rms_norm(x, y=_f16(M, K), want_y=False, want_q=True), "want_y is False"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, x, dx=_f16(M, K), want_dx=False), "want_dx is False"),
        (lambda: G.nvfp4_add_rms_norm_grad(x, x, dweight=torch.zeros(K), want_dweight=False), "want_dweight is False"),
    ]
    for fn, what in rows:
        with pytest.raises(ValueError, match=what):
            fn()


def test_rows_refuse_more_columns_than_a_launch_holds(L):
    """32 columns are a block of 256 threads for few rows, and a launch holds fewer than 2^32 threads along one axis."""
    call = lambda rows, M=4: L.nvfp4_linear_fp8_rows(fake, fake, M, C.byref(fp8_channel_weights(fake, fake, rows, 128)), fake, null)  # noqa: E731,E501
    for rows in ((1 << 29) - 240, 1 << 29, 1 << 30, (1 << 31) - 16):
        assert call(rows) == UNSUPPORTED and call(rows, 0) == UNSUPPORTED, rows
    assert call((1 << 29) - 256, 0) == OK
