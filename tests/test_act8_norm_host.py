"""CPU tests of the 8-bit activation copies and RMSNorm: the oracle against
torch's own casts and against finite differences, and the library's refusals
(fake pointers that no kernel ever sees)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import nf4_oracle as o

FAKE = 0x40000


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantised_b200 as pkg
    pkg.lib()
    return pkg


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).bfloat16()


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_oracle_codes_equal_torch_casts(code):
    """Exact quotients rounded by torch (round half to even; the float8 cast)."""
    rng = np.random.default_rng(1)
    x = _bf16(rng, 50, 64)
    x[:, ::7] *= 12.0
    x[3] = 0.0
    x[4, 0], x[4, 1:] = 127.0, torch.arange(63) + 0.5            # ties of the int8 code
    codes, scales = o.act8_encode(x.double().numpy(), code)
    c = x.double().abs().amax(1, keepdim=True)
    qt = torch.where(c > 0, x.double() * o.ACT8_TOP[code] / c, 0.0)
    want = torch.round(qt).to(torch.int8) if code == "int8" else qt.float().to(torch.float8_e4m3fn)
    got = torch.from_numpy(codes).reshape(50, 64)
    want = want if code == "int8" else want.view(torch.uint8)
    live = c[:, 0] > 0
    assert torch.equal(got[live], want[live])
    assert np.array_equal(scales, (c[:, 0].float() / o.ACT8_TOP[code]).numpy())


@pytest.mark.parametrize("code,bound", [("int8", 1 / 254), ("e4m3", 2.0 ** -4)])
def test_oracle_round_trip_error(code, bound):
    """int8: half a step, c / 254, for every value; E4M3: half a step of the
    value's own binade (2^-4 of it, and never below the subnormal step
    c / 448 2^-10); then half a step of bf16 (2^-8 of the value at most)."""
    rng = np.random.default_rng(2)
    x = _bf16(rng, 400, 64).double().numpy()
    y = o.act8_decode(*o.act8_encode(x, code), code).reshape(x.shape).astype(np.float64)
    c = np.abs(x).max(1, keepdims=True)
    half = bound * c if code == "int8" else np.maximum(bound * np.abs(x), c / 448 * 2.0 ** -10)
    assert (np.abs(y - x) <= half * (1 + 2.0 ** -8) + np.abs(x) * 2.0 ** -8 + 1e-30).all()


def test_oracle_nonfinite_block_reads_back_as_nan():
    x = np.ones((3, 64))
    x[0, 5], x[2, 7] = np.inf, np.nan
    for code in ("int8", "e4m3"):
        codes, scales = o.act8_encode(x, code)
        y = o.act8_decode(codes, scales, code).reshape(3, 64)
        assert np.isnan(y[[0, 2]]).all() and (y[1] == 1).all()


def test_oracle_rmsnorm_gradients_against_differences():
    rng = np.random.default_rng(3)
    h, w, dy, dr = rng.standard_normal((4, 24)), rng.standard_normal(24), rng.standard_normal((4, 24)), rng.standard_normal((4, 24))
    dh, dw = o.rmsnorm_backward(dy, h, w, 1e-3, dr)
    loss = lambda h, w: (o.rmsnorm(h, w, 1e-3) * dy + h * dr).sum()
    e = 1e-6
    for _ in range(20):
        i, j = rng.integers(4), rng.integers(24)
        d = np.zeros_like(h)
        d[i, j] = e
        assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * e) - dh[i, j]) < 1e-7
        assert abs((loss(h, w + d[i]) - loss(h, w - d[i])) / (2 * e) - dw[j]) < 1e-7


def test_oracle_swiglu_gradients_against_differences():
    rng = np.random.default_rng(4)
    g, u, dh = rng.standard_normal((3, 50)) * 3
    dg, du = o.swiglu_backward(dh, g, u)
    e = 1e-6
    f = lambda g, u: dh * o.silu(g) * u
    assert np.abs((f(g + e, u) - f(g - e, u)) / (2 * e) - dg).max() < 1e-7
    assert np.abs((f(g, u + e) - f(g, u - e)) / (2 * e) - du).max() < 1e-7


# ------------------------------------------------------------------- refusals
def test_sizes(q):
    assert q.qlora_act8_sizes(4, 128) == (512, 32)
    assert q.qlora_act8_sizes(0, 64) == (0, 0)
    E = q._lib
    L = q.lib()
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    size = lambda r, c: L.qlora_act8_sizes(r, c, ctypes.byref(a), ctypes.byref(b))
    assert size(4, 100) == E.QLORA_ERR_UNSUPPORTED
    assert size(-1, 64) == E.QLORA_ERR_SHAPE
    assert size(1 << 40, 1 << 40) == E.QLORA_ERR_SHAPE
    assert L.qlora_act8_sizes(4, 64, None, ctypes.byref(b)) == E.QLORA_ERR_NULL
    nsize = lambda m, d: L.qlora_rmsnorm_workspace_size(m, d, ctypes.byref(a))
    assert nsize(0, 64) == 0 and a.value == 0
    assert nsize(5, 64) == 0 and a.value >= 256
    assert nsize(-1, 64) == E.QLORA_ERR_SHAPE
    for d in (0, 4, 12, 16384 + 8):
        assert nsize(5, d) == E.QLORA_ERR_UNSUPPORTED
    assert L.qlora_rmsnorm_workspace_size(5, 64, None) == E.QLORA_ERR_NULL


def test_act8_argument_errors(q):
    L, E, V = q.lib(), q._lib, q._lib._Act8
    good = V(FAKE, FAKE, 4, 128, 0)
    for call in (lambda v, x=FAKE: L.qlora_act8_quantize(x, v, None),
                 lambda v, x=FAKE: L.qlora_act8_dequantize(v, x, None),
                 lambda v, x=FAKE: L.qlora_swiglu_forward_act8(FAKE, x, FAKE, v, v, None),
                 lambda v, x=FAKE: L.qlora_swiglu_backward_act8(FAKE, v, v, FAKE, x, None, None)):
        assert call(good, None) == E.QLORA_ERR_NULL
        assert call(good, FAKE + 8) == E.QLORA_ERR_ALIGN
        assert call(V(0, FAKE, 4, 128, 0)) == E.QLORA_ERR_NULL
        assert call(V(FAKE, 0, 4, 128, 0)) == E.QLORA_ERR_NULL
        assert call(V(FAKE + 4, FAKE, 4, 128, 0)) == E.QLORA_ERR_ALIGN
        assert call(V(FAKE, FAKE + 4, 4, 128, 0)) == E.QLORA_ERR_ALIGN
        assert call(V(FAKE, FAKE, -1, 128, 0)) == E.QLORA_ERR_SHAPE
        assert call(V(FAKE, FAKE, 4, 96, 0)) == E.QLORA_ERR_UNSUPPORTED
        assert call(V(FAKE, FAKE, 4, 128, 2)) == E.QLORA_ERR_UNSUPPORTED
        assert call(V(0, 0, 0, 128, 1), None) == E.QLORA_OK        # empty: nothing launched
    other = V(FAKE, FAKE, 4, 64, 0)
    coded = V(FAKE, FAKE, 4, 128, 1)
    for bad in (other, coded):
        assert L.qlora_swiglu_forward_act8(FAKE, FAKE, FAKE, good, bad, None) == E.QLORA_ERR_SHAPE
        assert L.qlora_swiglu_backward_act8(FAKE, good, bad, FAKE, FAKE, None, None) == E.QLORA_ERR_SHAPE


def test_linear_and_mlp_argument_errors(q):
    L, E, V, T = q.lib(), q._lib, q._lib._Act8, q._lib._Tensor
    w = T(FAKE, FAKE, FAKE, 256, 512)
    need = q.qlora_linear_workspace_size(64, 256, 512, 8)
    def back(x8=V(FAKE, FAKE, 64, 512, 0), dY=FAKE, r=8, n=need, dA=FAKE, t=None):
        return L.qlora_linear_backward_act8(dY, x8, w, FAKE, FAKE, r, 2.0, t, None, dA, FAKE, 0, FAKE, n, None)
    assert back(x8=V(FAKE, FAKE, 64, 256, 0)) == E.QLORA_ERR_SHAPE
    assert back(x8=V(0, FAKE, 64, 512, 0)) == E.QLORA_ERR_NULL
    assert back(x8=V(FAKE, FAKE, 64, 512, 3)) == E.QLORA_ERR_UNSUPPORTED
    assert back(dY=None) == E.QLORA_ERR_NULL
    assert back(r=12) == E.QLORA_ERR_UNSUPPORTED
    assert back(n=need - 1) == E.QLORA_ERR_WORKSPACE
    assert back(dA=FAKE + 8) == E.QLORA_ERR_ALIGN
    assert back(t=FAKE + 4) == E.QLORA_ERR_ALIGN

    mlp = q._lib._Mlp(T(FAKE, FAKE, FAKE, 256, 128), T(FAKE, FAKE, FAKE, 256, 128), T(FAKE, FAKE, FAKE, 128, 256),
                      FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 8)
    n = ctypes.c_size_t()
    assert L.qlora_mlp_workspace_size(64, mlp, ctypes.byref(n)) == 0
    S = q._lib._MlpSaved8
    copy = lambda rows=64, cols=256, code=0: V(FAKE, FAKE, rows, cols, code)
    grads = q._lib._MlpGrads(*([FAKE] * 6))
    def fwd(sv, X=FAKE, size=n.value):
        return L.qlora_mlp_forward_act8(X, mlp, 2.0, FAKE, sv, FAKE, size, None)
    def bwd(sv, x8=V(FAKE, FAKE, 64, 128, 0), size=n.value, g=grads):
        return L.qlora_mlp_backward_act8(FAKE, x8, mlp, 2.0, sv, FAKE, g, 0, FAKE, size, None)
    good = S(copy(), copy(), FAKE, FAKE, FAKE)
    for call in (fwd, bwd):
        assert call(S(copy(cols=128), copy(cols=128), FAKE, FAKE, FAKE)) == E.QLORA_ERR_SHAPE
        assert call(S(copy(), copy(code=1), FAKE, FAKE, FAKE)) == E.QLORA_ERR_SHAPE
        assert call(S(copy(), copy(), FAKE, None, FAKE)) == E.QLORA_ERR_NULL
        assert call(S(copy(), copy(), FAKE, FAKE + 4, FAKE)) == E.QLORA_ERR_ALIGN
        assert call(good, size=n.value - 1) == E.QLORA_ERR_WORKSPACE
    assert fwd(good, X=None) == E.QLORA_ERR_NULL
    assert bwd(good, x8=V(FAKE, FAKE, 63, 128, 0)) == E.QLORA_ERR_SHAPE
    assert bwd(good, x8=V(FAKE, FAKE, 64, 256, 0)) == E.QLORA_ERR_SHAPE
    assert bwd(good, g=q._lib._MlpGrads(*([FAKE] * 5 + [0]))) == E.QLORA_ERR_NULL
    assert bwd(good, g=q._lib._MlpGrads(*([FAKE] * 5 + [FAKE + 4]))) == E.QLORA_ERR_ALIGN


def test_rmsnorm_argument_errors(q):
    L, E, V = q.lib(), q._lib, q._lib._Act8
    def fwd(X=FAKE, R=None, w=FAKE, M=4, D=128, eps=1e-5, H=None, Y=FAKE, y8=None):
        return L.qlora_rmsnorm_forward(X, R, w, M, D, eps, H, Y, y8, None)
    assert fwd(X=None) == E.QLORA_ERR_NULL
    assert fwd(w=None) == E.QLORA_ERR_NULL
    assert fwd(Y=None) == E.QLORA_ERR_NULL
    for k in ("X", "R", "w", "H", "Y"):
        assert fwd(**{k: FAKE + 8}) == E.QLORA_ERR_ALIGN
    assert fwd(M=-1) == E.QLORA_ERR_SHAPE
    for D in (0, 4, 100, 16392):
        assert fwd(D=D) == E.QLORA_ERR_UNSUPPORTED
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fwd(eps=eps) == E.QLORA_ERR_UNSUPPORTED
    assert fwd(y8=V(FAKE, FAKE, 4, 64, 0)) == E.QLORA_ERR_SHAPE
    assert fwd(y8=V(FAKE, FAKE, 3, 128, 0)) == E.QLORA_ERR_SHAPE
    assert fwd(D=72, y8=V(FAKE, FAKE, 4, 72, 0)) == E.QLORA_ERR_UNSUPPORTED
    assert fwd(y8=V(FAKE, 0, 4, 128, 0)) == E.QLORA_ERR_NULL
    assert fwd(X=None, Y=None, M=0) == E.QLORA_OK

    def bwd(dY=FAKE, H=FAKE, dR=None, w=FAKE, M=4, D=128, eps=1e-5, dX=FAKE, dw=FAKE, ws=FAKE, n=1 << 30):
        return L.qlora_rmsnorm_backward(dY, H, dR, w, M, D, eps, dX, dw, 0, ws, n, None)
    for k in ("dY", "H", "w", "dX"):
        assert bwd(**{k: None}) == E.QLORA_ERR_NULL
    for k in ("dY", "H", "dR", "w", "dX", "dw", "ws"):
        assert bwd(**{k: FAKE + 8}) == E.QLORA_ERR_ALIGN
    assert bwd(ws=None) == E.QLORA_ERR_WORKSPACE
    assert bwd(n=16) == E.QLORA_ERR_WORKSPACE
    assert bwd(M=-2) == E.QLORA_ERR_SHAPE
    assert bwd(D=12) == E.QLORA_ERR_UNSUPPORTED
    assert bwd(M=0, dY=None, H=None, dX=None, dw=None, ws=None, n=0) == E.QLORA_OK


def test_python_refuses_before_the_library(q):
    """Tensors on the host, of another type, shape or layout."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.ones(128)
    for call in (lambda: q.qlora_rmsnorm_forward(x, w, 1e-5),
                 lambda: q.qlora_rmsnorm_backward(x, x, w, 1e-5),
                 lambda: q.qlora_act8_quantize(x),
                 lambda: q.qlora_swiglu_forward_act8(x, x),
                 lambda: q.qlora_swiglu_backward_act8(x, None, None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.QloraError):
        q.empty_act8(4, 100, device="cpu")
    x8 = q.empty_act8(4, 128, q.QLORA_ACT8_E4M3, device="cpu")
    assert x8.codes.dtype == torch.float8_e4m3fn and x8.nbytes == 512 + 32


def test_nf4_weights_of_another_type_are_refused(q):
    """The calls above count an NF4 weight's values; a half-width constant
    would be read past its end."""
    dev, n = torch.device("cpu"), q.qlora_quantized_sizes(64, 256)
    good = lambda: q.NF4Tensor(torch.zeros(n[0], dtype=torch.uint8), torch.zeros(n[1], dtype=torch.uint8),
                               torch.zeros(n[2] // 4), 64, 256)
    q._lib._nf4_struct(good(), dev, "w")
    w = good()
    w.scale_codes = w.scale_codes.view(torch.float8_e4m3fn)        # the codes under their own type
    q._lib._nf4_struct(w, dev, "w")
    for name, t in (("packed", torch.int16), ("packed", torch.float32), ("scale_codes", torch.bfloat16),
                    ("meta_scale", torch.float16), ("meta_scale", torch.bfloat16), ("meta_scale", torch.float64),
                    ("meta_scale", torch.int32)):
        w = good()
        setattr(w, name, getattr(w, name).to(t))
        with pytest.raises(ValueError, match=f"w.{name}"):
            q._lib._nf4_struct(w, dev, "w")
