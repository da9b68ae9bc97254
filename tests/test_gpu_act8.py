"""GPU tests of the 8-bit activation copies and their use in the backward
pass.  Codes, scales and the values read back are compared with the oracle
bit for bit.  The linear and MLP backwards are compared bit for bit with the
bf16 calls on the values read back, which the other tests hold to the oracle.
The SwiGLU outputs must lie within one bf16 rounding of the fp64 value widened
by the fp32 evaluation's error."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import nf4_oracle as o

from _parity import assert_close

pytestmark = pytest.mark.gpu

CODES = ["int8", "e4m3"]


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import bit_nf4_quantised_b200 as pkg
    pkg.lib()
    return pkg


def _code(q, name):
    return {"int8": q.QLORA_ACT8_INT8, "e4m3": q.QLORA_ACT8_E4M3}[name]


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1)


def _values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _same(a, b):
    """Equal bits, any NaN equal to any NaN."""
    a, b = np.asarray(a), np.asarray(b)
    nan = ((a & 0x7FFF) > 0x7F80) & ((b & 0x7FFF) > 0x7F80)
    return np.array_equal(a[~nan], b[~nan])


def _rows(rng, M, K):
    """Normal values with outlier columns, a row of zeros, tiny and huge rows."""
    x = rng.standard_normal((M, K), dtype=np.float32)
    x[:, ::37] *= 20.0
    if M > 4:
        x[1] = 0.0
        x[2] *= np.float32(2.0 ** -120)
        x[3] *= np.float32(2.0 ** 100)
        x[4] = np.round(x[4] * 8) / 2            # many equal magnitudes and code ties
        x[4, 0] = 127.0
    return torch.from_numpy(x).bfloat16()


def _inside(got_bits, exact, err):
    lo, hi = _values(o.bf16_rne_f64(exact - err)), _values(o.bf16_rne_f64(exact + err))
    g = _values(got_bits).reshape(exact.shape)
    ok = (g >= lo) & (g <= hi)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside, worst {np.abs(g - exact)[~ok].max()}"


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("M,K", [(1, 64), (1, 4096), (7, 192), (513, 1088), (3, 11008), (1000, 64), (2048, 4096)])
def test_copy_is_the_oracles(q, code, M, K):
    x = _rows(np.random.default_rng(M + K), M, K)
    x8 = q.qlora_act8_quantize(x.cuda(), _code(q, code))
    y = q.qlora_act8_dequantize(x8)
    codes, scales = o.act8_encode(x.double().numpy(), code)
    got = x8.codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(got, codes.view(np.uint8)), f"{(got != codes.view(np.uint8)).sum()} codes differ"
    assert np.array_equal(x8.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(_bits(y), o.act8_decode_bits(codes, scales, code))


@pytest.mark.parametrize("code", CODES)
def test_every_finite_magnitude(q, code):
    """Each bf16 magnitude as a block's largest, with fractions of it: from
    the subnormals to the largest finite value."""
    top = torch.arange(1, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = top[:, None].repeat(1, 64)
    x[:, 1:] = (x[:, 1:].double() * torch.linspace(-1, 1, 63, dtype=torch.float64)).bfloat16()
    x8 = q.qlora_act8_quantize(x.cuda(), _code(q, code))
    codes, scales = o.act8_encode(x.double().numpy(), code)
    assert np.array_equal(x8.codes.view(torch.uint8).cpu().numpy(), codes.view(np.uint8))
    assert np.array_equal(x8.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(_bits(q.qlora_act8_dequantize(x8)), o.act8_decode_bits(codes, scales, code))


@pytest.mark.parametrize("code", CODES)
def test_nonfinite_values_make_their_block_nan(q, code):
    x = torch.ones(6, 192, dtype=torch.bfloat16)
    x[0, 70], x[2, 0], x[5, 191] = float("inf"), float("nan"), float("-inf")
    x8 = q.qlora_act8_quantize(x.cuda(), _code(q, code))
    y = q.qlora_act8_dequantize(x8).cpu().float().reshape(6, 3, 64)
    bad = torch.zeros(6, 3, dtype=torch.bool)
    bad[0, 1] = bad[2, 0] = bad[5, 2] = True
    assert torch.isnan(y[bad]).all() and (y[~bad] == 1).all()


def test_empty_and_given_buffers(q):
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    x8 = q.qlora_act8_quantize(e)
    assert q.qlora_act8_dequantize(x8).shape == (0, 128)
    h, g8, u8 = q.qlora_swiglu_forward_act8(e, e)
    dg, du = q.qlora_swiglu_backward_act8(e, g8, u8)
    assert h.shape == dg.shape == du.shape == (0, 128)
    x = torch.randn(5, 128, device="cuda").bfloat16()
    # rows behind the given buffers stay as they were
    big = q.empty_act8(8, 128, q.QLORA_ACT8_INT8)
    big.codes.fill_(99)
    big.scales.fill_(7.0)
    part = q.Act8(big.codes[: 5 * 128], big.scales[: 5 * 2], 5, 128)
    q.qlora_act8_quantize(x, out=part)
    assert (big.codes[5 * 128:] == 99).all() and (big.scales[10:] == 7).all()
    with pytest.raises(ValueError):
        q.qlora_act8_quantize(x, out=big)
    with pytest.raises(ValueError):
        q.qlora_act8_quantize(x[:, :64])                       # strided
    with pytest.raises(ValueError):
        q.qlora_swiglu_forward_act8(x, x[:4])
    with pytest.raises(q.QloraError):
        q.qlora_act8_quantize(torch.zeros(4, 96, device="cuda").bfloat16())
    with pytest.raises(q.QloraError):                          # 2-byte aligned rows
        q.qlora_act8_quantize(torch.zeros(129, device="cuda").bfloat16()[1:].reshape(2, 64))


# --------------------------------------------------------------------- SwiGLU
# fp32 evaluation: the sigmoid within 2^-21 of itself (expf 2 ulp, one sum, one
# division), then at most five products: 2^-20 of each term, where silu' =
# s + s g (1 - s) has 1 - s off by 2^-23 at most.  For z < -88.72, exp(-z) is
# past fp32 and s is 0 in place of at most exp(-88.72) = 2^-128; |z| exp(z)
# falls with -z, so |z| s (and s (1 + |z|)) is then off by less than
# 90 2^-128 < 2^-121, times the other factors.
E = 2.0 ** -20
TINY = 2.0 ** -121


def _swiglu_check(q, code, M, F, hidden):
    rng = np.random.default_rng(M * F)
    g, u = _rows(rng, M, F), _rows(rng, M, F)
    if M > 4:
        g[0, :8] = torch.tensor([0.0, -0.0, 30.0, -30.0, 89.0, -89.0, 200.0, -200.0])
        g[3], u[3] = g[0], u[0]                    # huge rows overflow the product: tested elsewhere
    dh = torch.from_numpy(rng.standard_normal((M, F), dtype=np.float32)).bfloat16()
    H, g8, u8 = q.qlora_swiglu_forward_act8(g.cuda(), u.cuda(), _code(q, code))
    G, U = g.double().numpy(), u.double().numpy()
    with np.errstate(over="ignore"):
        _inside(_bits(H), o.silu(G) * U, E * np.abs(o.silu(G) * U) + TINY * (1 + np.abs(U)))
    for got, x in ((g8, g), (u8, u)):
        codes, scales = o.act8_encode(x.double().numpy(), code)
        assert np.array_equal(got.codes.view(torch.uint8).cpu().numpy(), codes.view(np.uint8))
        assert np.array_equal(got.scales.cpu().numpy(), scales)
    Hb = torch.empty_like(H) if hidden else None
    dG, dU = q.qlora_swiglu_backward_act8(dh.cuda(), g8, u8, H=Hb)
    gt = _values(_bits(q.qlora_act8_dequantize(g8))).reshape(M, F)
    ut = _values(_bits(q.qlora_act8_dequantize(u8))).reshape(M, F)
    d = dh.double().numpy()
    with np.errstate(over="ignore"):
        dg, du = o.swiglu_backward(d, gt, ut)
        s = 1 / (1 + np.exp(-gt))
        _inside(_bits(dG), dg, E * np.abs(d * ut) * s * (1 + np.abs(gt) * (1 - s)) + np.abs(d * ut * gt) * s * 2.0 ** -23 + TINY * (1 + np.abs(d * ut)))
        _inside(_bits(dU), du, E * np.abs(du) + TINY * (1 + np.abs(d)))
        if hidden:
            _inside(_bits(Hb), o.silu(gt) * ut, E * np.abs(o.silu(gt) * ut) + TINY * (1 + np.abs(ut)))


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("M,F", [(1, 64), (6, 128), (33, 1088), (257, 11008)])
def test_swiglu(q, code, M, F):
    _swiglu_check(q, code, M, F, hidden=M != 6)


def test_swiglu_in_place(q):
    g, u, dh = (torch.randn(9, 320, device="cuda").bfloat16() for _ in range(3))
    H, g8, u8 = q.qlora_swiglu_forward_act8(g, u)
    dG, dU = q.qlora_swiglu_backward_act8(dh, g8, u8)
    g2 = g.clone()
    H2, _, _ = q.qlora_swiglu_forward_act8(g2, u, H=g2)
    d2 = dh.clone()
    dG2, dU2 = q.qlora_swiglu_backward_act8(d2, g8, u8, dG=d2)
    assert torch.equal(H2, H) and torch.equal(dG2, dG) and torch.equal(dU2, dU)
    assert H2.data_ptr() == g2.data_ptr() and dG2.data_ptr() == d2.data_ptr()


# --------------------------------------------------- the adapted linear layer
def _layer(q, M, N, K, r, seed):
    rng = np.random.default_rng(seed)
    f = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32))
    W = 0.02 * f(N, K)
    w = q.qlora_quantize(W.cuda())
    A, B = (f(r, K) / K ** 0.5).bfloat16().cuda(), (0.01 * f(N, r)).bfloat16().cuda()
    X = _rows(rng, M, K)
    X[X.abs() > 1e10] = 1.0                        # keeps the products finite
    return w, W, A, B, X.cuda(), f(M, N).bfloat16().cuda()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("saved", [True, False])
@pytest.mark.parametrize("M,N,K,r", [(1, 8, 64, 8), (5, 72, 128, 16), (64, 256, 512, 8), (100, 264, 320, 24),
                                     (513, 640, 1088, 128), (1000, 128, 256, 64), (129, 256, 192, 72)])
def test_linear_backward_equals_the_one_on_the_values_read_back(q, code, saved, M, N, K, r):
    w, _, A, B, X, dY = _layer(q, M, N, K, r, M + N + K + r)
    x8 = q.qlora_act8_quantize(X, _code(q, code))
    Xt = q.qlora_act8_dequantize(x8)
    T = (X.float() @ A.float().t()).contiguous() if saved else None
    ws = q.workspace(M, N, K, r)
    got = q.qlora_linear_backward_act8(dY, x8, w, A, B, 2.0, T_saved=T, ws=ws)
    torch.cuda.synchronize()
    assert q.device_error_word(ws) == 0
    want = q.qlora_linear_backward(dY, Xt, w, A, B, 2.0, T_saved=T)
    for name, a, b in zip(("dX", "dA", "dB"), got, want):
        assert torch.equal(a, b), f"{name}: {(a != b).sum()} of {a.numel()} differ"


def test_linear_backward_against_the_oracle(q):
    M, N, K, r = 200, 264, 512, 16
    w, W, A, B, X, dY = _layer(q, M, N, K, r, 3)
    x8 = q.qlora_act8_quantize(X)
    dX, dA, dB = q.qlora_linear_backward_act8(dY, x8, w, A, B, 2.0)
    Wt = o.dequantize(*o.quantize(W.numpy()), N, K).astype(np.float64)
    codes, scales = o.act8_encode(X.double().cpu().numpy(), "int8")
    Xt = o.act8_decode(codes, scales, "int8").reshape(M, K).astype(np.float64)
    f = lambda t: t.double().cpu().numpy()
    rX, rA, rB, _ = o.linear_backward(f(dY), Xt, Wt, f(A), f(B), 2.0)
    for n, a, b in (("dX", dX, rX), ("dA", dA, rA), ("dB", dB, rB)):
        assert_close(n, a, b)


def test_linear_backward_accumulates_skips_dx_and_takes_no_tokens(q):
    M, N, K, r = 70, 128, 256, 16
    w, _, A, B, X, dY = _layer(q, M, N, K, r, 5)
    x8 = q.qlora_act8_quantize(X)
    _, dA, dB = q.qlora_linear_backward_act8(dY, x8, w, A, B, 2.0)
    a0, b0 = torch.ones_like(dA), torch.full_like(dB, -3.0)
    dX, a1, b1 = q.qlora_linear_backward_act8(dY, x8, w, A, B, 2.0, dA=a0, dB=b0, accumulate=True, want_dX=False)
    assert dX is None and torch.equal(a1, 1 + dA) and torch.equal(b1, -3 + dB)
    e8 = q.qlora_act8_quantize(X[:0])
    dX, a2, b2 = q.qlora_linear_backward_act8(dY[:0], e8, w, A, B, 2.0)
    assert dX.shape == (0, K) and not a2.any() and not b2.any()
    with pytest.raises(ValueError):
        q.qlora_linear_backward_act8(dY, x8, w, A, B, 2.0, accumulate=True)
    with pytest.raises(ValueError):
        q.qlora_linear_backward_act8(dY[:5], x8, w, A, B, 2.0)
    with pytest.raises(ValueError):
        q.qlora_linear_backward_act8(dY, x8, w, A, B, 2.0, T_saved=torch.zeros(M, r + 8, device="cuda"))


# -------------------------------------------------------------------- the MLP
def _mlp(q, M, D, F, r, seed):
    layers = [_layer(q, M, n, k, r, seed + i) for i, (n, k) in enumerate(((F, D), (F, D), (D, F)))]
    (wg, Wg, Ag, Bg, X, _), (wu, Wu, Au, Bu, _, _), (wd, Wd, Ad, Bd, _, dY) = layers
    f = lambda t: t.double().cpu().numpy()
    host = {n: (o.dequantize(*o.quantize(W.numpy()), *W.shape).astype(np.float64), f(A), f(B))
            for n, W, A, B in (("gate", Wg, Ag, Bg), ("up", Wu, Au, Bu), ("down", Wd, Ad, Bd))}
    X = torch.randn(M, D, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    return q.MLP(wg, wu, wd, Ag, Bg, Au, Bu, Ad, Bd), host, X, dY


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("M,D,F,r", [(100, 256, 640, 8), (12, 512, 768, 16), (513, 320, 1088, 24)])
def test_mlp(q, code, M, D, F, r):
    mlp, host, X, dY = _mlp(q, M, D, F, r, D + F)
    c, ws = _code(q, code), q.mlp_workspace(M, mlp)
    Y, saved = q.qlora_mlp_forward_act8(X, mlp, 2.0, c, ws=ws)
    torch.cuda.synchronize()
    assert q.device_error_word(ws) == 0
    assert torch.equal(Y, q.qlora_mlp_forward(X, mlp, 2.0))
    # what it keeps is what the layers' own calls give
    T = [torch.empty(M, r, device="cuda") for _ in range(3)]
    G = q.qlora_linear_forward(X, mlp.gate, mlp.A_gate, mlp.B_gate, 2.0, T_save=T[0])
    U = q.qlora_linear_forward(X, mlp.up, mlp.A_up, mlp.B_up, 2.0, T_save=T[1])
    H, g8, u8 = q.qlora_swiglu_forward_act8(G, U, c)
    q.qlora_linear_forward(H, mlp.down, mlp.A_down, mlp.B_down, 2.0, T_save=T[2])
    byte = lambda t: t.view(torch.uint8)
    for a, b in ((byte(saved.g.codes), byte(g8.codes)), (byte(saved.u.codes), byte(u8.codes)),
                 (saved.g.scales, g8.scales), (saved.u.scales, u8.scales), (saved.T_gate, T[0]),
                 (saved.T_up, T[1]), (saved.T_down, T[2])):
        assert torch.equal(a, b)
    x8 = q.qlora_act8_quantize(X, c)
    dX, grads = q.qlora_mlp_backward_act8(dY, x8, mlp, 2.0, saved, ws=ws)
    torch.cuda.synchronize()
    assert q.device_error_word(ws) == 0
    # the same from the parts
    Hb, dH0 = torch.empty_like(G), torch.zeros_like(G)
    q.qlora_swiglu_backward_act8(dH0, g8, u8, H=Hb)
    dH, dAd, dBd = q.qlora_linear_backward(dY, Hb, mlp.down, mlp.A_down, mlp.B_down, 2.0, T_saved=T[2])
    dG, dU = q.qlora_swiglu_backward_act8(dH, g8, u8)
    dXg, dAg, dBg = q.qlora_linear_backward_act8(dG, x8, mlp.gate, mlp.A_gate, mlp.B_gate, 2.0, T_saved=T[0])
    dXu, dAu, dBu = q.qlora_linear_backward_act8(dU, x8, mlp.up, mlp.A_up, mlp.B_up, 2.0, T_saved=T[1])
    assert torch.equal(dX, (dXg.float() + dXu.float()).bfloat16())
    for n, a, b in (("gate", dAg, dBg), ("up", dAu, dBu), ("down", dAd, dBd)):
        assert torch.equal(grads[f"dA_{n}"], a) and torch.equal(grads[f"dB_{n}"], b), n
    # and in 64 bits from the same copies
    val = lambda a8: _values(_bits(q.qlora_act8_dequantize(a8))).reshape(a8.rows, a8.cols)
    g, u, x, f = val(saved.g), val(saved.u), val(x8), lambda t: t.double().cpu().numpy()
    rdX, rg = o.mlp_backward(f(dY), x, host, 2.0, (g, u, o.silu(g) * u), bf16_activations=True)
    assert_close("dX", dX, rdX)
    for n in ("gate", "up", "down"):
        assert_close(f"dA_{n}", grads[f"dA_{n}"], rg[n][0])
        # T comes from the unrounded X and h, so dB differs by their 8-bit error
    # accumulation, and an empty batch
    twice = {k: v.clone() for k, v in grads.items()}
    q.qlora_mlp_backward_act8(dY, x8, mlp, 2.0, saved, grads=twice, accumulate=True)
    assert all(torch.equal(twice[k], 2 * grads[k]) for k in grads)
    Y0, s0 = q.qlora_mlp_forward_act8(X[:0], mlp, 2.0, c)
    dX0, g0 = q.qlora_mlp_backward_act8(dY[:0], q.qlora_act8_quantize(X[:0], c), mlp, 2.0, s0)
    assert Y0.shape == dX0.shape == (0, D) and not any(v.any() for v in g0.values())


def test_mlp_gradients_near_the_recomputing_backward(q):
    """int8 keeps each value within c / 254 of itself, c the largest of 64:
    about 2.5 of their rms, so an error of about 0.6% of it per value, in g, u
    and X each.  Gradients are sums of products with at most three such
    factors, so their relative error stays below 0.02 (three times 0.6%, and
    the bf16 roundings that both sides carry)."""
    M, D, F, r = 512, 512, 1024, 16
    mlp, _, X, dY = _mlp(q, M, D, F, r, 77)
    _, saved = q.qlora_mlp_forward_act8(X, mlp, 2.0)
    dX, g = q.qlora_mlp_backward_act8(dY, q.qlora_act8_quantize(X), mlp, 2.0, saved)
    rX, rg = q.qlora_mlp_backward(dY, X, mlp, 2.0)
    rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())
    assert rel(dX, rX) < 0.02
    for k in g:
        assert rel(g[k], rg[k]) < 0.02, (k, rel(g[k], rg[k]))
