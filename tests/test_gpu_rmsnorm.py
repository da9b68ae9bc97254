"""GPU tests of RMSNorm with the residual's addition, its 8-bit output and its
backward, against the oracle in fp64; and of a training step of the block
(norm, MLP from 8-bit copies, both backwards) as it would be used: eager, on
another stream, captured and replayed.

Bounds.  The sum of squares of a row is a sum of at most 40 sequential
fp32 additions per lane and then a tree over at most 32 lanes and 32 warps,
all terms positive: it is within (40 + 5 + 32 + 2) 2^-24 of itself, its root
within half of that; y takes three more roundings.  60 2^-24 = 2^-18 covers
them, then one rounding to bf16.  In the backward the sum of h t has the same
depth, relative to the sum of |h t|."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import nf4_oracle as o

from _threads import at_once

pytestmark = pytest.mark.gpu
E = 2.0 ** -18


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import bit_nf4_quantised_b200 as pkg
    pkg.lib()
    return pkg


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1)


def _values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _inside(t, exact, err):
    lo, hi = _values(o.bf16_rne_f64(exact - err)), _values(o.bf16_rne_f64(exact + err))
    g = t.double().cpu().numpy()
    ok = (g >= lo) & (g <= hi)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside"


def _f(t):
    return t.double().cpu().numpy()


def _inputs(M, D, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    x, r, dy, dr = (n(M, D).bfloat16().cuda() for _ in range(4))
    x[:, ::53] *= 30.0
    if M > 3:
        x[1], r[1] = 0.0, 0.0                       # a padding row
        x[2], r[2] = x[2] * 2.0 ** 40, r[2] * 2.0 ** 40
    return x, r, dy, dr, (1 + 0.3 * n(D)).cuda()


SHAPES = [(1, 8), (1, 4096), (3, 64), (5, 1024), (7, 1032), (33, 1088), (513, 320), (300, 2048), (149, 4096),
          (2, 16384), (200, 8200), (160, 16384), (1300, 768), (2500, 128)]


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("M,D", SHAPES)
def test_forward(q, M, D, res):
    x, r, _, _, w = _inputs(M, D, M + D)
    code = (q.QLORA_ACT8_INT8, q.QLORA_ACT8_E4M3)[M % 2]
    q8 = q.empty_act8(M, D, code) if D % 64 == 0 else None
    Y, H = q.qlora_rmsnorm_forward(x, w, 1e-5, residual=r if res else None, q8=q8)
    if res:
        assert torch.equal(H, (x.float() + r.float()).bfloat16())
    else:
        assert H is x
    exact = o.rmsnorm(_f(H), _f(w), float(np.float32(1e-5)))
    _inside(Y, exact, E * np.abs(exact))
    if q8 is not None:
        want = q.qlora_act8_quantize(Y, code)
        assert torch.equal(q8.codes.view(torch.uint8), want.codes.view(torch.uint8))
        assert torch.equal(q8.scales, want.scales)
        only = q.empty_act8(M, D, code)
        none, _ = q.qlora_rmsnorm_forward(x, w, 1e-5, residual=r if res else None, q8=only, want_Y=False)
        assert none is None and torch.equal(only.codes.view(torch.uint8), q8.codes.view(torch.uint8))
    # in place: the residual stream is overwritten, then x by y
    x2, r2 = x.clone(), r.clone()
    Y2, H2 = q.qlora_rmsnorm_forward(x2, w, 1e-5, residual=r2 if res else None, H=r2 if res else None, Y=x2)
    assert torch.equal(Y2, Y) and (not res or (torch.equal(r2, H) and H2 is r2))


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("M,D", SHAPES)
def test_backward(q, M, D, res):
    h, _, dy, dr, w = _inputs(M, D, M * 3 + D)
    dX, dw = q.qlora_rmsnorm_backward(dy, h, w, 1e-5, dres=dr if res else None)
    eps = float(np.float32(1e-5))
    H, G, W, R = _f(h), _f(dy), _f(w), _f(dr) if res else 0.0
    rx, rw = o.rmsnorm_backward(G, H, W, eps, R if res else None)
    rstd = 1 / np.sqrt((H * H).mean(1, keepdims=True) + eps)
    t = G * W
    size = rstd * (np.abs(t) + np.abs(H) * rstd ** 2 * np.abs(H * t).mean(1, keepdims=True)) + np.abs(R)
    _inside(dX, rx, 2 * E * size)
    # each partial sums its rows in order, then the partials are summed: at
    # most M additions, on terms with a relative error of 2^-18
    term = np.abs(G * H * rstd).sum(0)
    assert (np.abs(_f(dw) - rw) <= (E + (M + 8) * 2.0 ** -24) * term + 1e-37).all()
    # a frozen weight, accumulation, in place; and the same bytes again
    again, none = q.qlora_rmsnorm_backward(dy, h, w, 1e-5, dres=dr if res else None, want_dweight=False)
    assert none is None and torch.equal(again, dX)
    acc = torch.full((D,), 0.5, device="cuda")
    d2 = dy.clone()
    x2, _ = q.qlora_rmsnorm_backward(d2, h, w, 1e-5, dres=dr if res else None, dX=d2, dweight=acc, accumulate=True)
    assert x2 is d2 and torch.equal(d2, dX) and torch.equal(acc, 0.5 + dw)


@pytest.mark.parametrize("M,D", [(4000, 2056), (1500, 4096), (700, 16384)])
def test_many_rows_of_a_cta(q, M, D):
    """More rows than a persistent grid takes at once, past several rounds of
    its ring: the same bytes as the rows in two halves, which other CTAs take."""
    h, r, dy, dr, w = _inputs(M, D, M + D)
    q8 = q.empty_act8(M, D) if D % 64 == 0 else None
    Y, H = q.qlora_rmsnorm_forward(h, w, 1e-5, residual=r, q8=q8)
    dX, dw = q.qlora_rmsnorm_backward(dy, H, w, 1e-5, dres=dr)
    exact = o.rmsnorm(_f(H), _f(w), float(np.float32(1e-5)))
    _inside(Y, exact, E * np.abs(exact))
    k = M // 2 + 1
    for rows in (slice(0, k), slice(k, M)):
        p8 = q.empty_act8(rows.stop - rows.start, D) if q8 is not None else None
        Yp, Hp = q.qlora_rmsnorm_forward(h[rows], w, 1e-5, residual=r[rows], q8=p8)
        dXp, _ = q.qlora_rmsnorm_backward(dy[rows], Hp, w, 1e-5, dres=dr[rows], want_dweight=False)
        assert torch.equal(Yp, Y[rows]) and torch.equal(Hp, H[rows]) and torch.equal(dXp, dX[rows])
        if p8 is not None:
            assert torch.equal(p8.codes, q8.codes.view(M, D)[rows].reshape(-1))
            assert torch.equal(p8.scales, q8.scales.view(M, D // 64)[rows].reshape(-1))
    Hf, G = _f(H), _f(dy)
    term = G * Hf / np.sqrt((Hf * Hf).mean(1, keepdims=True) + float(np.float32(1e-5)))
    assert (np.abs(_f(dw) - term.sum(0)) <= (E + (M + 8) * 2.0 ** -24) * np.abs(term).sum(0) + 1e-37).all()


def test_zero_rows_and_empty_batches(q):
    w = torch.ones(256, device="cuda")
    z = torch.zeros(4, 256, device="cuda").bfloat16()
    Y, _ = q.qlora_rmsnorm_forward(z, w, 1e-6)
    assert not Y.any()
    e = z[:0]
    Y, H = q.qlora_rmsnorm_forward(e, w, 1e-6, residual=e)
    dX, dw = q.qlora_rmsnorm_backward(e, e, w, 1e-6)
    assert Y.shape == H.shape == dX.shape == (0, 256) and not dw.any()
    keep = torch.full((256,), 3.0, device="cuda")
    q.qlora_rmsnorm_backward(e, e, w, 1e-6, dweight=keep, accumulate=True)
    assert (keep == 3).all()


def test_nonfinite_rows_stay_in_their_rows(q):
    x, r, dy, dr, w = _inputs(200, 1088, 1)
    Y, _ = q.qlora_rmsnorm_forward(x, w, 1e-5)
    x2 = x.clone()
    x2[5, 3], x2[9, 0] = float("nan"), float("inf")
    q8 = q.empty_act8(200, 1088)
    Y2, _ = q.qlora_rmsnorm_forward(x2, w, 1e-5, q8=q8)
    ok = torch.ones(200, dtype=torch.bool, device="cuda")
    ok[5] = ok[9] = False
    assert torch.equal(Y2[ok], Y[ok]) and Y2[5].isnan().all() and Y2[9, 0].isnan() and not Y2[9, 1:].any()
    y8 = q.qlora_act8_dequantize(q8)
    assert y8[5].isnan().all() and y8[9, :64].isnan().all() and not y8[9, 64:].any() and y8[ok].isfinite().all()
    dX, _ = q.qlora_rmsnorm_backward(dy, x2, w, 1e-5)
    assert dX[ok].isfinite().all() and dX[5].isnan().all()


def test_refusals(q):
    x, r, dy, dr, w = _inputs(6, 128, 2)
    for bad in (lambda: q.qlora_rmsnorm_forward(x[:, :64], w[:64], 1e-5),                    # strided
                lambda: q.qlora_rmsnorm_forward(x, w.bfloat16(), 1e-5),
                lambda: q.qlora_rmsnorm_forward(x, w[:64], 1e-5),
                lambda: q.qlora_rmsnorm_forward(x, w, 1e-5, residual=r[:5]),
                lambda: q.qlora_rmsnorm_forward(x, w, 1e-5, q8=q.empty_act8(5, 128)),
                lambda: q.qlora_rmsnorm_forward(x.float(), w, 1e-5),
                lambda: q.qlora_rmsnorm_backward(dy, x[:5], w, 1e-5),
                lambda: q.qlora_rmsnorm_backward(dy, x, w, 1e-5, accumulate=True),
                lambda: q.qlora_rmsnorm_backward(dy, x, w, 1e-5, dweight=w[:64])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(q.QloraError):
        q.qlora_rmsnorm_forward(x, w, -1.0)
    with pytest.raises(q.QloraError):
        q.qlora_rmsnorm_backward(dy, x, w, 1e-5, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------------ the block's step
def _block(q, M, D, F, r, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).cuda()
    wt = [q.qlora_quantize(0.02 * n(a, b)) for a, b in ((F, D), (F, D), (D, F))]
    ab = []
    for a, b in ((F, D), (F, D), (D, F)):
        ab += [(n(r, b) / b ** 0.5).bfloat16(), (0.01 * n(a, r)).bfloat16()]
    mlp = q.MLP(*wt, *ab)
    x, res, dout = (n(M, D).bfloat16() for _ in range(3))
    return mlp, x, res, dout, 1 + 0.1 * n(D)


def _step(q, mlp, x, res, dout, w, code, ws, nws, stream=None):
    """out = mlp(norm(x + res)) ; gradients of x, the norm and the adapters
    for dout at the MLP's output and at the residual stream."""
    y8 = q.empty_act8(*x.shape, code)
    Y, H = q.qlora_rmsnorm_forward(x, w, 1e-5, residual=res, q8=y8, stream=stream)
    out, saved = q.qlora_mlp_forward_act8(Y, mlp, 2.0, code, ws=ws, stream=stream)
    dY, grads = q.qlora_mlp_backward_act8(dout, y8, mlp, 2.0, saved, ws=ws, stream=stream)
    dX, dw = q.qlora_rmsnorm_backward(dY, H, w, 1e-5, dres=dout, ws=nws, stream=stream)
    return [out, dX, dw] + [grads[k] for k in sorted(grads)], (Y, H, y8, saved, dY)


def _buffers(q, mlp, M, D):
    return q.mlp_workspace(M, mlp), torch.empty(q.qlora_rmsnorm_workspace_size(M, D), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_block_step_against_the_formulas(q, code):
    M, D, F, r = 130, 320, 640, 16
    c = {"int8": q.QLORA_ACT8_INT8, "e4m3": q.QLORA_ACT8_E4M3}[code]
    mlp, x, res, dout, w = _block(q, M, D, F, r, 9)
    outs, (Y, H, y8, saved, dY) = _step(q, mlp, x, res, dout, w, c, *_buffers(q, mlp, M, D))
    want = q.qlora_act8_quantize(Y, c)
    assert torch.equal(y8.codes.view(torch.uint8), want.codes.view(torch.uint8))
    assert torch.equal(outs[0], q.qlora_mlp_forward(Y, mlp, 2.0))
    rx, rw = o.rmsnorm_backward(_f(dY), _f(H), _f(w), float(np.float32(1e-5)), _f(dout))
    rel = lambda a, b: np.linalg.norm(_f(a) - b) / np.linalg.norm(b)
    assert rel(outs[1], rx) < 2.0 ** -8 and rel(outs[2], rw) < E + (M + 8) * 2.0 ** -24
    dY2, g2 = q.qlora_mlp_backward_act8(dout, y8, mlp, 2.0, saved)
    assert torch.equal(dY2, dY) and all(torch.equal(a, g2[k]) for a, k in zip(outs[3:], sorted(g2)))


def test_block_step_on_streams_and_captured(q):
    M, D, F, r = 96, 256, 512, 8
    mlp, x, res, dout, w = _block(q, M, D, F, r, 11)
    code = q.QLORA_ACT8_INT8
    ref, _ = _step(q, mlp, x, res, dout, w, code, *_buffers(q, mlp, M, D))
    torch.cuda.synchronize()
    # two steps at once on two streams, each with its own workspaces
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [_step(q, mlp, x, res, dout, w, code, *_buffers(q, mlp, M, D), stream=s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for outs, _ in runs:
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    # workspaces left to the calls, on another stream than the current one
    s = streams[0]
    Y, H = q.qlora_rmsnorm_forward(x, w, 1e-5, residual=res, stream=s)
    dX, dw = q.qlora_rmsnorm_backward(dout, H, w, 1e-5, stream=s.cuda_stream)
    s.synchronize()
    dX2, dw2 = q.qlora_rmsnorm_backward(dout, H, w, 1e-5)
    assert torch.equal(dX, dX2) and torch.equal(dw, dw2)
    # captured twice (two graphs over shared inputs), replayed in turn, the
    # second time on new inputs
    bufs = [_buffers(q, mlp, M, D) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(q, mlp, x, res, dout, w, code, *bufs[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs, kept = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kept.append(_step(q, mlp, x, res, dout, w, code, *b))
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for outs, _ in kept:
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    x.copy_(torch.randn_like(x))
    dout.mul_(0.5)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    new, _ = _step(q, mlp, x, res, dout, w, code, *_buffers(q, mlp, M, D))
    for outs, _ in kept:
        assert all(torch.equal(a, b) for a, b in zip(outs, new))
    assert not torch.equal(new[1], ref[1])


def test_host_threads_with_different_sizes(q):
    """Calls of one kernel whose rings differ in size, from several host
    threads at once: none is refused for the other's smaller ring."""
    fwd, bwd, keep = [], [], []
    for M, D in ((200, 8192), (200, 6400), (200, 7168), (200, 5120)):
        x, r, dy, dr, w = _inputs(M, D, D)
        Y, H = q.qlora_rmsnorm_forward(x, w, 1e-5, residual=r)
        dX, dw = q.qlora_rmsnorm_backward(dy, x, w, 1e-5, dres=dr)
        out = [torch.zeros_like(t) for t in (Y, H, dX, dw)]
        ws = torch.empty(q.qlora_rmsnorm_workspace_size(M, D), dtype=torch.uint8, device="cuda")
        keep.append((out, (Y, H, dX, dw), x, r, dy, dr, w, ws))
        p = lambda t: ctypes.c_void_p(t.data_ptr())
        fwd.append((q.lib().qlora_rmsnorm_forward,
                    (p(x), p(r), p(w), M, D, 1e-5, p(out[1]), p(out[0]), None, None)))
        bwd.append((q.lib().qlora_rmsnorm_backward,
                    (p(dy), p(x), p(dr), p(w), M, D, 1e-5, p(out[2]), p(out[3]), 0, p(ws), ws.numel(), None)))
    torch.cuda.synchronize()
    for calls in (fwd, bwd):
        assert at_once(calls, 5000) == [0] * len(calls)
    torch.cuda.synchronize()
    for out, ref, *_ in keep:
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
