"""GPU tests of the products of 1 to 16 tokens with a weight in any stored
format, against fp64 on the oracle's stored weight.

Bounds.  A code enters as an f16 value: within half a step, 2^-11 of itself
(FP4 and INT4 exactly).  An output adds, in fp32, at most 16 products inside
an MMA, 8 MMAs, 16 blocks or chunks per warp and slice of 4096 columns, 16
warps and the slices: fewer than 128 sequential additions of at most 2^-23
(the tensor core's accumulation may truncate), 2^-16 of the sum of
magnitudes; each product takes two more roundings of 2^-24 (the scale and its
decoding).  The LoRA term: sequential sums of at most K / 8 and r terms in
fp32.  Then one rounding to bf16."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from oracle import nf4_oracle as o

from _threads import at_once

pytestmark = pytest.mark.gpu

BOOKS = {"nf4": o.nf4_codebook()[0], "fp4": o.fp4_e2m1_codebook(), "int4": o.int4_codebook(),
         "dense": np.array([-1.0, -0.5, -0.2, -0.1, -0.05, -0.02, -0.01, 0.0, 0.01, 0.02, 0.05, 0.1, 0.2, 0.5, 0.75, 1.0],
                           np.float32),
         "grid8": np.linspace(-1.0, 1.0, 8).astype(np.float32),
         "big": np.array([-3e20, -1e20, 2e19, 5e20], np.float32)}
SCALES = ["fp32", "e4m3", "e5m2", "u8"]


@pytest.fixture(scope="module")
def q():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import bit_nf4_quantised_b200 as pkg
    pkg.lib()
    return pkg


def _fmt(q, book, block, scales):
    return q.Format(tuple(float(c) for c in BOOKS[book]), block, getattr(q, f"QLORA_SCALES_{scales.upper()}"))


def _store(N, K, book, block, scales, seed):
    """(device buffers, the weight in fp64) of a seeded weight, by the oracle."""
    rng = np.random.default_rng(seed)
    W = rng.standard_normal((N, K), dtype=np.float32) * np.float32(0.02)
    W *= np.exp2(rng.integers(-6, 4, (N, 1))).astype(np.float32)          # rows of different sizes
    if N > 3:
        W[2] = 0.0
    if book == "big":
        W /= np.float32(5e20)
    packed, sc, meta = o.quantize_fmt(W, BOOKS[book], block, scales)
    idx = o.unpack_nibbles(packed, packed.size * 2)
    c = np.asarray(sc, np.float64) if scales == "fp32" else o.dequantize_scales(sc, meta, fmt=scales).astype(np.float64)
    w = (BOOKS[book].astype(np.float64)[idx].reshape(-1, block) * c[:, None]).reshape(-1)[: N * K].reshape(N, K)
    dev = [torch.from_numpy(np.ascontiguousarray(t)).cuda() if t is not None else None
           for t in (packed, sc, None if scales == "fp32" else meta)]
    return dev, w


def _values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _check(q, M, N, K, book, block, scales, r=0, x=None, seed=0):
    dev, w = _store(N, K, book, block, scales, seed + N + K)
    g = torch.Generator().manual_seed(seed + M)
    n = lambda *s: torch.randn(*s, generator=g)
    if x is None:
        x = n(M, K)
        x[:, ::29] *= 15.0
        x = (x * torch.exp2(torch.randint(-30, 30, (M, 1), generator=g).float())).bfloat16()
    A = (n(r, K) / K ** 0.5).bfloat16() if r else None
    B = (0.05 * n(N, r)).bfloat16() if r else None
    c = lambda t: None if t is None else t.cuda()
    Y = q.qlora_linear_fmt_forward(x.cuda(), *dev, N, _fmt(q, book, block, scales), A=c(A), B=c(B), scale=2.0)
    X = x.double().numpy()
    exact, size = X @ w.T, np.abs(X) @ np.abs(w).T
    err = ((2.0 ** -11 if book not in ("fp4", "int4") else 0.0) + 2.0 ** -16) * size
    if r:
        a, b = A.double().numpy(), B.double().numpy()
        exact = exact + 2.0 * (X @ a.T) @ b.T
        err = err + (K / 8 + r + 16) * 2.0 ** -24 * 2.0 * (np.abs(X) @ np.abs(a).T) @ np.abs(b).T
    got = _values(Y.view(torch.int16).cpu().numpy().view(np.uint16))
    lo, hi = _values(o.bf16_rne_f64(exact - err)), _values(o.bf16_rne_f64(exact + err))
    ok = (got >= lo) & (got <= hi)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside"
    return Y


@pytest.mark.parametrize("scales", SCALES)
@pytest.mark.parametrize("block", [16, 32, 64, 128, 256, 4096])
@pytest.mark.parametrize("M", [1, 3, 8, 16])
def test_every_layout(q, M, block, scales):
    """Blocks inside, across and longer than a row's chunks, and rows of an
    odd number of 64-wide runs (K = 832: blocks of 128 and more begin in
    another half-chunk on every other row)."""
    book = list(BOOKS)[(M + block) % 5]
    _check(q, M, 203, 832, book, block, scales, r=8 if M == 3 else 0)


@pytest.mark.parametrize("M", range(1, 17))
def test_every_token_count(q, M):
    _check(q, M, 130, 1088, "nf4", (16, 32, 64, 512)[M % 4], SCALES[M % 3], r=(0, 16, 128)[M % 3])


@pytest.mark.parametrize("M,N,K,block", [(1, 1, 64, 64), (2, 5, 64, 16), (1, 4096, 64, 32), (4, 33, 128, 128), (1, 17, 192, 4096),
                                         (16, 9, 320, 32), (1, 300, 512, 64), (5, 1000, 256, 64), (1, 64, 28672, 64),
                                         (16, 40, 28672, 128), (16, 24, 11008, 16), (7, 600, 4096, 32), (2, 2049, 4160, 256)])
@pytest.mark.parametrize("r", [0, 24])
def test_shapes(q, M, N, K, block, r):
    _check(q, M, N, K, "nf4", block, SCALES[(M + N) % 4], r=r)


@pytest.mark.parametrize("M,N,K,block,scales,r", [(1, 200001, 64, 64, "e4m3", 0), (2, 60000, 512, 16, "fp32", 8), (16, 30000, 320, 32, "u8", 0),
                                                  (16, 2500, 4096, 64, "e5m2", 128), (13, 9001, 1024, 128, "fp32", 64),
                                                  (9, 700, 16384, 16, "fp32", 16), (8, 148 * 33, 2048, 256, "e4m3", 0)])
def test_many_rows(q, M, N, K, block, scales, r):
    """Many rows a CTA: several spans between barriers, ragged last units,
    slices with an adapter."""
    _check(q, M, N, K, "nf4", block, scales, r=r)


@pytest.mark.parametrize("book", list(BOOKS))
def test_codebooks(q, book):
    _check(q, 2, 300, 640, book, 64, "fp32")


def test_decode_shapes(q):
    """The decode weights' shapes, from a device-side store of the library."""
    for (M, N, K, block, scales) in ((1, 28672, 8192, 64, "e4m3"), (16, 8192, 28672, 32, "fp32")):
        f = _fmt(q, "nf4", block, scales)
        W = torch.randn(N, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.015
        packed, sc, meta = q.qlora_quantize_fmt(W, f)
        codes = torch.tensor(BOOKS["nf4"], device="cuda")
        x = torch.randn(M, K, device="cuda").bfloat16()
        Y = q.qlora_linear_fmt_forward(x, packed, sc, meta, N, f)
        rows = torch.randint(0, N, (200,), device="cuda").unique()
        rows = torch.cat([rows, torch.tensor([0, N - 1], device="cuda")])
        # these rows in fp64
        by = packed.reshape(N, K // 2)[rows].long()
        idx = torch.stack((by & 15, by >> 4), -1).reshape(len(rows), K)
        blk = (rows[:, None] * K + torch.arange(K, device="cuda")) // block
        if scales == "fp32":
            c = sc[blk].double()
        else:
            c = (sc.view(torch.float8_e4m3fn)[blk].float() * meta[blk // 256]).double()
        w = codes[idx].double() * c
        exact, size = x.double() @ w.t(), x.double().abs() @ w.abs().t()
        err = (2.0 ** -11 + 2.0 ** -16) * size + 2.0 ** -8 * exact.abs()
        assert ((Y[:, rows].double() - exact).abs() <= err).all()


def test_one_hot_rows_return_the_weight(q):
    """A single 1 in a token: the output is one code times its scale."""
    for book, block, scales in (("int4", 32, "fp32"), ("nf4", 64, "e4m3"), ("fp4", 16, "u8"), ("nf4", 256, "e5m2")):
        M, N, K = 16, 100, 448
        cols = np.random.default_rng(block).choice(K, M, replace=False)
        x = torch.zeros(M, K, dtype=torch.bfloat16)
        x[np.arange(M), cols] = 1.0
        _check(q, M, N, K, book, block, scales, x=x)


def test_extreme_activations(q):
    K = 512
    x = torch.zeros(6, K, dtype=torch.bfloat16)
    x[1] = torch.randn(K).bfloat16() * 2.0 ** -125                 # near the smallest normals
    x[2] = torch.randn(K).bfloat16() * 2.0 ** 110
    x[3, ::2], x[3, 1::2] = 2.0 ** 60, 2.0 ** 30                   # 2^30 apart
    x[4, 7] = 3.0e38
    x[5] = torch.tensor([2.0 ** -133] * K)                         # subnormal
    dev, w = _store(64, K, "int4", 64, "fp32", 5)
    Y = q.qlora_linear_fmt_forward(x.cuda(), *dev, 64, _fmt(q, "int4", 64, "fp32")).double().cpu().numpy()
    X = x.double().numpy()
    exact, size = X @ w.T, np.abs(X) @ np.abs(w).T
    top = np.abs(X).max(1, keepdims=True)
    # f16 activations: off by 2^-40 of the token's largest, per weight; fp32
    # outputs below 2^-126 lose their last bits
    err = 2.0 ** -16 * size + 2.0 ** -40 * top * np.abs(w).sum(1) + 2.0 ** -130
    lo, hi = _values(o.bf16_rne_f64(exact - err)), _values(o.bf16_rne_f64(exact + err))
    assert ((Y >= lo) & (Y <= hi)).all()
    assert not Y[0].any()


def test_nonfinite_activations_stay_in_their_token(q):
    K, N = 320, 70
    dev, w = _store(N, K, "int4", 64, "fp32", 6)
    f = _fmt(q, "int4", 64, "fp32")
    x = torch.randn(4, K).bfloat16()
    ref = q.qlora_linear_fmt_forward(x.cuda(), *dev, N, f)
    y = x.clone()
    y[1, 5], y[3, 300] = float("nan"), float("inf")
    got = q.qlora_linear_fmt_forward(y.cuda(), *dev, N, f)
    assert torch.equal(got[[0, 2]], ref[[0, 2]]) and got[1].isnan().all() and not got[3].isfinite().any()
    W = torch.from_numpy(w[:, 300])
    pos, neg = (W > 0).cuda(), (W < 0).cuda()
    assert (got[3][pos] == float("inf")).all() and (got[3][neg] == float("-inf")).all()


def test_rows_behind_the_output_and_given_buffers(q):
    N, K = 37, 256
    dev, _ = _store(N, K, "nf4", 64, "e4m3", 8)
    f = _fmt(q, "nf4", 64, "e4m3")
    x = torch.randn(3, K).bfloat16().cuda()
    A, B = torch.randn(8, K).bfloat16().cuda(), torch.randn(N, 8).bfloat16().cuda()
    buf = torch.full((5, N), 9.0, dtype=torch.bfloat16, device="cuda")
    n = q.qlora_linear_fmt_workspace_size(3, N, K, 8, f)
    ws = torch.full((n + 64,), 77, dtype=torch.uint8, device="cuda")
    Y = q.qlora_linear_fmt_forward(x, *dev, N, f, A=A, B=B, scale=0.5, Y=buf[:3], ws=ws[:n])
    assert torch.equal(Y, q.qlora_linear_fmt_forward(x, *dev, N, f, A=A, B=B, scale=0.5))
    assert (buf[3:] == 9).all() and (ws[n:] == 77).all()
    assert q.qlora_linear_fmt_forward(x[:0], *dev, N, f).shape == (0, N)
    for bad in (lambda: q.qlora_linear_fmt_forward(x, *dev, N + 1, f),
                lambda: q.qlora_linear_fmt_forward(x, *dev, N, f, A=A),
                lambda: q.qlora_linear_fmt_forward(x, *dev, N, f, A=A, B=B[:, :4].contiguous()),
                lambda: q.qlora_linear_fmt_forward(x.t().contiguous().t(), *dev, N, f),
                lambda: q.qlora_linear_fmt_forward(x, *dev, N, f, Y=buf)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: q.qlora_linear_fmt_forward(torch.zeros(17, K).bfloat16().cuda(), *dev, N, f),
                lambda: q.qlora_linear_fmt_forward(x, *dev, N, f, A=A, B=B, ws=ws[:16])):
        with pytest.raises(q.QloraError):
            bad()


def test_formats_that_are_refused(q):
    N, K = 37, 256
    dev, _ = _store(N, K, "nf4", 64, "e4m3", 8)
    good = _fmt(q, "nf4", 64, "e4m3")
    x = torch.randn(3, K).bfloat16().cuda()
    for codes, block, scales in ((good.codes, 0, good.scales), (good.codes, 48, good.scales), (good.codes, 8192, good.scales),
                                 (good.codes[::-1], 64, good.scales), ((0.0, float("nan")), 64, good.scales),
                                 ((0.0,), 64, good.scales), (good.codes, 64, 7), (good.codes, -64, good.scales)):
        with pytest.raises(q.QloraError):
            q.qlora_linear_fmt_forward(x, *dev, N, q.Format(codes, block, scales))
    assert q.qlora_linear_fmt_forward(x, *dev, N, q.Format(list(good.codes), 64, good.scales)).isfinite().all()


def test_same_bytes_streams_and_captured(q):
    """Repeated, concurrent, captured and replayed calls give the same bytes;
    two captured graphs keep their own workspaces."""
    N, K, r = 2000, 4096, 16
    f = _fmt(q, "nf4", 64, "e4m3")
    dev, _ = _store(N, K, "nf4", 64, "e4m3", 9)
    x = torch.randn(16, K).bfloat16().cuda()
    A, B = (torch.randn(r, K) / 64).bfloat16().cuda(), torch.randn(N, r).bfloat16().cuda()
    call = lambda **k: q.qlora_linear_fmt_forward(x, *dev, N, f, A=A, B=B, scale=2.0, **k)
    ref = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    runs = [call(stream=s) for s in streams * 4] + [call(stream=streams[0].cuda_stream)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y in runs)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    x.mul_(-1)
    for g in graphs * 3:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, -ref) for y in outs)


def test_decoding_through_the_block(q):
    """One token through the block on format variants: norm, gate and up
    products with adapters, SwiGLU, down product, each against the formula on
    the library's own previous output."""
    D, F, r = 512, 1088, 8
    fg, fd = _fmt(q, "nf4", 64, "e4m3"), _fmt(q, "int4", 128, "fp32")
    (g, wg), (u, wu), (d, wd) = _store(F, D, "nf4", 64, "e4m3", 1), _store(F, D, "nf4", 64, "e4m3", 2), _store(D, F, "int4", 128, "fp32", 3)
    gen = torch.Generator().manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=gen)
    A, B = (n(r, D) / D ** 0.5).bfloat16(), (0.05 * n(F, r)).bfloat16()
    for M in (1, 4):
        x, res = n(M, D).bfloat16().cuda(), n(M, D).bfloat16().cuda()
        y, h = q.qlora_rmsnorm_forward(x, torch.ones(D, device="cuda"), 1e-5, residual=res)
        G = q.qlora_linear_fmt_forward(y, *g, F, fg, A=A.cuda(), B=B.cuda(), scale=2.0)
        U = q.qlora_linear_fmt_forward(y, *u, F, fg)
        H, _, _ = q.qlora_swiglu_forward_act8(G, U)
        out = q.qlora_linear_fmt_forward(H, *d, D, fd)
        f = lambda t: t.double().cpu().numpy()
        rel = lambda a, b: np.linalg.norm(f(a) - b) / np.linalg.norm(b)
        step = 2.0 ** -8 + 2.0 ** -11                   # a rounding of bf16, and of the codes
        assert rel(y, o.rmsnorm(f(h), np.ones(D), 1e-5)) < step
        a, b = A.double().numpy(), B.double().numpy()
        assert rel(G, f(y) @ wg.T + 2 * (f(y) @ a.T) @ b.T) < step
        assert rel(U, f(y) @ wu.T) < step
        assert rel(H, o.silu(f(G)) * f(U)) < step
        assert rel(out, f(H) @ wd.T) < step


@pytest.mark.parametrize("M,block,scales", [(1, 64, "e4m3"), (4, 16, "fp32"), (12, 128, "fp32")])
def test_host_threads_with_different_sizes(q, M, block, scales):
    """Calls of one kernel whose plans of shared memory differ, from several
    host threads at once: none is refused for the other's smaller plan."""
    f = _fmt(q, "nf4", block, scales)
    st, calls, outs, refs = f.c_struct(), [], [], []
    for i, (N, K) in enumerate([(64, 256), (64, 28672), (64, 512), (300, 8192)]):
        dev, _ = _store(N, K, "nf4", block, scales, i)
        x = torch.randn(M, K).bfloat16().cuda()
        refs.append(q.qlora_linear_fmt_forward(x, *dev, N, f))
        outs.append((torch.empty_like(refs[-1]), x, dev))
        n = q.qlora_linear_fmt_workspace_size(M, N, K, 0, f)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        outs[-1] += (ws,)
        at = [None if t is None else ctypes.c_void_p(t.data_ptr()) for t in (x, *dev, outs[-1][0], ws)]
        calls.append((q.lib().qlora_linear_fmt_forward,
                      (at[0], M, *at[1:4], N, K, ctypes.byref(st), None, None, 0, 0.0, at[4], at[5], n, None)))
    torch.cuda.synchronize()
    assert at_once(calls, 5000) == [0] * len(calls)
    torch.cuda.synchronize()
    assert all(torch.equal(a[0], b) for a, b in zip(outs, refs))


@pytest.mark.parametrize("size,token", [(68, 80), (68, -80), (68, 100), (-80, -80), (-80, 80), (-80, -20), (-86, 100)])
def test_codebooks_and_tokens_of_any_size(q, size, token):
    """Codes of about 2^size, block scales that make weights of about 2^-6 of
    them, tokens of about 2^token: the factors taken out of codes and
    activations leave fp32's range together, the products do not.  The bounds
    are _check's, which no scale changes; the products stay above 2^-126."""
    N, K = 70, 448
    codes = (np.array([-3.0, -1.0, -0.4, 0.0, 0.2, 1.0, 5.0], np.float64) * 2.0 ** size).astype(np.float32)
    g = np.random.default_rng(abs(size) + abs(token))
    idx = g.integers(0, len(codes), N * K).astype(np.uint8)
    idx[2 * K: 3 * K] = 3                                     # a row of zeros
    c = np.exp2(g.uniform(-8, -4, N * K // 64) - size).astype(np.float32)
    w = (codes.astype(np.float64)[idx].reshape(-1, 64) * c.astype(np.float64)[:, None]).reshape(N, K)
    x = torch.from_numpy(g.standard_normal((3, K)) * 2.0 ** token).bfloat16()
    x[1] = 0.0
    packed = torch.from_numpy(idx[::2] | idx[1::2] << 4).cuda()
    f = q.Format(tuple(float(v) for v in codes), 64, q.QLORA_SCALES_FP32)
    Y = q.qlora_linear_fmt_forward(x.cuda(), packed, torch.from_numpy(c).cuda(), None, N, f).double().cpu().numpy()
    X = x.double().numpy()
    exact, err = X @ w.T, (2.0 ** -11 + 2.0 ** -16) * (np.abs(X) @ np.abs(w).T)
    lo, hi = _values(o.bf16_rne_f64(exact - err)), _values(o.bf16_rne_f64(exact + err))
    assert ((Y >= lo) & (Y <= hi)).all()
    assert not Y[1].any() and not Y[:, 2].any()


def test_activations_far_below_their_tokens_largest(q):
    """A value is exact down to 2^-28 of its token's largest; below that its
    f16 copy is off by half a step of the subnormals, 2^-25, where the largest
    is at least 2^14: 2^-39 of the largest.  A token below 2^-112 meets its
    factor's limit, 2^126, and is exact: bf16 values are multiples of 2^-133,
    so there of 2^-7, with 8 bits.  The largest value meets a weight of zero,
    so that it does not hide the others.  Outputs below 2^-126 are rounded to
    fp32's last step, 2^-149, on the way."""
    K, N = 64, 40
    dev, w = _store(N, K, "int4", 64, "fp32", 12)
    idx = o.unpack_nibbles(dev[0].cpu().numpy(), N * K).reshape(N, K).copy()
    idx[:, 0] = list(BOOKS["int4"]).index(0.0)
    w = w.copy()
    w[:, 0] = 0.0
    packed = torch.from_numpy(idx.reshape(-1)[::2] | idx.reshape(-1)[1::2] << 4).cuda()
    steps = 1 + torch.arange(K) / 128
    x = torch.stack([steps * 2.0 ** -28, steps * 2.0 ** -33,
                     torch.arange(1, K + 1) * 2.0 ** -120 / 100,                     # 2^-120.6 and below
                     torch.arange(K, 0, -1) * 2.0 ** -133]).bfloat16()               # subnormals
    x[:2, 0] = 1.0
    Y = q.qlora_linear_fmt_forward(x.cuda(), packed, dev[1], None, N, _fmt(q, "int4", 64, "fp32")).double().cpu().numpy()
    X = x.double().numpy()
    exact, err = X @ w.T, 2.0 ** -16 * (np.abs(X) @ np.abs(w).T) + 2.0 ** -149
    err[1] += 2.0 ** -39 * np.abs(w).sum(1)
    lo, hi = _values(o.bf16_rne_f64(exact - err)), _values(o.bf16_rne_f64(exact + err))
    assert ((Y >= lo) & (Y <= hi)).all()


def test_buffers_one_behind_the_other(q):
    """Buffers that touch but do not overlap are taken; a Y on X is refused."""
    M, N, K, r = 2, 64, 256, 8
    dev, _ = _store(N, K, "nf4", 64, "e4m3", 8)
    f = _fmt(q, "nf4", 64, "e4m3")
    x, A, B = (torch.randn(*s).bfloat16().cuda() for s in ((M, K), (r, K), (N, r)))
    ref = q.qlora_linear_fmt_forward(x, *dev, N, f, A=A, B=B, scale=2.0)
    one = torch.empty(M * K + M * N + r * K + N * r, dtype=torch.bfloat16, device="cuda")
    X1, Y1, A1, B1 = (t.view(s) for t, s in zip(one.split([M * K, M * N, r * K, N * r]), ((M, K), (M, N), (r, K), (N, r))))
    for a, b in ((X1, x), (A1, A), (B1, B)):
        a.copy_(b)
    assert torch.equal(q.qlora_linear_fmt_forward(X1, *dev, N, f, A=A1, B=B1, scale=2.0, Y=Y1), ref)
    assert torch.equal(X1, x) and torch.equal(A1, A) and torch.equal(B1, B)
    with pytest.raises(q.QloraError):
        q.qlora_linear_fmt_forward(X1, *dev, N, f, A=A1, B=B1, scale=2.0, Y=one[: M * N].view(M, N))
    assert torch.equal(X1, x)
