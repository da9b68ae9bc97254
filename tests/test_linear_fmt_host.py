"""CPU tests of the products with a weight in any stored format: sizes and
refusals (fake pointers that no kernel ever sees)."""
from __future__ import annotations

import ctypes
import pathlib
import re

import pytest
import torch

from oracle import nf4_oracle as o

FAKE = 0x40000


@pytest.fixture(scope="module")
def q():
    import bit_nf4_quantised_b200 as pkg
    pkg.lib()
    return pkg


def _fmt(q, block=64, scales=None, codes=None):
    return q.Format(tuple(float(c) for c in (o.nf4_codebook()[0] if codes is None else codes)), block,
                    q.QLORA_SCALES_E4M3 if scales is None else scales)


def test_workspace_sizes(q):
    f = _fmt(q)
    assert q.qlora_linear_fmt_workspace_size(0, 64, 64, 0, f) == 0
    assert q.qlora_linear_fmt_workspace_size(1, 4096, 4096, 0, f) == 0          # one kernel writes Y
    assert q.qlora_linear_fmt_workspace_size(1, 4096, 4096, 16, f) >= 4 * 16
    # activations that do not fit beside each other take slices and partials
    assert q.qlora_linear_fmt_workspace_size(16, 8192, 28672, 0, f) >= 2 * 4 * 16 * 8192
    L, E = q.lib(), q._lib
    n = ctypes.c_size_t()
    size = lambda M=1, N=64, K=64, r=0, f=f: L.qlora_linear_fmt_workspace_size(M, N, K, r, f.c_struct(), ctypes.byref(n))
    assert size() == E.QLORA_OK
    for bad in ({"M": 17}, {"K": 96}, {"K": 0}, {"N": 0}, {"r": 4}, {"r": 136}, {"N": 1 << 31}, {"K": 1 << 31},
                {"f": _fmt(q, block=8)}, {"f": _fmt(q, codes=[0.5])}, {"f": _fmt(q, scales=9)}):
        assert size(**bad) == E.QLORA_ERR_UNSUPPORTED, bad
    for bad in ({"M": -1}, {"N": -1}, {"K": -64}, {"r": -8}):
        assert size(**bad) in (E.QLORA_ERR_SHAPE, E.QLORA_ERR_UNSUPPORTED), bad
    assert L.qlora_linear_fmt_workspace_size(1, 64, 64, 0, f.c_struct(), None) == E.QLORA_ERR_NULL
    assert L.qlora_linear_fmt_workspace_size(1, 64, 64, 0, None, ctypes.byref(n)) == E.QLORA_ERR_NULL


def test_argument_errors(q):
    L, E = q.lib(), q._lib

    def call(X=FAKE, M=1, packed=FAKE, scales=FAKE, meta=FAKE, N=64, K=64, f=_fmt(q), A=None, B=None, r=0, Y=FAKE,
             ws=None, n=0):
        return L.qlora_linear_fmt_forward(X, M, packed, scales, meta, N, K, f.c_struct(), A, B, r, 2.0, Y, ws, n, None)
    for k in ("X", "packed", "scales", "meta", "Y"):
        assert call(**{k: None}) == E.QLORA_ERR_NULL
    for k in ("X", "packed", "Y"):
        assert call(**{k: FAKE + 8}) == E.QLORA_ERR_ALIGN
    for k in ("scales", "meta"):
        assert call(**{k: FAKE + 2}) == E.QLORA_ERR_ALIGN
    f32 = _fmt(q, 16, q.QLORA_SCALES_FP32)
    assert call(f=f32, scales=FAKE + 4, meta=None) == E.QLORA_ERR_ALIGN
    assert call(r=8, A=FAKE) == E.QLORA_ERR_NULL
    assert call(r=8, A=FAKE, B=FAKE + 8, ws=FAKE, n=1 << 20) == E.QLORA_ERR_ALIGN
    assert call(r=8, A=FAKE, B=FAKE) == E.QLORA_ERR_WORKSPACE
    assert call(r=8, A=FAKE, B=FAKE, ws=FAKE, n=16) == E.QLORA_ERR_WORKSPACE
    assert call(r=8, A=FAKE, B=FAKE, ws=FAKE + 16, n=1 << 20) == E.QLORA_ERR_ALIGN
    assert call(M=17) == E.QLORA_ERR_UNSUPPORTED
    assert call(K=32) == E.QLORA_ERR_UNSUPPORTED
    assert call(M=-1) == E.QLORA_ERR_SHAPE
    assert call(M=0, X=None, Y=None, packed=None, scales=None) == E.QLORA_OK


def test_python_refuses_before_the_library(q):
    x = torch.zeros(1, 64, dtype=torch.bfloat16)
    p, s, m = torch.zeros(64 * 32, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8), torch.zeros(1)
    with pytest.raises(ValueError):
        q.qlora_linear_fmt_forward(x, p, s, m, 64, _fmt(q))


def test_table_lookups_stay_behind_their_barrier():
    """An asm that reads memory without being volatile may be moved by the
    compiler to wherever its operands exist.  The code table's lookup is the
    only one here; its address is made of packed words, and those that are
    loaded before the table is complete pass through a volatile asm that
    clobbers memory, behind the barrier that completes it."""
    src = (pathlib.Path(__file__).parents[1] / "bit_nf4_quantised_b200" / "csrc" / "gemv_fmt.cu").read_text()
    free = [a for a in re.findall(r"\basm\s*\(.*?\);", src, re.S) if re.search(r"\bld\.", a)]
    assert len(free) == 1 and "kLut" in free[0]
    assert re.search(r"void ldg_weights\([^{]*\{\s*asm volatile\(", src)        # later words: volatile, so after it
    tie = re.search(r"void after_barrier\(uint4& v\) \{\s*asm volatile\((.*?)\);", src, re.S)
    assert tie and all(f'"+r"(v.{c})' in tie.group(1) for c in "xyzw") and '"memory"' in tie.group(1)
    filled = src.index("// code table: byte e of lane l")
    barrier = src.index("__syncthreads();", src.index("cp_async_wait<0>();", filled))
    tied = src.index("for (int i = 0; i < 8; ++i) after_barrier(buf[i >> 2][i & 3]);")
    assert filled < barrier < tied < src.index("auto code_pair") and "uint4 buf[2][4];" in src


@pytest.mark.parametrize("scales", ["E4M3", "FP32"])
def test_outputs_that_overlap_are_refused(q, scales):
    """Y and the workspace may lie on no input and not on each other: every
    CTA reads all of X, A and the constants while others already store."""
    L, E = q.lib(), q._lib
    f = _fmt(q, 16, getattr(q, f"QLORA_SCALES_{scales}"))
    M, N, K, r = 3, 40, 128, 8
    packed, sc, meta = q.qlora_format_sizes(N * K, f)
    need = q.qlora_linear_fmt_workspace_size(M, N, K, r, f)
    sizes = {"X": 2 * M * K, "packed": packed, "scales": sc, "meta": meta, "A": 2 * r * K, "B": 2 * N * r, "Y": 2 * M * N, "ws": need}
    at = {k: FAKE + 0x10000 * i for i, k in enumerate(sizes)}
    if not meta:
        sizes.pop("meta")
        at["meta"] = None

    def call(p):
        return L.qlora_linear_fmt_forward(p["X"], M, p["packed"], p["scales"], p["meta"], N, K, f.c_struct(), p["A"], p["B"], r, 2.0,
                                          p["Y"], p["ws"], need, None)
    for out in ("Y", "ws"):
        step = 16 if out == "Y" else 256
        for other in sizes:
            if other == out:
                continue
            first = at[other] - (sizes[out] - 1) // step * step                # the last place that still touches it
            last = at[other] + (sizes[other] - 1) // step * step
            for place in (at[other], first, last):
                assert call({**at, out: place}) == E.QLORA_ERR_UNSUPPORTED, (out, other, place - at[other])
