"""Host-side checks of the microscaled 4-bit operators (no GPU needed): hand-worked quantisations
of the 64-bit definitions that the GPU tests use, sizes, and refusals before any device work."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import fp4_helpers as ref
from conftest import ROOT
from fp4_helpers import MX, NV

FAKE = 0x100000  # never dereferenced: every call below fails validation, or does nothing
INVALID = 1


@pytest.fixture(scope="module")
def L():
    from post_weight_quantization_guided_b200 import build, fp4
    build.build_library()
    return fp4.lib()


def test_header_binding_and_library_agree(L):
    text = open(os.path.join(ROOT, "include", "lnq_fp4.h")).read()
    declared = sorted(set(re.findall(r"LNQ_API\s+[\w\s\*]*?\b(lnq_\w+)\s*\(", text)))
    import post_weight_quantization_guided_b200 as pkg
    from post_weight_quantization_guided_b200 import fp4
    assert declared == sorted(fp4.EXPORTED)
    for name in declared:
        assert hasattr(L, name) and hasattr(pkg, name), name


def test_row_pitches(L):
    for d in (1, 16, 127, 128, 129, 4096, 11008):
        assert L.lnq_fp4_code_bytes(d) == ref.pitch(d)
        assert L.lnq_fp4_scale_bytes(d, MX) == ref.pitch(d, MX)
        assert L.lnq_fp4_scale_bytes(d, NV) == ref.pitch(d, NV)
    assert L.lnq_fp4_code_bytes(0) == 0 and L.lnq_fp4_code_bytes((1 << 24) + 1) == 0
    assert L.lnq_fp4_scale_bytes(128, 2) == 0 and L.lnq_fp4_scale_bytes(-1, MX) == 0


def test_reference_by_hand():
    # MX: the largest is 5 -> scale 2^(2-2) = 1; ties go to the even code, 7 would saturate
    x = np.array([[5.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.3, -2.6, 0.0]])
    codes, scales = ref.quantize(x, MX)
    assert scales[0, 0] == 127 and list(ref.values(codes, scales, 10, MX)[0]) == [
        4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, -0.5, -3.0, 0.0]
    # a largest of 7.5 keeps the scale 1 and saturates to 6
    codes, scales = ref.quantize(np.array([[7.5, -7.5]]), MX)
    assert scales[0, 0] == 127 and list(ref.values(codes, scales, 2, MX)[0]) == [6.0, -6.0]
    # NV: amax / 6 = 1.1 lies between 1.0 and 1.125, nearer to 1.125 (byte 0x39)
    codes, scales = ref.quantize(np.array([[6.6, 1.0]]), NV)
    assert scales[0, 0] == 0x39 and list(ref.values(codes, scales, 2, NV)[0]) == [6.75, 1.125]
    # amax / 6 = 1.0625, half way between 1.0 and 1.125: the even byte, 0x38
    assert ref.quantize(np.array([[6.375]]), NV)[1][0, 0] == 0x38
    assert ref.E4M3[126] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6
    # a block with an infinity or a NaN reads back as NaN, the next block does not
    x = np.ones((1, 33)); x[0, 3] = np.inf
    codes, scales = ref.quantize(x, MX)
    v = ref.values(codes, scales, 33, MX)
    assert np.isnan(v[0, :32]).all() and v[0, 32] == 1.0


def _quantize(L, **kw):
    a = dict(x=FAKE, xt=1, rows=4, d=64, ldx=64, fmt=NV, t=FAKE, codes=FAKE, scales=FAKE)
    a.update(kw)
    return L.lnq_fp4_quantize(*[a[k] for k in ("x", "xt", "rows", "d", "ldx", "fmt", "t", "codes",
                                               "scales")], None)


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(xt=3), dict(xt=-1), dict(rows=-1), dict(rows=1 << 31), dict(d=0),
    dict(d=(1 << 24) + 1, ldx=1 << 25), dict(ldx=63), dict(fmt=2), dict(fmt=MX), dict(codes=None),
    dict(scales=None), dict(codes=FAKE + 8), dict(scales=FAKE + 4), dict(t=FAKE + 2),
    dict(x=FAKE + 1), dict(x=FAKE + 2, xt=0), dict(fmt=MX, t=None, scales=FAKE + 2),
])
def test_quantize_rejects_bad_arguments(L, kw):
    assert _quantize(L, **kw) == INVALID


@pytest.mark.parametrize("kw", [
    dict(codes=None), dict(scales=None), dict(rows=-1), dict(d=0), dict(fmt=7), dict(fmt=MX),
    dict(y=None), dict(yt=3), dict(ldy=63), dict(y=FAKE + 1), dict(codes=FAKE + 4),
])
def test_dequantize_rejects_bad_arguments(L, kw):
    a = dict(codes=FAKE, scales=FAKE, rows=4, d=64, fmt=NV, t=FAKE, y=FAKE, yt=1, ldy=64)
    a.update(kw)
    assert L.lnq_fp4_dequantize(*a.values(), None) == INVALID


@pytest.mark.parametrize("kw", [dict(x=None), dict(t=None), dict(d=0), dict(ldx=63), dict(xt=9),
                                dict(rows=-1), dict(t=FAKE + 1)])
def test_tensor_scale_rejects_bad_arguments(L, kw):
    a = dict(x=FAKE, xt=1, rows=4, d=64, ldx=64, t=FAKE)
    a.update(kw)
    assert L.lnq_fp4_tensor_scale(*a.values(), None) == INVALID


_GEMV = dict(x=FAKE, xt=1, n=4, ldx=64, codes=FAKE, scales=FAKE, t=FAKE, d_out=8, d_in=64, fmt=NV,
             y=FAKE, yt=1, ldy=8)
_GEMM = dict(ac=FAKE, asc=FAKE, ta=FAKE, n=4, codes=FAKE, scales=FAKE, t=FAKE, d_out=8, d_in=64,
             fmt=NV, y=FAKE, yt=1, ldy=8)
_SHARED = [dict(codes=None), dict(scales=None), dict(n=-1), dict(n=1 << 31), dict(d_out=0),
           dict(d_in=0), dict(fmt=2), dict(fmt=MX), dict(y=None), dict(yt=3), dict(ldy=7),
           dict(codes=FAKE + 8), dict(scales=FAKE + 4), dict(y=FAKE + 1), dict(t=FAKE + 1),
           dict(d_out=1 << 31, ldy=1 << 32), dict(d_in=(1 << 24) + 1, ldx=1 << 25)]


@pytest.mark.parametrize("kw", _SHARED + [dict(x=None), dict(xt=3), dict(ldx=63), dict(x=FAKE + 1)])
def test_gemv_rejects_bad_arguments(L, kw):
    a = {**_GEMV, **{k: v for k, v in kw.items() if k in _GEMV}}
    assert L.lnq_fp4_gemv(*a.values(), None) == INVALID
    v = list(a.values())
    assert L.lnq_fp4_grouped_gemv(*v[:4], FAKE, 3, *v[4:], None) == INVALID


@pytest.mark.parametrize("kw", _SHARED + [dict(ac=None), dict(asc=None), dict(ac=FAKE + 8),
                                          dict(asc=FAKE + 4), dict(ta=FAKE + 1)])
def test_gemm_rejects_bad_arguments(L, kw):
    a = {**_GEMM, **{k: v for k, v in kw.items() if k in _GEMM}}
    assert L.lnq_fp4_gemm(*a.values(), None) == INVALID
    v = list(a.values())
    assert L.lnq_fp4_grouped_gemm(*v[:4], FAKE, 3, *v[4:], None) == INVALID


@pytest.mark.parametrize("offsets,experts", [(None, 3), (FAKE + 2, 3), (FAKE, 0), (FAKE, 1025),
                                             (FAKE, -1)])
def test_grouped_products_reject_bad_groups(L, offsets, experts):
    g, m = list(_GEMV.values()), list(_GEMM.values())
    assert L.lnq_fp4_grouped_gemv(*g[:4], offsets, experts, *g[4:], None) == INVALID
    assert L.lnq_fp4_grouped_gemm(*m[:4], offsets, experts, *m[4:], None) == INVALID


def test_no_rows_is_a_call_that_does_nothing(L):
    assert _quantize(L, rows=0, x=None, codes=None, scales=None) == 0
    a = {**_GEMV, "n": 0, "x": None, "y": None}
    assert L.lnq_fp4_gemv(*a.values(), None) == 0
    m = {**_GEMM, "n": 0, "ac": None, "asc": None, "y": None}
    assert L.lnq_fp4_gemm(*m.values(), None) == 0
    assert L.lnq_fp4_dequantize(None, None, 0, 64, MX, None, None, 0, 64, None) == 0


def test_binding_refuses_host_tensors(L):
    import post_weight_quantization_guided_b200 as pkg
    x = torch.zeros(4, 128)
    codes = torch.zeros(8, 64, dtype=torch.uint8)
    scales = torch.zeros(8, 8, dtype=torch.uint8)
    off = torch.zeros(2, dtype=torch.int32)
    calls = [lambda: pkg.lnq_fp4_tensor_scale(x),
             lambda: pkg.lnq_fp4_quantize(x, NV),
             lambda: pkg.lnq_fp4_dequantize(codes, scales, 128, NV),
             lambda: pkg.lnq_fp4_gemv(x, codes, scales, NV),
             lambda: pkg.lnq_fp4_grouped_gemv(x, off, codes[None], scales[None], NV),
             lambda: pkg.lnq_fp4_gemm(codes, scales, codes, scales, 128, NV),
             lambda: pkg.lnq_fp4_grouped_gemm(codes, scales, off, codes[None], scales[None], 128,
                                              NV)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
