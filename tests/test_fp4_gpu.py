"""The microscaled 4-bit operators against their definitions in 64 bits (needs a B200).

Quantised bytes are compared for equality. Products are compared in two ways. With operands whose
every partial sum is a multiple of 1/8 below 2^20 (24 bits hold it), 32-bit sums are exact in any
order, and the results have to be equal. With random operands a sum of K exact products may be off
by one part in 2^23 of the sum of magnitudes S at each of its K additions (an addition that
truncates), and the matrix scales and the rounding to the output's type add their half steps:
    |y - y64| <= (K + 4) 2^-23 S + eps / 2 |y64|.
"""
import numpy as np
import pytest
import torch

import fp4_helpers as ref
from fp4_helpers import MX, NV

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def lnq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_weight_quantization_guided_b200 import build
    build.build_library()
    import post_weight_quantization_guided_b200 as pkg
    yield pkg
    assert pkg.lnq_fp4_check() == 0  # no bounded wait gave up in any test


def _rng(*key):
    return np.random.default_rng([abs(hash(str(k))) % (1 << 32) if isinstance(k, str) else int(k)
                                  for k in key])


def dev(a, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype) if dtype is not None \
        else torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


def strided(x, extra=0, shift=0):
    """A copy of the matrix x whose rows are `extra` elements further apart, `shift` elements into
    its storage."""
    rows, d = x.shape
    buf = torch.full((rows * (d + extra) + shift + 8,), float("nan"), dtype=x.dtype, device="cuda")
    v = buf[shift:shift + rows * (d + extra)].view(rows, d + extra)[:, :d]
    v.copy_(x)
    return v


def f64(t):
    return t.double().cpu().numpy()


def check_quantized(lnq, x, fmt, t=None):
    ts = None if t is None else torch.tensor([t], dtype=torch.float32, device="cuda")
    rows, d = x.shape
    codes = torch.full((rows, ref.pitch(d)), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, ref.pitch(d, fmt)), 0xCD, dtype=torch.uint8, device="cuda")
    lnq.lnq_fp4_quantize(x, fmt, tensor_scale=ts, codes=codes, scales=scales)
    want_c, want_s = ref.quantize(f64(x), fmt, 1.0 if t is None else float(np.float32(t)))
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    assert ref.codes_equal(codes.cpu().numpy(), want_c)


# ------------------------------------------------------------------------------- quantisation

@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 15), (2, 16), (5, 31), (1, 32), (4, 33), (3, 127),
                                    (7, 128), (2, 130), (3, 257), (130, 544), (2, 16389)])
def test_quantize_shapes(lnq, fmt, dtype, rows, d):
    x = dev(_rng(rows, d).standard_normal((rows, d)) * 3, dtype)
    check_quantized(lnq, x, fmt)
    if fmt == NV:
        check_quantized(lnq, x, fmt, 0.0123)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("extra,shift", [(0, 1), (3, 0), (8, 0), (5, 3), (8, 8)])
def test_quantize_strided_rows(lnq, fmt, dtype, extra, shift):
    x = dev(_rng(1).standard_normal((9, 200)), dtype)
    check_quantized(lnq, strided(x, extra, shift), fmt)


@pytest.mark.parametrize("fmt,t", [(MX, None)] + [(NV, v) for v in (
    None, 1.0, 0.25, 1 / 3, 0.00171, 1234.5, 2.0 ** -99, 2.0 ** -101, 2.0 ** 114, 2.0 ** 116,
    1e-38, 1e-45, 3.4e38)])
def test_quantize_at_the_borders(lnq, fmt, t):
    """Elements on, and one 32-bit step to either side of, every border of two codes, for block
    scales on, and next to, the borders of two scales."""
    step = 1.0 if t is None else float(np.float32(t))
    rows = []
    borders = (ref.LEVELS[1:] + ref.LEVELS[:-1]) / 2
    with np.errstate(over="ignore", under="ignore"):
        for s in (2.0 ** -9, 2.0 ** -7 * 1.25, 0.6875, 1.0, 1.125, 1.75, 52.0, 448.0):
            for top in (6.0, 6.375, 6.4, 5.5):
                base = np.float32([top * s * step] + [b * s * step for b in borders])
                r = np.concatenate([base, np.nextafter(base[1:], np.float32(0)), -base[1:2]])
                up = np.concatenate([base, np.nextafter(base[1:], np.float32(np.inf)), -base[1:2]])
                for a in (r, up):
                    a = np.where(np.isfinite(a), a, np.float32(0))
                    rows.append(np.concatenate([a, a[:1] * 0])[:16])
    x = np.concatenate([np.array(rows)] * 2, 1) if fmt == MX else np.array(rows)
    check_quantized(lnq, dev(x.astype(np.float32)), fmt, t)
    # the same numbers in 16 bits, where ties are frequent
    for dtype in (torch.bfloat16, torch.float16):
        h = dev(x.astype(np.float32)).to(dtype)
        check_quantized(lnq, torch.where(h.isfinite(), h, 0), fmt, t)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quantize_ties_are_dense(lnq, fmt):
    """Small multiples of 1/8: every fourth quotient or so is a tie."""
    x = _rng(5).integers(-48, 49, (64, 512)) / 8.0
    check_quantized(lnq, dev(x, torch.bfloat16), fmt)
    if fmt == NV:
        check_quantized(lnq, dev(x, torch.float32), fmt, 0.5)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_quantize_special_values(lnq, fmt):
    x = _rng(2).standard_normal((12, 96)).astype(np.float32)
    x[0] = 0
    x[1, 40:] = -0.0
    x[2, 5] = np.nan
    x[3, 37] = np.inf
    x[4, 95] = -np.inf
    x[5] *= 1e-40            # subnormal
    x[6] *= 3e38 / 5
    x[7, :32] = 1e-45
    x[8, 3] = np.float32(3.4028235e38)
    x[9] *= 1e30
    x[10] *= 1e-30
    x = np.where(np.isinf(x) & (np.arange(12)[:, None] > 4), 3e38, x)
    for t in ([None] if fmt == MX else [None, 1e-3, 1e30, 1e-36]):
        check_quantized(lnq, dev(x), fmt, t)


@pytest.mark.parametrize("t", [0.0, -1.0, float("nan"), float("inf"), -float("inf")])
def test_quantize_bad_matrix_scale_gives_nan(lnq, t):
    x = torch.randn(3, 40, device="cuda")
    check_quantized(lnq, x, NV, t)
    ts = torch.tensor([t], device="cuda")
    codes, scales = lnq.lnq_fp4_quantize(x, NV, tensor_scale=ts)
    assert lnq.lnq_fp4_dequantize(codes, scales, 40, NV).isnan().all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t", [None, 0.37])
def test_dequantize_every_code_and_scale(lnq, fmt, dtype, t):
    if fmt == MX and t is not None:
        t = None
    B = ref.BLOCK[fmt]
    n = 256 if fmt == MX else 128
    d = B * 2 + 5
    codes = np.zeros((n, ref.pitch(d)), dtype=np.uint8)
    codes[:, :d // 2 + 1] = _rng(3).integers(0, 256, (n, d // 2 + 1))
    codes[:, :8] = np.arange(0, 256, 34)[:8]
    scales = np.full((n, ref.pitch(d, fmt)), 0, dtype=np.uint8)
    scales[:, 0], scales[:, 1], scales[:, 2] = np.arange(n), np.arange(n)[::-1], (np.arange(n) * 7) % n
    ts = None if t is None else torch.tensor([t], device="cuda")
    y = torch.full((n, d + 3), 7.0, dtype=dtype, device="cuda")
    out = y[:, :d]
    lnq.lnq_fp4_dequantize(dev(codes), dev(scales), d, fmt, tensor_scale=ts, y=out)
    assert (y[:, d:] == 7.0).all()
    want = ref.values(codes, scales, d, fmt)
    with np.errstate(over="ignore", invalid="ignore"):
        if t is not None:
            want = (want * float(np.float32(t))).astype(np.float32)
        want = torch.from_numpy(want).float().to(dtype)
    got = out.cpu()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got, nan=0.0, posinf=9e4, neginf=-9e4),
                       torch.nan_to_num(want, nan=0.0, posinf=9e4, neginf=-9e4))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,d,extra", [(1, 1, 0), (5, 33, 0), (70, 1000, 5), (300, 4096, 0)])
def test_tensor_scale(lnq, dtype, rows, d, extra):
    x = strided(dev(_rng(rows, d).standard_normal((rows, d)), dtype), extra)
    want = float(np.float32(x.double().abs().max().item() / 2688))
    assert lnq.lnq_fp4_tensor_scale(x).item() == want
    x[0, 0] = float("inf")
    x[-1, -1] = float("nan")
    fin = x.double()[x.isfinite()]
    want = float(np.float32(fin.abs().max().item() / 2688)) if fin.numel() else 1.0
    assert lnq.lnq_fp4_tensor_scale(x).item() == want


def test_tensor_scale_of_nothing(lnq):
    assert lnq.lnq_fp4_tensor_scale(torch.zeros(4, 70, device="cuda")).item() == 1.0
    assert lnq.lnq_fp4_tensor_scale(torch.zeros(0, 70, device="cuda")).item() == 1.0
    # a largest element whose quotient rounds to zero
    assert lnq.lnq_fp4_tensor_scale(torch.full((1, 3), 1e-44, device="cuda")).item() == 1.0


def test_round_trip_at_the_matrix_scale(lnq):
    """With the matrix's own t every element comes back within the bound below."""
    x = torch.randn(64, 700, device="cuda") * torch.logspace(-3, 2, 64, device="cuda")[:, None]
    t = lnq.lnq_fp4_tensor_scale(x)
    codes, scales = lnq.lnq_fp4_quantize(x, NV, tensor_scale=t)
    y = lnq.lnq_fp4_dequantize(codes, scales, 700, NV, tensor_scale=t)
    top = torch.nn.functional.pad(x, (0, 4)).abs().view(64, 44, 16).amax(-1)
    # q = top / (6 t) is at most 448 (1 + 2^-24), and its E4M3 number s is off by at most
    # h = max(q / 16, 2^-10) (half a step: 2^-4 of the value, or half the least number). Codes
    # are at most 2 apart, so an element within 6 s t comes back within s t <= (q + h) t; one above
    # it (at most top = 6 q t) comes back as 6 s t, off by at most 6 (q - s) t <= 6 h t.
    h = torch.maximum(top / 96, 2.0 ** -10 * t)
    bound = torch.maximum(top / 6 + h, 6 * h)
    err = torch.nn.functional.pad((x - y).abs(), (0, 4)).view(64, 44, 16).amax(-1)
    assert (err <= bound * 1.0001).all()


# ----------------------------------------------------------------------------------- products

def _operand(rng, rows, d, dtype, exact):
    x = rng.integers(-2, 3, (rows, d)).astype(np.float64) if exact \
        else rng.standard_normal((rows, d))
    return dev(x, dtype)


def check_product(y, x64, w64, scale=1.0, exact=False, rows=None):
    """y against x64 w64^T * scale (both in 64 bits), within the tolerance above."""
    got = f64(y)
    want = x64 @ w64.T * scale
    if exact:
        want = torch.from_numpy(want).to(y.dtype).double().numpy()
        np.testing.assert_array_equal(got, want)
        return
    K = x64.shape[1]
    S = np.abs(x64) @ np.abs(w64).T * abs(scale)
    tol = (K + 4) * 2.0 ** -23 * S + torch.finfo(y.dtype).eps / 2 * np.abs(want)
    # below the least normal number of the type a step no longer shrinks with the value
    tol = tol + torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,d_in,d_out", [
    (1, 1, 1), (1, 16, 3), (2, 31, 17), (3, 33, 16), (4, 128, 40), (5, 130, 33), (7, 257, 100),
    (8, 1024, 64), (9, 1000, 31), (16, 384, 50), (17, 640, 16), (33, 200, 70), (1, 4096, 256),
    (2, 11008, 48), (70, 96, 20)])
@pytest.mark.parametrize("exact", [True, False])
def test_gemv(lnq, fmt, dtype, n, d_in, d_out, exact):
    rng = _rng(n, d_in, d_out)
    x = _operand(rng, n, d_in, dtype, exact)
    codes, scales = ref.random_stored(rng, (d_out,), d_in, fmt, exact)
    t = None if fmt == MX or exact else 0.37
    ts = None if t is None else torch.tensor([t], device="cuda")
    w = ref.values(codes, scales, d_in, fmt)
    for out in ([torch.float32] if exact else TYPES):
        y = lnq.lnq_fp4_gemv(x, dev(codes), dev(scales), fmt, tensor_scale=ts, dtype=out)
        check_product(y, f64(x), w, 1.0 if t is None else float(np.float32(t)), exact)


@pytest.mark.parametrize("fmt,dtype,n,d_in,d_out,experts", [
    (MX, torch.float32, 5, 8200, 5001, 1), (NV, torch.bfloat16, 1, 4100, 9001, 1),
    (NV, torch.float16, 20, 5000, 2600, 1), (MX, torch.bfloat16, 9, 12000, 1500, 1),
    (NV, torch.bfloat16, 7, 2100, 4700, 3), (MX, torch.float32, 11, 900, 4700, 3)])
def test_gemv_many_tiles(lnq, fmt, dtype, n, d_in, d_out, experts):
    """Several rounds of tiles to a CTA, the last one not full; K shared among warps and CTAs."""
    rng = _rng(n, d_in, d_out)
    x = _operand(rng, n, d_in, dtype, True)
    codes, scales = ref.random_stored(rng, (experts, d_out), d_in, fmt, True)
    if experts == 1:
        y = lnq.lnq_fp4_gemv(x, dev(codes[0]), dev(scales[0]), fmt, dtype=torch.float32)
        ends = [0, n]
    else:
        ends = [0, 4, 4, n]
        y = lnq.lnq_fp4_grouped_gemv(x, dev(np.array(ends, np.int32)), dev(codes), dev(scales), fmt,
                                     dtype=torch.float32)
    for e in range(experts):
        rows = slice(ends[e], ends[e + 1])
        if ends[e + 1] > ends[e]:
            check_product(y[rows], f64(x)[rows], ref.values(codes[e], scales[e], d_in, fmt), exact=True)


def test_gemv_strided(lnq):
    rng = _rng(9)
    for dtype in TYPES:
        for extra, shift in ((1, 0), (8, 0), (0, 1), (3, 5)):
            x = strided(_operand(rng, 6, 300, dtype, True), extra, shift)
            codes, scales = ref.random_stored(rng, (37,), 300, MX, True)
            y = torch.full((6, 50), -1.0, device="cuda")
            lnq.lnq_fp4_gemv(x, dev(codes), dev(scales), MX, y=y[:, 5:42])
            check_product(y[:, 5:42], f64(x), ref.values(codes, scales, 300, MX), exact=True)
            assert (y[:, :5] == -1).all() and (y[:, 42:] == -1).all()


def test_gemv_32_bit_activations_are_not_rounded(lnq):
    """x = 1 + 2^-23 and its like: products keep all 24 bits of x."""
    d = 64
    x = torch.zeros(3, d, device="cuda")
    x[0, 5], x[1, 6], x[2, 63] = 1 + 2.0 ** -23, -(3 + 2.0 ** -21), 2.0 ** -100 * (1 + 2.0 ** -20)
    codes = np.full((4, ref.pitch(d)), 0x22, dtype=np.uint8)  # every code 1.0
    scales = np.full((4, ref.pitch(d, MX)), 127, dtype=np.uint8)
    y = lnq.lnq_fp4_gemv(x, dev(codes), dev(scales), MX)
    assert torch.equal(y, x.sum(1, keepdim=True).expand(3, 4))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 11])
def test_gemv_extreme_mx_scales(lnq, dtype, n):
    """Scales from the whole range of powers of two, mixed within rows; the products stay in range
    through x. Bits of x below 2^-133 and results below the 32-bit normal range may be cut off."""
    rng = _rng(13, n)
    d_in, d_out = 416, 24
    codes, scales = ref.random_stored(rng, (d_out,), d_in, MX)
    scales[:, :13] = np.where(rng.random((d_out, 13)) < 0.6, rng.integers(100, 130, (d_out, 13)),
                              rng.integers(0, 255, (d_out, 13)))
    scales[3, :13], scales[4, :13], scales[5, 1:13] = 0, 254, 1
    block = np.arange(d_in) // 32
    x = rng.standard_normal((n, d_in)) * 2.0 ** rng.integers(-20, 3, 13)[block]
    xt = dev(x, dtype)
    w = ref.values(codes, scales, d_in, MX)
    y = f64(lnq.lnq_fp4_gemv(xt, dev(codes), dev(scales), MX, dtype=torch.float32))
    want = f64(xt) @ w.T
    S = np.abs(f64(xt)) @ np.abs(w).T
    top = float(torch.finfo(torch.float32).max)
    sure = S < top / 2  # no partial sum overflows
    tol = (d_in + 4) * 2.0 ** -23 * S + 2.0 ** -126
    assert sure.mean() > 0.3
    assert (np.abs(y - want) <= tol)[sure].all()
    with np.errstate(invalid="ignore"):
        assert (np.isinf(y) | np.isnan(y) | (np.abs(y - want) <= tol))[~sure].all()


@pytest.mark.parametrize("byte", [0, 1, 2, 8, 9, 130, 131, 253, 254])
def test_gemv_smallest_and_largest_mx_scales(lnq, byte):
    """Whole rows at one end of the scales, against x at the other end: equal on exact sums."""
    rng = _rng(15, byte)
    codes, scales = ref.random_stored(rng, (20,), 300, MX)
    scales[:, :10] = byte
    x = rng.integers(-2, 3, (3, 300)) * 2.0 ** (100 if byte < 127 else -100)
    y = lnq.lnq_fp4_gemv(dev(x, torch.bfloat16), dev(codes), dev(scales), MX, dtype=torch.float32)
    check_product(y, x, ref.values(codes, scales, 300, MX), exact=True)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_products_with_nan_scales(lnq, fmt):
    """A NaN block of one row of either operand makes that row's (column's) outputs NaN, no other."""
    rng = _rng(11)
    n, d_in, d_out = 5, 300, 40
    codes, scales = ref.random_stored(rng, (d_out,), d_in, fmt, True)
    scales[7, 2] = 255 if fmt == MX else 127
    x = _operand(rng, n, d_in, torch.bfloat16, True)
    y = f64(lnq.lnq_fp4_gemv(x, dev(codes), dev(scales), fmt))
    assert np.isnan(y[:, 7]).all() and np.isfinite(np.delete(y, 7, 1)).all()
    ac, as_ = ref.random_stored(rng, (n,), d_in, fmt, True)
    as_[3, 1] = 255 if fmt == MX else 127
    y = f64(lnq.lnq_fp4_gemm(dev(ac), dev(as_), dev(codes), dev(scales), d_in, fmt))
    bad = np.zeros((n, d_out), bool)
    bad[3], bad[:, 7] = True, True
    np.testing.assert_array_equal(np.isnan(y), bad)


@pytest.mark.parametrize("dtype", TYPES)
def test_gemv_infinite_activations(lnq, dtype):
    """An infinity or NaN in x reaches that row of y alone."""
    rng = _rng(12)
    codes = np.full((24, ref.pitch(200)), 0x22, dtype=np.uint8)
    scales = np.full((24, ref.pitch(200, MX)), 127, dtype=np.uint8)
    x = _operand(rng, 4, 200, dtype, True)
    x[1, 17] = float("inf")
    x[2, 199] = float("nan")
    y = lnq.lnq_fp4_gemv(x, dev(codes), dev(scales), MX, dtype=torch.float32)
    assert (y[1] == float("inf")).all() and y[2].isnan().all()
    assert y[0].isfinite().all() and y[3].isfinite().all()


GEMM_SHAPES = [(1, 1, 1), (1, 64, 128), (2, 31, 17), (3, 33, 130), (16, 128, 128), (17, 256, 129),
               (64, 200, 300), (127, 257, 127), (128, 512, 256), (129, 1000, 64), (200, 96, 520),
               (255, 640, 384), (257, 768, 257), (300, 4096, 200), (5, 11008, 136)]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("n,d_in,d_out", GEMM_SHAPES)
@pytest.mark.parametrize("exact", [True, False])
def test_gemm(lnq, fmt, out, n, d_in, d_out, exact):
    rng = _rng(n, d_in, d_out, 1)
    ac, as_ = ref.random_stored(rng, (n,), d_in, fmt, exact)
    if exact:  # whole and half numbers up to 2: sums of a few thousand products stay exact
        ac &= 0x33
        ac |= (rng.integers(0, 256, ac.shape, dtype=np.uint8) & 0x88)
        as_[:] = 127 if fmt == MX else 56
        if d_in % 2:
            ac[:, d_in // 2] &= 15
    wc, ws = ref.random_stored(rng, (d_out,), d_in, fmt, exact)
    if exact:
        wc &= 0xBB
    ta = None if fmt == MX or exact else 0.37
    tb = None if fmt == MX or exact else 0.0021
    sa = None if ta is None else torch.tensor([ta], device="cuda")
    sb = None if tb is None else torch.tensor([tb], device="cuda")
    y = lnq.lnq_fp4_gemm(dev(ac), dev(as_), dev(wc), dev(ws), d_in, fmt, a_scale=sa, b_scale=sb,
                         dtype=out)
    scale = 1.0 if ta is None else float(np.float32(ta)) * float(np.float32(tb))
    check_product(y, ref.values(ac, as_, d_in, fmt), ref.values(wc, ws, d_in, fmt), scale, exact)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("n,d_in,d_out", [(2100, 700, 5000), (5000, 256, 1100), (31, 900, 20000),
                                          (100, 2944, 9000), (60, 1408, 12000), (1300, 11008, 777)])
def test_gemm_many_tiles(lnq, fmt, n, d_in, d_out):
    """More tiles than run at once, for every tile width and both ways of loading scales; equality
    on exact sums, in 64 bits on the device."""
    rng = _rng(n, d_in, d_out, 2)
    ac, as_ = ref.random_stored(rng, (n,), d_in, fmt, True)
    ac &= 0x33
    as_[:] = 127 if fmt == MX else 56
    if d_in > 4000:
        ac &= 0x11
    wc, ws = ref.random_stored(rng, (d_out,), d_in, fmt, True)
    x = dev(ref.values(ac, as_, d_in, fmt))
    want = x @ dev(ref.values(wc, ws, d_in, fmt)).T
    assert want.abs().max() < 2 ** 20
    y = lnq.lnq_fp4_gemm(dev(ac), dev(as_), dev(wc), dev(ws), d_in, fmt, dtype=torch.float32)
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_grouped_gemm_many_tiles(lnq, fmt):
    rng = _rng(34)
    E, d_in, d_out = 9, 520, 1500
    sizes = [300, 0, 1, 1700, 128, 129, 33, 700, 64]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n = int(off[-1])
    ac, as_ = ref.random_stored(rng, (n,), d_in, fmt, True)
    ac &= 0x33
    as_[:] = 127 if fmt == MX else 56
    wc, ws = ref.random_stored(rng, (E, d_out), d_in, fmt, True)
    x = dev(ref.values(ac, as_, d_in, fmt))
    y = lnq.lnq_fp4_grouped_gemm(dev(ac), dev(as_), dev(off), dev(wc), dev(ws), d_in, fmt,
                                 dtype=torch.float32)
    for e in range(E):
        want = x[off[e]:off[e + 1]] @ dev(ref.values(wc[e], ws[e], d_in, fmt)).T
        assert torch.equal(y[off[e]:off[e + 1]].double(), want)


def test_gemm_extreme_mx_scales(lnq):
    """Small scales on one side against large ones on the other."""
    rng = _rng(14)
    n, d_in, d_out = 20, 512, 140
    ac, as_ = ref.random_stored(rng, (n,), d_in, MX)
    wc, ws = ref.random_stored(rng, (d_out,), d_in, MX)
    as_[:, :16] = rng.integers(0, 12, (n, 16))
    ws[:, :16] = rng.integers(242, 255, (d_out, 16))
    y = lnq.lnq_fp4_gemm(dev(ac), dev(as_), dev(wc), dev(ws), d_in, MX, dtype=torch.float32)
    check_product(y, ref.values(ac, as_, d_in, MX), ref.values(wc, ws, d_in, MX))


def test_gemm_writes_only_its_columns(lnq):
    rng = _rng(21)
    ac, as_ = ref.random_stored(rng, (150,), 300, NV)
    wc, ws = ref.random_stored(rng, (140,), 300, NV)
    for out in TYPES:
        y = torch.full((152, 161), -1.0, dtype=out, device="cuda")
        part = y[1:151, 7:147]
        lnq.lnq_fp4_gemm(dev(ac), dev(as_), dev(wc), dev(ws), 300, NV, y=part,
                         a_scale=torch.tensor([1e-3], device="cuda"))
        check_product(part, ref.values(ac, as_, 300, NV), ref.values(wc, ws, 300, NV),
                      float(np.float32(1e-3)))
        part.fill_(-1.0)
        assert (y == -1.0).all()


OFFSETS = [
    [0, 5, 5, 9, 40],              # an empty group
    [3, 10, 30, 35, 38],           # rows before the first group and behind the last
    [0, 0, 0, 0, 40],              # one group has all
    [40, 40, 40, 40, 40],          # nobody has any
    [0, 1, 2, 3, 4],               # single rows
    [-5, 7, 3, 60, 20],            # not in order and out of range: limited
]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("offsets", OFFSETS)
def test_grouped_gemv(lnq, fmt, offsets):
    rng = _rng(31)
    n, E, d_in, d_out = 40, 4, 290, 50
    wc, ws = ref.random_stored(rng, (E, d_out), d_in, fmt, True)
    t = None if fmt == MX else torch.tensor([0.5, 1.0, 2.0, 4.0], device="cuda")
    for dtype in TYPES:
        x = _operand(rng, n, d_in, dtype, True)
        y = torch.full((n, d_out), -77.0, device="cuda")
        lnq.lnq_fp4_grouped_gemv(x, dev(np.int32(offsets)), dev(wc), dev(ws), fmt, tensor_scale=t,
                                 y=y)
        want = np.full((n, d_out), -77.0)
        for e, (a, b) in enumerate(ref.groups(offsets, n)):
            s = 1.0 if t is None else t[e].item()
            want[a:b] = f64(x)[a:b] @ ref.values(wc[e], ws[e], d_in, fmt).T * s
        np.testing.assert_array_equal(f64(y), want)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("factor", [1, 11])
@pytest.mark.parametrize("offsets", OFFSETS)
def test_grouped_gemm(lnq, fmt, factor, offsets):
    rng = _rng(32)
    n, E, d_in, d_out = 40 * factor, 4, 290, 150
    offsets = [o * factor for o in offsets]
    wc, ws = ref.random_stored(rng, (E, d_out), d_in, fmt, True)
    ac, as_ = ref.random_stored(rng, (n,), d_in, fmt, True)
    ac &= 0x33
    as_[:] = 127 if fmt == MX else 56
    t = None if fmt == MX else torch.tensor([0.5, 1.0, 2.0, 4.0], device="cuda")
    y = torch.full((n, d_out), -77.0, device="cuda")
    lnq.lnq_fp4_grouped_gemm(dev(ac), dev(as_), dev(np.int32(offsets)), dev(wc), dev(ws), d_in,
                             fmt, b_scale=t, y=y)
    x = ref.values(ac, as_, d_in, fmt)
    want = np.full((n, d_out), -77.0)
    for e, (a, b) in enumerate(ref.groups(offsets, n)):
        s = 1.0 if t is None else t[e].item()
        want[a:b] = x[a:b] @ ref.values(wc[e], ws[e], d_in, fmt).T * s
    np.testing.assert_array_equal(f64(y), want)


@pytest.mark.parametrize("experts", [1, 33, 300, 1024])
def test_grouped_products_with_many_experts(lnq, experts):
    rng = _rng(33, experts)
    d_in, d_out = 64, 20
    sizes = rng.integers(0, 4, experts)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n = max(1, int(offsets[-1]))
    wc, ws = ref.random_stored(rng, (experts, d_out), d_in, MX, True)
    ac, as_ = ref.random_stored(rng, (n,), d_in, MX, True)
    x = ref.values(ac, as_, d_in, MX)
    want = np.zeros((n, d_out))
    for e, (a, b) in enumerate(ref.groups(offsets, n)):
        want[a:b] = x[a:b] @ ref.values(wc[e], ws[e], d_in, MX).T
    y = torch.zeros((n, d_out), device="cuda")
    lnq.lnq_fp4_grouped_gemm(dev(ac), dev(as_), dev(offsets), dev(wc), dev(ws), d_in, MX, y=y)
    np.testing.assert_array_equal(f64(y), want)
    y.zero_()
    lnq.lnq_fp4_grouped_gemv(dev(x, torch.float32), dev(offsets), dev(wc), dev(ws), MX, y=y)
    np.testing.assert_array_equal(f64(y), want)


# ------------------------------------------------------------------------------- used together

def _linear(lnq, x, t, w, s, tw, d_in):
    codes, scales = lnq.lnq_fp4_quantize(x, NV, tensor_scale=t)
    return lnq.lnq_fp4_gemm(codes, scales, w, s, d_in, NV, a_scale=t, b_scale=tw, dtype=x.dtype)


def test_linear_layer_end_to_end(lnq):
    """Weights quantised with their own matrix scale, activations with theirs, multiplied: against
    the product of the read-back matrices in 64 bits; and the few-row product of the same."""
    torch.manual_seed(0)
    x = torch.randn(150, 600, device="cuda").bfloat16()
    W = torch.randn(260, 600, device="cuda") * 0.02
    tw, t = lnq.lnq_fp4_tensor_scale(W), lnq.lnq_fp4_tensor_scale(x)
    w, s = lnq.lnq_fp4_quantize(W, NV, tensor_scale=tw)
    Wq = f64(lnq.lnq_fp4_dequantize(w, s, 600, NV)) * tw.item()
    codes, scales = lnq.lnq_fp4_quantize(x, NV, tensor_scale=t)
    xq = f64(lnq.lnq_fp4_dequantize(codes, scales, 600, NV)) * t.item()
    check_product(_linear(lnq, x, t, w, s, tw, 600), xq, Wq)
    check_product(lnq.lnq_fp4_gemv(x[:3], w, s, NV, tensor_scale=tw), f64(x[:3]), Wq)


def test_experts_end_to_end(lnq):
    torch.manual_seed(1)
    E, n, d, h = 6, 210, 256, 384
    off = torch.tensor([0, 40, 40, 41, 170, 200, 210], dtype=torch.int32, device="cuda")
    x = torch.randn(n, d, device="cuda").half()
    W = torch.randn(E * h, d, device="cuda") * 0.05
    w, s = lnq.lnq_fp4_quantize(W, MX)
    Wq = f64(lnq.lnq_fp4_dequantize(w, s, d, MX)).reshape(E, h, d)
    w, s = w.view(E, h, -1), s.view(E, h, -1)
    codes, scales = lnq.lnq_fp4_quantize(x, MX)
    xq = f64(lnq.lnq_fp4_dequantize(codes, scales, d, MX))
    y = lnq.lnq_fp4_grouped_gemm(codes, scales, off, w, s, d, MX, dtype=torch.float16)
    z = lnq.lnq_fp4_grouped_gemv(x, off, w, s, MX)
    for e in range(E):
        a, b = off[e].item(), off[e + 1].item()
        if a < b:
            check_product(y[a:b], xq[a:b], Wq[e])
            check_product(z[a:b], f64(x)[a:b], Wq[e])


def test_captured_and_replayed_on_another_stream(lnq):
    torch.manual_seed(2)
    x = torch.randn(33, 512, device="cuda").bfloat16()
    W = torch.randn(200, 512, device="cuda")
    t, tw = torch.tensor([0.002], device="cuda"), lnq.lnq_fp4_tensor_scale(W)
    w, s = lnq.lnq_fp4_quantize(W, NV, tensor_scale=tw)
    eager = _linear(lnq, x, t, w, s, tw, 512)
    few = lnq.lnq_fp4_gemv(x[:2], w, s, NV, tensor_scale=tw)
    scale = lnq.lnq_fp4_tensor_scale(x)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, _linear(lnq, x, t, w, s, tw, 512),
                           lnq.lnq_fp4_gemv(x[:2], w, s, NV, tensor_scale=tw),
                           lnq.lnq_fp4_tensor_scale(x)))
    x2 = torch.randn(33, 512, device="cuda").bfloat16()
    before = x.clone()
    x.copy_(x2)
    want = [_linear(lnq, x, t, w, s, tw, 512), lnq.lnq_fp4_gemv(x[:2], w, s, NV, tensor_scale=tw),
            lnq.lnq_fp4_tensor_scale(x)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for (g, *_), st in zip(graphs, streams):  # both at once
        with torch.cuda.stream(st):
            g.replay()
    torch.cuda.synchronize()
    for _, *got in graphs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    x.copy_(before)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for a, b in zip(graphs[0][1:], (eager, few, scale)):
        assert torch.equal(a, b)


def test_results_do_not_change_from_run_to_run(lnq):
    torch.manual_seed(3)
    x = torch.randn(48, 4096, device="cuda").bfloat16()
    W = torch.randn(640, 4096, device="cuda")
    w, s = lnq.lnq_fp4_quantize(W, MX)
    codes, scales = lnq.lnq_fp4_quantize(x, MX)
    y = lnq.lnq_fp4_gemm(codes, scales, w, s, 4096, MX, dtype=torch.float32)
    z = lnq.lnq_fp4_gemv(x[:9], w, s, MX, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(y, lnq.lnq_fp4_gemm(codes, scales, w, s, 4096, MX, dtype=torch.float32))
        assert torch.equal(z, lnq.lnq_fp4_gemv(x[:9], w, s, MX, dtype=torch.float32))


@pytest.mark.parametrize("n,d_in,d_out", [(20, 1024, 300), (60, 2048, 500), (128, 512, 9000),
                                          (300, 1000, 700), (40, 2944, 300)])
def test_a_wait_that_gives_up_is_reported(lnq, n, d_in, d_out):
    """With no time for any wait, the product returns, the check says so once, and the next call is
    whole again."""
    rng = _rng(41, n)
    ac, as_ = ref.random_stored(rng, (n,), d_in, NV, True)
    ac &= 0x33
    as_[:] = 56
    wc, ws = ref.random_stored(rng, (d_out,), d_in, NV, True)
    args = [dev(v) for v in (ac, as_, wc, ws)]
    want = dev(ref.values(ac, as_, d_in, NV)) @ dev(ref.values(wc, ws, d_in, NV)).T
    assert lnq.lnq_fp4_check() == 0
    lnq.lnq_set_wait_limit(0)
    try:
        lnq.lnq_fp4_gemm(*args, d_in, NV, dtype=torch.float32)
        assert lnq.lnq_fp4_check() == 5  # LNQ_ERR_TIMEOUT
    finally:
        lnq.lnq_set_wait_limit(-1)
    assert lnq.lnq_fp4_check() == 0
    assert torch.equal(lnq.lnq_fp4_gemm(*args, d_in, NV, dtype=torch.float32).double(), want)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_scales_at_their_least_alignment(lnq, fmt):
    """Matrices that begin one row into their storage: scales 4 (MX) or 8 (NV) bytes off 16."""
    rng = _rng(42)
    for d_in in (100, 300, 512):
        ac, as_ = ref.random_stored(rng, (41,), d_in, fmt, True)
        ac &= 0x33
        as_[:] = 127 if fmt == MX else 56
        wc, ws = ref.random_stored(rng, (131,), d_in, fmt, True)
        a, sa, w, sw = [dev(v)[1:] for v in (ac, as_, wc, ws)]
        x, v = ref.values(ac[1:], as_[1:], d_in, fmt), ref.values(wc[1:], ws[1:], d_in, fmt)
        check_product(lnq.lnq_fp4_gemm(a, sa, w, sw, d_in, fmt, dtype=torch.float32), x, v, exact=True)
        check_product(lnq.lnq_fp4_gemv(dev(x, torch.float32)[:5], w, sw, fmt), x[:5], v, exact=True)
        assert np.array_equal(f64(lnq.lnq_fp4_dequantize(w, sw, d_in, fmt)), v)


def test_a_stream_given_by_the_caller(lnq):
    x = torch.randn(64, 256, device="cuda")
    w, s = lnq.lnq_fp4_quantize(x, MX)
    want = lnq.lnq_fp4_gemv(x[:4], w, s, MX)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = torch.zeros(4, 64, device="cuda")
    torch.cuda.synchronize()
    lnq.lnq_fp4_gemv(x[:4], w, s, MX, y=y, stream=st)
    st.synchronize()
    assert torch.equal(y, want)


def test_matrices_beyond_32_bits(lnq):
    """Codes, activations and results whose offsets pass 2^32 bytes: the last rows are those of
    small calls."""
    d, rows = 4096, 1_150_000                        # 9.4 GB of bf16, 2.4 GB of codes
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    x[:] = torch.randn(d, device="cuda")
    x[-3:] = torch.randn(3, d, device="cuda")
    codes, scales = lnq.lnq_fp4_quantize(x, MX)
    c3, s3 = lnq.lnq_fp4_quantize(x[-3:].clone(), MX)
    assert torch.equal(codes[-3:], c3) and torch.equal(scales[-3:], s3)
    x.zero_()
    lnq.lnq_fp4_dequantize(codes, scales, d, MX, y=x)
    assert torch.equal(x[-3:], lnq.lnq_fp4_dequantize(c3, s3, d, MX, dtype=torch.bfloat16))
    top = lnq.lnq_fp4_tensor_scale(x)
    x[-1, -1] = 1000.0
    assert lnq.lnq_fp4_tensor_scale(x).item() == float(np.float32(1000.0 / 2688)) != top.item()
    del x
    # as weights: 1.15 million outputs
    a = torch.randn(2, d, device="cuda").bfloat16()
    ac, as_ = lnq.lnq_fp4_quantize(a, MX)
    assert torch.equal(lnq.lnq_fp4_gemm(ac, as_, codes, scales, d, MX)[:, -3:],
                       lnq.lnq_fp4_gemm(ac, as_, c3, s3, d, MX))
    check_product(lnq.lnq_fp4_gemv(a, codes, scales, MX)[:, -3:], f64(a),
                  f64(lnq.lnq_fp4_dequantize(c3, s3, d, MX)))
    # as activations: 1.15 million rows, 3000 outputs (6.9 GB)
    w, s = lnq.lnq_fp4_quantize(torch.randn(3000, d, device="cuda"), MX)
    y = lnq.lnq_fp4_gemm(codes, scales, w, s, d, MX)
    assert torch.equal(y[-3:], lnq.lnq_fp4_gemm(codes[-259:], scales[-259:], w, s, d, MX)[-3:])


def test_no_rows(lnq):
    for fmt in (MX, NV):
        x = torch.zeros(0, 100, device="cuda")
        codes, scales = lnq.lnq_fp4_quantize(x, fmt)
        assert codes.shape == (0, 64) and scales.shape == (0, ref.pitch(100, fmt))
        assert lnq.lnq_fp4_dequantize(codes, scales, 100, fmt).shape == (0, 100)
        w = torch.zeros(5, 64, dtype=torch.uint8, device="cuda")
        s = torch.zeros(5, ref.pitch(100, fmt), dtype=torch.uint8, device="cuda")
        assert lnq.lnq_fp4_gemv(x, w, s, fmt).shape == (0, 5)
        assert lnq.lnq_fp4_gemm(codes, scales, w, s, 100, fmt).shape == (0, 5)


def test_binding_refusals(lnq):
    x = torch.zeros(4, 128, device="cuda")
    codes, scales = lnq.lnq_fp4_quantize(x, NV)
    mx_codes, mx_scales = lnq.lnq_fp4_quantize(x, MX)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    t = torch.ones(1, device="cuda")
    bad = [
        lambda: lnq.lnq_fp4_quantize(x.double(), NV),
        lambda: lnq.lnq_fp4_quantize(x[0], NV),
        lambda: lnq.lnq_fp4_quantize(x.T, NV),
        lambda: lnq.lnq_fp4_quantize(x[:1].expand(4, 128), NV),
        lambda: lnq.lnq_fp4_quantize(x, 2),
        lambda: lnq.lnq_fp4_quantize(x, MX, tensor_scale=t),
        lambda: lnq.lnq_fp4_quantize(x, NV, tensor_scale=t.double()),
        lambda: lnq.lnq_fp4_quantize(x, NV, tensor_scale=torch.ones(2, device="cuda")),
        lambda: lnq.lnq_fp4_quantize(x, NV, codes=codes[:3]),
        lambda: lnq.lnq_fp4_dequantize(codes, scales, 129, NV),
        lambda: lnq.lnq_fp4_dequantize(codes, mx_scales, 128, NV),
        lambda: lnq.lnq_fp4_dequantize(codes, scales, 128, NV, dtype=torch.int8),
        lambda: lnq.lnq_fp4_gemv(x[:, :100], codes[:, :32], scales, NV),
        lambda: lnq.lnq_fp4_gemv(x, codes[None], scales[None], NV),
        lambda: lnq.lnq_fp4_gemv(x, codes, scales, NV, y=torch.zeros(4, 5, device="cuda")),
        lambda: lnq.lnq_fp4_grouped_gemv(x, off, codes[None], scales[None], NV),
        lambda: lnq.lnq_fp4_grouped_gemv(x, off.long(), codes.view(2, 2, 64), scales.view(2, 2, 8),
                                         NV),
        lambda: lnq.lnq_fp4_gemm(codes, scales, mx_codes, mx_scales, 128, NV),
        lambda: lnq.lnq_fp4_gemm(codes, scales, codes, scales, 0, NV),
        lambda: lnq.lnq_fp4_gemm(codes, scales, codes, scales, 128, NV, a_scale=torch.ones(4)),
        lambda: lnq.lnq_fp4_grouped_gemm(codes, scales, off, codes.view(2, 2, 64),
                                         scales.view(2, 2, 8), 128, NV, b_scale=t),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
