"""The 4-bit products with block scales that differ by row and by block in both operands, over powers
of two from 2^-8 to 2^10 in every sum (needs a B200).

A scale that reaches the wrong row or block shows as a wrong number: blocks with large scales have few
nonzero codes, so that all partial sums are multiples of 2^-8 below 2^16. 24 bits hold them, sums are
exact in 32 bits in any order, and results have to be equal. The shapes take tiles of every width, with
the scales loaded by TMA and by plain loads."""
import numpy as np
import pytest
import torch

import fp4_helpers as ref
from fp4_helpers import MX, NV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lnq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_weight_quantization_guided_b200 import build
    build.build_library()
    import post_weight_quantization_guided_b200 as pkg
    yield pkg
    assert pkg.lnq_fp4_check() == 0


def stored(rng, lead, d, fmt, exps, most):
    """Random matrices [*lead][d]: block k has the scale 2^exps[k], or twice that, row by row, and
    about most[k] nonzero codes out of +-1 and +-2; NaN scales behind the row."""
    B, pad = ref.BLOCK[fmt], ref.pitch(d, fmt)
    blocks = exps.shape[0]
    code = rng.choice(np.array([2, 4, 10, 12], np.uint8), (*lead, pad * B))
    keep = np.zeros(pad)
    keep[:blocks] = most / B
    code = np.where(rng.random(code.shape) < np.repeat(keep, B), code, 0).astype(np.uint8)
    code[..., d:] = 0
    e = exps + rng.integers(0, 2, (*lead, blocks))
    scales = np.full((*lead, pad), 255 if fmt == MX else 127, dtype=np.uint8)
    scales[..., :blocks] = e + 127 if fmt == MX else (e + 7) * 8
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def operands(fmt, n, d, lead):
    rng = np.random.default_rng([fmt, n, d, *lead])
    e = rng.permutation(np.arange(-(-d // ref.BLOCK[fmt])) % 17 - 8)  # a block's product of scales
    most = np.clip(2.0 ** (4 - e), 1, ref.BLOCK[fmt])
    ea = e // 2
    a, sa = stored(rng, (n,), d, fmt, ea, most)
    w, sw = stored(rng, lead, d, fmt, e - ea, np.full(e.shape, ref.BLOCK[fmt]))
    return a, sa, w, sw


def exact(x, v):
    """x v^T in 64 bits on the device, where 32-bit sums are exact."""
    x, v = torch.from_numpy(x).cuda(), torch.from_numpy(v).cuda()
    assert (x.abs() @ v.abs().T).max() < 2 ** 16
    return x @ v.T


SHAPES = [  # rows of a tile: 32, 64, 128, 256, each with rows of scales of whole 16 bytes and not
    (70, 2048, 3000), (70, 1900, 3000), (128, 1024, 9000), (128, 1100, 9000),
    (600, 1024, 2500), (700, 1100, 2500), (2000, 1024, 3000), (2000, 1100, 3000)]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_gemm_scales_of_rows_and_blocks(lnq, fmt, n, d_in, d_out):
    a, sa, w, sw = operands(fmt, n, d_in, (d_out,))
    want = exact(ref.values(a, sa, d_in, fmt), ref.values(w, sw, d_in, fmt))
    args = [torch.from_numpy(v).cuda() for v in (a, sa, w, sw)]
    y = lnq.lnq_fp4_gemm(*args, d_in, fmt, dtype=torch.float32)
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("d_in", [1024, 1100])
@pytest.mark.parametrize("sizes", [[20, 0, 33, 61, 3, 1], [70, 129, 1, 0, 64, 40], [300, 5, 0, 411, 256]])
def test_grouped_gemm_scales_of_rows_and_blocks(lnq, fmt, d_in, sizes):
    """Groups that begin anywhere in a tile's 128 rows of scales; tiles of 64, 128 and 256 rows."""
    ends = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32) + 7  # rows before the first group
    n, E, d_out = int(ends[-1]) + 5, len(sizes), 600
    a, sa, w, sw = operands(fmt, n, d_in, (E, d_out))
    x, v = ref.values(a, sa, d_in, fmt), ref.values(w, sw, d_in, fmt)
    args = [torch.from_numpy(u).cuda() for u in (a, sa, ends, w, sw)]
    y = torch.full((n, d_out), -77.0, device="cuda")
    lnq.lnq_fp4_grouped_gemm(*args, d_in, fmt, y=y)
    want = torch.full((n, d_out), -77.0, dtype=torch.float64, device="cuda")
    for e in range(E):
        if sizes[e]:
            want[ends[e]:ends[e + 1]] = exact(x[ends[e]:ends[e + 1]], v[e])
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("n,d_in,d_out", [(1, 2048, 3000), (7, 1900, 700), (16, 4000, 2000)])
def test_gemv_scales_of_rows_and_blocks(lnq, fmt, n, d_in, d_out):
    a, sa, w, sw = operands(fmt, n, d_in, (d_out,))
    x = ref.values(a, sa, d_in, fmt)
    want = exact(x, ref.values(w, sw, d_in, fmt))
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        y = lnq.lnq_fp4_gemv(torch.from_numpy(x).cuda().to(dtype), *[torch.from_numpy(v).cuda() for v in (w, sw)],
                             fmt, dtype=torch.float32)
        assert torch.equal(y.double(), want)
