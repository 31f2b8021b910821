"""The 4-bit products where numbers leave the ordinary range (needs a B200): matrix scales t from the
whole of the 32-bit range, with results inside it.

All sums here are exact in 32 bits in any order (multiples of one power of two, below 2^20 of it), and
a matrix scale that is a power of two keeps them exact, so the results have to be equal."""
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("log_t", [127, 125, 122, 121, 120, 60, 0, -60, -126, -135, -149])
def test_gemv_at_every_matrix_scale(lnq, dtype, log_t):
    """Sums of about 2^9 steps, the step 2^-log_t / 8: results of about 1 to 100."""
    rng = np.random.default_rng([7, log_t + 200])
    n, d_in, d_out = 3, 200, 40
    codes, scales = ref.random_stored(rng, (d_out,), d_in, NV, True)
    x = rng.integers(-2, 3, (n, d_in)).astype(np.float64)
    x[1] = 0
    move = max(-120, min(120, log_t))  # what is left of t beyond that stays in the result
    t = torch.tensor([2.0 ** log_t], dtype=torch.float32, device="cuda")
    xt = dev(x * 2.0 ** -move).to(dtype)
    y = lnq.lnq_fp4_gemv(xt, dev(codes), dev(scales), NV, tensor_scale=t, dtype=torch.float32)
    want = x @ ref.values(codes, scales, d_in, NV).T * 2.0 ** (log_t - move)
    np.testing.assert_array_equal(y.double().cpu().numpy(), want)
    off = torch.tensor([0, 1, n], dtype=torch.int32, device="cuda")
    y = lnq.lnq_fp4_grouped_gemv(xt, off, dev(np.stack([codes, codes])), dev(np.stack([scales, scales])),
                                 NV, tensor_scale=torch.cat([t, t]), dtype=torch.float32)
    np.testing.assert_array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("n,d_in", [(20, 200), (20, 1024), (300, 300), (600, 520)])
@pytest.mark.parametrize("log_a,log_w", [
    (0, 0), (100, -100), (-100, 100), (127, -127), (-127, 127), (-149, 127), (127, -149), (-140, 120),
    (120, -110), (-110, 120), (60, 60), (63, 50), (-60, -50), (127, 0), (0, -120), (-130, 10),
    (-100, -40), (-149, -149), (127, 127)])
def test_gemm_at_every_pair_of_matrix_scales(lnq, n, d_in, log_a, log_w):
    """Whatever the product of the sum with one of the two scales would be: sums below 2^13 in steps
    of 1/8, which are 32-bit numbers after the scales too, or too large for them (infinite), or for
    (-149, -149) too small (zero)."""
    rng = np.random.default_rng([8, n, d_in])
    d_out = 150
    ac, as_ = ref.random_stored(rng, (n,), d_in, NV, True)
    ac &= 0x33
    as_[:] = 56
    wc, ws = ref.random_stored(rng, (d_out,), d_in, NV, True)
    total = ref.values(ac, as_, d_in, NV) @ ref.values(wc, ws, d_in, NV).T
    assert np.abs(total).max() < 2 ** 13
    with np.errstate(over="ignore", under="ignore"):
        want = (total * 2.0 ** (log_a + log_w)).astype(np.float32).astype(np.float64)
    ta, tw = [torch.tensor([2.0 ** v], dtype=torch.float32, device="cuda") for v in (log_a, log_w)]
    a = [dev(v) for v in (ac, as_, wc, ws)]
    y = lnq.lnq_fp4_gemm(*a, d_in, NV, a_scale=ta, b_scale=tw, dtype=torch.float32)
    np.testing.assert_array_equal(y.double().cpu().numpy(), want)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    y = lnq.lnq_fp4_grouped_gemm(a[0], a[1], off, a[2][None], a[3][None], d_in, NV, a_scale=ta, b_scale=tw,
                                 dtype=torch.float32)
    np.testing.assert_array_equal(y.double().cpu().numpy(), want)
