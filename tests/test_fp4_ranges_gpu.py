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
