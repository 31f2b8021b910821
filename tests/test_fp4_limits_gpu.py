"""The 4-bit operators at the ends of what the header allows, and several callers at once (needs a
B200)."""
import threading

import numpy as np
import pytest
import torch

import fp4_helpers as ref
from fp4_helpers import MX, NV

pytestmark = pytest.mark.gpu

MAX_D = 1 << 24


@pytest.fixture(scope="module")
def lnq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_weight_quantization_guided_b200 import build
    build.build_library()
    import post_weight_quantization_guided_b200 as pkg
    yield pkg
    assert pkg.lnq_fp4_check() == 0


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("d", [MAX_D, MAX_D - 77])
def test_longest_rows(lnq, fmt, d):
    """Rows of 2^24 elements: quantised bytes as defined, and products of sparse rows, whose sums are
    whole numbers below 2^14."""
    rng = np.random.default_rng([9, fmt, d])
    x = torch.randn(1, d, device="cuda").bfloat16()
    codes, scales = lnq.lnq_fp4_quantize(x, fmt)
    want_c, want_s = ref.quantize(x.double().cpu().numpy(), fmt)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert ref.codes_equal(codes.cpu().numpy(), want_c)
    back = lnq.lnq_fp4_dequantize(codes, scales, d, fmt)
    assert np.array_equal(back.double().cpu().numpy(), ref.values(want_c, want_s, d, fmt))
    del x, codes, scales, back

    def sparse(rows):
        at = np.unique(np.concatenate([rng.integers(0, d, 2000), [0, 1, d // 2, d - 2, d - 1]]))
        v = np.zeros((rows, d), np.float32)
        v[:, at] = rng.choice([-2, -1, 0, 1, 2], (rows, at.size))
        return v, at

    (a, at), n, d_out = sparse(3), 3, 5
    w = np.zeros((d_out, d), np.float32)
    w[:, at] = rng.choice([-2, -1, 1, 2], (d_out, at.size))
    want = a[:, at].astype(np.float64) @ w[:, at].T
    one = 127 if fmt == MX else 56

    def stored(v):
        code = np.zeros((v.shape[0], ref.pitch(d) * 2), np.uint8)
        code[:, :d] = np.where(v < 0, 8, 0) + 2 * np.abs(v)
        s = np.full((v.shape[0], ref.pitch(d, fmt)), one, np.uint8)
        return [torch.from_numpy(u).cuda() for u in (code[:, 0::2] | (code[:, 1::2] << 4), s)]

    ac, as_ = stored(a)
    wc, ws = stored(w)
    off = torch.tensor([0, 1, n], dtype=torch.int32, device="cuda")
    y = [lnq.lnq_fp4_gemm(ac, as_, wc, ws, d, fmt, dtype=torch.float32),
         lnq.lnq_fp4_grouped_gemm(ac, as_, off, torch.stack([wc, wc]), torch.stack([ws, ws]), d, fmt,
                                  dtype=torch.float32)]
    for dtype in (torch.float32, torch.bfloat16):
        xd = torch.from_numpy(a).cuda().to(dtype)
        y.append(lnq.lnq_fp4_gemv(xd, wc, ws, fmt, dtype=torch.float32))
        y.append(lnq.lnq_fp4_grouped_gemv(xd, off, torch.stack([wc, wc]), torch.stack([ws, ws]), fmt,
                                          dtype=torch.float32))
    for got in y:
        assert np.array_equal(got.double().cpu().numpy(), want)


def test_threads_on_streams_of_their_own(lnq):
    """Four host threads, each with a stream, all operators at once: every call gives what it gives
    alone. (Sizes with and without split sums, clusters and TMA scales.)"""
    torch.manual_seed(4)
    cases = []
    for fmt, n, d, d_out in [(MX, 5, 11008, 700), (NV, 40, 2048, 900), (MX, 300, 1000, 2000), (NV, 1, 4096, 4096)]:
        x = torch.randn(n, d, device="cuda").bfloat16()
        t = torch.tensor([0.01], device="cuda") if fmt == NV else None
        w, s = lnq.lnq_fp4_quantize(torch.randn(d_out, d, device="cuda"), fmt, tensor_scale=t)
        off = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda")
        w2, s2 = w.view(2, d_out // 2, -1), s.view(2, d_out // 2, -1)
        t2 = None if t is None else t.repeat(2)

        def work(st, fmt=fmt, x=x, t=t, w=w, s=s, off=off, w2=w2, s2=s2, t2=t2, d=d):
            c, q = lnq.lnq_fp4_quantize(x, fmt, tensor_scale=t, stream=st)
            return (c, q, lnq.lnq_fp4_tensor_scale(x, stream=st),
                    lnq.lnq_fp4_dequantize(c, q, d, fmt, tensor_scale=t, stream=st),
                    lnq.lnq_fp4_gemv(x, w, s, fmt, tensor_scale=t, stream=st),
                    lnq.lnq_fp4_grouped_gemv(x, off, w2, s2, fmt, tensor_scale=t2, stream=st),
                    lnq.lnq_fp4_gemm(c, q, w, s, d, fmt, a_scale=t, b_scale=t, stream=st),
                    lnq.lnq_fp4_grouped_gemm(c, q, off, w2, s2, d, fmt, a_scale=t, b_scale=t2, stream=st))

        cases.append((work, [v.clone() for v in work(None)]))
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream() for _ in cases]

    def run(k):
        try:
            for i in range(60):
                work, want = cases[(k + i) % len(cases)]
                got = work(streams[k])
                streams[k].synchronize()
                wrong.extend((k, i, j) for j, (a, b) in enumerate(zip(got, want))
                             if not torch.equal(a.view(torch.uint8).cpu(), b.view(torch.uint8).cpu()))
        except Exception as error:  # a thread's exception is the test's
            wrong.append(error)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(cases))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong
    assert all(lnq.lnq_fp4_check(stream=st) == 0 for st in streams)
