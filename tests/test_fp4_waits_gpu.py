"""Waits of the 4-bit products that give up (needs a B200): the next product, started behind the
one that gave up with nothing in between, is whole."""
import numpy as np
import pytest
import torch

import fp4_helpers as ref
from fp4_helpers import MX, NV

pytestmark = pytest.mark.gpu

TIMEOUT = 5  # LNQ_ERR_TIMEOUT


@pytest.fixture(scope="module")
def lnq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_weight_quantization_guided_b200 import build
    build.build_library()
    import post_weight_quantization_guided_b200 as pkg
    yield pkg
    pkg.lnq_set_wait_limit(-1)
    assert pkg.lnq_fp4_check() == 0


def operands(fmt, n, d_in, d_out, experts=None):
    """Device operands whose products are exact in 32 bits, and the result in 64 bits for one
    matrix."""
    rng = np.random.default_rng([fmt, n, d_in, d_out])
    ac, as_ = ref.random_stored(rng, (n,), d_in, fmt, True)
    ac &= 0x33
    as_[:] = 127 if fmt == MX else 56
    lead = (d_out,) if experts is None else (experts, d_out)
    wc, ws = ref.random_stored(rng, lead, d_in, fmt, True)
    a, sa, w, sw = [torch.from_numpy(v).cuda() for v in (ac, as_, wc, ws)]
    x = torch.from_numpy(ref.values(ac, as_, d_in, fmt)).cuda()
    v = torch.from_numpy(ref.values(wc, ws, d_in, fmt)).cuda()
    return a, sa, w, sw, x, v


# fewer stages than the ring holds and many, split K and not, tiles of every width, many tiles to a
# pair, scales by TMA and by plain loads
SHAPES = [(1, 64, 128), (20, 1024, 300), (60, 2048, 500), (128, 512, 9000), (300, 1000, 700),
          (40, 2944, 300), (16, 11008, 4096), (2000, 1024, 3000), (700, 300, 4000)]


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("n,d_in,d_out", SHAPES)
def test_the_product_behind_one_that_gave_up_is_whole(lnq, fmt, n, d_in, d_out):
    a, sa, w, sw, x, v = operands(fmt, n, d_in, d_out)
    want = (x @ v.T).float()
    assert lnq.lnq_fp4_check() == 0
    bad, good = torch.empty_like(want), torch.empty_like(want)
    for limit in (0, 0, 0, 300, 1500, 4000, 10000):
        lnq.lnq_set_wait_limit(limit)
        try:
            lnq.lnq_fp4_gemm(a, sa, w, sw, d_in, fmt, y=bad)
        finally:
            lnq.lnq_set_wait_limit(-1)
        lnq.lnq_fp4_gemm(a, sa, w, sw, d_in, fmt, y=good)
        status = lnq.lnq_fp4_check()
        assert status == TIMEOUT if limit == 0 else status in (0, TIMEOUT)
        assert torch.equal(good, want)
        if status == 0:
            assert torch.equal(bad, want)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_the_grouped_product_behind_one_that_gave_up_is_whole(lnq, fmt):
    sizes = [300, 0, 1, 170, 128, 33]
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    a, sa, w, sw, x, v = operands(fmt, int(off[-1]), 1032, 700, len(sizes))
    o = torch.from_numpy(off).cuda()
    want = torch.cat([x[off[e]:off[e + 1]] @ v[e].T for e in range(len(sizes))]).float()
    for limit in (0, 0, 500, 3000):
        lnq.lnq_set_wait_limit(limit)
        try:
            lnq.lnq_fp4_grouped_gemm(a, sa, o, w, sw, 1032, fmt, dtype=torch.float32)
        finally:
            lnq.lnq_set_wait_limit(-1)
        y = lnq.lnq_fp4_grouped_gemm(a, sa, o, w, sw, 1032, fmt, dtype=torch.float32)
        assert lnq.lnq_fp4_check() in ((TIMEOUT,) if limit == 0 else (0, TIMEOUT))
        assert torch.equal(y, want)


# --------------------------------------------------------------------------- who is told of it

def _gives_up(lnq, args, stream=None):
    lnq.lnq_set_wait_limit(0)
    try:
        return lnq.lnq_fp4_gemm(*args, 1024, MX, stream=stream)
    finally:
        lnq.lnq_set_wait_limit(-1)


@pytest.fixture()
def args(lnq):
    a = operands(MX, 20, 1024, 300)[:4]
    torch.cuda.synchronize()
    yield a
    lnq.lnq_fp4_check()  # the default stream has been told of all


def test_each_of_two_streams_has_its_own_report(lnq, args):
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, other):
        lnq.lnq_fp4_check(stream=st)
    _gives_up(lnq, args, s)
    lnq.lnq_fp4_gemm(*args, 1024, MX, stream=other)
    assert lnq.lnq_fp4_check(stream=other) == 0         # its product is whole, and it takes
    assert lnq.lnq_fp4_check(stream=s) == TIMEOUT       # nothing from the other stream's report
    assert lnq.lnq_fp4_check(stream=s) == 0
    assert lnq.lnq_fp4_check() == TIMEOUT               # the default stream's: of the device
    assert lnq.lnq_fp4_check() == 0


def test_a_report_on_the_default_stream_takes_none_from_a_stream(lnq, args):
    s = torch.cuda.Stream()
    lnq.lnq_fp4_check(stream=s)
    _gives_up(lnq, args, s)
    s.synchronize()
    assert lnq.lnq_fp4_check() == TIMEOUT
    assert lnq.lnq_fp4_check(stream=s) == TIMEOUT
    _gives_up(lnq, args)
    assert lnq.lnq_fp4_check(stream=s) == 0             # called on the default stream
    assert lnq.lnq_fp4_check() == TIMEOUT


def test_a_captured_product_is_reported_where_it_runs(lnq, args):
    graph, s, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    lnq.lnq_set_wait_limit(0)
    try:
        with torch.cuda.graph(graph):
            lnq.lnq_fp4_gemm(*args, 1024, MX)
    finally:
        lnq.lnq_set_wait_limit(-1)
    for st in (s, other, None):
        lnq.lnq_fp4_check(stream=st)
        assert lnq.lnq_fp4_check(stream=st) == 0
    with torch.cuda.stream(s):
        graph.replay()
    for st in (s, other, None):
        assert lnq.lnq_fp4_check(stream=st) == TIMEOUT
        assert lnq.lnq_fp4_check(stream=st) == 0


def test_two_threads_check_while_one_products_give_up(lnq, args):
    """One caller checks all the time; every give-up of the other is reported to the other."""
    import threading
    s, noisy = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, noisy):
        lnq.lnq_fp4_check(stream=st)
    stop, seen = threading.Event(), []

    def watch():
        while not stop.is_set():
            seen.append(lnq.lnq_fp4_check(stream=noisy))

    th = threading.Thread(target=watch)
    th.start()
    try:
        for _ in range(50):
            _gives_up(lnq, args, s)
            assert lnq.lnq_fp4_check(stream=s) == TIMEOUT
    finally:
        stop.set()
        th.join()
    assert seen and not any(seen)
