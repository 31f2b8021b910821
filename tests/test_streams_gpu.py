"""Calls on a stream given by the caller: what the binding allocates is that stream's memory, not a
block that work on the current stream may still be using (needs a B200)."""
import pytest
import torch

from fp4_helpers import MX, NV

pytestmark = pytest.mark.gpu

D = 2048


@pytest.fixture(scope="module")
def lnq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_weight_quantization_guided_b200 import build
    build.build_library()
    import post_weight_quantization_guided_b200 as pkg
    return pkg


@pytest.fixture(scope="module")
def calls(lnq):
    """{name: call(stream) -> its outputs}"""
    torch.manual_seed(0)
    x = torch.randn(D, D, device="cuda")
    w, s = lnq.lnq_fp4_quantize(x, MX)
    off = torch.tensor([0, D // 2, D], dtype=torch.int32, device="cuda")
    grouped = (w.view(2, D // 2, -1), s.view(2, D // 2, -1))
    Xb, W = x.bfloat16(), x[:1024].contiguous()
    C, Q = lnq.lnq_init_codebook(W, 16)
    P = lnq.lnq_pack_codes(Q, 4)
    F = lnq.lnq_build_fisher(Xb, None, 1)
    torch.cuda.synchronize()
    return {
        "quantize": lambda st: lnq.lnq_fp4_quantize(x, NV, stream=st),
        "dequantize": lambda st: lnq.lnq_fp4_dequantize(w, s, D, MX, stream=st),
        "tensor_scale": lambda st: lnq.lnq_fp4_tensor_scale(x, stream=st),
        "gemv": lambda st: lnq.lnq_fp4_gemv(x[:256], w, s, MX, stream=st),
        "grouped_gemv": lambda st: lnq.lnq_fp4_grouped_gemv(x, off, *grouped, MX, stream=st),
        "gemm": lambda st: lnq.lnq_fp4_gemm(w, s, w, s, D, MX, stream=st),
        "grouped_gemm": lambda st: lnq.lnq_fp4_grouped_gemm(w, s, off, *grouped, D, MX, stream=st),
        "build_fisher": lambda st: lnq.lnq_build_fisher(Xb, None, 1, stream=st),
        "build_fisher_noalloc": lambda st: lnq.lnq_build_fisher_noalloc(Xb, None, 1, stream=st),
        "init_codebook": lambda st: lnq.lnq_init_codebook(W, 16, stream=st),
        "objective": lambda st: lnq.lnq_objective(F, W, C, Q, stream=st),
        "pack_codes": lambda st: lnq.lnq_pack_codes(Q, 4, stream=st),
        "lut_gemv": lambda st: lnq.lnq_lut_gemv(x[:8], P, C, D, stream=st),
    }


NAMES = ["quantize", "dequantize", "tensor_scale", "gemv", "grouped_gemv", "gemm", "grouped_gemm",
         "build_fisher", "build_fisher_noalloc", "init_codebook", "objective", "pack_codes",
         "lut_gemv"]


def _outputs(v):
    return v if isinstance(v, tuple) else (v,)


@pytest.mark.parametrize("name", NAMES)
def test_no_block_of_the_current_stream_is_taken(calls, name):
    """The current stream still has to read tensors that the program has dropped; a call on another
    stream, run meanwhile, leaves their memory alone."""
    call, st = calls[name], torch.cuda.Stream()
    want = [t.clone() for t in _outputs(call(None))]
    torch.cuda.synchronize()
    # tensors of the outputs' sizes, several of each, read only after a while and dropped at once
    dropped = [torch.full((t.numel() * t.element_size(),), 7, dtype=torch.uint8, device="cuda")
               for t in want for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    copies = [t.clone() for t in dropped]
    del dropped
    got = _outputs(call(st))
    st.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert all((c == 7).all() for c in copies)


def test_a_workspace_is_the_streams_memory(lnq):
    from post_weight_quantization_guided_b200 import binding
    size = dict(d_in=1024, d_out=1024, groups=1, m=16)
    a = binding.workspace(binding.LNQ_OP_QUANTIZE_ROWS, **size)
    ptr = a.data_ptr()
    del a
    b = binding.workspace(binding.LNQ_OP_QUANTIZE_ROWS, **size, stream=torch.cuda.Stream())
    assert b.data_ptr() != ptr
    del b
    assert binding.workspace(binding.LNQ_OP_QUANTIZE_ROWS, **size).data_ptr() == ptr
