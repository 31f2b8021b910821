"""Cases for timing and checking the microscaled 4-bit floating-point operators.

Weights and activations are stored as 4-bit floating-point codes (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6
and their negatives, two per byte, even element in the low half) with one 8-bit scale per block of
consecutive elements of a row, in two formats:

  mx   blocks of 32, the scale a power of two (E8M0)
  nv   blocks of 16, the scale an E4M3 number, with one 32-bit scale for the whole matrix

Operators: quantising a matrix (with the matrix scale where the format has one) and reading it
back; the product of a few activation rows with quantised weights; the product of two quantised
matrices, the activations quantised in the call; and both products with the rows grouped by expert.

`run` computes each operator in plain torch operations, or, where `own` is set, through this
repository's entry points. `exact` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

BLOCK = {"mx": 32, "nv": 16}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token's activations on their way into a 4-bit product
        {"name": "quantize_one_token", "op": "quantize", "fmt": "nv", "dtype": "f16", "rows": 1,
         "d": 4096, "matrix_scale": False},
        # a down projection's weights, quantised once for serving
        {"name": "quantize_weights", "op": "quantize", "fmt": "mx", "dtype": "f32", "rows": 4096,
         "d": 11008, "matrix_scale": False},
        # a calibration batch of activations, with the matrix scale found from the data
        {"name": "quantize_tokens", "op": "quantize", "fmt": "nv", "dtype": "bf16", "rows": 16384,
         "d": 4096, "matrix_scale": True},
        # one decoded token through a q projection
        {"name": "gemv_one_token", "op": "gemv", "fmt": "nv", "dtype": "bf16", "n": 1,
         "d_in": 4096, "d_out": 4096},
        # a small batch of decoded tokens, 32-bit activations, an odd number of outputs
        {"name": "gemv_batch", "op": "gemv", "fmt": "mx", "dtype": "f32", "n": 7,
         "d_in": 11008, "d_out": 4101},
        # a short prompt through a q projection
        {"name": "gemm_short", "op": "gemm", "fmt": "nv", "dtype": "f16", "n": 64,
         "d_in": 4096, "d_out": 4096},
        # a prompt of odd length through a down projection
        {"name": "gemm_prompt", "op": "gemm", "fmt": "mx", "dtype": "bf16", "n": 777,
         "d_in": 11008, "d_out": 4096},
        # the largest: a batch of prompts through an up projection
        {"name": "gemm_batch", "op": "gemm", "fmt": "nv", "dtype": "bf16", "n": 16384,
         "d_in": 4096, "d_out": 14336},
        # prompts routed over eight experts
        {"name": "experts_prompt", "op": "grouped_gemm", "fmt": "nv", "dtype": "bf16", "n": 4096,
         "experts": 8, "d_in": 4096, "d_out": 14336, "skew": 0.5},
        # few rows over many small experts, some of them without any
        {"name": "experts_ragged", "op": "grouped_gemm", "fmt": "mx", "dtype": "f16", "n": 1000,
         "experts": 64, "d_in": 2048, "d_out": 1408, "skew": 1.0},
        # eight decoded tokens, two experts each
        {"name": "experts_decode", "op": "grouped_gemv", "fmt": "nv", "dtype": "bf16", "n": 16,
         "experts": 8, "d_in": 4096, "d_out": 14336, "skew": 0.5},
        # decoded tokens over many small experts
        {"name": "experts_decode_small", "op": "grouped_gemv", "fmt": "mx", "dtype": "f32", "n": 24,
         "experts": 64, "d_in": 2048, "d_out": 1408, "skew": 0.5},
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantize", "gemv", "gemm", "grouped_gemm", "grouped_gemv"])
    case = {"op": op, "fmt": rng.choice(["mx", "nv"]), "dtype": rng.choice(["bf16", "f16", "f32"])}
    if op == "quantize":
        d = size(32, 14336)
        case |= {"rows": size(1, min(32768, 67_000_000 // d)), "d": d,
                 "matrix_scale": case["fmt"] == "nv" and rng.random() < 0.5}
        return case
    if op == "gemv":
        return case | {"n": rng.randint(1, 16), "d_in": size(64, 14336), "d_out": size(64, 14336)}
    if op == "gemm":
        return case | {"n": size(1, 8192), "d_in": size(64, 11008), "d_out": size(64, 14336)}
    case |= {"experts": size(2, 128), "d_in": size(256, 4096), "skew": rng.choice([0.0, 0.5, 1.0])}
    case["d_out"] = size(128, min(14336, 400_000_000 // (case["experts"] * case["d_in"])))
    case["n"] = size(1, 64) if op == "grouped_gemv" else size(16, 4096)
    return case


# ------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _activations(rows, d, dtype, g):
    """Normal values with one column in 128 twenty times as large, as activations have them."""
    x = torch.randn(rows, d, generator=g, device="cuda")
    x = x * torch.where(torch.rand(d, generator=g, device="cuda") < 1 / 128, 20.0, 1.0)
    return x.to(DTYPES[dtype])


def _weights(rows, d, g):
    """Student-t values (5 degrees of freedom) of standard deviation 0.02."""
    z = torch.randn(rows, d, generator=g, device="cuda")
    chi2 = torch.randn(rows, d, 5, generator=g, device="cuda").square_().sum(-1)
    return z / (chi2 / 5).sqrt_() * (0.02 * math.sqrt(3 / 5))


def _quantized_weights(experts, rows, d, fmt, g):
    """Stored codes [experts][rows][.], scales and matrix scales of random weights."""
    codes, scales, of_matrix = [], [], []
    for _ in range(experts):
        w = _weights(rows, d, g)
        t = w.abs().max() / 2688 if fmt == "nv" else None
        q, s = _quantize_plain(w, fmt, t)
        codes.append(_pack(q))
        scales.append(_store_scales(s, fmt))
        of_matrix.append(t)
    return (torch.stack(codes), torch.stack(scales), torch.stack(of_matrix) if fmt == "nv" else None)


def _group_sizes(case):
    """Rows per expert, largest first: shares that fall as rank ** -skew, whole numbers, sum n."""
    p = [(e + 1) ** -case["skew"] for e in range(case["experts"])]
    share = [case["n"] * v / sum(p) for v in p]
    sizes = [int(v) for v in share]
    order = sorted(range(len(p)), key=lambda e: sizes[e] - share[e])
    for e in order[:case["n"] - sum(sizes)]:
        sizes[e] += 1
    return sizes


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case)
    if case["op"] == "quantize":
        if case["dtype"] == "f32":
            state["x"] = _weights(case["rows"], case["d"], g)
        else:
            state["x"] = _activations(case["rows"], case["d"], case["dtype"], g)
        # without a matrix scale of its own, the matrix comes with the one found in calibration
        state["x_scale"] = (state["x"].abs().max().float() / 2688).reshape(1)
        return state
    state["x"] = _activations(case["n"], case["d_in"], case["dtype"], g)
    state["x_scale"] = (state["x"].abs().max().float() / 2688).reshape(1)
    experts = case.get("experts", 1)
    w, s, t = _quantized_weights(experts, case["d_out"], case["d_in"], case["fmt"], g)
    if "experts" not in case:
        w, s = w[0], s[0]
    state |= {"w_codes": w, "w_scales": s, "w_scale": t}
    if "experts" in case:
        sizes = torch.tensor(_group_sizes(case), device="cuda")
        sizes = sizes[torch.randperm(experts, generator=g, device="cuda")]
        offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = sizes.cumsum(0)
        state |= {"offsets": offsets, "most": max(_group_sizes(case))}
    return state


# ------------------------------------------------------------------------------------------
# The plain form
# ------------------------------------------------------------------------------------------
def _blocks(x, fmt):
    """x [..., d] as [..., blocks, block], zeros behind the row's end."""
    b = BLOCK[fmt]
    x = torch.nn.functional.pad(x, (0, -x.shape[-1] % b))
    return x.unflatten(-1, (-1, b))


def _round_to(x, quantum):
    """The multiple of quantum (a power of two) nearest x, ties to the even one."""
    return torch.round(x / quantum) * quantum


def _quantize_plain(x, fmt, t=None):
    """(E2M1 values [rows][d], scales [rows][blocks]) in 32 bits; quotients in 64 bits, which
    decide exactly at the borders between two codes."""
    xb = _blocks(x.double(), fmt)
    top = xb.abs().amax(-1)
    if fmt == "mx":
        # frexp gives top = m 2^e with m in [0.5, 1): the leading bit's exponent is e - 1
        scale = torch.exp2((torch.frexp(top)[1] - 3).clamp(-127, 125).double())
        scale = torch.where(top > 0, scale, 2.0 ** -127)
        step = scale
    else:
        q = top / (6 * t.double())
        e = (torch.frexp(q)[1] - 1).clamp(-6, 8)
        scale = _round_to(q, torch.exp2((e - 3).double())).clamp(max=448.0)
        step = scale * t.double()
    q = torch.where(step[..., None] > 0, xb / step[..., None], 0.0)
    a = q.abs()
    a = torch.where(a < 2, _round_to(a, 0.5), torch.where(a < 4, _round_to(a, 1.0), _round_to(a, 2.0)))
    a = a.clamp(max=6.0)
    q = torch.where(xb < 0, -a, a).flatten(-2)[..., :x.shape[-1]]
    return q.float(), scale.float()


def _pack(q):
    """E2M1 values [rows][d] as stored codes [rows][64 ceil(d / 128)]."""
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * (q < 0).to(torch.uint8)
    code = torch.nn.functional.pad(code, (0, -q.shape[-1] % 128))
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _store_scales(s, fmt):
    """Scales [rows][blocks] as stored bytes, the row padded to whole 128 elements."""
    if fmt == "mx":
        byte = (torch.frexp(s.double())[1] + 126).to(torch.uint8)
    else:
        byte = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.nn.functional.pad(byte, (0, -byte.shape[-1] % (128 // BLOCK[fmt])))


def _values(codes, scales, fmt, d, t=None):
    """The 32-bit values [..., d] that stored codes and scales stand for."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)[..., :d]
    q = table[q.int()]
    if fmt == "mx":
        s = torch.exp2(scales.double() - 127).float()
    else:
        s = scales.view(torch.float8_e4m3fn).float()
    v = (_blocks(q, fmt) * s[..., :-(-d // BLOCK[fmt]), None]).flatten(-2)[..., :d]
    return v if t is None else v * t


def _quantized_values(x, fmt, t):
    q, s = _quantize_plain(x, fmt, t)
    v = (_blocks(q, fmt) * s[..., None]).flatten(-2)[..., :x.shape[-1]]
    return v * t if fmt == "nv" else v


def _places(offsets, n):
    """Each row's expert and its place among that expert's rows."""
    rows = torch.arange(n, device="cuda", dtype=offsets.dtype)
    expert = torch.searchsorted(offsets, rows, right=True) - 1
    return expert, rows - offsets[expert]


def _plain(state):
    fmt, x = state["fmt"], state["x"]
    if state["op"] == "quantize":
        t = state["x_scale"]
        if state["matrix_scale"]:
            t = (x.abs().max().double() / 2688).float().reshape(1)
        y = _quantized_values(x, fmt, t).to(x.dtype)
        return (y, t) if state["matrix_scale"] else (y,)
    v = x.float() if state["op"].endswith("gemv") else _quantized_values(x, fmt, state["x_scale"])
    t = state["w_scale"]
    w = _values(state["w_codes"], state["w_scales"], fmt, state["d_in"],
                t if t is None or "experts" not in state else t[:, None, None])
    if "experts" not in state:
        return (v @ w.mT).to(x.dtype)
    expert, place = _places(state["offsets"], state["n"])
    rows = torch.zeros(state["experts"], state["most"], state["d_in"], device="cuda")
    rows[expert, place] = v
    return (rows @ w.mT)[expert, place].to(x.dtype)


# ------------------------------------------------------------------------------------------
# The framework's operators
# ------------------------------------------------------------------------------------------
def _own(state):
    import post_weight_quantization_guided_b200 as lnq
    fmt = lnq.LNQ_FP4_MX if state["fmt"] == "mx" else lnq.LNQ_FP4_NV
    x, op = state["x"], state["op"]
    t = state["x_scale"] if state["fmt"] == "nv" else None
    if op == "quantize":
        if state["matrix_scale"]:
            t = lnq.lnq_fp4_tensor_scale(x)
        codes, scales = lnq.lnq_fp4_quantize(x, fmt, tensor_scale=t)
        y = lnq.lnq_fp4_dequantize(codes, scales, x.shape[1], fmt, tensor_scale=t, dtype=x.dtype)
        return (y, t) if state["matrix_scale"] else (y,)
    w, s, tw = state["w_codes"], state["w_scales"], state["w_scale"]
    if op == "gemv":
        return lnq.lnq_fp4_gemv(x, w, s, fmt, tensor_scale=tw)
    if op == "grouped_gemv":
        return lnq.lnq_fp4_grouped_gemv(x, state["offsets"], w, s, fmt, tensor_scale=tw)
    codes, scales = lnq.lnq_fp4_quantize(x, fmt, tensor_scale=t)
    if op == "gemm":
        return lnq.lnq_fp4_gemm(codes, scales, w, s, state["d_in"], fmt, a_scale=t, b_scale=tw,
                                dtype=x.dtype)
    return lnq.lnq_fp4_grouped_gemm(codes, scales, state["offsets"], w, s, state["d_in"], fmt,
                                    a_scale=t, b_scale=tw, dtype=x.dtype)


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------
# What a pass cannot do without, and its outputs in 64 bits
# ------------------------------------------------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "quantize":
        n = case["rows"] * case["d"]
        return {"bytes": 2 * size * n, "flops": 0}
    d_in, d_out, n = case["d_in"], case["d_out"], case["n"]
    matrices = sum(k > 0 for k in _group_sizes(case)) if "experts" in case else 1
    weights = matrices * d_out * (d_in // 2 + d_in // BLOCK[case["fmt"]])
    return {"bytes": weights + size * n * (d_in + d_out), "flops": 2 * n * d_in * d_out}


def _quantized_exact(x, fmt, t):
    """Quantised values in 64 bits: each code found between the exact borders of its neighbours."""
    x = _blocks(x.double(), fmt)
    levels = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    border = (levels[1:] + levels[:-1]) / 2
    top = x.abs().amax(-1, keepdim=True)
    if fmt == "mx":
        powers = torch.exp2(torch.arange(-125, 128, dtype=torch.float64, device="cuda"))
        # the scale is 2^-2 times the largest power of two that is not above the block's largest
        step = torch.exp2(torch.searchsorted(powers, top, right=True).double() - 128)
    else:
        bytes_ = torch.arange(127, dtype=torch.uint8, device="cuda")
        e4m3 = bytes_.view(torch.float8_e4m3fn).double()
        middle = (e4m3[1:] + e4m3[:-1]) / 2 * (6 * t.double())
        low, high = torch.searchsorted(middle, top), torch.searchsorted(middle, top, right=True)
        step = e4m3[torch.where(low % 2 == 0, low, high)] * t.double()
    a, code = x.abs(), torch.zeros(x.shape, dtype=torch.int8, device="cuda")
    for k in range(7):  # a tie goes to the even code: up from an odd code, and down to an even one
        limit = border[k] * step
        code += (a >= limit if k % 2 else a > limit).to(torch.int8)
    v = levels[code.int()] * step
    return torch.where(x < 0, -v, v).flatten(-2)


def _values_exact(codes, scales, fmt, d, t):
    """Stored values in 64 bits, from the sign, exponent and mantissa bits."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    e, m = ((nib >> 1) & 3).double(), (nib & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1)) * torch.where(nib >= 8, -1.0, 1.0)
    if fmt == "mx":
        s = torch.exp2(scales.double() - 127)
    else:
        e, m = ((scales >> 3) & 15).double(), (scales & 7).double()
        s = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7)) * t.double()
    return (v * s.repeat_interleave(BLOCK[fmt], -1))[..., :d]


def exact(case, seed):
    state = prepare(case, seed)
    fmt, x = state["fmt"], state["x"]
    if case["op"] == "quantize":
        t = state["x_scale"]
        if case["matrix_scale"]:  # the scale is by definition a 32-bit number
            t = (x.abs().max().double() / 2688).float().reshape(1)
        y = _quantized_exact(x, fmt, t)[:, :case["d"]]
        return (y, t.double()) if case["matrix_scale"] else (y,)
    v = x.double()
    if not case["op"].endswith("gemv"):
        v = _quantized_exact(x, fmt, state["x_scale"])[:, :case["d_in"]]
    codes, scales, t = state["w_codes"], state["w_scales"], state["w_scale"]
    if "experts" not in case:
        return v @ _values_exact(codes, scales, fmt, case["d_in"], t).mT
    y = torch.zeros(case["n"], case["d_out"], dtype=torch.float64, device="cuda")
    at = state["offsets"].tolist()
    for e in range(case["experts"]):
        w = _values_exact(codes[e], scales[e], fmt, case["d_in"], None if t is None else t[e])
        y[at[e]:at[e + 1]] = v[at[e]:at[e + 1]] @ w.mT
    return y
