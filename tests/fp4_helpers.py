"""The microscaled 4-bit formats in 64-bit numpy, from their definitions, for the tests."""
import numpy as np

MX, NV = 0, 1
BLOCK = {MX: 32, NV: 16}
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_b = np.arange(127)
# E4M3 numbers of the bytes 0 .. 126: four exponent bits (bias 7), three mantissa bits
E4M3 = np.where(_b < 8, _b / 8 * 2.0 ** -6, (1 + _b % 8 / 8) * 2.0 ** (_b // 8 - 7.0))


def pitch(d, fmt=None):
    """Bytes per row of codes, or of scales."""
    pad = -(-d // 128)
    return pad * 64 if fmt is None else pad * 128 // BLOCK[fmt]


def nearest_even(a, levels, step):
    """Index of the level l with l * step nearest a (elementwise, a >= 0), ties to the even index;
    borders of two levels times step are exact in 64 bits."""
    border = (levels[1:] + levels[:-1]) / 2
    idx = np.zeros(a.shape, dtype=np.int64)
    for k, b in enumerate(border):
        limit = b * step
        idx += np.where(k % 2 == 1, a >= limit, a > limit)
    return idx


def quantize(x, fmt, t=1.0):
    """(codes, scales) bytes of the matrix x (float64 [rows][d]), as the header defines them."""
    rows, d = x.shape
    B = BLOCK[fmt]
    nb = pitch(d, fmt)
    xp = np.zeros((rows, nb * B))
    xp[:, :d] = x
    xb = xp.reshape(rows, nb, B)
    top = np.abs(xb).max(-1)
    bad = ~np.isfinite(xb).all(-1)
    top = np.where(bad, 0.0, top)
    if fmt == MX:
        e = np.floor(np.log2(np.where(top > 0, top, 1.0)))
        e = np.where(2.0 ** e > top, e - 1, np.where(2.0 ** (e + 1) <= top, e + 1, e))
        byte = np.where(top > 0, np.clip(e - 2, -127, 125) + 127, 0).astype(np.int64)
        step = 2.0 ** (byte - 127.0)
        nan_byte = 255
    else:
        if not (t > 0 and np.isfinite(t)):
            bad[:] = True
            t = 1.0
        byte = nearest_even(top, E4M3, 6 * t)
        step = E4M3[byte] * t
        nan_byte = 127
    a = np.abs(np.where(np.isfinite(xb), xb, 0.0))
    code = nearest_even(a, LEVELS, step[..., None])
    code = np.where(step[..., None] > 0, code, 0)
    code = np.where(bad[..., None], 0, code)
    code = np.where((code > 0) & (xb < 0), code + 8, code)
    byte = np.where(bad, nan_byte, byte)
    code = code.reshape(rows, -1)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    byte = np.where(np.arange(nb) * B < d, byte, 0)
    return codes, byte.astype(np.uint8)


def codes_equal(a, b):
    """Whether two code arrays agree, a zero's sign aside."""
    def nib(c):
        n = np.stack([c & 15, c >> 4], -1)
        return np.where(n == 8, 0, n)
    return np.array_equal(nib(a), nib(b))


def scale_values(scales, fmt):
    s = scales.astype(np.int64)
    if fmt == MX:
        return np.where(s == 255, np.nan, 2.0 ** (s - 127.0))
    return np.append(E4M3, np.nan)[s & 127]


def values(codes, scales, d, fmt, t=1.0):
    """float64 [..., d] that (codes, scales) stand for."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)[..., :d]
    v = LEVELS[n & 7] * np.where(n >= 8, -1.0, 1.0)
    s = np.repeat(scale_values(scales, fmt), BLOCK[fmt], -1)[..., :d]
    return v * s * t


def random_stored(rng, lead, d, fmt, exact=False):
    """Random stored matrices [*lead][d] with arbitrary bytes behind each row. exact: values are
    small multiples of 1/4, so that 32-bit sums of a few thousand products of them and of whole
    numbers are exact."""
    codes = rng.integers(0, 256, (*lead, pitch(d)), dtype=np.uint8)
    if d % 2:
        codes[..., d // 2] &= 15
    if exact:
        exps = rng.integers(-1, 2, (*lead, pitch(d, fmt)))
        scales = (exps + 127 if fmt == MX else (exps + 7) * 8).astype(np.uint8)
    elif fmt == MX:
        scales = rng.integers(118, 128, (*lead, pitch(d, fmt)), dtype=np.uint8)
    else:
        scales = rng.integers(0, 127, (*lead, pitch(d, fmt)), dtype=np.uint8)
    blocks = -(-d // BLOCK[fmt])
    if not exact:  # behind the row: NaN scales, which nothing may read
        scales[..., blocks:] = 255 if fmt == MX else 127
    return codes, scales


def groups(offsets, n):
    """The rows of each group, as the header limits the offsets."""
    top, out = 0, []
    lim = []
    for o in offsets:
        top = max(top, min(int(o), n))
        lim.append(top)
    for e in range(len(lim) - 1):
        out.append((lim[e], lim[e + 1]))
    return out
