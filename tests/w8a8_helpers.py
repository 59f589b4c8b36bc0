"""Plain implementations, in 64 bits, of the operators on int8 activations,
and inputs for them."""
import numpy as np


def quantize_rows(x):
    """Codes, scales and code sums of the rows of x by the definition: every
    step one fp32 operation, which float64 followed by one rounding to fp32
    reproduces for a quotient of two fp32 values."""
    x = np.asarray(x, dtype=np.float64)
    scale = (np.abs(x).max(axis=1) / 127.0).astype(np.float32)
    s = scale.astype(np.float64)[:, None]
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = (x / s).astype(np.float32).astype(np.float64)
    q = np.where(s > 0, np.clip(np.rint(ratio), -127, 127), 0.0)
    return q.astype(np.int8), scale, q.sum(axis=1).astype(np.int32)


def linear(q, xs, w, scales, zeros=None, bias=None):
    """s_m s_n sum q (w - z) + b in float64; the integer sum is exact there."""
    wz = w.astype(np.float64)
    if zeros is not None:
        wz = wz - zeros.astype(np.float64)
    prod = (q.astype(np.float64) @ wz) * xs.astype(np.float64)[:, None] * scales.astype(np.float64)
    return prod + (0.0 if bias is None else bias.astype(np.float64)), prod


def bound(y, prod):
    """How far the fp16 result may be off: the sum rounded to fp32 and its
    product with s_m (2^-24 each, relative to the product part), one fused
    multiply-add (2^-24 of y), one rounding to fp16 (2^-11 of the rounded
    value, 2^-25 absolute below fp16's normal range).  2^-22 covers the fp32
    steps and their products."""
    return 2.0 ** -11 * np.abs(y) + 2.0 ** -22 * (np.abs(prod) + np.abs(y)) + 2.0 ** -25


def assert_linear(got, y, prod, what=""):
    err = np.abs(got.astype(np.float64) - y)
    worst = float((err / bound(y, prod)).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: worst error / bound {worst:.3f}"


def operands(M, K, N, seed, lead=(), asym=False, bias=False):
    """(q, xs, sums, w, scales, zeros, bias): full-range codes."""
    rng = np.random.default_rng(seed)
    q = rng.integers(-128, 128, (M, K)).astype(np.int8)
    xs = (0.01 + rng.random(M)).astype(np.float32) / 127
    sums = q.sum(axis=1, dtype=np.int64).astype(np.int32)
    w = rng.integers(-128, 128, lead + (K, N)).astype(np.int8)
    scales = ((0.5 + rng.random(lead + (N,))) / 127).astype(np.float16)
    zeros = rng.integers(-128, 128, lead + (N,)).astype(np.int8) if asym else None
    b = rng.normal(0, 1, lead + (N,)).astype(np.float16) if bias else None
    return q, xs, sums, w, scales, zeros, b


def pitched(torch, q):
    """q [M, K] on the GPU with rows on 16-byte boundaries; what lies between
    the rows is not zero."""
    M, K = q.shape
    wide = torch.full((M, (K + 15) // 16 * 16), 77, dtype=torch.int8, device="cuda")
    wide[:, :K] = torch.from_numpy(q).cuda()
    return wide[:, :K]
