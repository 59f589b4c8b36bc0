"""Rows with NaN or infinities through the per-token quantizers and the W8A8
linears: they stay visible, and only in their own rows."""
import numpy as np
import pytest

from tests.gpu_helpers import to_gpu, to_np, w8
from tests.w8a8_helpers import operands, quantize_rows

pytestmark = pytest.mark.gpu


def _definition(x):
    """Codes, scales and sums: NaN rows have a NaN scale and codes of 0, rows
    with infinities an infinite scale and codes of 127 sign(x) for those."""
    x = np.asarray(x, dtype=np.float64)
    nan, inf = np.isnan(x).any(axis=1), np.isinf(x).any(axis=1)
    q, s, sums = quantize_rows(np.where((nan | inf)[:, None], 0.0, x))
    q[inf] = np.where(np.isinf(x[inf]), 127 * np.sign(x[inf]), 0)
    q[nan] = 0
    s[inf] = np.inf
    s[nan] = np.nan
    return q, s, q.sum(axis=1, dtype=np.int32)


def _same(x, got):
    q, s, sums = (to_np(t) for t in got)
    qo, so, sumo = _definition(x)
    assert np.array_equal(s, so, equal_nan=True)
    assert np.array_equal(q, qo) and np.array_equal(sums, sumo)


def _spoil(X, rng):
    """NaN, +inf, -inf, both infinities, and NaN beside infinity, at the first,
    the last and a random place; a row of NaN and a row of infinities alone."""
    M, K = X.shape
    plans = [[(0, np.nan)], [(K - 1, np.nan)], [(0, np.inf)], [(K - 1, -np.inf)], [(1, np.inf), (K - 2, -np.inf)],
             [(0, np.inf), (K - 1, np.nan)], [(int(rng.integers(K)), np.nan)], [(int(rng.integers(K)), -np.inf)]]
    rows = rng.permutation(M)
    for r, plan in zip(rows, plans):
        for k, v in plan:
            X[r, k] = v
    if M > len(plans) + 4:
        X[rows[-1]] = np.nan
        X[rows[-2]] = np.inf
        X[rows[-3]] = -np.inf
        X[rows[-4]] = 0
        X[rows[-4], K // 2] = np.nan
    return X


# every width of block and number of values a thread, and rows read twice
SIZES = [(1, 8), (9, 256), (20, 1024), (1000, 1024), (40, 4096), (40, 8192), (30, 13696), (20, 20000), (700, 2048),
         (700, 6144), (620, 10000), (620, 16384)]


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("M,K", SIZES)
def test_quantize(M, K, dtype):
    rng = np.random.default_rng(M + K)
    X = _spoil(rng.normal(0, 1, (M, K)).astype(dtype), rng)
    _same(X, w8().quantize_tokens(to_gpu(X)))


def test_finite_values_beside_an_infinity_have_code_zero():
    # up to the largest finite one
    X = np.full((2, 64), np.finfo(np.float32).max, np.float32)
    X[0, 5], X[1, 5] = np.inf, -np.inf
    X[:, 6:20] *= -1
    _same(X, w8().quantize_tokens(to_gpu(X)))


@pytest.mark.parametrize("M,K", [(M, K) for M, K in SIZES if (M, K) != (20, 20000)] + [(1000, 13696), (3, 16392)])
def test_swiglu(M, K):
    rng = np.random.default_rng(M * 3 + K)
    H = rng.normal(0, 2, (M, 2 * K)).astype(np.float16)
    H[:, :K] = np.where(H[:, :K] == 0, 1, H[:, :K])
    G, U = H[:, :K], H[:, K:]
    nan, inf, plus = [], [], []
    rows = list(rng.permutation(M))
    for r, (half, k, v) in zip(rows, [(G, 0, np.nan), (U, K - 1, np.nan), (G, K - 1, np.inf), (G, 3, -np.inf),
                                      (U, 0, np.inf), (U, 5, -np.inf), (G, int(rng.integers(K)), np.inf)]):
        half[r, k] = v
        other = (U if half is G else G)[r, k]
        if np.isnan(v) or (half is G and v == -np.inf) or other == 0:
            nan.append(r)
        else:
            inf.append(r)
            plus.append((k, v * other > 0))
    q, s, sums = (to_np(t) for t in w8().swiglu_quantize_tokens(to_gpu(H)))
    assert np.all(np.isnan(s[nan])) and np.all(q[nan] == 0) and np.all(sums[nan] == 0)
    assert np.all(np.isposinf(s[inf]))
    for r, (k, up) in zip(inf, plus):
        expect = np.zeros(K, np.int8)
        expect[k] = 127 if up else -127
        assert np.array_equal(q[r], expect) and sums[r] == expect[k]
    keep = np.setdiff1d(np.arange(M), nan + inf)
    assert np.all(np.isfinite(s[keep]))


@pytest.mark.parametrize("M,K,N", [(6, 1024, 136), (60, 512, 264), (200, 1032, 136), (600, 1032, 4200), (20, 256, 16384)])
def test_outputs_of_such_rows_are_not_finite(M, K, N):
    import torch
    m = w8()
    rng = np.random.default_rng(M)
    X = rng.normal(0, 1, (M, K)).astype(np.float16)
    _, _, _, w, scales, zeros, b = operands(M, K, N, M, asym=True, bias=True)
    packed = m.prepack(to_gpu(w))
    tail = dict(bias=to_gpu(b), zeros=to_gpu(zeros))
    xq, xs, sums = m.quantize_tokens(to_gpu(X))
    clean = to_np(m.linear_w8a8(xq, xs, sums, packed, to_gpu(scales), **tail))
    X[1, 7], X[3, K - 1], X[5, 0] = np.nan, np.inf, -np.inf
    xq, xs, sums = m.quantize_tokens(to_gpu(X))
    dense = to_np(m.linear_w8a8(xq, xs, sums, packed, to_gpu(scales), **tail))
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    grouped = to_np(m.linear_w8a8_grouped(xq, xs, sums, offsets, packed[None], to_gpu(scales)[None], bias=tail["bias"][None],
                                          zeros=tail["zeros"][None]))
    keep = np.setdiff1d(np.arange(M), [1, 3, 5])
    for Y in (dense, grouped):
        assert np.all(np.isnan(Y[1])) and not np.any(np.isfinite(Y[[3, 5]]))
        assert np.array_equal(Y[keep], clean[keep])
