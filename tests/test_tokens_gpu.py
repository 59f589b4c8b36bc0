"""Per-token quantization on the GPU: codes, scales and code sums equal the
definition bit for bit; the SwiGLU form within the error of its fp32 steps."""
import numpy as np
import pytest

from tests.gpu_helpers import to_gpu, to_np, w8
from tests.w8a8_helpers import quantize_rows

pytestmark = pytest.mark.gpu


def _check(X, got):
    q, s, sums = (to_np(t) for t in got)
    qo, so, sumo = quantize_rows(X)
    assert np.array_equal(s.view(np.uint32), so.view(np.uint32))
    bad = np.argwhere(q != qo)
    assert bad.size == 0, f"{len(bad)} codes differ, first at {tuple(bad[0])}"
    assert np.array_equal(sums, sumo)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("M,K", [(1, 8), (1, 4096), (7, 24), (9, 504), (8, 512), (65, 520), (33, 1000), (17, 1024),
                                 (3, 2048), (5, 4096), (4, 4104), (2, 8192), (3, 13696), (2, 16384), (2, 16392),
                                 (3, 40000), (1000, 64), (300, 768), (1001, 1032), (700, 4096), (449, 13696),
                                 (601, 16384), (460, 16400)])
def test_codes_scales_sums(M, K, dtype):
    rng = np.random.default_rng(M * 100003 + K)
    X = rng.normal(0, 1, (M, K)) * np.where(rng.random(K) < 0.01, 10, 1)
    _check(X.astype(dtype), w8().quantize_tokens(to_gpu(X.astype(dtype))))


@pytest.mark.parametrize("K", [256, 4096, 20000])
def test_rounding_boundaries(K):
    # halves and their neighbours of every level, for scales that are and are
    # not powers of two
    rng = np.random.default_rng(K)
    rows = []
    for s in (2.0 ** -7, 1.0, 0.1, 3.7e-5, 1.3e7):
        half = (rng.integers(-127, 127, K) + 0.5).astype(np.float32) * np.float32(s)
        step = rng.integers(-2, 3, K)
        for _ in range(2):
            half = np.where(step > 0, np.nextafter(half, np.float32(np.inf)),
                            np.where(step < 0, np.nextafter(half, np.float32(-np.inf)), half))
            step = step - np.sign(step)
        half[0] = np.float32(127) * np.float32(s)
        rows.append(half)
    X = np.stack(rows).astype(np.float32)
    _check(X, w8().quantize_tokens(to_gpu(X)))


def test_fp16_ties():
    # fp16 values at exact halves of the row maximum's 127 steps
    X = np.tile(np.arange(-127, 128, dtype=np.float16) / 2, (4, 5))[:, :1272]
    X[:, 0] = [127, 63.5, 254, 2]
    _check(X, w8().quantize_tokens(to_gpu(X)))


def test_zero_tiny_and_huge_rows():
    rng = np.random.default_rng(3)
    X = rng.normal(0, 1, (8, 1000)).astype(np.float32)
    X[1] = 0
    X[2] *= np.float32(1e-38)      # subnormal scale
    X[3] *= np.float32(1e-42)      # scale of a few units in the last place
    X[4] = 0
    X[4, 17] = np.float32(1e-45)   # scale rounds to zero
    X[5] *= np.float32(1e37)
    X[6, 999] = np.float32(3.4e38)
    X[7] = -0.0
    _check(X, w8().quantize_tokens(to_gpu(X)))
    with np.errstate(over="ignore"):
        H = X.astype(np.float16)
    H[6, 999] = 65504
    finite = [0, 1, 2, 3, 4, 6, 7]   # row 5 is past fp16's range: infinities, outside the contract
    _check(H[finite], [t[finite] for t in w8().quantize_tokens(to_gpu(H))])


def test_a_row_that_is_not_finite_spoils_only_itself():
    rng = np.random.default_rng(4)
    X = rng.normal(0, 1, (9, 520)).astype(np.float16)
    want = quantize_rows(X)
    X[2, 7], X[5, 0] = np.nan, np.inf
    q, s, sums = (to_np(t) for t in w8().quantize_tokens(to_gpu(X)))
    keep = [0, 1, 3, 4, 6, 7, 8]
    assert np.array_equal(q[keep], want[0][keep]) and np.array_equal(s[keep], want[1][keep])
    assert np.array_equal(sums[keep], want[2][keep])


def test_strided_rows_and_given_outputs():
    import torch
    m = w8()
    rng = np.random.default_rng(5)
    for K, lead in ((1000, 8), (4096, 4096)):
        wide = rng.normal(0, 1, (6, K + 2 * lead)).astype(np.float16)
        g = to_gpu(wide)
        _check(wide[:, lead:lead + K], m.quantize_tokens(g[:, lead:lead + K]))
        buf = torch.full((6, K + 40 + (-(K + 40)) % 16), 55, dtype=torch.int8, device="cuda")
        s = torch.full((8,), -1.0, device="cuda")
        c = torch.full((8,), -1, dtype=torch.int32, device="cuda")
        out = m.quantize_tokens(g[::2, lead:lead + K], q=buf[:3, :K], scales=s[:3], sums=c[:3])
        _check(wide[::2, lead:lead + K], out)
        # nothing beside the rows is written
        assert bool((buf[:3, K:] == 55).all()) and bool((buf[3:] == 55).all())
        assert bool((s[3:] == -1).all()) and bool((c[3:] == -1).all())


def test_no_rows():
    import torch
    q, s, sums = w8().quantize_tokens(torch.empty((0, 64), dtype=torch.float16, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,) and sums.shape == (0,)


@pytest.mark.parametrize("M,K", [(1, 8), (5, 264), (3, 512), (16, 1000), (4, 4096), (16, 13696), (2, 16400), (200, 344),
                                 (1001, 1032), (700, 4096), (449, 13696), (450, 16384)])
def test_swiglu(M, K):
    rng = np.random.default_rng(M * 7 + K)
    H = rng.normal(0, 2, (M, 2 * K)).astype(np.float16)
    H[0, 0], H[0, 1], H[0, 2] = -60000, 60000, -20    # exp overflows, underflows
    H[0, K:K + 3] = 1
    if M > 1:
        H[1, :K] = 0                                   # a row of zeros
    q, s, sums = (to_np(t) for t in w8().swiglu_quantize_tokens(to_gpu(H)))
    g, u = H[:, :K].astype(np.float64), H[:, K:].astype(np.float64)
    h = g / (1 + np.exp(np.minimum(-g, 700))) * u
    # fp32 steps: exp within 2^-22 of its value (two units in the last
    # place), the sum, the quotient and the product 2^-24 each: h is within
    # 2^-21; the scale adds its own rounding
    scale = np.abs(h).max(axis=1) / 127
    assert np.all(np.abs(s - scale) <= 2.0 ** -20 * scale)
    # a code is the nearest integer to a quotient within 127 2^-20 of h / s,
    # itself rounded by at most 2^-18 more
    with np.errstate(divide="ignore", invalid="ignore"):
        ratio = np.where(s[:, None] > 0, h / s.astype(np.float64)[:, None], 0)
    assert np.all(np.abs(q - ratio) <= 0.5 + 2.0 ** -12)
    assert np.array_equal(sums, q.sum(axis=1, dtype=np.int64).astype(np.int32))


def test_swiglu_strided_rows():
    rng = np.random.default_rng(8)
    wide = rng.normal(0, 2, (6, 2 * 520 + 16)).astype(np.float16)
    m = w8()
    g = to_gpu(wide)
    a = [to_np(t) for t in m.swiglu_quantize_tokens(g[1::2, 8:8 + 1040])]
    b = [to_np(t) for t in m.swiglu_quantize_tokens(to_gpu(np.ascontiguousarray(wide[1::2, 8:1048])))]
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_refusals():
    import torch
    m = w8()
    X = torch.zeros((4, 64), dtype=torch.float16, device="cuda")
    for bad in (X.cpu(), X[0], X.t(), X.to(torch.bfloat16), X.to(torch.int8)):
        with pytest.raises(ValueError):
            m.quantize_tokens(bad)
    for bad in (X[:, :60], X[:, 4:], torch.zeros((4, 68), dtype=torch.float16, device="cuda")[:, :64]):
        with pytest.raises(m.W8Error):
            m.quantize_tokens(bad)
    with pytest.raises(ValueError):
        m.quantize_tokens(X, q=torch.empty((4, 32), dtype=torch.int8, device="cuda"))
    with pytest.raises(m.W8Error):
        m.quantize_tokens(X, q=torch.empty((4, 72), dtype=torch.int8, device="cuda")[:, :64])
    with pytest.raises(m.W8Error):
        m.quantize_tokens(X, q=X.view(torch.int8)[:, :64])   # inside X
    for bad in (X.float(), X[:, :63]):
        with pytest.raises(ValueError):
            m.swiglu_quantize_tokens(bad)


def test_swiglu_every_gate_value():
    # one row for each finite fp16 gate g: its only product sets the row's
    # scale, which shows h = g / (1 + exp(-g)) u to a unit in the last place.
    # The steps after CUDA's exp (here through torch) are correctly rounded:
    # float64 and one rounding give the same.
    import torch
    g = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.float16)
    g = g[torch.isfinite(g)]
    e = torch.exp(-g.float()).cpu().numpy()
    gate = g.cpu().numpy().astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        silu = (gate / (np.float32(1) + e).astype(np.float64)).astype(np.float32)
    for u in (1.0, 127.0, 0.3):
        H = torch.zeros((g.numel(), 16), dtype=torch.float16, device="cuda")
        H[:, 3] = g
        H[:, 11] = u
        _, s, sums = (to_np(t) for t in w8().swiglu_quantize_tokens(H))
        h = (silu.astype(np.float64) * np.float64(np.float16(u))).astype(np.float32)
        want = (np.abs(h).astype(np.float64) / 127).astype(np.float32)
        assert np.array_equal(s, want)
        assert np.array_equal(np.abs(sums), np.where(want > 0, 127, 0))
