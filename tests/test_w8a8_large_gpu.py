"""Int8-activation operators on tensors whose offsets pass 32 bits: rows on
both sides of 2^31 elements against 64-bit sums on the GPU."""
import pytest

from tests.gpu_helpers import w8

pytestmark = pytest.mark.gpu


def _rows(M, row_elements):
    """The first and last rows and those around 2^31 and 2^32 elements."""
    near = {0, 1, M - 2, M - 1}
    for e in (2 ** 31, 2 ** 32):
        near |= {r for r in (e // row_elements - 1, e // row_elements, e // row_elements + 1) if 0 <= r < M}
    return sorted(near)


def _check(Y, rows, q, xs, w, scales):
    """Y[r] against the sum in float64 (exact: |sum| < 2^53), within the bound
    of its roundings: 2^-11 of y for fp16, 2^-22 for the fp32 steps."""
    import torch
    acc = q[rows].double() @ w.double()
    y = acc * xs[rows].double()[:, None] * scales.double()
    err = (Y[rows].double() - y).abs()
    assert bool((err <= 2.0 ** -11 * y.abs() + 2.0 ** -21 * y.abs() + 2.0 ** -25).all())


@pytest.mark.parametrize("op", ["plain", "swiglu"])
def test_tokens(op):
    import torch
    m = w8()
    M, K = 140000, 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    f = m.quantize_tokens if op == "plain" else m.swiglu_quantize_tokens
    X = torch.empty((M, K), dtype=torch.float16, device="cuda").normal_(generator=g)
    q, s, sums = f(X)
    rows = _rows(M, K)
    one = [f(X[r:r + 1]) for r in rows]        # the same rows, alone
    assert torch.equal(q[rows], torch.cat([o[0] for o in one]))
    assert torch.equal(s[rows], torch.cat([o[1] for o in one])) and torch.equal(sums[rows], torch.cat([o[2] for o in one]))
    assert torch.equal(sums, q.sum(1, dtype=torch.int64).to(torch.int32))


@pytest.mark.parametrize("M,N,grouped", [(140000, 16384, False), (140000, 16384, True), (2400, 1 << 20, False),
                                         (2100, 1 << 20, True)])
def test_outputs(M, N, grouped):
    import torch
    m = w8()
    K = 64
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (K, N), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand((M,), generator=g, device="cuda") / 127
    scales = torch.rand((N,), generator=g, device="cuda").half()
    sums = q.sum(1, dtype=torch.int64).to(torch.int32)
    packed = m.prepack(w)
    if grouped:
        at = torch.tensor([0, M // 3, M], dtype=torch.int32, device="cuda")
        Y = m.linear_w8a8_grouped(q, xs, sums, at, packed.expand(2, -1).contiguous(), scales.expand(2, -1).contiguous())
    else:
        Y = m.linear_w8a8(q, xs, sums, packed, scales)
    _check(Y, _rows(M, N), q, xs, w, scales)
    assert m.device_status() == 0


@pytest.mark.parametrize("T", [40, 400, 4000])
def test_weights(T):
    # 40 experts of 8192 x 16384: 5.4 GB of packed weights
    import torch
    m = w8()
    E, K, N = 40, 8192, 16384
    g = torch.Generator(device="cuda").manual_seed(T)
    w = [torch.randint(-128, 128, (K, N), generator=g, device="cuda", dtype=torch.int8) for _ in range(E)]
    packed = torch.stack([m.prepack(e) for e in w])
    q = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.rand((T,), generator=g, device="cuda") / 127
    scales = torch.rand((E, N), generator=g, device="cuda").half() / 64
    at = torch.arange(E + 1, device="cuda") * T // E
    Y = m.linear_w8a8_grouped(q, xs, q.sum(1, dtype=torch.int64).to(torch.int32), at.to(torch.int32), packed, scales)
    for e in (0, 14, 15, 16, 30, 31, 32, 33, E - 1):
        rows = torch.arange(int(at[e]), int(at[e + 1]), device="cuda")
        _check(Y, rows, q, xs, w[e], scales[e])
    # one weight past 2^32 bytes: 65536 x 65664
    if T == 40:
        del w, packed, Y
        K, N = 65536, 65664
        w = torch.randint(-128, 128, (K, N), generator=g, device="cuda", dtype=torch.int8)
        q = torch.randint(-128, 128, (3, K), generator=g, device="cuda", dtype=torch.int8)
        scales = torch.rand((N,), generator=g, device="cuda").half() / 64
        Y = m.linear_w8a8(q, xs[:3].clone(), q.sum(1, dtype=torch.int64).to(torch.int32), m.prepack(w), scales)
        for n0 in (0, 32768, N - 128):     # the last of them lie past 2^32 bytes
            c = slice(n0, n0 + 128)
            _check(Y[:, c], [0, 1, 2], q, xs, w[:, c], scales[c])
    assert m.device_status() == 0
