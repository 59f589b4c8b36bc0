"""The W8A8 linear and its grouped form on the GPU against exact sums."""
import numpy as np
import pytest

from tests.gpu_helpers import SEED, to_gpu, to_np, w8
from tests.w8a8_helpers import assert_linear, linear, operands, pitched

pytestmark = pytest.mark.gpu


def _gpu(a):
    return None if a is None else to_gpu(a)


def _run(ops):
    import torch
    m = w8()
    q, xs, sums, w, scales, zeros, b = ops
    return m.linear_w8a8(pitched(torch, q), _gpu(xs), _gpu(sums), m.prepack(_gpu(w)), _gpu(scales), bias=_gpu(b),
                         zeros=_gpu(zeros))


def _check(ops, got, what=""):
    q, xs, _, w, scales, zeros, b = ops
    y, prod = linear(q, xs, w, scales, zeros, b)
    assert_linear(to_np(got), y, prod, what)


SHAPES = [(8, 8), (64, 128), (72, 136), (256, 512), (1000, 264), (4096, 384), (13696, 136), (640, 2048)]


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 200, 256, 257, 300, 513, 1100])
@pytest.mark.parametrize("K,N", SHAPES)
def test_linear(M, K, N):
    asym, bias = (M + K) % 3 == 0, M % 2 == 1
    ops = operands(M, K, N, M * 31 + K + N, asym=asym, bias=bias)
    _check(ops, _run(ops), f"M={M} K={K} N={N}")


@pytest.mark.parametrize("M,K,N", [(1, 4096, 27392), (16, 13696, 4096), (100, 4096, 4608), (4096, 768, 2304)])
def test_linear_full_sizes(M, K, N):
    ops = operands(M, K, N, M + K + N, asym=True, bias=True)
    _check(ops, _run(ops), f"M={M} K={K} N={N}")


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("x,w,z", [(-128, -128, 127), (-128, 127, -128), (127, -128, 127), (127, 127, -128)])
def test_largest_sums(M, x, w, z):
    # the longest allowed K with every product at its extreme: no sum wraps
    K, N = 65536, 8
    q = np.full((M, K), x, np.int8)
    ops = (q, np.full(M, 2.0 ** -20, np.float32), q.sum(1, dtype=np.int64).astype(np.int32), np.full((K, N), w, np.int8),
           np.full(N, 2.0 ** -8, np.float16), np.full(N, z, np.int8), None)
    _check(ops, _run(ops))


@pytest.mark.parametrize("M", [5, 40, 100, 300])
def test_small_integers_are_exact(M):
    rng = np.random.default_rng(M)
    K, N = 520, 136
    q = rng.integers(-1, 2, (M, K)).astype(np.int8)
    w = rng.integers(-1, 2, (K, N)).astype(np.int8)
    ops = (q, np.ones(M, np.float32), q.sum(1, dtype=np.int32), w, np.ones(N, np.float16), None, None)
    got = to_np(_run(ops)).astype(np.int64)
    assert np.array_equal(got, q.astype(np.int64) @ w.astype(np.int64))


def test_zero_scales_give_the_bias():
    ops = list(operands(40, 256, 136, 9, bias=True))
    ops[1] = np.zeros(40, np.float32)
    assert np.array_equal(to_np(_run(ops)), np.tile(ops[6], (40, 1)))


def test_from_quantized_weights_and_tokens():
    # the whole path from fp weights and activations, both code forms
    import synthetic
    m = w8()
    K, N = 1000, 264
    W = synthetic.weights(K, N, SEED, 7000, outlier_frac=0.001)
    X = synthetic.activations(70, K, SEED, 7001)
    xq, xs, sums = m.quantize_tokens(to_gpu(X))
    q, s = m.quantize(to_gpu(W))
    y, prod = linear(to_np(xq), to_np(xs), to_np(q), to_np(s))
    assert_linear(to_np(m.linear_w8a8(xq, xs, sums, m.prepack(q), s)), y, prod)
    qa, sa, za = m.quantize_asym(to_gpu(W))
    y, prod = linear(to_np(xq), to_np(xs), to_np(qa), to_np(sa), to_np(za))
    got = to_np(m.linear_w8a8(xq, xs, sums, m.prepack(qa), sa, zeros=za))
    assert_linear(got, y, prod)
    # and it is the product: each activation is off by at most half its step
    # and each weight by at most half its own (plus the rounding of the scale
    # and the zero point), so the sum over K is off by less than this
    ref = X.astype(np.float64) @ W.astype(np.float64)
    ax, aw = np.abs(X).astype(np.float64), np.abs(W).astype(np.float64)
    ex, ew = 0.501 * to_np(xs).astype(np.float64)[:, None], 0.51 * to_np(sa).astype(np.float64)
    off = ax.sum(1)[:, None] * ew + ex * aw.sum(0) + K * ex * ew + 2.0 ** -10 * np.abs(ref) + 1e-3
    assert np.all(np.abs(got - ref) <= off)
    layer = m.W8A8Linear(to_gpu(W))
    assert np.array_equal(to_np(layer(to_gpu(X))), to_np(m.linear_w8a8(xq, xs, sums, layer.packed, layer.scales)))


def test_calls_in_turn_with_the_w8a16_linear():
    # the kernels of both activation widths follow one another on one stream,
    # each launched while the one before ends; every call twice
    import torch
    m = w8()
    for M, K, N in [(1, 4096, 384), (20, 13696, 136), (300, 1000, 2048), (4, 4096, 4096), (129, 2048, 384)]:
        ops = operands(M, K, N, M, bias=True)
        first = to_np(_run(ops))
        X = torch.randn((M, K), device="cuda").half()
        packed, scales = m.prepack(_gpu(ops[3])), _gpu(ops[4])
        a = to_np(m.linear(X, packed, scales))
        assert np.array_equal(first, to_np(_run(ops)))
        assert np.array_equal(a, to_np(m.linear(X, packed, scales)))
        _check(ops, torch.from_numpy(first).cuda())
    assert m.device_status() == 0


def test_pitched_codes_slice():
    # codes that are a slice of a wider buffer
    import torch
    m = w8()
    ops = operands(50, 512, 136, 11)
    wide = torch.full((50, 1024), 99, dtype=torch.int8, device="cuda")
    wide[:, 256:768] = _gpu(ops[0])
    got = m.linear_w8a8(wide[:, 256:768], _gpu(ops[1]), _gpu(ops[2]), m.prepack(_gpu(ops[3])), _gpu(ops[4]))
    _check(ops, got)


# ---------------------------------------------------------------- groups
def _grouped(counts, K, N, seed, before=0, behind=0, asym=False, bias=False):
    """Runs a grouped call and checks every row of Y."""
    import torch
    m = w8()
    E, M = len(counts), before + sum(counts) + behind
    q, xs, sums, w, scales, zeros, b = operands(M, K, N, seed, lead=(E,), asym=asym, bias=bias)
    offsets = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    packed = torch.stack([m.prepack(_gpu(w[e])) for e in range(E)])
    out = torch.full((M, N), 3.5, dtype=torch.float16, device="cuda")
    got = to_np(m.linear_w8a8_grouped(pitched(torch, q), _gpu(xs), _gpu(sums), _gpu(offsets), packed, _gpu(scales),
                                      bias=_gpu(b), zeros=_gpu(zeros), out=out))
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        y, prod = linear(q[r], xs[r], w[e], scales[e], None if zeros is None else zeros[e], None if b is None else b[e])
        assert_linear(got[r], y, prod, f"group {e} of {E}")
    assert np.all(got[:offsets[0]] == 3.5) and np.all(got[offsets[-1]:] == 3.5)
    assert m.device_status() == 0


@pytest.mark.parametrize("counts", [
    [1], [0, 5], [5, 0], [0, 0, 3, 0, 0], [1, 1, 1, 1], [16, 17, 15, 0, 1], [128, 129, 127], [3, 500, 0, 40],
    [256, 255, 257, 64], [0, 0, 0], [700, 1, 0, 1, 2], [32] * 16, [2, 0] * 20])
@pytest.mark.parametrize("K,N", [(64, 128), (264, 392), (1000, 136), (2048, 1024)])
def test_grouped(counts, K, N):
    if sum(counts) == 0:
        _grouped(counts, K, N, 5, behind=40)
        return
    n = len(counts) + sum(counts)
    _grouped(counts, K, N, n + K, before=n % 3, behind=(n % 5) * 7, asym=n % 2 == 0, bias=n % 3 == 0)


@pytest.mark.parametrize("mean", [4, 5, 16, 17, 96, 97])
def test_grouped_kernel_borders(mean):
    # mean groups on both sides of each border, one group with most of the rows
    for counts in ([mean] * 3, [0, 3 * mean - 1, 1], [3 * mean, 0, 0]):
        _grouped(counts, 1032, 264, mean, asym=mean % 2 == 0, bias=True)


def test_grouped_many_groups():
    rng = np.random.default_rng(1)
    _grouped(list(rng.integers(0, 4, 1024)), 64, 128, 21, behind=3, bias=True)
    _grouped([0] * 1023 + [9], 72, 136, 22)


def test_grouped_no_rows():
    import torch
    m = w8()
    out = m.linear_w8a8_grouped(torch.empty((0, 64), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"),
                                torch.empty(0, dtype=torch.int32, device="cuda"),
                                torch.zeros(3, dtype=torch.int32, device="cuda"),
                                torch.zeros((2, 8192), dtype=torch.uint8, device="cuda"),
                                torch.zeros((2, 128), dtype=torch.float16, device="cuda"))
    assert out.shape == (0, 128)


def test_grouped_equals_the_linear_of_each_group():
    import torch
    m = w8()
    q, xs, sums, w, scales, _, b = operands(300, 1000, 264, 33, lead=(3,), bias=True)
    packed = torch.stack([m.prepack(_gpu(w[e])) for e in range(3)])
    g = [pitched(torch, q), _gpu(xs), _gpu(sums)]
    at = [0, 90, 110, 300]
    Y = m.linear_w8a8_grouped(*g, _gpu(np.array(at, np.int32)), packed, _gpu(scales), bias=_gpu(b))
    for e in range(3):
        r = slice(at[e], at[e + 1])
        # scales and sums of a group start anywhere: copies on 16-byte boundaries
        one = m.linear_w8a8(g[0][r], g[1][r].clone(), g[2][r].clone(), packed[e], _gpu(scales[e]), bias=_gpu(b[e]))
        assert np.array_equal(to_np(Y[r]), to_np(one))


def test_offsets_outside_the_rows_are_clamped():
    # the kernel takes every offset into [0, M]; a group that ends before it
    # begins is empty
    import torch
    m = w8()
    M, K, N = 40, 264, 136
    q, xs, sums, w, scales, _, _ = operands(M, K, N, 44, lead=(3,))
    packed = torch.stack([m.prepack(_gpu(w[e])) for e in range(3)])
    for at, groups in (([-5, 10, 10, 400], {0: (0, 10), 2: (10, 40)}), ([2, 30, 20, 20], {0: (2, 30)}),
                       ([50, 60, -1, 5], {2: (0, 5)})):
        out = torch.full((M, N), 3.5, dtype=torch.float16, device="cuda")
        got = to_np(m.linear_w8a8_grouped(pitched(torch, q), _gpu(xs), _gpu(sums), _gpu(np.array(at, np.int32)), packed,
                                          _gpu(scales), out=out))
        left = np.ones(M, bool)
        for e, (a, b) in groups.items():
            y, prod = linear(q[a:b], xs[a:b], w[e], scales[e])
            assert_linear(got[a:b], y, prod)
            left[a:b] = False
        assert np.all(got[left] == 3.5)
    assert m.device_status() == 0


# ---------------------------------------------------------------- streams, graphs, the path together
def test_gated_mlp_of_experts_in_a_graph():
    """quantize -> grouped gate/up -> SwiGLU + quantize -> grouped down, eagerly,
    on another stream, and captured and replayed on changed inputs."""
    import torch
    m = w8()
    E, K, F, T = 4, 512, 344, 150
    rng = np.random.default_rng(6)
    W1 = [m.quantize(to_gpu(rng.normal(0, 0.02, (K, 2 * F)).astype(np.float32))) for _ in range(E)]
    W2 = [m.quantize(to_gpu(rng.normal(0, 0.02, (F, K)).astype(np.float32))) for _ in range(E)]
    p1, s1 = torch.stack([m.prepack(q) for q, _ in W1]), torch.stack([s for _, s in W1])
    p2, s2 = torch.stack([m.prepack(q) for q, _ in W2]), torch.stack([s for _, s in W2])
    X = to_gpu(rng.normal(0, 1, (T, K)).astype(np.float16))
    offsets = to_gpu(np.array([0, 60, 60, 149, 150], np.int32))

    def mlp():
        xq, xs, sums = m.quantize_tokens(X)
        H = m.linear_w8a8_grouped(xq, xs, sums, offsets, p1, s1)
        hq, hs, hsums = m.swiglu_quantize_tokens(H)
        return H, hq, hs, m.linear_w8a8_grouped(hq, hs, hsums, offsets, p2, s2)

    def check(out):
        H, hq, hs, Y = (to_np(t) for t in out)
        x, at = to_np(X), to_np(offsets)
        xq, xs, _ = __import__("tests.w8a8_helpers", fromlist=["x"]).quantize_rows(x)
        for e in range(E):
            r = slice(at[e], at[e + 1])
            assert_linear(H[r], *linear(xq[r], xs[r], to_np(W1[e][0]), to_np(W1[e][1])))
            assert_linear(Y[r], *linear(hq[r], hs[r], to_np(W2[e][0]), to_np(W2[e][1])))

    check(mlp())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = mlp()
    torch.cuda.current_stream().wait_stream(side)
    check(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = mlp()
    for seed in range(3):
        X.copy_(torch.from_numpy(np.random.default_rng(seed).normal(0, 1, (T, K)).astype(np.float16)))
        cut = sorted(np.random.default_rng(seed).integers(0, T + 1, E - 1).tolist())
        offsets.copy_(torch.tensor([0] + cut + [T], dtype=torch.int32))
        graph.replay()
        check(captured)
    assert m.device_status() == 0


def test_two_graphs_replayed_at_once():
    # no call keeps scratch: replays of two graphs may overlap on the GPU
    import torch
    m = w8()
    ops = [operands(9, 4096, 4096, s, bias=True) for s in (1, 2)]
    args = [(pitched(torch, o[0]), _gpu(o[1]), _gpu(o[2]), m.prepack(_gpu(o[3])), _gpu(o[4]), _gpu(o[6])) for o in ops]
    graphs, outs = [], []
    for a in args:
        m.linear_w8a8(*a)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(20):
                y = m.linear_w8a8(*a)
        graphs.append(g)
        outs.append(y)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, y in zip(ops, outs):
        _check(o, y)
    assert m.device_status() == 0


def test_refusals():
    import torch
    m = w8()
    q, xs, sums, w, scales, zeros, b = (_gpu(a) for a in operands(20, 128, 136, 1, asym=True, bias=True))
    packed = m.prepack(w)
    good = dict(q=q, x_scales=xs, x_sums=sums, packed=packed, scales=scales, bias=b, zeros=zeros)
    m.linear_w8a8(**good)
    for name, bad in [("q", q.cpu()), ("q", q.half()), ("q", q.t()), ("x_scales", xs[:19]), ("x_scales", xs.double()),
                      ("x_sums", sums.long()), ("packed", packed[:-1]), ("packed", packed.view(torch.int8)),
                      ("scales", scales.float()), ("bias", b.float()), ("bias", b[:128]), ("zeros", zeros.int()),
                      ("scales", scales.cpu()), ("x_scales", torch.zeros((20, 2), device="cuda")[:, 0])]:
        with pytest.raises(ValueError):
            m.linear_w8a8(**{**good, name: bad})
    with pytest.raises(ValueError):
        m.linear_w8a8(**good, out=torch.empty((20, 128), dtype=torch.float16, device="cuda"))
    with pytest.raises(m.W8Error):   # rows not on 16-byte boundaries
        m.linear_w8a8(**{**good, "q": torch.zeros((20, 136), dtype=torch.int8, device="cuda")[:, :128]})
    offsets = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    grouped = dict(good, packed=packed[None], scales=scales[None], bias=b[None], zeros=zeros[None], offsets=offsets)
    m.linear_w8a8_grouped(**grouped)
    for name, bad in [("offsets", offsets.long()), ("offsets", offsets[:1]), ("offsets", offsets.cpu()),
                      ("scales", scales), ("packed", packed), ("bias", b), ("zeros", zeros)]:
        with pytest.raises(ValueError):
            m.linear_w8a8_grouped(**{**grouped, name: bad})


def _log_size(rng, lo, hi, step=1):
    return max(step, int(round(np.exp(rng.uniform(np.log(lo), np.log(hi))) / step)) * step)


@pytest.mark.parametrize("seed", range(48))
def test_linear_random_sizes(seed):
    # every kernel and the borders between them
    rng = np.random.default_rng(1000 + seed)
    while True:
        M, K, N = _log_size(rng, 1, 3000), _log_size(rng, 8, 9000, 8), _log_size(rng, 8, 24000, 8)
        if M * K * N <= 3e9:
            break
    ops = operands(M, K, N, seed, asym=bool(rng.integers(2)), bias=bool(rng.integers(2)))
    _check(ops, _run(ops), f"M={M} K={K} N={N}")


@pytest.mark.parametrize("seed", range(24))
def test_grouped_random_sizes(seed):
    rng = np.random.default_rng(2000 + seed)
    E, K, N = _log_size(rng, 1, 40), _log_size(rng, 8, 2000, 8), _log_size(rng, 8, 3000, 8)
    most = max(1, int(min(1500, 2e9 / (K * N))))
    share = rng.dirichlet(np.full(E, 0.5))
    counts = rng.multinomial(rng.integers(1, most + 1), share).tolist()
    _grouped(counts, K, N, seed, before=int(rng.integers(0, 4)), behind=int(rng.integers(0, 300)),
             asym=bool(rng.integers(2)), bias=bool(rng.integers(2)))


def test_two_streams_at_once():
    # calls of every kernel, eagerly on two streams that overlap on the GPU
    import torch
    m = w8()
    shapes = [(1, 4096, 4096), (40, 1024, 16384), (200, 4096, 1024), (700, 1024, 4096), (5, 13696, 1024)]
    ops = [operands(M, K, N, i) for i, (M, K, N) in enumerate(shapes)]
    args = [(pitched(torch, o[0]), _gpu(o[1]), _gpu(o[2]), m.prepack(_gpu(o[3])), _gpu(o[4])) for o in ops]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for turn in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append([m.linear_w8a8(*a) for a in args])
    torch.cuda.synchronize()
    first = [to_np(y) for y in outs[0]]
    for y, o in zip(outs[0], ops):
        _check(o, y)
    for got in outs[1:]:
        assert all(np.array_equal(to_np(y), f) for y, f in zip(got, first))
    assert m.device_status() == 0
