"""Every kernel of the W8A8 linear at the sizes where it can go wrong, each
case with the kernel it is for: 1000 x (1 whole tiles on single SMs, 2
clusters, 3 pairs of SMs) + tokens of a tile."""
import numpy as np
import pytest

from tests.gpu_helpers import to_gpu, to_np, w8
from tests.w8a8_helpers import assert_linear, linear, operands, pitched

pytestmark = pytest.mark.gpu

# Pairs of SMs.  4968 and 4872 channels are 39 blocks of 128, the last of 104
# and of 8 channels: the last pair has one block, which its second SM computes
# too and must not store.  5008 are 40 blocks, the last of 16.  1032 and 1016
# features are 17 and 16 weight tiles, the last of 8 and of 56.
PAIR = [(M, 1032, 4968) for M in (385, 400, 415, 417, 511, 512, 513, 527, 529, 543, 545, 640, 767, 768)]
PAIR += [(M, K, N) for M in (447, 512, 513) for K, N in ((1016, 4872), (1024, 5008), (1032, 4872), (1016, 5120))]
PAIR += [(4000, 104, 7976), (4096, 128, 8064), (400, 13696, 4968), (513, 4040, 4872), (1500, 1032, 8168), (300, 64, 8040)]
# Single SMs: whole tiles where there are many, clusters where there are few.
TILES = [(M, K, 9608, 1000 + t) for M, t in ((1, 16), (16, 16), (17, 32), (32, 32), (33, 64), (64, 64), (65, 128), (127, 128),
                                            (128, 128)) for K in (520, 1032)]
TILES += [(M, 1032, 4968, 1128) for M in (129, 160, 255, 256)] + [(3, 65536, 9608, 1016), (140, 13696, 4968, 1128), (700, 2056, 2104, 1128)]
CLUSTER = [(M, K, N, 2000 + t) for M, t in ((1, 16), (15, 16), (17, 32), (31, 32), (33, 64), (63, 64), (65, 128), (127, 128))
           for K, N in ((2056, 1096), (4040, 4232), (4040, 2184), (13696, 136), (8200, 9096))]
CLUSTER += [(129, 4104, 1032, 2128), (257, 4104, 1032, 2128), (200, 13696, 4096, 2128)]
CASES = [c + (3256,) for c in PAIR] + TILES + CLUSTER

# Groups: all rows in the second of so many groups that the mean one is what the
# kernel is for.
GROUPED = [(M, E, K, N, 3000 + t) for M, E, t in ((1, 1, 128), (17, 1, 128), (31, 1, 128), (33, 1, 128), (63, 1, 128), (65, 1, 128),
                                                 (96, 1, 128), (127, 2, 128), (129, 2, 128), (160, 2, 128), (161, 2, 128),
                                                 (255, 3, 128), (257, 3, 128), (289, 4, 128), (385, 5, 128), (700, 8, 128),
                                                 (97, 1, 256), (129, 1, 256), (255, 1, 256), (257, 1, 256), (287, 1, 256),
                                                 (289, 2, 256), (513, 2, 256))
           for K, N in ((1016, 392), (776, 264)) if M > 16 * E or (M > 4 * E and K < 1024)]
GROUPED += [(M, E, 1032, N, 1000 + t) for M, E, t in ((1, 1, 16), (15, 4, 16), (17, 5, 16), (33, 10, 16), (5, 1, 32), (31, 2, 32),
                                                     (33, 3, 32), (65, 5, 32)) for N in (136, 392)]
GROUPED += [(300, 4, 72, 9608, 3128), (200, 1, 4104, 2440, 3256), (600, 7, 4104, 2440, 3128)]


@pytest.mark.parametrize("M,K,N,kernel", CASES)
def test_kernel(M, K, N, kernel):
    import torch
    m = w8()
    assert m.load_library().w8_test_w8a8_kernel(M, K, N, 0) == kernel
    seed = M + 3 * K + 7 * N
    q, xs, sums, w, scales, zeros, b = operands(M, K, N, seed, asym=seed % 3 == 0, bias=seed % 2 == 0)
    # rows before and behind the outputs, which no tile may touch
    out = torch.full((M + 2, N), 3.5, dtype=torch.float16, device="cuda")
    m.linear_w8a8(pitched(torch, q), to_gpu(xs), to_gpu(sums), m.prepack(to_gpu(w)), to_gpu(scales),
                  bias=None if b is None else to_gpu(b), zeros=None if zeros is None else to_gpu(zeros), out=out[1:M + 1])
    got = to_np(out)
    assert np.all(got[0] == 3.5) and np.all(got[M + 1] == 3.5)
    assert_linear(got[1:M + 1], *linear(q, xs, w, scales, zeros, b))
    assert m.device_status() == 0


@pytest.mark.parametrize("M,E,K,N,kernel", GROUPED)
def test_grouped_kernel(M, E, K, N, kernel):
    import torch
    m = w8()
    assert m.load_library().w8_test_w8a8_kernel(M, K, N, E) == kernel
    seed = M + 3 * K + 7 * N + E
    q, xs, sums, w, scales, zeros, b = operands(M, K, N, seed, lead=(E,), asym=seed % 3 == 0, bias=seed % 2 == 0)
    one = 1 if E > 1 else 0
    at = torch.tensor([0] * (one + 1) + [M] * (E - one), dtype=torch.int32, device="cuda")
    out = torch.full((M + 2, N), 3.5, dtype=torch.float16, device="cuda")
    m.linear_w8a8_grouped(pitched(torch, q), to_gpu(xs), to_gpu(sums), at, torch.stack([m.prepack(to_gpu(e)) for e in w]),
                          to_gpu(scales), bias=None if b is None else to_gpu(b),
                          zeros=None if zeros is None else to_gpu(zeros), out=out[1:M + 1])
    got = to_np(out)
    assert np.all(got[0] == 3.5) and np.all(got[M + 1] == 3.5)
    assert_linear(got[1:M + 1], *linear(q, xs, w[one], scales[one], None if zeros is None else zeros[one],
                                        None if b is None else b[one]))
    assert m.device_status() == 0


EXTREMES = [(-128, -128, 127), (-128, 127, -128), (127, -128, 127), (127, 127, -128)]
K_MAX = 65536


def _extreme(x, w, z, N, runs):
    """Every product at its extreme, at the longest K: no sum wraps.  runs: (M,
    groups, kernel); one weight serves them all."""
    import torch
    m = w8()
    packed = m.prepack(torch.full((K_MAX, N), w, dtype=torch.int8, device="cuda"))
    exact = np.float64(K_MAX * x * (w - z)) * 2.0 ** -28
    for M, groups, kernel in runs:
        assert m.load_library().w8_test_w8a8_kernel(M, K_MAX, N, groups) == kernel
        q = torch.full((M, K_MAX), x, dtype=torch.int8, device="cuda")
        xs = torch.full((M,), 2.0 ** -20, device="cuda")
        sums = torch.full((M,), K_MAX * x, dtype=torch.int32, device="cuda")
        lead = (groups,) if groups else ()
        scales = torch.full(lead + (N,), 2.0 ** -8, dtype=torch.float16, device="cuda")
        zeros = torch.full(lead + (N,), z, dtype=torch.int8, device="cuda")
        if groups:
            at = torch.tensor([M * e // groups for e in range(groups + 1)], dtype=torch.int32, device="cuda")
            y = m.linear_w8a8_grouped(q, xs, sums, at, packed.expand(groups, -1).contiguous(), scales, zeros=zeros)
        else:
            y = m.linear_w8a8(q, xs, sums, packed, scales, zeros=zeros)
        got = to_np(y)
        assert_linear(got, np.full((M, N), exact), np.full((M, N), exact), f"M={M} groups={groups}")
    assert m.device_status() == 0


@pytest.mark.parametrize("x,w,z", EXTREMES)
def test_largest_sums_on_single_sms(x, w, z):
    _extreme(x, w, z, 9608, [(3, 0, 1016), (20, 0, 1032), (40, 0, 1064), (100, 0, 1128)])


@pytest.mark.parametrize("x,w,z", EXTREMES)
def test_largest_sums_on_pairs(x, w, z):
    # (with tiles of 128 tokens at this K only in the grouped form, below)
    _extreme(x, w, z, 4872, [(400, 0, 3256)])


@pytest.mark.parametrize("x,w,z", EXTREMES)
def test_largest_sums_of_groups(x, w, z):
    _extreme(x, w, z, 264, [(7, 2, 1016), (20, 2, 1032), (100, 2, 3128), (300, 2, 3256)])


# The fastest kernel of each as measured when the rule was made; an earlier rule
# took clusters for the first four and pairs with tiles of 128 tokens for the fifth.
@pytest.mark.parametrize("M,K,N,kernel", [(16, 512, 9216, 1016), (64, 512, 9216, 1064), (128, 512, 9216, 1128), (512, 768, 2304, 1128),
                                          (512, 4096, 4096, 1128), (1, 4096, 4096, 2016), (48, 13696, 4096, 2064),
                                          (128, 4096, 4096, 2128), (1, 4096, 27392, 1016), (1024, 4096, 4096, 3256),
                                          (4096, 768, 2304, 3256), (2048, 4096, 27392, 3256)])
def test_choice(M, K, N, kernel):
    assert w8().load_library().w8_test_w8a8_kernel(M, K, N, 0) == kernel
