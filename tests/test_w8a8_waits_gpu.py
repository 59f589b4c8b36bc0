"""The bounded waits of the W8A8 kernels: their second begins when the kernel
before has ended, and one that runs out leaves the outputs as they were."""
import pytest

from tests.gpu_helpers import to_gpu, to_np, w8
from tests.w8a8_helpers import assert_linear, linear, operands, pitched

pytestmark = pytest.mark.gpu

LONG_NS = 1_300_000_000     # more than a wait's one second


# (M, K, N, groups): clusters, whole tiles on single SMs with few and many
# tokens, pairs of SMs, and the groups' kernels
@pytest.mark.parametrize("M,K,N,E", [(3, 4096, 256, 0), (100, 4096, 1024, 0), (5, 256, 16384, 0), (140, 1032, 4968, 0),
                                     (520, 1032, 4968, 0), (6, 1024, 264, 3), (40, 1024, 264, 2), (300, 520, 264, 2)])
def test_a_long_kernel_before_does_not_use_up_the_wait(M, K, N, E):
    import torch
    m = w8()
    q, xs, sums, w, scales, zeros, b = operands(M, K, N, M + N, lead=(E,) if E else (), asym=True, bias=True)
    args = [pitched(torch, q), to_gpu(xs), to_gpu(sums)]
    tail = dict(bias=to_gpu(b), zeros=to_gpu(zeros), out=torch.full((M, N), 3.5, dtype=torch.float16, device="cuda"))
    if E:
        at = [M * e // E for e in range(E + 1)]
        args += [torch.tensor(at, dtype=torch.int32, device="cuda"),
                 torch.stack([m.prepack(to_gpu(w[e])) for e in range(E)]), to_gpu(scales)]
        f = m.linear_w8a8_grouped
    else:
        args += [m.prepack(to_gpu(w)), to_gpu(scales)]
        f = m.linear_w8a8
    f(*args, **tail)
    first = to_np(tail["out"])
    tail["out"].fill_(3.5)
    assert m.device_status() == 0
    m.test_bounded_wait(LONG_NS)
    got = f(*args, **tail)
    # the one wait that ran out is that of the kernel before
    assert (m.device_status() >> 8) & 0xFF == 0xEE
    assert (to_np(got) == first).all()
    for e in range(max(E, 1)):
        r = slice(at[e], at[e + 1]) if E else slice(0, M)
        i = e if E else ()
        assert_linear(first[r], *linear(q[r], xs[r], w[i], scales[i], zeros[i], b[i]))


# clusters of 8, 4 and 2 blocks; the last with two token tiles
@pytest.mark.parametrize("M,K,N", [(3, 4096, 256), (100, 1024, 1032), (20, 512, 4096), (150, 2048, 1024)])
def test_a_cluster_that_gives_up_stores_nothing(M, K, N):
    import torch
    m = w8()
    lib = m.load_library()
    q, xs, sums, w, scales, _, _ = operands(M, K, N, M + N)
    a = [pitched(torch, q), to_gpu(xs), to_gpu(sums), m.prepack(to_gpu(w)), to_gpu(scales)]
    out = torch.full((M, N), 3.5, dtype=torch.float16, device="cuda")
    assert m.device_status() == 0
    m._call(lib.w8_test_w8a8_cluster_stall, "w8_test_w8a8_cluster_stall", out.device, m._raw_stream(out.device),
            a[0].data_ptr(), a[0].stride(0), *[t.data_ptr() for t in a[1:]], out.data_ptr(), M, K, N)
    status = m.device_status()
    assert status & 1 and 0x60 <= (status >> 8) & 0xFF <= 0x64
    assert bool((out == 3.5).all())
    # the GPU and the next call are as before
    got = to_np(m.linear_w8a8(*a, out=out))
    assert_linear(got, *linear(q, xs, w, scales))
    assert m.device_status() == 0


def test_the_stalled_form_needs_clusters():
    import torch
    m = w8()
    lib = m.load_library()
    for M, K, N in ((3, 192, 256), (3, 4096, 27392)):
        q, xs, sums = torch.zeros((M, K), dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda")
        packed = torch.zeros(m.prepacked_bytes(K, N), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(N, dtype=torch.float16, device="cuda")
        out = torch.empty((M, N), dtype=torch.float16, device="cuda")
        with pytest.raises(m.W8Error):
            m._call(lib.w8_test_w8a8_cluster_stall, "w8_test_w8a8_cluster_stall", out.device, m._raw_stream(out.device),
                    q.data_ptr(), K, xs.data_ptr(), sums.data_ptr(), packed.data_ptr(), scales.data_ptr(), out.data_ptr(),
                    M, K, N)
