"""The committed ncu traffic belongs to the W8A16 kernels as they stand: the
bench line reports it only while their sources are unchanged, so a change that
is not theirs must not touch those sources."""
import pytest

import bench

KERNELS = {"decode_kernel": "decode.cuh", "prefill2_kernel": "prefill2.cuh", "quantize_kernel": "quantize.cuh"}


@pytest.mark.parametrize("kernel", sorted(KERNELS))
def test_bench_line_has_its_traffic(kernel):
    traffic = bench.measured_traffic(kernel, [KERNELS[kernel], "common.cuh"])
    assert traffic is not None and traffic > 1e8
