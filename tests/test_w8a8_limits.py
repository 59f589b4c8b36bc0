"""Sizes at which a row's code sum would leave 32 bits are refused on the host
(no GPU needed; no call here gets past its arguments)."""
import ctypes

import pytest

A, B, C, D = (ctypes.c_void_p(0x1000000000 * i) for i in range(1, 5))
UNALIGNED = ctypes.c_void_p(0x1000000008)
MOST = (2 ** 31 - 1) // 127 // 8 * 8      # 16909320


def test_longest_row_of_the_quantizers(w8lib):
    assert 127 * MOST < 2 ** 31 <= 127 * (MOST + 8)
    for K, status in ((MOST, -3), (MOST + 8, -2), (2 ** 30 - 8, -2), (2 ** 62, -2), (2 ** 63 - 8, -2)):
        wide = min(2 * K, 2 ** 40)
        assert w8lib.w8_quantize_per_token(UNALIGNED, 1, wide, 1, K, B, wide, C, D, None) == status, K
        assert w8lib.w8_swiglu_quantize_per_token(UNALIGNED, wide, 1, K, B, wide, C, D, None) == status, K


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
def test_the_longest_row_sums_exactly(sign):
    import torch
    import int8_weight_only_b200 as m
    X = torch.full((1, MOST), 2.5 * sign, dtype=torch.float16, device="cuda")
    q, s, sums = m.quantize_tokens(X)
    assert bool((q == 127 * sign).all()) and int(sums[0]) == 127 * sign * MOST
    assert float(s[0]) == float(torch.tensor(2.5) / torch.tensor(127.0))
    with pytest.raises(m.W8Error):
        m.quantize_tokens(torch.zeros((1, MOST + 8), dtype=torch.float16, device="cuda"))
