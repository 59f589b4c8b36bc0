"""What the binding of the int8-activation operators lets through to the
kernels, with stand-ins for CUDA tensors (no GPU needed)."""
import pytest
import torch

import int8_weight_only_b200 as m


class FakeCuda:
    """A CPU tensor that says it is on a GPU."""

    def __init__(self, t):
        self.inner = t

    is_cuda = True
    device = torch.device("cuda", 0)

    def __getattr__(self, name):
        return getattr(self.inner, name)

    def __getitem__(self, i):
        return FakeCuda(self.inner[i])

    def new_empty(self, shape, dtype):
        return FakeCuda(torch.empty(shape, dtype=dtype))


def fake(shape, dtype):
    return FakeCuda(torch.empty(shape, dtype=dtype))


@pytest.fixture
def calls(monkeypatch):
    """The argument lists that reach the library."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return name

    monkeypatch.setattr(m, "load_library", lambda: Lib())
    monkeypatch.setattr(m, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(m, "_call", lambda fn, what, device, stream, *args: seen.append((what, args)))
    return seen


OPERATORS = [("quantize_tokens", 1), ("swiglu_quantize_tokens", 2)]


@pytest.mark.parametrize("op,wide", OPERATORS)
@pytest.mark.parametrize("M", [1, 3])
@pytest.mark.parametrize("K", [64, 72])
def test_given_codes_with_adjacent_columns_are_taken(calls, op, wide, M, K):
    X = fake((M, wide * K), torch.float16)
    for q in (None, fake((M, 80), torch.int8)[:, :K]):
        got, scales, sums = getattr(m, op)(X, q=q)
        assert got.shape == (M, K) and scales.shape == (M,) and sums.shape == (M,)
        assert q is None or got is q
    assert [c[0] for c in calls] == ["w8_" + op.replace("_tokens", "_per_token")] * 2


@pytest.mark.parametrize("op,wide", OPERATORS)
@pytest.mark.parametrize("M", [1, 3])
def test_given_codes_whose_columns_are_apart_are_refused(calls, op, wide, M):
    # the kernels write K bytes from the first one on, whatever the strides
    K = 64
    X = fake((M, wide * K), torch.float16)
    for q in (FakeCuda(torch.empty((K, 16), dtype=torch.int8)[:, :M].t()),
              fake((M, 2 * K), torch.int8)[:, ::2], FakeCuda(torch.empty((1, 1), dtype=torch.int8).expand(M, K))):
        assert q.shape == (M, K)
        with pytest.raises(ValueError):
            getattr(m, op)(X, q=q)
    assert not calls


@pytest.mark.gpu
def test_given_codes_on_the_gpu():
    K = 64
    X = torch.randn((1, 2 * K), device="cuda").half()
    wide = torch.full((K, 16), 99, dtype=torch.int8, device="cuda")
    for op, H in (("quantize_tokens", X[:, :K]), ("swiglu_quantize_tokens", X)):
        for q in (wide[:, :1].t(), wide.view(-1)[:2 * K:2].view(1, K), wide[:1, :1].expand(1, K)):
            with pytest.raises(ValueError):
                getattr(m, op)(H, q=q)
        assert bool((wide == 99).all())
        want, given = getattr(m, op)(H), getattr(m, op)(H, q=wide.view(-1)[:K].view(1, K))
        assert all(torch.equal(a, b) for a, b in zip(want, given))
        assert bool((wide.view(-1)[K:] == 99).all())
        wide.fill_(99)
