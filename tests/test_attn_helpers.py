"""The tensor-level helpers' own checks on the CPU: what the C entries are given."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_top_gb300 as sv  # noqa: E402


class OnGpu:
    """A CPU tensor that says it is on the GPU; nothing reads it."""
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


def tokens(t, H, D):
    return sv._tokens(OnGpu(t), "q", H, D, (torch.bfloat16,))


def zeros(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_token_strides():
    assert tokens(zeros(2, 3, 4, 64), 4, 64) == 256
    assert tokens(zeros(2, 3, 9, 64)[:, :, 2:6], 4, 64) == 576       # of a wider projection
    assert tokens(zeros(5, 1, 9, 64)[:, :, 2:6], 4, 64) == 576       # single tokens
    assert tokens(zeros(1, 1, 4, 64).expand(1, 1, 4, 64), 4, 64) == 256


@pytest.mark.parametrize("B,N", [(4, 1), (1, 5), (4, 5)])
def test_expanded_tokens_are_refused(B, N):
    """One token's storage seen as many: a step of 0, which the C entries take
    for packed tokens, would read past it."""
    with pytest.raises(ValueError):
        tokens(zeros(1, 1, 4, 64).expand(B, N, 4, 64), 4, 64)


def test_overlapping_and_uneven_tokens_are_refused():
    with pytest.raises(ValueError):
        tokens(torch.as_strided(zeros(2000), (2, 3, 4, 64), (600, 200, 64, 1)), 4, 64)
    with pytest.raises(ValueError):
        tokens(torch.as_strided(zeros(9000), (2, 3, 4, 64), (1000, 256, 64, 1)), 4, 64)
    with pytest.raises(ValueError):
        tokens(zeros(2, 3, 64, 4).transpose(2, 3), 4, 64)
