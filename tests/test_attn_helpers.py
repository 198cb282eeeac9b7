"""The tensor-level helpers' own checks on the CPU: what the C entries are given."""
import contextlib
import copy
import types

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_top_gb300 as sv  # noqa: E402


class OnGpu:
    """A CPU tensor that says it is on the GPU; nothing reads it."""
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        if name.startswith("_"):
            raise AttributeError(name)
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


@pytest.mark.parametrize("given", [False, True])
def test_a_calls_own_tensors_are_made_on_its_stream(monkeypatch, given):
    """With `stream`, the workspace is zeroed, and it and the outputs are
    allocated, on that stream: made on the current one, the workspace would be
    handed out again while the other stream still works on it."""
    stream, within, made = types.SimpleNamespace(cuda_stream=5), [], []

    @contextlib.contextmanager
    def entered(s):
        within.append(s)
        yield
        within.pop()

    def note(real):
        def f(*args, **kw):
            made.append(list(within))
            return OnGpu(real(*args, **kw))
        return f

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch, "empty", note(torch.empty))
    monkeypatch.setattr(sv, "new_workspace", note(lambda n, device: torch.zeros(n, dtype=torch.uint8)))
    calls = []
    monkeypatch.setattr(sv, "spec_attn_tree", lambda *args: calls.append(args))
    monkeypatch.setattr(sv, "spec_attn_workspace_size", lambda *args: 64)
    monkeypatch.setattr(sv, "spec_kv_read", lambda *args: calls.append(args))
    cache = types.SimpleNamespace(descriptor=sv.CacheDescriptor(None, None, None, None, 1, 2, 16, 64, 0))
    ints = OnGpu(torch.zeros((2, 1), dtype=torch.int32))
    one = OnGpu(torch.zeros(2, dtype=torch.int32))
    sv.attn_tree(OnGpu(zeros(2, 3, 4, 64)), cache, ints, one, lse=True, stream=stream if given else None)
    sv.kv_read(cache, ints, one, 4, stream=stream if given else None)
    assert made == [[stream] if given else []] * 5  # out, lse, workspace; k, v
    assert [c[-1] for c in calls] == [5 if given else 0] * 2


def test_copies_of_a_cache_have_descriptors_of_their_own():
    def pool():
        return OnGpu(zeros(3, 2, 16, 64))

    a, k = sv.KVCache(pool(), pool()), pool()
    for b in (a._replace(k=k), sv.KVCache._make((k, a.v, None, None)), copy.deepcopy(a), copy.copy(a)):
        assert type(b) is sv.KVCache
        assert (b.descriptor.k, b.descriptor.v) == (b.k.data_ptr(), b.v.data_ptr())
        assert (b.descriptor.num_pages, b.descriptor.page) == (3, 16)
    assert a._replace(k=k).k is k
    with pytest.raises(ValueError):
        a._replace(k=OnGpu(zeros(3, 2, 16, 128)))
