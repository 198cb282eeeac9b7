"""What the tensor helpers of the rotary, latent-cache and log-probability calls hand to the C entries, and what
they refuse; without a GPU."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_top_gb300 as sv  # noqa: E402


class OnGpu:
    """A CPU tensor that says it is on a GPU; nothing reads it."""
    is_cuda = True

    def __init__(self, t, index=0):
        self._t, self._index = t, index

    def get_device(self):
        return self._index

    def unsqueeze(self, dim):
        return OnGpu(self._t.unsqueeze(dim), self._index)

    def __getattr__(self, name):
        if name.startswith("_"):
            raise AttributeError(name)
        return getattr(self._t, name)


def made(*shape, dtype=torch.bfloat16, index=0):
    return OnGpu(torch.zeros(shape, dtype=dtype), index)


def ints(*shape, index=0):
    return made(*shape, dtype=torch.int32, index=index)


@pytest.fixture
def calls(monkeypatch):
    """The C entries' arguments by name; device 0 is current, its stream's handle is 7."""
    got = {}
    for name in ("spec_rope", "spec_kv_append_rope", "spec_latent_append", "spec_latent_attn", "spec_verify_logprobs"):
        monkeypatch.setattr(sv, name, lambda *args, _n=name: got.setdefault(_n, []).append(args))
    monkeypatch.setattr(sv, "spec_latent_workspace_size", lambda *args: 64)
    monkeypatch.setattr(sv, "spec_verify_logprobs_workspace_size", lambda *args: 64)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 7, raising=False)
    return got


def latent_cache(index=0):
    return types.SimpleNamespace(descriptor=sv.LatentDescriptor(None, 3, 16, 128, 64), data=made(3, 16, 192, index=index))


def kv_cache(index=0):
    return types.SimpleNamespace(descriptor=sv.CacheDescriptor(None, None, None, None, 3, 2, 16, 64, 0),
                                 k=made(3, 2, 16, 64, index=index))


def freqs(rot=64, index=0):
    return made(rot // 2, dtype=torch.int64, index=index)


def every(index=0, stream=None):
    """One call of each helper with its tensors on device `index`."""
    def one(shape, **kw):
        return made(*shape, index=index, **kw)

    table, lens, pos = ints(2, 1, index=index), ints(2, index=index), ints(2, 3, index=index)
    return [
        lambda: sv.rope(one((2, 3, 4, 64)), freqs(index=index), pos, out=one((2, 3, 4, 64)), stream=stream),
        lambda: sv.kv_append_rope(kv_cache(index), table, lens, one((2, 3, 2, 64)), one((2, 3, 2, 64)), freqs(index=index),
                                  q=one((2, 3, 4, 64)), out_q=one((2, 3, 4, 64)), pos=pos, stream=stream),
        lambda: sv.latent_append(latent_cache(index), table, lens, one((2, 3, 128)), one((2, 3, 64)), freqs(index=index),
                                 stream=stream),
        lambda: sv.latent_attn(one((2, 3, 4, 192)), latent_cache(index), table, lens, 1.0, out=one((2, 3, 4, 128)),
                               workspace=one((64,), dtype=torch.uint8), stream=stream),
    ]


def test_stream_and_device(calls):
    side = types.SimpleNamespace(cuda_stream=5)
    for stream, handle in ((None, 7), (side, 5)):
        calls.clear()
        for call in every(stream=stream):
            call()
        assert sorted(calls) == ["spec_kv_append_rope", "spec_latent_append", "spec_latent_attn", "spec_rope"]
        assert all(args[-1] == handle for some in calls.values() for args in some)
    calls.clear()
    for call in every(index=1):  # not the current device: the kernel would run on another one's stream
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not calls


def test_tensors_of_two_devices_are_refused(calls):
    x, pos = made(2, 3, 4, 64), ints(2, 3)
    out = made(2, 3, 4, 64)
    for bad in (lambda: sv.rope(x, freqs(index=1), pos, out=out), lambda: sv.rope(x, freqs(), ints(2, 3, index=1), out=out),
                lambda: sv.rope(x, freqs(), pos, out=made(2, 3, 4, 64, index=1))):
        with pytest.raises(ValueError):
            bad()
    table, lens, k = ints(2, 1), ints(2), made(2, 3, 2, 64)
    for kw in (dict(v=made(2, 3, 2, 64, index=1)), dict(cache=kv_cache(1)), dict(table=ints(2, 1, index=1)),
               dict(q=made(2, 3, 4, 64, index=1)), dict(lens=ints(2, index=1))):
        a = dict(cache=kv_cache(), table=table, lens=lens, v=k, q=None) | kw
        with pytest.raises(ValueError):
            sv.kv_append_rope(a["cache"], a["table"], a["lens"], k, a["v"], freqs(), q=a["q"])
    q, ws = made(2, 3, 4, 192), made(64, dtype=torch.uint8)
    for kw in (dict(cache=latent_cache(1)), dict(table=ints(2, 1, index=1)), dict(lens=ints(2, index=1)),
               dict(mask=made(2, 3, 3, dtype=torch.uint8, index=1)), dict(out=made(2, 3, 4, 128, index=1)),
               dict(lse=made(2, 3, 4, dtype=torch.float32, index=1)), dict(ws=made(64, dtype=torch.uint8, index=1))):
        a = dict(cache=latent_cache(), table=table, lens=lens, mask=None, out=made(2, 3, 4, 128), lse=None, ws=ws) | kw
        with pytest.raises(ValueError):
            sv.latent_attn(q, a["cache"], a["table"], a["lens"], 1.0, mask=a["mask"], out=a["out"], lse=a["lse"],
                           workspace=a["ws"])
    with pytest.raises(ValueError):
        sv.logprobs(made(2, 3, 50), ints(2, 3, index=1))
    with pytest.raises(ValueError):
        sv.logprobs(made(2, 3, 50), ints(2, 3), rows=ints(2, 3, index=1))
    with pytest.raises(ValueError):
        sv.logprobs(made(2, 3, 50), ints(2, 3), workspace=made(64, dtype=torch.uint8, index=1))
    assert not calls


def test_workspaces_that_hold_less_than_they_count_are_refused(calls):
    """The kernels would write past an expanded workspace's one element."""
    for ws in (OnGpu(torch.zeros(1, dtype=torch.uint8).expand(64)), OnGpu(torch.zeros(128, dtype=torch.uint8)[::2])):
        with pytest.raises(ValueError, match="workspace"):
            sv.latent_attn(made(2, 3, 4, 192), latent_cache(), ints(2, 1), ints(2), 1.0, out=made(2, 3, 4, 128), workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            sv.logprobs(made(2, 3, 50), ints(2, 3), workspace=ws)
    assert not calls


def test_strides_and_counts(calls):
    """Parts of one projection come with its stride; rows set the entries' count."""
    wide = torch.zeros((2, 3, 4 * 192 + 192), dtype=torch.bfloat16)
    c, r = OnGpu(wide[..., 768:896]), OnGpu(wide[..., 896:960])
    sv.latent_append(latent_cache(), ints(2, 1), ints(2), c, r, freqs(), rows=ints(2, 5), interleaved=True)
    (a,) = calls["spec_latent_append"]
    assert (a[5], a[7], a[12]) == (960, 960, sv.SPEC_ROPE_INTERLEAVED) and a[13:16] == (2, 3, 5)
    q = OnGpu(wide[..., :768].unflatten(2, (4, 192)))
    sv.latent_attn(q, latent_cache(), ints(2, 1), ints(2), 0.5, out=made(2, 3, 4, 128), workspace=made(64, dtype=torch.uint8))
    (a,) = calls["spec_latent_attn"]
    assert a[5] == 960 and a[7:11] == (2, 3, 4, 0.5)
    for bad in (dict(c=made(2, 3, 64)), dict(r=made(2, 4, 64)), dict(r=made(2, 3, 64, dtype=torch.float32)), dict(f=freqs(32))):
        k = dict(c=made(2, 3, 128), r=made(2, 3, 64), f=freqs()) | bad
        with pytest.raises(ValueError):
            sv.latent_append(latent_cache(), ints(2, 1), ints(2), k["c"], k["r"], k["f"])


@pytest.mark.parametrize("given", [False, True])
def test_a_calls_own_tensors_are_made_on_its_stream(monkeypatch, calls, given):
    """Made on the current stream, a workspace would be handed out again while the given one still works on it."""
    stream, within, where = types.SimpleNamespace(cuda_stream=5), [], []

    @contextlib.contextmanager
    def entered(s):
        within.append(s)
        yield
        within.pop()

    def note(*args, **kw):
        where.append(list(within))
        return made(1)

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch, "empty", note)
    monkeypatch.setattr(torch, "empty_like", note)
    monkeypatch.setattr(sv, "new_workspace", note)
    kw = dict(stream=stream if given else None)
    sv.rope(made(2, 3, 4, 64), freqs(), ints(2, 3), **kw)
    sv.kv_append_rope(kv_cache(), ints(2, 1), ints(2), made(2, 3, 2, 64), made(2, 3, 2, 64), freqs(), q=made(2, 3, 4, 64), **kw)
    sv.latent_attn(made(2, 3, 4, 192), latent_cache(), ints(2, 1), ints(2), 1.0, lse=True, **kw)
    sv.logprobs(made(2, 3, 50), ints(2, 3), top=4, **kw)
    assert where == [[stream] if given else []] * 11  # out; out_q; out, lse, workspace; five results, workspace
    assert all(args[-1] == (5 if given else 7) for some in calls.values() for args in some)
