"""Refusals of the rotary, latent and log-probability entries on the CPU: turned
down on the host before any CUDA call; and the frequencies, which are host work."""
import ctypes
import decimal
import math

import numpy as np
import pytest

import speculative_decoding_verification_top_gb300 as sv
import target_reference as ref

P = 4096  # a fake pointer, aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def kv(**kw):
    a = dict(k=P, v=P, k_exp=P, v_exp=P, num_pages=4, Hkv=2, page=16, D=64, dtype=sv.SPEC_E4M3)
    a.update(kw)
    return ctypes.byref(sv.CacheDescriptor(*[a[n] for n, _ in sv.CacheDescriptor._fields_]))


def latent(**kw):
    a = dict(data=P, num_pages=4, page=16, C=512, R=64)
    a.update(kw)
    return ctypes.byref(sv.LatentDescriptor(*[a[n] for n, _ in sv.LatentDescriptor._fields_]))


def rope(**kw):
    a = dict(x=P, xs=0, out=2 * P, os=0, freqs=P, rot=64, first=0, amp=1.0, layout=0, inverse=0, pos=P, B=0, N=3,
             H=4, D=128, dtype=1)
    a.update(kw)
    rc = sv.lib().spec_rope(*[a[k] for k in ("x", "xs", "out", "os", "freqs", "rot", "first", "amp", "layout", "inverse",
                                             "pos", "B", "N", "H", "D", "dtype")], None)
    assert rc < 0 or 0 in (a["B"], a["N"])
    return rc


def append(c=None, **kw):
    a = dict(table=P, width=3, starts=P, k=P, v=P, stride=0, rows=None, pos=None, freqs=P, rot=64, amp=1.0, layout=0,
             q=None, qs=0, out_q=None, os=0, B=0, N=3, M=3, Hq=4, dtype=1)
    a.update(kw)
    rc = sv.lib().spec_kv_append_rope(c or kv(), *[a[k] for k in (
        "table", "width", "starts", "k", "v", "stride", "rows", "pos", "freqs", "rot", "amp", "layout", "q", "qs", "out_q",
        "os", "B", "N", "M", "Hq", "dtype")], None)
    assert rc < 0 or 0 in (a["B"], a["N"], a["M"], a["width"])
    return rc


def put(cache=None, **kw):
    a = dict(table=P, width=3, starts=P, c=P, cs=0, r=P, rs=0, rows=None, pos=None, freqs=P, amp=1.0, layout=0, B=0, N=3,
             M=3, dtype=1)
    a.update(kw)
    rc = sv.lib().spec_latent_append(cache or latent(), *[a[k] for k in (
        "table", "width", "starts", "c", "cs", "r", "rs", "rows", "pos", "freqs", "amp", "layout", "B", "N", "M",
        "dtype")], None)
    assert rc < 0 or 0 in (a["B"], a["N"], a["M"], a["width"])
    return rc


def attn(c=None, **kw):
    a = dict(table=P, width=3, lens=P, q=P, stride=0, mask=None, B=0, N=3, H=4, scale=1.0, out=P, lse=None, ws=P,
             ws_bytes=4)
    a.update(kw)
    rc = sv.lib().spec_latent_attn(c or latent(), *[a[k] for k in (
        "table", "width", "lens", "q", "stride", "mask", "B", "N", "H", "scale", "out", "lse", "ws", "ws_bytes")], None)
    assert rc < 0 or a["B"] == 0
    return rc


def logprobs(**kw):
    a = dict(x=P, tokens=P, rows=None, B=0, N=3, M=3, V=100, T=1.0, top=5, dtype=1, lp=P, ent=None, rank=None, ids=P,
             best=P, ws=P, ws_bytes=4)
    a.update(kw)
    rc = sv.lib().spec_verify_logprobs(*[a[k] for k in (
        "x", "tokens", "rows", "B", "N", "M", "V", "T", "top", "dtype", "lp", "ent", "rank", "ids", "best", "ws",
        "ws_bytes")], None)
    assert rc < 0 or 0 in (a["B"], a["M"])
    return rc


def test_rope():
    assert rope() == 0
    assert rope(B=-1) == -2
    assert rope(D=120) == -2
    assert rope(D=1040, rot=64) == -2
    assert rope(rot=0) == -2
    assert rope(rot=24) == -2
    assert rope(rot=144) == -2
    assert rope(first=8) == -2
    assert rope(first=80) == -2
    assert rope(H=0) == -2
    assert rope(B=1 << 20, N=1 << 20) == -2
    assert rope(xs=508) == -2                     # under H * D
    assert rope(os=516) == -2                     # not a multiple of 8
    assert rope(out=P, os=520) == -2              # in place with another stride
    assert rope(layout=2) == -5
    assert rope(amp=float("nan")) == -3
    assert rope(dtype=2) == -4
    assert rope(B=2, x=None) == -1
    assert rope(B=2, out=None) == -1
    assert rope(B=2, freqs=None) == -1
    assert rope(B=2, pos=None) == -1
    assert rope(B=2, x=P + 8) == -6
    assert rope(B=2, freqs=P + 8) == -6
    assert rope(B=2, pos=P + 2) == -6


def test_append():
    assert append() == 0
    assert append(kv(D=96)) == -2
    assert append(kv(dtype=0)) == -4
    assert append(rot=128) == -2                  # wider than the head
    assert append(M=2) == -2                      # M != N without rows
    assert append(stride=64) == -2
    assert append(q=P, out_q=P, Hq=0) == -2
    assert append(q=P, out_q=P, qs=128) == -2
    assert append(q=P, out_q=P, qs=264) == -2     # in place with another stride
    assert append(q=P, out_q=P, rows=P) == -3
    assert append(layout=-1) == -5
    assert append(amp=float("inf")) == -3
    assert append(dtype=2) == -4
    assert append(B=2, q=P) == -1
    assert append(B=2, out_q=P) == -1
    assert append(B=2, freqs=None) == -1
    assert append(B=2, starts=None) == -1
    assert append(B=2, v=P + 4) == -6
    assert append(B=2, pos=P + 1) == -6
    assert append(B=2, q=P, out_q=P + 8) == -6
    assert append(B=2, width=0, table=None) == 0


def test_overlapping_outputs():
    """An output that shares elements with what other threads still read."""
    n = 6 * 512 * 2  # bytes of the default call's six packed tokens
    for d in (16, 1024, n - 16, 16 - n):
        assert rope(B=2, x=4 * P, out=4 * P + d) == -2
    assert rope(B=2, out=P + n - 16, dtype=0) == -2      # fp32: twice as long
    assert rope(B=2, xs=1024, os=1024, out=P + 1008) == -2   # a token's stride is 2048 bytes, its elements 1024
    assert rope(B=2, xs=1024, os=1024, out=P + 1040) == -2
    assert rope(B=2, xs=1024, os=1040, out=P + 1024) == -2   # strides that differ
    assert rope(B=1 << 15, N=1 << 15, H=1, D=16, rot=16, xs=1 << 40, os=1 << 40, out=P + 16) == -2  # past 64 bits
    # tokens of 4 heads of 64 between others' 4: out_q over the keys, the values, beside them, over the queries
    far = 1 << 20
    a = dict(B=2, q=far, out_q=4 * far, qs=512, os=512, k=2 * far, v=3 * far, stride=512, Hq=4)
    for out_q, os in ((2 * far + 16, 512), (3 * far + 240, 512), (3 * far - 496, 512), (far + 16, 512), (2 * far + 512, 520)):
        assert append(kv(D=64, dtype=1), **{**a, "out_q": out_q, "os": os}) == -2


def test_latent_append():
    assert put() == 0
    assert put(latent(C=192)) == -2
    assert put(latent(R=32)) == -2
    assert put(latent(page=48)) == -2
    assert put(latent(num_pages=0)) == -2
    assert put(latent(data=None)) == -1
    assert put(latent(data=P + 8)) == -6
    assert put(cs=256) == -2
    assert put(rs=60) == -2
    assert put(M=2) == -2
    assert put(N=-1) == -2
    assert put(layout=3) == -5
    assert put(dtype=2) == -4
    assert put(B=2, c=None) == -1
    assert put(B=2, r=P + 8) == -6
    assert put(B=2, rows=P + 2, M=2) == -6


def test_latent_attention():
    assert attn() == 0
    assert attn(latent(C=96)) == -2
    assert attn(N=0) == -2
    assert attn(N=1025) == -2
    assert attn(H=0) == -2
    assert attn(H=1025) == -2
    assert attn(B=1 << 20, N=1024) == -2
    assert attn(width=1 << 28) == -2
    assert attn(stride=2300) == -2
    assert attn(scale=float("inf")) == -3
    assert attn(B=2, lens=None) == -1
    assert attn(B=2, q=None) == -1
    assert attn(B=2, out=None) == -1
    assert attn(B=2, q=P + 8) == -6
    assert attn(B=2, lse=P + 2) == -6
    assert attn(B=2, ws=None) == -7
    assert attn(B=2, ws=P + 4, ws_bytes=1 << 40) == -6


def test_latent_rows():
    """As many query rows as the header allows, and one more."""
    for B, N, H in ((128, 128, 128), (1 << 10, 1 << 10, 1 << 10), (1 << 30, 1, 1), (1 << 20, 4, 256)):
        assert sv.spec_latent_workspace_size(B, N, H, 512) > 0
        assert attn(B=B, N=N, H=H, ws=None) == -7
    for B, N, H in (((1 << 10) + 1, 1 << 10, 1 << 10), ((1 << 30) + 1, 1, 1), ((1 << 31) - 1, 1024, 1024)):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_latent_workspace_size(B, N, H, 512)
        assert attn(B=B, N=N, H=H, ws=None) == -2


def test_latent_workspace():
    assert 0 < sv.spec_latent_workspace_size(1, 1, 16, 512) <= sv.spec_latent_workspace_size(64, 6, 32, 512)
    for args in [(-1, 1, 4, 512), (1, 0, 4, 512), (1, 1, 0, 512), (1, 1, 4, 96), (1, 1025, 4, 512)]:
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_latent_workspace_size(*args)


def test_logprobs():
    assert logprobs() == 0
    assert logprobs(B=-1) == -2
    assert logprobs(N=0) == -2
    assert logprobs(M=4) == -2                    # more entries than rows without `rows`
    assert logprobs(M=4, rows=P) == 0
    assert logprobs(V=0) == -2
    assert logprobs(V=(1 << 22) + 1) == -2
    assert logprobs(top=33) == -2
    assert logprobs(V=4) == -2                    # top > V
    assert logprobs(T=0.0) == -3
    assert logprobs(T=float("nan")) == -3
    assert logprobs(T=1e-40) == -3                # 1 / T is not finite
    assert logprobs(dtype=2) == -4
    assert logprobs(B=2, x=None) == -1
    assert logprobs(B=2, tokens=None) == -1
    assert logprobs(B=2, lp=None) == -1
    assert logprobs(B=2, ids=None) == -1
    assert logprobs(B=2, best=None) == -1
    assert logprobs(B=2, x=P + 1) == -6
    assert logprobs(B=2, x=P + 2, dtype=0) == -6
    assert logprobs(B=2, rank=P + 2) == -6
    assert logprobs(B=2) == -7                    # the fake workspace holds 4 bytes
    assert logprobs(B=2, top=0, ids=None, best=None) == -7


@pytest.mark.parametrize("rot,base,scaling,args", [
    (64, 10000.0, "plain", (1.0, 0, 0.0, 0.0)), (128, 500000.0, "linear", (4.0, 0, 0.0, 0.0)),
    (16, 10000.0, "turns", (8.0, 8192, 1.0, 4.0)), (128, 500000.0, "turns", (8.0, 8192, 1.0, 4.0)),
    (64, 10000.0, "index", (40.0, 4096, 1.0, 32.0)), (128, 1e6, "index", (4.0, 32768, 1.0, 32.0))])
def test_frequencies(rot, base, scaling, args):
    got = (ctypes.c_uint64 * (rot // 2))()
    sv.spec_rope_freqs(rot, base, sv.SCALINGS[scaling], *args, ctypes.addressof(got))
    want = ref.frequencies(rot, base, scaling, *args)
    # powers, logarithms and quotients in 64 bits: a few roundings of 2^-53 each; the
    # fixed point is off by half a step, 2^-65 of a turn
    assert np.allclose(np.array(got[:], np.float64) / 2.0 ** 64 * (2 * np.pi), want, rtol=2.0 ** -48,
                       atol=2 * np.pi * 2.0 ** -65)


PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.mark.parametrize("rot,base,scaling,args", [
    (64, 10000.0, "plain", (1.0, 0, 0.0, 0.0)), (128, 5e5, "plain", (1.0, 0, 0.0, 0.0)), (16, 1.5, "plain", (1.0, 0, 0.0, 0.0)),
    (1024, 1e30, "plain", (1.0, 0, 0.0, 0.0)), (1024, 1 + 2.0 ** -40, "plain", (1.0, 0, 0.0, 0.0)),
    (128, 5e5, "linear", (3.7, 0, 0.0, 0.0)), (128, 5e5, "turns", (8.0, 8192, 1.0, 4.0)),
    (64, 10000.0, "turns", (40.0, 4096, 0.1, 31.9)), (64, 1e30, "turns", (40.0, 1e30, 1e-301, 1e-300)),
    (64, 1e30, "turns", (2.0, 1.0, 1e-20, 1.0)), (64, 3.0, "turns", (40.0, 7e29, 1e-300, 1e30)), (64, 10000.0, "index", (40.0, 4096, 1.0, 32.0)),
    (1024, 1e6, "index", (4.3, 32768, 1.0, 32.0))])
def test_frequencies_to_the_last_bit(rot, base, scaling, args):
    """The nearest integers to 2^64 theta / (2 pi): a frequency's error grows with the position."""
    got = (ctypes.c_uint64 * (rot // 2))()
    sv.spec_rope_freqs(rot, base, sv.SCALINGS[scaling], *args, ctypes.addressof(got))
    factor, original, low, high = args
    D = decimal.Decimal
    with decimal.localcontext() as c:
        c.prec = 70
        for i in range(rot // 2):
            theta, w = (D(base).ln() * -2 * i / rot).exp(), D(0)
            if scaling == "turns":
                w = (D(original) * theta / (2 * PI) - D(low)) / (D(high) - D(low))
            elif scaling == "index":
                at = [rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (high, low)]
                a, b = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
                w = 1 - min(D(1), max(D(0), (i - a) / D(max(b - a, 1))))
            w = min(D(1), max(D(0), w))
            if scaling != "plain":
                theta *= w + (1 - w) / D(factor)
            # half a step, and what two doubles are off by after a thousand operations: 2^-94 of less than 2^62
            assert abs(got[i] - theta / (2 * PI) * 2 ** 64) <= D("0.5") + D(2) ** -32


def test_frequency_refusals():
    got = (ctypes.c_uint64 * 512)()
    at = ctypes.addressof(got)

    def call(rot=64, base=10000.0, scaling=0, factor=1.0, original=0, low=0.0, high=0.0, to=at):
        return sv.lib().spec_rope_freqs(rot, base, scaling, factor, original, low, high, to)

    assert call() == 0 and call(rot=1024) == 0
    assert call(to=None) == -1
    assert call(rot=8) == call(rot=24) == call(rot=1040) == -2
    assert call(base=1.0) == call(base=float("nan")) == call(base=float("inf")) == -3
    assert call(scaling=4) == call(scaling=-1) == -5
    assert call(scaling=1, factor=0.5) == -3
    assert call(scaling=2, factor=2.0) == -3
    assert call(scaling=2, factor=2.0, original=4096, low=4.0, high=1.0) == -3
    assert call(scaling=3, factor=2.0, original=4096, low=1.0, high=32.0) == 0


def test_helper_refusals():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        sv.rope_freqs(64, scaling="quadratic", device="cpu")
    with pytest.raises(sv.SpecVerifyError):
        sv.rope_freqs(24, device="cpu")
    with pytest.raises(ValueError):
        sv.LatentCache(torch.zeros((2, 16, 576), dtype=torch.bfloat16))  # not on a GPU
    freqs = sv.rope_freqs(64, device="cpu")
    assert freqs.shape == (32,) and freqs.dtype == torch.int64
    with pytest.raises(ValueError):
        sv.rope(torch.zeros((1, 1, 1, 64)), freqs, torch.zeros((1, 1), dtype=torch.int32))
