"""Refusals of include/spec_attn.h's entries on the CPU: every case below is
turned down on the host before any CUDA call, with nothing enqueued."""
import ctypes

import pytest

import speculative_decoding_verification_top_gb300 as sv

P = 4096  # a fake pointer, aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def cache(**kw):
    a = dict(k=P, v=P, k_exp=P, v_exp=P, num_pages=4, Hkv=2, page=16, D=64, dtype=sv.SPEC_E4M3)
    a.update(kw)
    return ctypes.byref(sv.CacheDescriptor(*[a[n] for n, _ in sv.CacheDescriptor._fields_]))


def append(c=None, **kw):
    a = dict(table=P, width=3, starts=P, k=P, v=P, stride=0, rows=None, B=0, N=3, M=3,
             dtype=sv.SPEC_BF16)
    a.update(kw)
    rc = sv.lib().spec_kv_append(c or cache(), a["table"], a["width"], a["starts"], a["k"], a["v"],
                                 a["stride"], a["rows"], a["B"], a["N"], a["M"], a["dtype"], None)
    assert rc < 0 or 0 in (a["B"], a["N"], a["M"], a["width"])
    return rc


def read(c=None, **kw):
    a = dict(table=P, width=3, starts=P, k=P, v=P, B=0, M=3, dtype=sv.SPEC_BF16)
    a.update(kw)
    rc = sv.lib().spec_kv_read(c or cache(), a["table"], a["width"], a["starts"], a["k"], a["v"],
                               a["B"], a["M"], a["dtype"], None)
    assert rc < 0 or 0 in (a["B"], a["M"]) or not (a["k"] or a["v"])
    return rc


def attn(c=None, **kw):
    a = dict(stable=P, slen=20, table=P, width=3, lens=P, q=P, stride=0, mask=None, pos=None,
             slopes=None, B=0, N=3, Hq=4, scale=1.0, cap=0.0, window=0, dtype=sv.SPEC_BF16, out=P,
             lse=None, ws=P, ws_bytes=4)
    a.update(kw)
    rc = sv.lib().spec_attn_shared(
        c or cache(), a["stable"], a["slen"], a["table"], a["width"], a["lens"], a["q"], a["stride"],
        a["mask"], a["pos"], a["slopes"], a["B"], a["N"], a["Hq"], a["scale"], a["cap"], a["window"],
        a["dtype"], a["out"], a["lse"], a["ws"], a["ws_bytes"], None)
    assert rc < 0 or a["B"] == 0
    return rc


@pytest.mark.parametrize("call", [append, read, attn])
def test_cache_descriptor(call):
    assert call(cache(dtype=0)) == -4
    assert call(cache(dtype=3)) == -4
    assert call(cache(num_pages=0)) == -2
    assert call(cache(Hkv=0)) == -2
    assert call(cache(Hkv=1025)) == -2
    assert call(cache(page=48)) == -2
    assert call(cache(page=256)) == -2
    assert call(cache(D=96)) == -2
    assert call(cache(k=None)) == -1
    assert call(cache(v=None)) == -1
    assert call(cache(k_exp=None)) == -1
    assert call(cache(k=P + 8)) == -6
    assert call(cache(v_exp=P + 2)) == -6
    assert call(cache(k_exp=None, v_exp=None, dtype=sv.SPEC_BF16)) == 0
    assert call() == 0  # B = 0: nothing to do


def test_append_arguments():
    assert append(B=-1) == -2
    assert append(N=-1) == -2
    assert append(B=2, M=2) == -2             # M != N without rows
    assert append(B=2, stride=64) == -2       # under Hkv * D
    assert append(B=2, stride=132) == -2      # not a multiple of 8
    assert append(B=2, dtype=sv.SPEC_E4M3) == -4
    assert append(B=2, table=None) == -1
    assert append(B=2, starts=None) == -1
    assert append(B=2, k=None) == -1
    assert append(B=2, k=P + 8) == -6
    assert append(B=2, rows=P + 2) == -6
    assert append(B=2, N=0, M=0, k=None) == 0
    assert append(B=2, width=0, table=None) == 0


def test_read_arguments():
    assert read(B=-1) == -2
    assert read(M=-1) == -2
    assert read(B=2, dtype=2) == -4
    assert read(B=2, starts=None) == -1
    assert read(B=2, k=P + 4) == -6
    assert read(B=2, k=None, v=None) == 0


def test_attention_arguments():
    assert attn(B=-1) == -2
    assert attn(N=0) == -2
    assert attn(N=sv_max_nodes() + 1) == -2
    assert attn(Hq=3) == -2
    assert attn(Hq=0) == -2
    assert attn(slen=-1) == -2
    assert attn(width=-1) == -2
    assert attn(width=1 << 28) == -2
    assert attn(stride=128) == -2             # under Hq * D
    assert attn(stride=260) == -2
    assert attn(dtype=sv.SPEC_F32) == -4
    assert attn(scale=float("nan")) == -3
    assert attn(cap=-1.0) == -3
    assert attn(cap=float("inf")) == -3
    assert attn(window=-1) == -3
    assert attn(B=2, stable=None) == -1
    assert attn(B=2, table=None) == -1
    assert attn(B=2, lens=None) == -1
    assert attn(B=2, q=None) == -1
    assert attn(B=2, out=None) == -1
    assert attn(B=2, q=P + 8) == -6
    assert attn(B=2, out=P + 2) == -6
    assert attn(B=2, pos=P + 1) == -6
    assert attn(B=2, ws=None) == -7
    assert attn(B=2) == -7                    # the fake workspace holds 4 bytes
    assert attn(B=2, ws=P + 4, ws_bytes=1 << 40) == -6


def sv_max_nodes():
    return 1024


def test_workspace_size():
    a = sv.spec_attn_workspace_size(1, 1, 4, 2, 64)
    assert 0 < a <= sv.spec_attn_workspace_size(64, 6, 32, 8, 128)
    for args in [(-1, 1, 4, 2, 64), (1, 0, 4, 2, 64), (1, 1, 4, 3, 64), (1, 1, 4, 2, 96),
                 (1, 1025, 4, 2, 64)]:
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_attn_workspace_size(*args)


def test_status_string():
    assert "page" in sv.spec_verify_status_string(sv.SPEC_DATA_PAGE_RANGE)
