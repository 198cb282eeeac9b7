"""The paged cache on the GPU against the plain 64-bit form: written values
and exponents exact, untouched positions untouched, reading exact."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

import attn_reference as ref  # noqa: E402
import speculative_decoding_verification_top_gb300 as sv  # noqa: E402

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def random_cache(rng, n, H, page, D, e4m3):
    """A cache of random contents, and its numpy copy (bytes or bf16 bits)."""
    c = sv.new_cache(n, H, page, D, DEV, e4m3)
    if e4m3:
        for t in (c.k, c.v):
            t.view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 127, t.shape).astype(np.uint8)))
        for t in (c.k_exp, c.v_exp):
            t.copy_(torch.from_numpy(rng.integers(-9, 3, t.shape).astype(np.int8)))
    else:
        for t in (c.k, c.v):
            t.copy_(torch.from_numpy(rng.normal(size=t.shape).astype(np.float32)))
    return c


def raw(cache):
    out = {}
    for name in ("k", "v", "k_exp", "v_exp"):
        t = getattr(cache, name)
        if t is not None:
            out[name] = t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy().copy()
    return out


def page_tables(rng, B, width, n):
    return rng.permutation(n)[:B * width].reshape(B, width).astype(np.int32)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,H,page,B,N", [(64, 1, 16, 1, 1), (64, 3, 16, 3, 5), (128, 2, 64, 2, 37),
                                         (128, 8, 32, 5, 6), (64, 5, 128, 2, 131)])
def test_append_and_read(e4m3, dtype, D, H, page, B, N):
    rng = np.random.default_rng([D, H, page, N])
    width = (N + 40) // page + 2
    n = B * width + 2
    c = random_cache(rng, n, H, page, D, e4m3)
    before = raw(c)
    table = page_tables(rng, B, width, n)
    starts = rng.integers(-3, 40, B).astype(np.int32)  # some tokens fall before position 0
    x = {w: dev(rng.normal(size=(B, N, H, D)) * 2.0 ** rng.integers(-20, 20, (B, N, H, 1)), dtype)
         for w in "kv"}
    x["k"][0, 0, 0] = 0.0
    x["v"][-1, -1, -1, 3] = float("nan")
    x["v"][-1, -1, -1, 5] = -float("inf")
    sv.kv_append(c, dev(table), dev(starts), x["k"], x["v"])
    got_k, got_v = sv.kv_read(c, dev(table), dev(starts), N, dtype=torch.float32)
    half_k, half_v = sv.kv_read(c, dev(table), dev(starts), N)
    torch.cuda.synchronize()
    want = {k: v.copy() for k, v in before.items()}
    for w, got, half in (("k", got_k, half_k), ("v", got_v, half_v)):
        src = x[w].double().cpu().numpy()
        full = np.zeros((B, N, H, D))
        for b in range(B):
            for t in range(N):
                p = int(starts[b]) + t
                if p < 0:
                    continue
                pid, slot = int(table[b, p // page]), p % page
                if e4m3:
                    y, e = ref.quantise(src[b, t])
                    want[w + "_exp"][pid, :, slot] = e.astype(np.int8).view(np.uint8)
                    byte = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
                    want[w][pid, :, slot] = np.where(np.isnan(y), 0x7f, byte)
                    full[b, t] = y * 2.0 ** e[:, None].astype(float)
                else:
                    r = torch.from_numpy(src[b, t]).float().to(torch.bfloat16)
                    want[w][pid, :, slot] = r.view(torch.int16).numpy()
                    full[b, t] = r.double().numpy()
        np.testing.assert_array_equal(got.double().cpu().numpy(), full)
        np.testing.assert_array_equal(half.double().cpu().numpy(), full)  # exact in bf16 too
    after = raw(c)
    for name in want:
        if not e4m3:  # NaN payloads may differ in bits: compare those as NaN
            a, b = (torch.from_numpy(z[name]).view(torch.bfloat16).float().numpy() for z in (after, want))
            np.testing.assert_array_equal(a, b)
        else:
            np.testing.assert_array_equal(after[name], want[name], err_msg=name)


def test_append_extremes():
    """Rows at the ends of fp32's range: exponents stay in [-120, 120]."""
    D, c = 64, sv.new_cache(1, 1, 16, 64, DEV, e4m3=True)
    rows = np.zeros((1, 5, 1, D), np.float32)
    rows[0, 0] = np.float32(3.4e38)
    rows[0, 1] = np.float32(1e-45)
    rows[0, 2, 0, 7] = -np.float32(448.0)
    rows[0, 3, 0, 7] = np.nextafter(np.float32(448.0), np.float32(1e9))
    rows[0, 4, 0, 1] = np.inf
    t, s = dev(np.zeros((1, 1), np.int32)), dev(np.zeros(1, np.int32))
    sv.kv_append(c, t, s, dev(rows), dev(rows))
    assert c.k_exp[0, 0, :5].tolist() == [120, -120, 0, 1, 0]
    k, _ = sv.kv_read(c, t, s, 5, dtype=torch.float32)
    assert k[0, 2, 0, 7] == -448 and k[0, 3, 0, 7] == 448 and torch.isnan(k[0, 4, 0, 1])
    assert k[0, 0, 0, 0] == 256 * 2.0 ** 120 and torch.all(k[0, 1] == 0)


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_pick_tokens_and_bad_entries_are_skipped(e4m3):
    rng = np.random.default_rng(7)
    B, N, M, H, page, D = 4, 9, 4, 2, 16, 64
    c = random_cache(rng, 12, H, page, D, e4m3)
    before = raw(c)
    table = page_tables(rng, B, 2, 12)
    table[2] = [-1, 12]                       # no such pages
    starts = np.array([3, 30, 5, 14], np.int32)  # sequence 1 leaves its table after two tokens
    rows = np.array([[0, 2, 8, -1], [1, 2, 3, 4], [0, 1, 2, 3], [9, -1, 100, 5]], np.int32)
    x = dev(rng.normal(size=(B, N, H, D)), torch.bfloat16)
    sv.kv_append(c, dev(table), dev(starts), x, x, rows=dev(rows))
    after = raw(c)
    live = {(0, 3): 0, (0, 4): 2, (0, 5): 8, (1, 30): 1, (1, 31): 2, (3, 17): 5}
    touched = np.zeros(before["k"].shape[:3], bool)
    for (b, p), r in live.items():
        pid, slot = table[b, p // page], p % page
        touched[pid, :, slot] = True
        one = sv.kv_read(c, dev(table[b:b + 1]), dev(np.array([p], np.int32)), 1, dtype=torch.float32)[0]
        src = x[b, r].double().cpu().numpy()
        if e4m3:
            y, e = ref.quantise(src)
            src = y * 2.0 ** e[:, None].astype(float)
        np.testing.assert_array_equal(one[0, 0].double().cpu().numpy(), src)
    for name in before:
        np.testing.assert_array_equal(after[name][~touched], before[name][~touched])


def test_read_out_of_range_is_zero():
    c = random_cache(np.random.default_rng(3), 2, 1, 16, 64, False)
    t = dev(np.array([[0, 5]], np.int32))
    k, v = sv.kv_read(c, t, dev(np.array([-2], np.int32)), 40)
    assert torch.all(k[0, :2] == 0) and torch.all(k[0, 18:] == 0) and torch.all(v[0, 18:] == 0)
    assert torch.equal(k[0, 2:18, 0], c.k[0, 0])


def test_strided_tokens_and_other_stream():
    """k and v as slices of one wide projection, on a side stream."""
    rng = np.random.default_rng(5)
    B, N, H, D = 3, 7, 2, 64
    wide = dev(rng.normal(size=(B, N, 5 * H * D)), torch.bfloat16)
    k, v = (wide[..., i * H * D:(i + 1) * H * D].unflatten(-1, (H, D)) for i in (1, 4))
    t, s = dev(page_tables(rng, B, 1, 5)), dev(np.array([0, 4, 9], np.int32))
    a, b = sv.new_cache(5, H, 16, D, DEV, True), sv.new_cache(5, H, 16, D, DEV, True)
    sv.kv_append(a, t, s, k.contiguous(), v.contiguous())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    sv.kv_append(b, t, s, k, v, stream=st)
    st.synchronize()
    for x, y in zip(raw(a).values(), raw(b).values()):
        np.testing.assert_array_equal(x, y)
    with pytest.raises(ValueError):
        sv.kv_append(a, t, s, k.transpose(2, 3), v.transpose(2, 3))
    with pytest.raises(ValueError):
        sv.kv_append(a, t, s, k, v.contiguous())


def test_empty_calls():
    c = sv.new_cache(1, 1, 16, 64, DEV)
    none = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    x = torch.zeros((0, 3, 1, 64), dtype=torch.bfloat16, device=DEV)
    sv.kv_append(c, none, none[:, 0].contiguous(), x, x)
    k, _ = sv.kv_read(c, none, none[:, 0].contiguous(), 3)
    assert k.shape == (0, 3, 1, 64)
