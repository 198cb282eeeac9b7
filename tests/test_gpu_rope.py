"""Rotary positions on the GPU against the 64-bit form: queries, keys on their way
into the paged cache, and a latent cache's rows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

import attn_reference as attn_ref  # noqa: E402
import speculative_decoding_verification_top_gb300 as sv  # noqa: E402
import target_reference as ref  # noqa: E402

DEV = "cuda:0"
HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2
                               else torch.int32).cpu().numpy()


def check(got, want, size, dtype):
    """got (a tensor) within the turn's rounding and its type's of want."""
    bound = size * ref.TURN + np.abs(want) * (HALF_BF16 if dtype == torch.bfloat16 else 0.0)
    # an element that stays is exact; a turned one may fall under the smallest normal
    assert np.all(np.abs(host(got) - want) <= bound * (1 + 2.0 ** -20))


def positions(rng, B, N, far):
    p = rng.integers(0, far, (B, N)).astype(np.int32)
    p[0, 0] = far - 1
    return p


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,N,H,D,rot,first,far", [
    (1, 1, 1, 16, 16, 0, 1), (2, 3, 5, 64, 64, 0, 100), (3, 1, 7, 128, 32, 96, 131072), (1, 5, 2, 576, 64, 512, 9000),
    (2, 130, 4, 128, 128, 0, 2 ** 31), (4, 1500, 12, 64, 48, 16, 5000), (1, 2, 3, 1024, 1024, 0, 4000)])
def test_rope(dtype, interleaved, B, N, H, D, rot, first, far):
    rng = np.random.default_rng([B, N, H, D])
    freqs = sv.rope_freqs(rot, 10000.0, "turns", 8.0, 8192, 1.0, 4.0)
    f = freqs.cpu().numpy()
    x, pos = dev(rng.normal(size=(B, N, H, D)), dtype), positions(rng, B, N, far)
    got = sv.rope(x, freqs, dev(pos), first=first, amplitude=1.25, interleaved=interleaved)
    want, size = ref.turned(host(x), pos, f, first, interleaved, 1.25)
    check(got, want, size, dtype)
    stay = np.ones(D, bool)
    stay[first:first + rot] = False
    assert np.array_equal(bits(got)[..., stay], bits(x)[..., stay])
    back = sv.rope(x, freqs, dev(pos), first=first, interleaved=interleaved, inverse=True)
    want, size = ref.turned(host(x), pos, f, first, interleaved, 1.0, True)
    check(back, want, size, dtype)
    y = x.clone()  # in place: the same bits
    assert sv.rope(y, freqs, dev(pos), first=first, amplitude=1.25, interleaved=interleaved, out=y) is y
    assert np.array_equal(bits(y), bits(got))


def test_rope_strides_and_negative_positions():
    """Parts of a wider projection, into a part of a wider tensor; left padding."""
    rng = np.random.default_rng(3)
    freqs = sv.rope_freqs(64)
    wide = dev(rng.normal(size=(2, 7, 640)), torch.bfloat16)
    x = wide[..., 128:384].unflatten(-1, (4, 64))
    room = torch.full((2, 7, 512), 3.0, dtype=torch.bfloat16, device=DEV)
    out = room[..., 256:].unflatten(-1, (4, 64))
    pos = np.arange(14, dtype=np.int32).reshape(2, 7) - 9
    sv.rope(x, freqs, dev(pos), out=out)
    want, size = ref.turned(host(x), pos, freqs.cpu().numpy(), 0, False)
    check(out, want, size, torch.bfloat16)
    assert bool((room[..., :256] == 3.0).all())
    with pytest.raises(ValueError):
        sv.rope(x[:, :, :, ::2], sv.rope_freqs(32), dev(pos))
    with pytest.raises(ValueError):
        sv.rope(x.transpose(0, 1), freqs, dev(pos.T.copy()))
    with pytest.raises(ValueError):
        sv.rope(x, freqs.int(), dev(pos))


def tables(rng, B, width, n):
    return rng.permutation(n)[:B * width].reshape(B, width).astype(np.int32)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,Hkv,Hq,rot,page,B,N,interleaved,by_pos", [
    (64, 1, 1, 64, 16, 1, 1, False, False), (64, 3, 6, 32, 16, 3, 5, True, True), (128, 2, 4, 128, 64, 2, 37, False, True),
    (128, 8, 32, 16, 32, 5, 6, False, False), (64, 5, 5, 48, 128, 2, 131, True, False),
    (128, 6, 6, 128, 16, 8, 1700, False, True)])
def test_append(e4m3, dtype, D, Hkv, Hq, rot, page, B, N, interleaved, by_pos):
    rng = np.random.default_rng([D, Hkv, page, N])
    width = (N + 40) // page + 2
    n = B * width + 2
    cache = sv.new_cache(n, Hkv, page, D, DEV, e4m3)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(7)
    table, starts = tables(rng, B, width, n), rng.integers(-3, 40, B).astype(np.int32)
    k, v = (dev(rng.normal(size=(B, N, Hkv, D)) * 2.0 ** rng.integers(-9, 9, (B, N, Hkv, 1)), dtype) for _ in "kv")
    q = dev(rng.normal(size=(B, N, Hq, D)), dtype)
    at = starts[:, None] + np.arange(N, dtype=np.int32)
    pos = at + 1000 if by_pos else at
    freqs = sv.rope_freqs(rot)
    f = freqs.cpu().numpy()
    got_q = sv.kv_append_rope(cache, dev(table), dev(starts), k, v, freqs, q=q, pos=dev(pos) if by_pos else None,
                              amplitude=0.75, interleaved=interleaved)
    want, size = ref.turned(host(q), pos, f, 0, interleaved, 0.75)
    check(got_q, want, size, dtype)
    want, size = ref.turned(host(k), pos, f, 0, interleaved, 0.75)
    got_k, got_v = sv.kv_read(cache, dev(table), dev(starts), N, dtype=torch.float32)
    held = (at >= 0) & (at < width * page)
    gk, gv = host(got_k)[held], host(got_v)[held]
    if not e4m3:
        bound = size * ref.TURN + np.abs(want) * HALF_BF16
        assert np.all(np.abs(gk - want[held]) <= bound[held] * (1 + 2.0 ** -20))
        wv = host(v.to(torch.bfloat16))[held]
        assert np.array_equal(gv, wv)
    else:
        # half a step of a byte: 2^-4 of it, or of the smallest normal's step under that;
        # the exponent is of a maximum that may be off by the turn's rounding
        _, e = attn_ref.quantise(want * (1 + 2.0 ** -20))
        step = np.maximum(np.abs(want) * 2.0 ** -4, 2.0 ** (e[..., None] - 10.0))
        assert np.all(np.abs(gk - want[held]) <= (step + size * ref.TURN)[held] * (1 + 2.0 ** -18))
        wv, e = attn_ref.quantise(host(v))
        assert np.array_equal(gv, (wv * 2.0 ** e[..., None])[held])
    # the pages nobody names are untouched
    other = np.setdiff1d(np.arange(n), np.unique(table))
    for t in (cache.k, cache.v):
        assert bool((t.view(torch.uint8)[torch.from_numpy(other).to(DEV)] == 7).all())


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_like_rope_then_append(e4m3):
    """One call gives what spec_rope in fp32 and spec_kv_append give one after the other, bit for bit."""
    rng = np.random.default_rng(8)
    B, N, Hkv, D, page = 3, 9, 4, 128, 16
    k, v = (dev(rng.normal(size=(B, N, Hkv, D)), torch.float32) for _ in "kv")
    table, starts = dev(np.arange(B * 3, dtype=np.int32).reshape(B, 3)), dev(np.array([0, 5, 30], np.int32))
    pos = (starts[:, None] + torch.arange(N, device=DEV)).int().contiguous()
    freqs = sv.rope_freqs(64)
    one, two = (sv.new_cache(9, Hkv, page, D, DEV, e4m3) for _ in range(2))
    sv.kv_append_rope(one, table, starts, k, v, freqs, amplitude=1.5)
    sv.kv_append(two, table, starts, sv.rope(k, freqs, pos, amplitude=1.5), v)
    for a, b in zip(one, two):
        assert a is None or np.array_equal(bits(a), bits(b))


def test_append_path():
    """The accepted path's keys: turned to their nodes' position indices, -1 skipped."""
    rng = np.random.default_rng(4)
    B, N, Hkv, D, page = 2, 21, 2, 64, 16
    k, v = (dev(rng.normal(size=(B, N, Hkv, D)), torch.bfloat16) for _ in "kv")
    rows = np.array([[0, 2, 9, -1], [0, -1, -1, -1]], np.int32)
    pos = rng.integers(0, 100, (B, N)).astype(np.int32)
    cache = sv.new_cache(6, Hkv, page, D, DEV)
    starts = np.array([14, 40], np.int32)
    table = np.arange(6, dtype=np.int32).reshape(2, 3)
    freqs = sv.rope_freqs(64)
    sv.kv_append_rope(cache, dev(table), dev(starts), k, v, freqs, rows=dev(rows), pos=dev(pos))
    got_k, got_v = sv.kv_read(cache, dev(table), dev(starts), 4, dtype=torch.float32)
    want, size = ref.turned(host(k), pos, freqs.cpu().numpy(), 0, False)
    for b in range(B):
        for t, r in enumerate(rows[b]):
            if r < 0:
                assert not got_k[b, t].any() and not got_v[b, t].any()
                continue
            bound = size[b, r] * ref.TURN + np.abs(want[b, r]) * HALF_BF16
            assert np.all(np.abs(host(got_k)[b, t] - want[b, r]) <= bound * (1 + 2.0 ** -20))
            assert np.array_equal(host(got_v)[b, t], host(v)[b, r])
    with pytest.raises(sv.SpecVerifyError):
        sv.kv_append_rope(cache, dev(table), dev(starts), k, v, freqs, q=k, rows=dev(rows))


def test_append_bad_pages_and_non_finite():
    """Bad pages and positions past the table are skipped; an infinite key becomes the NaN byte."""
    B, N, Hkv, D = 1, 6, 1, 64
    k = torch.ones((B, N, Hkv, D), device=DEV)
    k[0, 1, 0, 3] = float("inf")
    cache = sv.new_cache(2, Hkv, 16, D, DEV, True)
    freqs = sv.rope_freqs(64)
    table = dev(np.array([[0, 9]], np.int32))
    sv.kv_append_rope(cache, table, dev(np.array([12], np.int32)), k, k, freqs)
    raw = cache.k.view(torch.uint8)[0, 0].cpu().numpy()
    assert not raw[:12].any() and raw[12].any()
    assert np.array_equal(np.flatnonzero((raw[13] & 127) == 127), [3, 35])  # the pair of element 3
    assert not cache.k.view(torch.uint8)[1].any()
    assert not bool(cache.v.view(torch.uint8)[1].any())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("C,page,B,N,interleaved,turn", [
    (512, 64, 2, 5, True, True), (128, 16, 3, 37, False, True), (256, 128, 1, 1, True, False), (512, 32, 4, 300, False, True)])
def test_latent_append(dtype, C, page, B, N, interleaved, turn):
    rng = np.random.default_rng([C, page, N])
    width = (N + 40) // page + 2
    n = B * width + 1
    cache = sv.new_latent_cache(n, page, C, DEV)
    cache.data.fill_(5.0)
    table, starts = tables(rng, B, width, n), rng.integers(-2, 40, B).astype(np.int32)
    wide = dev(rng.normal(size=(B, N, C + 128)), dtype)
    c, r = wide[..., :C], wide[..., C + 64:]
    at = starts[:, None] + np.arange(N, dtype=np.int32)
    freqs = sv.rope_freqs(64, 10000.0, "linear", 4.0) if turn else None
    sv.latent_append(cache, dev(table), dev(starts), c, r, freqs, interleaved=interleaved, amplitude=0.5)
    data = host(cache.data)
    seen = np.zeros(data.shape[:2], bool)
    want, size = (ref.turned(host(r)[:, :, None], at, freqs.cpu().numpy(), 0, interleaved, 0.5) if turn
                  else (host(r.to(torch.bfloat16))[:, :, None], np.zeros((B, N, 1, 64))))
    wc = host(c.to(torch.bfloat16))
    for b in range(B):
        for t in range(N):
            if not 0 <= at[b, t] < width * page:
                continue
            p, s = table[b, at[b, t] // page], at[b, t] % page
            seen[p, s] = True
            assert np.array_equal(data[p, s, :C], wc[b, t])
            bound = size[b, t, 0] * ref.TURN + np.abs(want[b, t, 0]) * (HALF_BF16 if turn else 0.0)
            assert np.all(np.abs(data[p, s, C:] - want[b, t, 0]) <= bound * (1 + 2.0 ** -20))
    assert np.all(data[~seen] == 5.0)


def test_latent_append_path():
    rng = np.random.default_rng(5)
    c, r = dev(rng.normal(size=(2, 7, 128)), torch.bfloat16), dev(rng.normal(size=(2, 7, 64)), torch.bfloat16)
    rows, pos = np.array([[0, 4, -1], [0, 1, 6]], np.int32), rng.integers(0, 50, (2, 7)).astype(np.int32)
    cache = sv.new_latent_cache(2, 16, 128, DEV)
    freqs = sv.rope_freqs(64)
    sv.latent_append(cache, dev(np.array([[1], [0]], np.int32)), dev(np.array([3, 14], np.int32)), c, r, freqs,
                     rows=dev(rows), pos=dev(pos))
    want, size = ref.turned(host(r)[:, :, None], pos, freqs.cpu().numpy(), 0, False)
    data, used = host(cache.data), []
    for b, page, t, token in ((0, 1, 3, 0), (0, 1, 4, 4), (1, 0, 14, 0), (1, 0, 15, 1)):  # the sixth falls past the table
        assert np.array_equal(data[page, t, :128], host(c)[b, token])
        bound = size[b, token, 0] * ref.TURN + np.abs(want[b, token, 0]) * HALF_BF16
        assert np.all(np.abs(data[page, t, 128:] - want[b, token, 0]) <= bound * (1 + 2.0 ** -20))
        used.append((page, t))
    for page in range(2):
        for t in range(16):
            assert (page, t) in used or not data[page, t].any()


def test_captured():
    """A captured call follows new positions."""
    x = torch.randn((2, 3, 4, 64), device=DEV)
    freqs, pos = sv.rope_freqs(64), torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.rope(x, freqs, pos, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.rope(x, freqs, pos, out=out)
    pos.fill_(77)
    graph.replay()
    assert torch.equal(out, sv.rope(x, freqs, pos))


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_past_32_bits(e4m3):
    """A cache of more than 2^31 elements, its last pages written and read back."""
    n, Hkv, page, D = 33000, 8, 64, 128  # 65536 elements a page
    shape = (n, Hkv, page, D)
    if e4m3:
        k, v = (torch.empty(shape, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in "kv")
        ke, ve = (torch.empty(shape[:3], dtype=torch.int8, device=DEV) for _ in "kv")
    else:
        k, v = (torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in "kv")
        ke = ve = None
    assert k.numel() > 2 ** 31
    big, small = sv.KVCache(k, v, ke, ve), sv.new_cache(2, Hkv, page, D, DEV, e4m3=e4m3)
    x = torch.randn((1, 100, Hkv, D), device=DEV).to(torch.bfloat16)
    freqs, zero = sv.rope_freqs(D), dev(np.zeros(1, np.int32))
    got = []
    for cache, table in ((big, [[n - 1, n - 2]]), (small, [[0, 1]])):
        table = dev(np.array(table, np.int32))
        q = sv.kv_append_rope(cache, table, zero, x, x, freqs, q=x)
        got.append((q, *sv.kv_read(cache, table, zero, 100)))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_a_step_captured():
    """Rotated queries and keys and the attention that reads both, in one captured graph: each waits for the one ahead."""
    B, N, H, Hkv, D, page = 3, 5, 8, 2, 64, 16
    g = torch.Generator(DEV)
    g.manual_seed(3)
    cache = sv.new_cache(40, Hkv, page, D, DEV)
    table = torch.arange(39, dtype=torch.int32, device=DEV).view(B, 13)
    freqs = sv.rope_freqs(D)
    held = torch.tensor([100, 7, 64], dtype=torch.int32, device=DEV)
    lens = held + N
    x = [torch.randn((B, N, h, D), generator=g, device=DEV).bfloat16() for h in (H, Hkv, Hkv)]
    old = torch.randn((B, 120, Hkv, D), generator=g, device=DEV).bfloat16()
    sv.kv_append(cache, table, held - held, old, old)

    def step(q, k, v):
        q = sv.kv_append_rope(cache, table, held, k, v, freqs, q=q)
        return sv.attn_tree(q, cache, table, lens)

    step(*x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*x)
    for _ in range(5):
        for t in x:
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        pos = held[:, None] + torch.arange(N, dtype=torch.int32, device=DEV)
        sv.kv_append(cache, table, held, sv.rope(x[1], freqs, pos), x[2])
        assert torch.equal(got, sv.attn_tree(sv.rope(x[0], freqs, pos), cache, table, lens))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_outputs_beside_inputs(dtype):
    """Outputs between the parts of one projection, and in place; outputs over what is still read are refused."""
    rng = np.random.default_rng(12)
    B, N, Hq, Hkv, D = 3, 5, 6, 2, 64
    freqs, table, starts = sv.rope_freqs(D), dev(np.arange(6, dtype=np.int32).reshape(3, 2)), dev(np.array([0, 3, 9], np.int32))
    wide = dev(rng.normal(size=(B, N, 2 * Hq + 2 * Hkv, D)), dtype)
    q, spare, k, v = wide.split((Hq, Hq, Hkv, Hkv), 2)
    pos = (starts[:, None] + torch.arange(N, device=DEV)).int()
    want = sv.rope(q.contiguous(), freqs, pos)
    assert torch.equal(sv.rope(q, freqs, pos, out=spare), want) and torch.equal(spare, want)
    spare.zero_()
    caches = [sv.new_cache(6, Hkv, 16, D, DEV) for _ in range(2)]
    sv.kv_append_rope(caches[0], table, starts, k.contiguous(), v.contiguous(), freqs)
    assert torch.equal(sv.kv_append_rope(caches[1], table, starts, k, v, freqs, q=q, out_q=spare), want)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    before = wide.clone()
    for bad in (wide[:, :, 1:Hq + 1], wide[:, :, Hq - 1:2 * Hq - 1]):
        with pytest.raises(sv.SpecVerifyError):
            sv.rope(q, freqs, pos, out=bad)
        with pytest.raises(sv.SpecVerifyError):
            sv.kv_append_rope(caches[1], table, starts, k, v, freqs, q=q, out_q=bad)
    with pytest.raises(sv.SpecVerifyError):
        sv.kv_append_rope(caches[1], table, starts, k, v, freqs, q=q, out_q=wide[:, :, Hq + 1:2 * Hq + 1])
    assert torch.equal(wide, before)
    assert sv.rope(q, freqs, pos, out=q) is q and torch.equal(q, want)
