"""Attention over a latent cache on the GPU against the 64-bit form."""
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

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


def seen_by(N, length, mask):
    s = np.ones((N, length), bool)
    among = np.tril(np.ones((N, N), bool)) if mask is None else mask != 0
    s[:, length - min(N, length):] = among[:, N - min(N, length):]
    return s


def make(rng, B, N, H, C, page, lens, mask=None, big=1.0):
    width = max(1, -(-max(lens) // page))
    n = B * width + 2
    cache = sv.new_latent_cache(n, page, C, DEV)
    cache.data.copy_(torch.randn(cache.data.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(int(rng.integers(99999)))) * big)
    table = rng.permutation(n)[:B * width].reshape(B, width).astype(np.int32)
    q = dev(rng.normal(size=(B, N, H, C + 64)), torch.bfloat16)
    return cache, table, q, None if mask is None else dev(mask.astype(np.uint8))


def check(got, lse, cache, table, q, lens, scale, mask=None, some=None):
    C, page = cache.descriptor.C, cache.descriptor.page
    data, q, got, lse = host(cache.data), host(q), host(got), host(lse)
    for b in range(len(lens)):
        j = np.arange(lens[b])
        K = data[table[b][j // page], j % page]
        seen = seen_by(q.shape[1], lens[b], None if mask is None else mask[b])
        heads = range(q.shape[2]) if some is None else some
        want, wl, spread, size = ref.latent(q[b][:, list(heads)], K, C, seen, scale)
        g, gl = got[b][:, list(heads)], lse[b][:, list(heads)]
        # a score: C + 64 products and sums in fp32, and its factor; the maximum's too
        ds = np.where(np.isfinite(wl), size * (C + 72) * 2.0 ** -24, 0.0)
        assert np.array_equal(np.isneginf(wl), np.isneginf(gl))
        fin = np.isfinite(wl)
        # the sum of weights: at most 2^-12 off (128 sums of 2^-24 a tile and its rescaling)
        assert np.all(np.abs(gl[fin] - wl[fin]) <= (2 * ds + 2.0 ** -12)[fin] + np.abs(wl[fin]) * 2.0 ** -22)
        # weights rounded to bf16, the sum's and scores' errors, the output's rounding
        bound = spread * (HALF_BF16 + 4 * ds[..., None] + 2.0 ** -11) + np.abs(want) * HALF_BF16
        nan = np.isnan(want)
        assert np.array_equal(nan, np.isnan(g))
        inf = np.isinf(want)
        assert np.array_equal(g[inf], want[inf])
        ok = ~nan & ~inf
        assert np.all(np.abs(g - want)[ok] <= bound[ok] + 1e-30)


def call(q, cache, table, lens, scale, mask=None):
    ws = sv.new_workspace(sv.spec_latent_workspace_size(q.shape[0], q.shape[1], q.shape[2], cache.descriptor.C), DEV)
    ws[256:].fill_(255)  # any state past the error word
    out, lse = sv.latent_attn(q, cache, dev(table), dev(np.array(lens, np.int32)), scale, mask=mask, lse=True, workspace=ws)
    return out, lse, sv.last_error(ws)


def trees(rng, B, N):
    m = np.zeros((B, N, N), np.uint8)
    for b in range(B):
        for n in range(N):
            if n:
                m[b, n] = m[b, rng.integers(max(0, n - 5), n)]
            m[b, n, n] = 1
    return m


@pytest.mark.parametrize("B,N,H,C,page,lens", [
    (1, 1, 1, 512, 16, [1]), (1, 1, 16, 512, 64, [63]), (1, 1, 16, 512, 64, [64]), (2, 1, 16, 256, 32, [65, 2]),
    (1, 2, 128, 512, 64, [129]), (3, 6, 32, 512, 64, [6, 200, 77]), (2, 3, 20, 128, 128, [300, 3]),
    (1, 8, 7, 512, 16, [1000]), (4, 1, 64, 128, 16, [5, 128, 129, 700]), (2, 5, 13, 256, 128, [130, 127]),
    (1, 4, 65, 512, 32, [513]), (5, 6, 128, 512, 64, [70, 64, 6, 333, 128])])
def test_chain(B, N, H, C, page, lens):
    rng = np.random.default_rng([B, N, H, C])
    cache, table, q, _ = make(rng, B, N, H, C, page, lens)
    scale = 192 ** -0.5
    out, lse, err = call(q, cache, table, lens, scale)
    assert err == 0
    check(out, lse, cache, table, q, lens, scale, some=range(0, H, max(1, H // 9)))
    again, _, _ = call(q, cache, table, lens, scale)
    assert torch.equal(out, again)


@pytest.mark.parametrize("B,N,H,C,page,lens", [
    (1, 9, 4, 512, 16, [9]), (2, 21, 16, 512, 64, [100, 64]), (1, 85, 8, 256, 32, [300]), (3, 70, 3, 128, 128, [70, 150, 71]),
    (1, 130, 16, 512, 64, [400])])
def test_tree(B, N, H, C, page, lens):
    rng = np.random.default_rng([B, N, H, C, 1])
    mask = trees(rng, B, N)
    mask[0, N // 2] = 0  # a node that sees only the context
    cache, table, q, m = make(rng, B, N, H, C, page, lens, mask)
    out, lse, err = call(q, cache, table, lens, 0.07, m)
    assert err == 0
    check(out, lse, cache, table, q, lens, 0.07, mask, some=range(0, H, max(1, H // 3)))


@pytest.mark.parametrize("H,lens", [(16, [20000]), (128, [6001, 9, 3000])])
def test_long(H, lens):
    """Units cut into many shares, joined."""
    rng = np.random.default_rng(H)
    B = len(lens)
    cache, table, q, _ = make(rng, B, 2, H, 512, 64, lens)
    out, lse, err = call(q, cache, table, lens, 192 ** -0.5)
    assert err == 0
    check(out, lse, cache, table, q, lens, 192 ** -0.5, some=range(0, H, max(1, H // 4)))


def test_large_scores():
    """Maxima that grow tile by tile, a negative and a zero scale."""
    rng = np.random.default_rng(1)
    lens = [500]
    cache, table, q, _ = make(rng, 1, 2, 16, 512, 16, lens)
    for t in range(32):
        cache.data[int(table[0, t])].mul_(0.2 * (t + 1))
    for scale in (0.5, -0.5, 0.0):
        out, lse, _ = call(q, cache, table, lens, scale)
        check(out, lse, cache, table, q, lens, scale)


def test_nothing_seen_and_empty():
    """Masks that leave a row empty, lengths of zero, and rows of other sequences as they were."""
    rng = np.random.default_rng(2)
    mask = np.zeros((3, 4, 4), np.uint8)
    mask[1] = np.tril(np.ones((4, 4)))
    cache, table, q, m = make(rng, 3, 4, 16, 512, 16, [4, 20, 1], mask)
    lens = [4, 20, 0]
    out, lse, err = call(q, cache, table, lens, 0.1, m)
    assert err == 0
    assert not out[0].any() and bool(torch.isneginf(lse[0]).all())
    assert not out[2].any() and bool(torch.isneginf(lse[2]).all())
    check(out[:2], lse[:2], cache, table[:2], q[:2], lens[:2], 0.1, mask[:2])


def test_unseen_not_finite():
    """What a row does not see adds nothing whatever it holds; what it sees does."""
    rng = np.random.default_rng(3)
    N, lens = 6, [70, 134]
    mask = np.tril(np.ones((2, N, N), np.uint8))
    cache, table, q, m = make(rng, 2, N, 16, 512, 16, lens, mask)
    for b in range(2):  # behind the last position, and the last new token
        for j, x in ((lens[b] - 1, float("nan")), (lens[b] - 2, float("inf"))):
            if b == 0:
                cache.data[int(table[b, j // 16]), j % 16] = x
        last = lens[b] % 16
        if last:
            cache.data[int(table[b, lens[b] // 16]), last:] = float("nan")
    out, lse, err = call(q, cache, table, lens, 0.1, m)
    assert err == 0
    assert bool(torch.isfinite(out[0, :N - 2]).all()) and bool(torch.isnan(out[0, N - 1]).all())
    assert bool(torch.isfinite(out[1]).all())
    check(out[:, :N - 2], lse[:, :N - 2], cache, table, q[:, :N - 2].contiguous(), [n - 2 for n in lens], 0.1,
          mask[:, :N - 2, :N - 2])
    # an infinite latent element that is seen with a finite score
    cache, table, q, _ = make(rng, 1, 3, 16, 128, 16, [40])
    cache.data[int(table[0, 2]), 5, 7] = float("inf")  # position 37: the first new token
    q[..., 7] = 0.0
    q[0, :, :, 7] = 1e-30
    out, lse, err = call(q, cache, table, [40], 0.1)
    # its score is infinite for all that see it: NaN
    assert bool(torch.isnan(out).all())


def test_bad_lengths_and_pages():
    rng = np.random.default_rng(4)
    lens = [40, 40, 40, 40]
    cache, table, q, _ = make(rng, 4, 2, 16, 512, 16, lens)
    want, _, _ = call(q, cache, table, lens, 0.1)
    bad = table.copy()
    bad[1, 1] = cache.descriptor.num_pages
    bad[2, 2] = -1
    out, lse, err = call(q, cache, bad, [40, 40, 40, 49], 0.1)
    assert err == sv.SPEC_DATA_PAGE_RANGE
    assert torch.equal(out[0], want[0])
    for b in (1, 2, 3):
        assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all())
    out, _, err = call(q, cache, bad, [40, 16, 32, -1], 0.1)
    assert err == sv.SPEC_DATA_PAGE_RANGE
    assert bool(torch.isfinite(out[:3]).all()) and bool(torch.isnan(out[3]).all())


def test_strides_streams_and_captured():
    """Queries inside a wider projection, another stream, and a captured call that follows the lengths."""
    rng = np.random.default_rng(5)
    lens = [100, 37]
    cache, table, q, _ = make(rng, 2, 3, 16, 256, 32, lens)
    want, _, _ = call(q, cache, table, lens, 0.1)
    wide = torch.zeros((2, 3, 16 * 320 + 64), dtype=torch.bfloat16, device=DEV)
    part = wide[..., 64:].unflatten(-1, (16, 320))
    part.copy_(q)
    t, n = dev(table), dev(np.array(lens, np.int32))
    assert torch.equal(sv.latent_attn(part, cache, t, n, 0.1), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = sv.latent_attn(part, cache, t, n, 0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    ws = sv.new_workspace(sv.spec_latent_workspace_size(2, 3, 16, 256), DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.latent_attn(part, cache, t, n, 0.1, out=out, workspace=ws)
    n.copy_(torch.tensor([20, 90], device=DEV))
    table[1] = table[0]
    t.copy_(dev(table))
    graph.replay()
    assert torch.equal(out, sv.latent_attn(q, cache, t, n, 0.1)) and sv.last_error(ws) == 0
    with pytest.raises(ValueError):
        sv.latent_attn(q[..., :256], cache, t, n, 0.1)


def test_append_attend_verify():
    """The run of a step: rotate, append, attend, and the accepted path appended again gives plain decoding's cache."""
    rng = np.random.default_rng(6)
    C, page, H, held = 128, 16, 16, 30
    parents = np.array([-1, 0, 0, 1, 3], np.int32)
    N = len(parents)
    cache = sv.new_latent_cache(4, page, C, DEV)
    plain = sv.new_latent_cache(4, page, C, DEV)
    table = dev(np.arange(4, dtype=np.int32)[None])
    freqs = sv.rope_freqs(64)
    zero = dev(np.zeros(1, np.int32))
    c, r = dev(rng.normal(size=(1, held, C)), torch.bfloat16), dev(rng.normal(size=(1, held, 64)), torch.bfloat16)
    for x in (cache, plain):
        sv.latent_append(x, table, zero, c, r, freqs, interleaved=True)
    mask, _, pos = sv.tree_mask(dev(parents[None]), dev(np.array([held], np.int32)))
    c, r = dev(rng.normal(size=(1, N, C)), torch.bfloat16), dev(rng.normal(size=(1, N, 64)), torch.bfloat16)
    q = dev(rng.normal(size=(1, N, H, C + 64)), torch.bfloat16)
    q = sv.rope(q, freqs, pos, first=C, interleaved=True)
    start = dev(np.array([held], np.int32))
    sv.latent_append(cache, table, start, c, r, freqs, pos=pos, interleaved=True)
    out = sv.latent_attn(q, cache, table, start + N, 0.1, mask=mask)
    path = dev(np.array([[0, 1, 3, 4, -1]], np.int32))
    sv.latent_append(cache, table, start, c, r, freqs, rows=path, pos=pos, interleaved=True)
    on = [0, 1, 3, 4]
    sv.latent_append(plain, table, start, c[:, on].contiguous(), r[:, on].contiguous(), freqs, interleaved=True)
    assert torch.equal(cache.data.flatten(0, 1)[:held + 4], plain.data.flatten(0, 1)[:held + 4])
    one = sv.latent_attn(q[:, on].contiguous(), plain, table, start + 4, 0.1)
    # the same values in another order of positions: twice the forms' own distance
    assert float((out[:, on] - one).float().abs().max()) <= 2.0 ** -6 * float(one.float().abs().max())


@pytest.mark.parametrize("C,page", [(128, 16), (256, 64), (512, 32), (512, 128)])
def test_bad_pages_among_many_sequences(C, page):
    """Many short sequences a CTA, some with a bad page: those fail, and no others, call after call."""
    rng = np.random.default_rng([C, page])
    B = 700
    lens = rng.integers(1, 150, B).tolist()
    lens[3] = lens[-1] = 140
    cache, table, q, _ = make(rng, B, 2, 16, C, page, lens)
    want, wl, err = call(q, cache, table, lens, 0.05)
    assert err == 0
    bad = np.zeros(B, bool)
    bad[[3, B - 1]] = bad[rng.choice(B, 40, replace=False)] = True
    broken = table.copy()
    for b in np.flatnonzero(bad):
        broken[b, rng.integers(0, -(-lens[b] // page))] = rng.choice([-1, cache.descriptor.num_pages])
    at = torch.from_numpy(bad).to(DEV)
    for _ in range(3):
        out, lse, err = call(q, cache, broken, lens, 0.05)
        assert err == sv.SPEC_DATA_PAGE_RANGE
        assert bool(torch.isnan(out[at]).all()) and bool(torch.isnan(lse[at]).all())
        assert torch.equal(out[~at], want[~at]) and torch.equal(lse[~at], wl[~at])


@pytest.mark.parametrize("B,N,H,C,page,longest,tree", [
    (30, 6, 32, 512, 64, 4000, False), (9, 40, 20, 512, 16, 3000, True), (64, 1, 16, 256, 32, 2500, False),
    (12, 24, 64, 128, 128, 5000, True)])
def test_same_bits(B, N, H, C, page, longest, tree):
    """Results do not depend on timing: calls back to back, with others between, give the same bits."""
    rng = np.random.default_rng([B, N, H, C, 7])
    lens = rng.integers(N, longest, B).tolist()
    mask = trees(rng, B, N) if tree else None
    cache, table, q, m = make(rng, B, N, H, C, page, lens, mask)
    t, n = dev(table), dev(np.array(lens, np.int32))
    ws = sv.new_workspace(sv.spec_latent_workspace_size(B, N, H, C), DEV)
    out, lse = sv.latent_attn(q, cache, t, n, 0.06, mask=m, lse=True, workspace=ws)
    check(out[:2], lse[:2], cache, table[:2], q[:2], lens[:2], 0.06, None if mask is None else mask[:2], some=range(0, H, 7))
    short = dev(np.minimum(lens, N + 3).astype(np.int32))
    for i in range(25):
        if i % 3 == 0:
            sv.latent_attn(q, cache, t, short, 0.06, mask=m, workspace=ws)
        again, again_lse = sv.latent_attn(q, cache, t, n, 0.06, mask=m, lse=True, workspace=ws)
        assert torch.equal(again, out) and torch.equal(again_lse, lse)
    assert sv.last_error(ws) == 0


def test_past_32_bits():
    """A cache of more than 2^31 elements, its last pages in use."""
    C, page, n = 512, 64, 58300  # 58300 * 64 * 576 elements
    cache = sv.LatentCache(torch.empty((n, page, C + 64), dtype=torch.bfloat16, device=DEV))
    assert cache.data.numel() > 2 ** 31
    rng = np.random.default_rng(8)
    lens, table = [130], (n - 1 - np.arange(3, dtype=np.int32))[None]
    c, r = dev(rng.normal(size=(1, 130, C)), torch.bfloat16), dev(rng.normal(size=(1, 130, 64)), torch.bfloat16)
    sv.latent_append(cache, dev(table), dev(np.zeros(1, np.int32)), c, r)
    got = cache.data[n - 3:].flip(0).flatten(0, 1)[:130]
    assert torch.equal(got, torch.cat((c[0], r[0]), -1))
    q = dev(rng.normal(size=(1, 2, 16, C + 64)), torch.bfloat16)
    out, lse, err = call(q, cache, table, lens, 0.06)
    assert err == 0
    few = types.SimpleNamespace(data=cache.data[n - 3:], descriptor=cache.descriptor)
    check(out, lse, few, table - (n - 3), q, lens, 0.06)


def test_two_graphs_and_two_streams():
    """Two captured calls that share a workspace, replayed in turn; two streams with a workspace each, at once."""
    rng = np.random.default_rng(9)
    made_ = []
    for C, lens in ((512, [900, 40, 333]), (128, [70, 1500, 8])):
        cache, table, q, _ = make(rng, 3, 4, 32, C, 32, lens)
        made_.append((q, cache, dev(table), dev(np.array(lens, np.int32))))
    want = [sv.latent_attn(q, c, t, n, 0.06) for q, c, t, n in made_]
    size = max(sv.spec_latent_workspace_size(3, 4, 32, C) for C in (512, 128))
    ws = sv.new_workspace(size, DEV)
    graphs, outs = [], []
    for q, c, t, n in made_:
        out = torch.empty(q.shape[:3] + (c.descriptor.C,), dtype=q.dtype, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.latent_attn(q, c, t, n, 0.06, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for i in (0, 1, 1, 0, 1, 0, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
    assert sv.last_error(ws) == 0
    sides = [torch.cuda.Stream() for _ in made_]
    spaces = [sv.new_workspace(size, DEV) for _ in made_]
    torch.cuda.synchronize()
    for _ in range(20):
        for (q, c, t, n), out, s, w in zip(made_, outs, sides, spaces):
            sv.latent_attn(q, c, t, n, 0.06, out=out, workspace=w, stream=s)
    torch.cuda.synchronize()
    for out, w, o in zip(outs, want, spaces):
        assert torch.equal(out, w) and sv.last_error(o) == 0


ONE, SPLIT, MANY = [40], [2560], [134] * 304  # one tile; a tile a share, joined; whole units, two a share


@pytest.mark.parametrize("C", [128, 256, 512])
@pytest.mark.parametrize("lens,where", [
    (ONE, [36]), (ONE, [5, 39]), (SPLIT, [200]), (SPLIT, range(192, 256)), (SPLIT, [2557]), (SPLIT, [3, 2554]),
    (MANY, [10]), (MANY, range(64)), (MANY, range(128)), (MANY, [131]), ([6], range(6)), ([70], range(70))])
def test_infinite_latents(C, lens, where):
    """Seen infinite elements whose score is -inf: their weight is 0 and 0 * inf makes the element NaN, wherever the
    position lies; the row's others are as without the position, and a row without another is NaN."""
    rng = np.random.default_rng([C, len(lens), lens[0], len(where)])
    N, H, marks = 6, 8, (0, len(lens) - 4 if len(lens) > 4 else 0)
    cache, table, q, _ = make(rng, len(lens), N, H, C, 32, lens)
    at = [7, C - 3]
    x = q[..., at].float().abs() + 0.25
    for sign, scale in ((1.0, 0.07), (-1.0, 0.07), (1.0, -0.07)):
        q[..., at] = (-x if sign * scale > 0 else x).to(q.dtype)
        for b in marks:
            for i, j in enumerate(where):
                cache.data[int(table[b, j // 32]), j % 32, at[i % 2]] = sign * float("inf")
        out, lse, err = call(q, cache, table, lens, scale)
        assert err == 0
        for b in {*marks, len(lens) // 2}:
            K, j = host(cache.data[torch.from_numpy(table[b]).to(DEV).long()]).reshape(-1, C + 64)[:lens[b]], np.arange(lens[b])
            odd, seen = ~np.isfinite(K), seen_by(N, lens[b], None)
            finite = ~odd.any(-1)
            assert finite.all() == (b not in marks)
            want, wl, spread, size = ref.latent(host(q[b]), np.where(odd, 0.0, K), C, seen & finite, scale)
            for i in range(N):
                nan = odd[j[seen[i]], :C].any(0) | (not (seen[i] & finite).any())
                got, gl = host(out[b, i]), host(lse[b, i])
                assert np.array_equal(np.isnan(got), np.broadcast_to(nan, got.shape))
                assert np.array_equal(np.isneginf(gl), np.isneginf(wl[i]))
                some, ds = np.isfinite(wl[i]), size[i] * (C + 72) * 2.0 ** -24  # as in check()
                off, bound = np.abs(gl[some] - wl[i][some]), np.abs(wl[i][some]) * 2.0 ** -22
                assert np.all(off <= 2 * ds[some] + 2.0 ** -12 + bound)
                bound = spread[i] * (HALF_BF16 + 4 * ds[:, None] + 2.0 ** -11) + np.abs(want[i]) * HALF_BF16
                assert np.all((np.abs(got - want[i]) <= bound + 1e-30)[:, ~nan])


@pytest.mark.parametrize("C", [128, 256, 512])
@pytest.mark.parametrize("N,H,lens,tree", [
    (40, 4, [1, 5, 39, 40, 17], False), (40, 4, [1, 5, 39, 40, 17], True), (130, 3, [70, 129, 1, 64, 65], False),
    (130, 3, [70, 129, 1, 64, 65], True), (6, 16, [1, 2, 5] * 70, False)])
def test_shorter_than_the_new_tokens(C, N, H, lens, tree):
    """Caches that hold the last new tokens only: the first tokens see nothing, beside rows of the unit that do."""
    rng = np.random.default_rng([C, N, len(lens), tree])
    mask = trees(rng, len(lens), N) if tree else None
    cache, table, q, m = make(rng, len(lens), N, H, C, 16, lens, mask)
    out, lse, err = call(q, cache, table, lens, 0.07, m)
    assert err == 0
    if not tree:
        for b, n in enumerate(lens):
            assert not out[b, :N - n].any() and bool(torch.isneginf(lse[b, :N - n]).all())
            assert bool(torch.isfinite(lse[b, N - n:]).all())
    few = slice(0, 5)
    check(out[few], lse[few], cache, table[few], q[few], lens[few], 0.07, None if mask is None else mask[few])


@pytest.mark.parametrize("B,N,H", [(129, 128, 128), (2200000, 1, 1)])
def test_many_rows(B, N, H):
    """More than 2^21 query rows: long trees of many heads, and many short sequences, the last ones among them."""
    rng = np.random.default_rng([B, N, H])
    cache, _, _, _ = make(rng, 1, 1, 1, 128, 16, [16 * 40])
    # sequences share their pages: each starts at one of 16 of them
    table = ((np.arange(B)[:, None] * 7 + np.arange(16 if N > 1 else 1)) % 40).astype(np.int32)
    lens = np.minimum(N + np.arange(B) % 90, 16 * table.shape[1]).astype(np.int32)
    if N == 1:
        lens = (np.arange(B) % 17).astype(np.int32)
    q = torch.randn((B, N, H, 192), dtype=torch.bfloat16, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    out, lse, err = call(q, cache, table, lens, 0.07)
    assert err == 0
    few = [0, 1, B // 2, B - 2, B - 1]
    check(out[few], lse[few], cache, table[few], q[few], lens[few], 0.07, some=range(0, H, 31))
    assert not out[lens == 0].any()
