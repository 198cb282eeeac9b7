"""The target pass's attention on the GPU against the plain 64-bit form.

Tolerance of an output element, from the arithmetic (fixed before the first
run): the result's rounding to bf16 gives 2^-9 |out|; rounding each weight to
bf16 gives at most 2^-9 sum p |v|, to two e4m3 terms at most 2^-8 sum p |v|
plus an absolute 2^-15 of the largest weight per position ("floor"); fp32
scores of magnitude up to ~30 and sums give under 2^-14 of sum p |v|.  The
bounds below are twice the sum of these.  lse: fp32 scores and sums, 4e-4
absolute.
"""
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
TABLE = ref.e4m3_table()


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


class Problem:
    """Seeded inputs; every position no sequence holds is NaN."""

    def __init__(self, seed, lens, N, Hq, H, D, page, e4m3, shared=0, tree=False, slack=1):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.N, self.Hq, self.H, self.D, self.page = lens, N, Hq, H, D, page
        self.shared, self.B = shared, len(lens)
        B = self.B
        width = max([1] + [-(-n // page) for n in lens]) + slack
        sp = -(-shared // page)
        n = B * width + sp + 2
        ids = rng.permutation(n)
        self.table = ids[:B * width].reshape(B, width).astype(np.int32)
        self.stable = ids[B * width:B * width + sp].astype(np.int32)
        self.cache = sv.new_cache(n, H, page, D, DEV, e4m3)
        for t in (self.cache.k, self.cache.v):
            (t.view(torch.uint8).fill_(0x7f) if e4m3 else t.fill_(float("nan")))
        if e4m3:
            self.cache.k_exp.fill_(77)
            self.cache.v_exp.fill_(-77)
        self.K, self.V = [], []
        for tab, count in [(self.table[b], lens[b]) for b in range(B)] + [(self.stable, shared)]:
            kv = []
            for t, ex in ((self.cache.k, self.cache.k_exp), (self.cache.v, self.cache.v_exp)):
                x = rng.normal(size=(count, H, D)).astype(np.float32)
                x *= rng.choice([0.5, 1.0, 2.0], size=(count, H, 1))
                pid, slot = ref.positions(tab, page, count)
                pid, slot = dev(pid.astype(np.int64)), dev(slot.astype(np.int64))
                if e4m3:
                    y, e = ref.quantise(x)
                    b8 = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8)
                    t.view(torch.uint8)[pid, :, slot] = b8.to(DEV)
                    ex[pid, :, slot] = dev(e.astype(np.int8))
                    kv.append(y * 2.0 ** e[..., None].astype(float))
                else:
                    r = torch.from_numpy(x).to(torch.bfloat16)
                    t[pid, :, slot] = r.to(DEV)
                    kv.append(r.double().numpy())
            self.K.append(kv[0])
            self.V.append(kv[1])
        self.Ks, self.Vs = self.K.pop(), self.V.pop()
        self.q = dev(rng.normal(size=(B, N, Hq, D)), torch.bfloat16)
        self.mask = self.pos = None
        if tree:
            m, p = np.zeros((B, N, N), np.uint8), np.zeros((B, N), np.int32)
            for b in range(B):
                for i in range(N):
                    if i:
                        par = int(rng.integers(max(0, i - 6), i))
                        m[b, i], p[b, i] = m[b, par], p[b, par] + 1
                    m[b, i, i] = 1
                p[b] += shared + lens[b] - N
            self.mask, self.pos = m, p

    def run(self, lse=True, workspace=None, stream=None, q=None, **kw):
        args = (dev(self.table), dev(np.asarray(self.lens, np.int32)))
        kw.update(mask=None if self.mask is None else dev(self.mask),
                  pos=None if self.pos is None else dev(self.pos), lse=lse, workspace=workspace,
                  stream=stream)
        if kw.get("slopes") is not None:
            kw["slopes"] = dev(np.asarray(kw["slopes"], np.float32))
        q = self.q if q is None else q
        if stream is not None:
            torch.cuda.synchronize()
        if self.shared:
            return sv.attn_shared(q, self.cache, dev(self.stable), self.shared, *args, **kw)
        return sv.attn_tree(q, self.cache, *args, **kw)

    def want(self, b, scale=None, cap=0.0, window=0, slopes=None):
        N, L, Ls = self.N, self.lens[b], self.shared
        K, V = np.concatenate((self.Ks, self.K[b])), np.concatenate((self.Vs, self.V[b]))
        first = L - N
        pos = Ls + first + np.arange(N) if self.pos is None else self.pos[b].astype(np.int64)
        jpos = np.arange(Ls + L)
        seen = np.ones((N, Ls + L), bool)
        for c in range(N):
            if first + c < 0:
                continue
            j = Ls + first + c
            jpos[j] = pos[c]
            seen[:, j] = (np.arange(N) >= c) if self.mask is None else self.mask[b][:, c] != 0
        if self.mask is None:
            for i in range(N):
                if first + i < 0 and not Ls:
                    assert not seen[i].any()
        far = pos[:, None] - jpos[None, :]
        if window:
            seen &= far < window
        scale = self.D ** -0.5 if scale is None else scale
        return ref.attention(self.q[b].double().cpu().numpy(), K, V, seen, far, slopes, scale, cap)

    def check(self, only=None, **kw):
        out, lse = self.run(**kw)
        torch.cuda.synchronize()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        e4m3 = self.cache.k.dtype == torch.float8_e4m3fn
        for b in range(self.B) if only is None else only:
            o, e, spread, floor = self.want(b, **kw)
            tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -7 + 2.0 ** -13 if e4m3 else 2.0 ** -8 + 2.0 ** -13) * spread
            tol += 2.0 ** -14 * floor if e4m3 else 0.0
            assert np.all(np.isfinite(out[b])), "sequence %d: not finite" % b
            worst = np.max(np.abs(out[b] - o) - tol)
            assert worst <= 0, "sequence %d: off by %g over the bound" % (b, worst)
            fin = np.isfinite(e)
            np.testing.assert_array_equal(lse[b][~fin], e[~fin])
            assert np.all(np.abs(lse[b][fin] - e[fin]) <= 4e-4)


SHAPES = [  # lens, N, Hq, Hkv, D, page
    ([1], 1, 1, 1, 64, 16),
    ([5, 0, 17], 1, 4, 2, 64, 16),
    ([2, 300, 129, 128, 127], 3, 8, 2, 128, 64),
    ([700, 1, 64, 0, 333], 6, 32, 8, 128, 64),
    ([511, 515], 4, 28, 4, 128, 32),
    ([400, 257], 5, 12, 12, 64, 128),
    ([390, 100], 40, 8, 1, 128, 16),   # 320 rows a key/value head
    ([200, 333], 130, 4, 2, 64, 32),   # more new tokens than a tile
    ([600, 70, 129, 12], 12, 8, 2, 128, 64),   # 48 rows a key/value head
    ([300, 31, 256], 16, 4, 1, 64, 16),        # 64 rows
    ([500, 27, 260], 25, 12, 4, 128, 32),      # 75 rows
    ([260, 131], 32, 8, 2, 64, 128),           # 128 rows
    ([129, 400], 43, 12, 4, 128, 64),          # 129 rows: a unit of two row tiles
    ([3, 1, 2] * 100, 1, 2, 1, 64, 16),        # many short sequences
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_chain(shape, e4m3):
    Problem(1, *shape, e4m3).check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("opts", [dict(cap=5.0), dict(window=40), dict(slopes=True), dict(scale=0.3),
                                  dict(cap=20.0, window=130, slopes=True, scale=-0.2)])
@pytest.mark.parametrize("tree", [False, True])
def test_options(opts, tree, e4m3):
    opts = dict(opts)
    if opts.get("slopes"):
        opts["slopes"] = 2.0 ** -np.arange(1, 9)
    Problem(2, [300, 85, 200], 85 if tree else 7, 8, 2, 64 if tree else 128, 32, e4m3, tree=tree).check(**opts)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Ls,lens,N,Hq,H,D,page,tree", [
    (1, [1, 4, 2], 1, 4, 2, 64, 16, False),
    (333, [6, 200, 41, 9], 6, 8, 2, 128, 64, False),
    (640, [30, 77], 21, 16, 2, 64, 32, True),
    (129, [90, 0, 88], 85, 8, 2, 128, 16, True),
    (257, [7] * 40, 6, 8, 1, 128, 64, False),    # 1920 rows over the prefix
])
def test_shared(Ls, lens, N, Hq, H, D, page, tree, e4m3):
    if tree:
        lens = [n if n == 0 or n >= N else N for n in lens]
    p = Problem(3, lens, N, Hq, H, D, page, e4m3, shared=Ls, tree=tree)
    p.check()
    p.check(cap=8.0, window=100, slopes=0.5 ** np.arange(Hq))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("N,Hq,H", [(10, 4, 1), (25, 4, 1), (60, 8, 2)])
def test_windows_over_groups_of_rows(N, Hq, H, e4m3):
    """Windows that cut tiles and leave some out, by cache position and by
    tree position, for 40, 100 and 240 rows a head."""
    for tree in (False, True):
        p = Problem(20, [700, 200, 61], N, Hq, H, 64, 32, e4m3, tree=tree)
        for window in (1, 64, 150):
            p.check(window=window)
    p = Problem(21, [300, 77], N, Hq, H, 128, 64, e4m3, shared=400)
    p.check(window=350)


def test_a_tree_of_many_nodes():
    Problem(22, [1400, 900], 700, 2, 1, 64, 64, False, tree=True).check(only=[1])


def test_shared_equals_the_same_cache_held_apart():
    """A prefix of whole pages given as the shared one or at the head of each
    table: the same attention."""
    p = Problem(4, [100, 37, 64], 5, 8, 2, 128, 32, False, shared=96)
    a, la = p.run()
    table = np.concatenate((np.broadcast_to(p.stable, (3, 3)), p.table), 1)
    b, lb = sv.attn_tree(p.q, p.cache, dev(table), dev(np.array([n + 96 for n in p.lens], np.int32)), lse=True)
    assert torch.allclose(la, lb, atol=4e-4, rtol=0)
    assert torch.allclose(a.float(), b.float(), atol=2 ** -6, rtol=2 ** -6)


@pytest.mark.parametrize("e4m3", [False, True])
def test_split_along_a_long_cache(e4m3):
    Problem(5, [9000], 2, 4, 1, 128, 64, e4m3).check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_see_nothing(e4m3):
    """All-zero mask rows (a malformed tree's) with no context, and padding."""
    p = Problem(6, [9, 40, 5], 9, 4, 2, 64, 16, e4m3, tree=True)
    p.mask[0] = 0
    p.mask[1, 3] = 0
    p.check()
    out, lse = p.run()
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -np.inf)
    p.check(window=1)  # only positions with an index of at least the token's own


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("e4m3", [False, True])
def test_masked_places_may_hold_anything(bad, e4m3):
    """A tree node's key and value are not finite: only the nodes that see it
    change, and where its value is infinite they do."""
    p = Problem(7, [50, 33], 20, 4, 2, 128, 16, e4m3, tree=True)
    good, _ = p.run()
    c = 7
    for b in range(2):
        j = p.lens[b] - p.N + c
        pid, slot = int(p.table[b, j // p.page]), j % p.page
        for t in (p.cache.k, p.cache.v):
            if e4m3:
                t.view(torch.uint8)[pid, :, slot, 3] = 0x7f
            else:
                t[pid, :, slot, 3] = bad
    out, _ = p.run()
    for b in range(2):
        sees = p.mask[b][:, c] != 0
        assert torch.equal(out[b, ~sees], good[b, ~sees])
        assert not torch.isfinite(out[b, sees]).all(-1).any()


@pytest.mark.parametrize("e4m3", [False, True])
def test_an_infinite_value_stays_in_its_column(e4m3):
    """Only the value is not finite: the nodes that see it get it in that
    column and ordinary numbers in the others."""
    p = Problem(17, [50, 33], 20, 4, 2, 128, 16, e4m3, tree=True)
    good, _ = p.run()
    c = 7
    for b in range(2):
        j = p.lens[b] - p.N + c
        pid, slot = int(p.table[b, j // p.page]), j % p.page
        if e4m3:
            p.cache.v.view(torch.uint8)[pid, :, slot, 3] = 0x7f
        else:
            p.cache.v[pid, :, slot, 3] = -float("inf")
    out, _ = p.run()
    for b in range(2):
        sees = p.mask[b][:, c] != 0
        assert torch.equal(out[b, ~sees], good[b, ~sees])
        col = out[b, sees][..., 3]
        assert torch.isnan(col).all() if e4m3 else (col == -float("inf")).all()
        rest = [d for d in range(128) if d != 3]
        assert torch.equal(out[b, sees][..., rest], good[b, sees][..., rest])


def test_large_scores_and_equal_scores():
    """Scores of magnitude ~1e3 (one position takes everything), and all
    equal (a plain mean)."""
    p = Problem(8, [300, 129], 3, 8, 2, 128, 64, False)
    out, lse = p.run(scale=30.0)
    for b in range(2):
        o, e, spread, _ = p.want(b, scale=30.0)
        # scores are fp32 sums of magnitude ~1e3: 1e-3 absolute, so weights are good to 0.2%
        assert np.all(np.abs(out[b].double().cpu().numpy() - o) <= 2.0 ** -6 * spread + 2.0 ** -8)
    p.q.zero_()
    p.check()


def test_deterministic_and_on_a_side_stream():
    p = Problem(9, [900, 300, 77], 6, 32, 8, 128, 64, True)
    ws = sv.new_workspace(sv.spec_attn_workspace_size(3, 6, 32, 8, 128), DEV)
    a, la = p.run(workspace=ws)
    for _ in range(3):
        b, lb = p.run(workspace=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)
    st = torch.cuda.Stream()
    c, lc = p.run(workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(a, c) and torch.equal(la, lc)
    assert sv.last_error(ws) == 0


def test_strided_queries():
    p = Problem(10, [100, 64], 4, 8, 2, 64, 16, False)
    wide = torch.zeros((2, 4, 12, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, :, 2:10] = p.q
    a, _ = p.run()
    b, _ = p.run(q=wide[:, :, 2:10])
    assert torch.equal(a, b)


def test_lengths_and_pages_out_of_range():
    """A length past the table, a negative one and a bad page id fail their
    own sequences: NaN, and the error bit; the others are untouched."""
    p = Problem(11, [200, 90, 150, 60, 70], 3, 8, 2, 128, 32, False)
    good, _ = p.run()
    lens = list(p.lens)
    p.lens = [200, 10 ** 6, 150, -4, 70]
    p.table[2, 1] = 10 ** 6
    p.table[4, 3] = -1  # past what sequence 4 needs: never followed
    ws = sv.new_workspace(sv.spec_attn_workspace_size(5, 3, 8, 2, 128), DEV)
    out, lse = p.run(workspace=ws)
    assert torch.equal(out[0], good[0]) and torch.equal(out[4], good[4])
    for b in (1, 2, 3):
        assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
    assert sv.last_error(ws) == sv.SPEC_DATA_PAGE_RANGE
    assert sv.last_error(ws) == 0
    p.lens = lens
    s = Problem(12, [40, 9], 3, 8, 2, 128, 32, True, shared=100)
    s.stable[2] = -7
    out, _ = s.run(workspace=ws)
    assert torch.isnan(out).all()
    assert sv.last_error(ws) == sv.SPEC_DATA_PAGE_RANGE


def test_empty_batch():
    c = sv.new_cache(1, 2, 16, 64, DEV)
    q = torch.zeros((0, 3, 4, 64), dtype=torch.bfloat16, device=DEV)
    none = torch.zeros((0, 1), dtype=torch.int32, device=DEV)
    assert sv.attn_tree(q, c, none, none[:, 0].contiguous()).shape == (0, 3, 4, 64)


def test_graph_capture():
    """The call captured into a graph follows lengths that change between
    replays."""
    p = Problem(13, [300, 200], 3, 8, 2, 128, 64, False)
    ws = sv.new_workspace(sv.spec_attn_workspace_size(2, 3, 8, 2, 128), DEV)
    table, lens = dev(p.table), dev(np.array([300, 200], np.int32))
    out = torch.empty_like(p.q)
    sv.attn_tree(p.q, p.cache, table, lens, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.attn_tree(p.q, p.cache, table, lens, out=out, workspace=ws)
    lens.copy_(torch.tensor([130, 7], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    want = sv.attn_tree(p.q, p.cache, table, lens, workspace=ws)
    assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements: the pages at its end."""
    H, page, D = 8, 128, 128
    n = (1 << 32) // (H * page * D) + 16
    if torch.cuda.mem_get_info()[0] < 4 * n * H * page * D + (8 << 30):
        pytest.skip("needs 17 GiB and some room")
    k = torch.empty((n, H, page, D), dtype=torch.bfloat16, device=DEV)
    c = sv.KVCache(k, torch.empty_like(k), None, None)
    rng = np.random.default_rng(14)
    x = {w: dev(rng.normal(size=(1, 200, H, D)), torch.bfloat16) for w in "kv"}
    far, near = (dev(np.array([t], np.int32)) for t in ([n - 1, n - 3], [0, 1]))
    zero, lens = dev(np.zeros(1, np.int32)), dev(np.array([200], np.int32))
    q = dev(rng.normal(size=(1, 2, 16, D)), torch.bfloat16)
    got = []
    for t in (far, near):
        sv.kv_append(c, t, zero, x["k"], x["v"])
        a, b = sv.kv_read(c, t, zero, 200)
        assert torch.equal(a, x["k"]) and torch.equal(b, x["v"])
        got.append(sv.attn_tree(q, c, t, lens))
    assert torch.equal(*got)
