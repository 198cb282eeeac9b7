"""Attention calls whose work is long enough that every multiprocessor takes
segments of ten tiles and more, so that the kernels' rings of slots go round,
maxima outgrow their reference again and again, and page tables are read on.
Every place that no sequence holds is NaN, in the page tails too.  Against the
definition in 64 bits, for a few of the sequences.

Tolerances as in test_gpu_attn.py, from the same arithmetic.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

import speculative_decoding_verification_top_gb300 as sv  # noqa: E402

DEV = "cuda:0"
B, H = 32, 8


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


class Batch:
    """B sequences of 1500 to 2999 positions; keys grow from a tenth to four
    times along each, so that the largest score keeps rising."""

    def __init__(self, seed, N, G, D, page, e4m3, shared=0, least=1500, most=3000, small=1.0):
        g = torch.Generator(DEV).manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.N, self.G, self.D, self.shared, self.e4m3, self.rng = N, G, D, shared, e4m3, rng
        lens = rng.integers(max(N, least), max(N + 1, most), B)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        most, width = int(lens.max()), -(-int(lens.max()) // page)
        sp = -(-shared // page)
        n = B * width + sp + 1
        ids = torch.randperm(n, generator=g, device=DEV).int()
        self.table = ids[:B * width].view(B, width).contiguous()
        self.stable = ids[B * width:B * width + sp].contiguous()
        self.cache = sv.new_cache(n, H, page, D, DEV, e4m3)
        for t in (self.cache.k, self.cache.v):
            (t.view(torch.uint8).fill_(0x7f) if e4m3 else t.fill_(float("nan")))
        if e4m3:
            self.cache.k_exp.fill_(77)
            self.cache.v_exp.fill_(-77)

        def fill(table, count, lens):
            b = table.shape[0]
            k, v = (torch.randn((b, count, H, D), generator=g, device=DEV) for _ in "kv")
            k *= torch.linspace(0.1, 4.0, count, device=DEV)[:, None, None]
            if small != 1.0:  # values of that size, every third a row of zeros
                v *= small
                v[:, ::3] = 0.0
            t = torch.arange(count, dtype=torch.int32, device=DEV).expand(b, count)
            rows = torch.where(t < lens[:, None], t, -1).int().contiguous()
            sv.kv_append(self.cache, table, torch.zeros(b, dtype=torch.int32, device=DEV), k.bfloat16(),
                         v.bfloat16(), rows=rows)

        fill(self.table, most, self.lens)
        if shared:
            fill(self.stable.view(1, sp), shared, torch.full((1,), shared, device=DEV))
        self.q = torch.randn((B, N, H * G, D), generator=g, device=DEV).bfloat16()
        self.ws = sv.new_workspace(sv.spec_attn_workspace_size(B, N, H * G, H, D), DEV)

    def tree(self):
        """Every sequence's mask and positions of one random tree, and the tree's mask."""
        N = self.N
        m, p = np.zeros((N, N), np.uint8), np.zeros(N, np.int64)
        for i in range(N):
            if i:
                par = int(self.rng.integers(max(0, i - 6), i))
                m[i], p[i] = m[par], p[par] + 1
            m[i, i] = 1
        pos = torch.from_numpy(p).to(DEV) + (self.lens - N + self.shared)[:, None]
        return torch.from_numpy(m).to(DEV).expand(B, N, N).contiguous(), pos.int().contiguous()

    def run(self, **kw):
        if self.shared:
            return sv.attn_shared(self.q, self.cache, self.stable, self.shared, self.table, self.lens, lse=True,
                                  workspace=self.ws, **kw)
        return sv.attn_tree(self.q, self.cache, self.table, self.lens, lse=True, workspace=self.ws, **kw)

    def held(self, table, count):
        zero = torch.zeros(1, dtype=torch.int32, device=DEV)
        return [x[0].double() for x in sv.kv_read(self.cache, table.view(1, -1), zero, count, dtype=torch.float32)]

    def want(self, b, mask=None, pos=None, window=0, scale=None, slopes=None, cap=0.0):
        """out, lse, sum p |v| and sum |v| / sum e^(s - max s), heads first."""
        N, G, D, L, Ls = self.N, self.G, self.D, int(self.lens[b]), self.shared
        K, V = self.held(self.table[b], L)
        if Ls:
            first = self.held(self.stable, Ls)
            K, V = torch.cat((first[0], K)), torch.cat((first[1], V))
        K, V = (x.nan_to_num(0.0, 0.0, 0.0).transpose(0, 1) for x in (K, V))  # [H, all, D]; unseen, or not checked
        jpos = torch.arange(Ls + L, device=DEV)
        ipos = jpos[-N:].clone() if pos is None else pos[b].long()
        jpos[-N:] = ipos
        seen = torch.ones((N, Ls + L), dtype=torch.bool, device=DEV)
        seen[:, -N:] = torch.ones((N, N), device=DEV).tril() > 0 if mask is None else mask[b] != 0
        far = ipos[:, None] - jpos[None, :]
        if window:
            seen &= far < window
        q = self.q[b].double().view(N, H, G, D).permute(1, 0, 2, 3).reshape(H, N * G, D)
        s = q @ K.transpose(1, 2) * (D ** -0.5 if scale is None else scale)
        if cap:
            s = cap * torch.tanh(s / cap)
        s = s.view(H, N, G, -1)
        if slopes is not None:
            s = s - slopes.double().view(H, 1, G, 1) * far[None, :, None, :]
        s = s.masked_fill(~seen[None, :, None, :], -torch.inf).view(H, N * G, -1)
        m = s.amax(-1, keepdim=True)
        w = torch.exp(s - m)
        l = w.sum(-1, keepdim=True)
        there = seen.repeat_interleave(G, 0).double()

        def by_token(x):
            return x.view(H, N, G, -1).transpose(0, 1).reshape(N, H * G, -1)

        return (by_token(w @ V / l), by_token(m + l.log())[..., 0], by_token(w @ V.abs() / l),
                by_token(there @ V.abs() / l))

    def check(self, skip=None, floored=True, **kw):
        """skip [N]: nodes that are not compared, but must not be finite.  floored:
        over an e4m3 cache an absolute error per position is allowed."""
        out, lse = self.run(**kw)
        again = self.run(**kw)
        every = slice(None) if skip is None else ~skip
        assert torch.equal(out[:, every], again[0][:, every]) and torch.equal(lse[:, every], again[1][:, every])
        assert torch.isfinite(out[:, every]).all() and torch.isfinite(lse[:, every]).all()
        if skip is not None:
            assert not torch.isfinite(out[:, skip]).any()
        for b in (0, 13, B - 1):
            o, e, spread, floor = self.want(b, **kw)
            tol = 2.0 ** -8 * o.abs()
            if self.e4m3 and floored:
                tol += (2.0 ** -7 + 2.0 ** -13) * spread + 2.0 ** -14 * floor
            else:
                tol += (2.0 ** -8 + 2.0 ** -13) * spread
            over = ((out[b].double() - o).abs() - tol)[every].max()
            assert over <= 0, "sequence %d: off by %g over the bound" % (b, over)
            assert (lse[b].double() - e)[every].abs().max() <= 4e-4
        assert sv.last_error(self.ws) == 0


ROWS = [(1, 4), (6, 4), (12, 4), (16, 4), (25, 4), (64, 4)]  # new tokens, query heads a key/value head


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", ROWS)
def test_many_tiles_a_segment(N, G, D, e4m3):
    p = Batch(1, N, G, D, 16, e4m3)
    p.check()                                   # scores up to ~20, rising
    p.check(scale=D ** -0.5 / 16)               # nearly equal weights
    p.check(window=1077)                        # starts within a tile
    p.check(slopes=2.0 ** -torch.arange(1.0, H * G + 1, device=DEV), cap=25.0)
    mask, pos = p.tree()
    p.check(mask=mask, pos=pos)
    if N == 1:
        return
    # A node whose key and value are not finite: the nodes that do not see it are as before.
    c = N // 2
    place = (p.lens - N + c).long()
    page = p.table.gather(1, (place // 16)[:, None])[:, 0].long()
    for t in (p.cache.k, p.cache.v):
        if e4m3:
            t.view(torch.uint8)[page, :, place % 16] = 0x7f
        else:
            t[page, :, place % 16] = float("inf")
    p.check(mask=mask, pos=pos, skip=mask[0, :, c] != 0)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("N,G,D,page", [(2, 1, 128, 64), (6, 4, 128, 64), (20, 2, 64, 32)])
def test_a_long_prefix_under_a_batch(N, G, D, page, e4m3):
    """64, 768 and 1280 rows over 12100 positions, own caches of up to 300."""
    p = Batch(2, N, G, D, page, e4m3, shared=12100, least=1, most=300)
    p.check()
    p.check(window=12200)
    mask, pos = p.tree()
    p.check(mask=mask, pos=pos, scale=D ** -0.5 / 16)
