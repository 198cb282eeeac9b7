"""Attention and cache reads at the ends of what their arguments may hold."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

import speculative_decoding_verification_top_gb300 as sv  # noqa: E402
from test_gpu_attn import DEV, Problem, dev  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def test_read_keeps_exponents_within_the_written_range():
    """Exponents past +-120, which no append writes, count as +-120, as in the attention."""
    c = sv.new_cache(1, 1, 16, 64, DEV, e4m3=True)
    c.k.view(torch.uint8).fill_(0x38)  # 1.0
    c.v.view(torch.uint8).fill_(0xb8)  # -1.0
    odd = [-128, -127, -121, -120, 0, 120, 121, 127]
    for t in (c.k_exp, c.v_exp):
        t[0, 0, :8] = torch.tensor(odd, dtype=torch.int8)
    zero = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    want = 2.0 ** torch.tensor(odd, dtype=torch.float64).clamp(-120, 120)
    for dtype in (torch.float32, torch.bfloat16):
        k, v = sv.kv_read(c, zero, zero[0], 8, dtype=dtype)
        assert torch.equal(k[0, :, 0].double().cpu(), want[:, None].expand(8, 64))
        assert torch.equal(v[0, :, 0].double().cpu(), -want[:, None].expand(8, 64))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("N,Hq,H", [(3, 4, 2), (24, 4, 2), (40, 8, 2)])
def test_a_query_that_is_not_finite(N, Hq, H, e4m3, bad):
    """Scores of both infinities, or NaN: no number comes out, whatever the
    cache's type; the other rows are as before."""
    p = Problem(30, [200, 90], N, Hq, H, 128, 32, e4m3)
    if e4m3:  # small keys: no score overflows by itself
        p.cache.k_exp.sub_(40)
    else:
        p.cache.k.mul_(2.0 ** -40)
    good, _ = p.run()
    p.q[1, 2, 1, 5] = bad
    out, lse = p.run()
    assert torch.isnan(out[1, 2, 1]).all() and torch.isnan(lse[1, 2, 1])
    good[1, 2, 1] = out[1, 2, 1] = 0
    assert torch.equal(out, good)


@pytest.mark.parametrize("cap", [1e3, 1e5, 1e9, 1e20, 3e38])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("N", [3, 40])
def test_a_cap_far_above_the_scores(N, e4m3, cap):
    """cap tanh(s / cap) is then nearly s."""
    Problem(31, [300, 129], N, 8, 2, 64, 64, e4m3).check(cap=cap)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("N,Hq,H,tree", [(1, 2, 1, False), (3, 8, 2, False), (24, 8, 2, True)])
def test_a_window_leaves_out_most_of_a_prefix(N, Hq, H, tree, e4m3):
    """Right results, and tiles of the prefix that no row's window reaches are
    not taken: their page ids may be anything."""
    p = Problem(32, [40, 130, 24], N, Hq, H, 64, 32, e4m3, shared=900, tree=tree)
    ws = sv.new_workspace(sv.spec_attn_workspace_size(3, N, Hq, H, 64), DEV)
    for window in (1, 30, 100, 400, 1000, 2000):
        p.check(window=window)
    pages = p.stable.copy()
    for window in (30, 300):
        least = 900 if p.pos is None else min(int(x.min()) for x in p.pos)
        if p.pos is None:
            least = 900 + min(p.lens) - N
        first = max(0, least - window + 1)
        p.stable = pages.copy()
        p.stable[:min(first, 900) // 128 * 4] = -1  # whole tiles of 128 positions before it
        assert (p.stable == -1).any()
        out, lse = p.run(window=window, workspace=ws)
        assert sv.last_error(ws) == 0
        p.stable = pages
        want, want_lse = p.run(window=window)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_a_window_past_the_whole_prefix():
    """No tile of the prefix is left."""
    p = Problem(33, [400, 700, 200], 4, 8, 2, 128, 16, False, shared=300)
    out, lse = p.run(window=50)
    for b in range(3):
        o, e, spread, _ = p.want(b, window=50)
        got = out[b].double().cpu().numpy()
        assert np.all(np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -13) * spread)
        assert np.all(np.abs(lse[b].double().cpu().numpy() - e) <= 4e-4)
    alone = sv.attn_tree(p.q[:2].contiguous(), p.cache, dev(p.table[:2]), dev(np.array([400, 700], np.int32)),
                         pos=dev(np.array([[396, 397, 398, 399], [696, 697, 698, 699]], np.int32)), window=50)
    assert torch.allclose(out[:2].float(), alone.float(), atol=2 ** -6, rtol=2 ** -6)
