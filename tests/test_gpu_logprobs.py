"""Log probabilities, entropies, ranks and top tokens on the GPU against the 64-bit
form."""
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


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def check(x, tokens, rows, T, top, got):
    """x [B, N, V] as the kernel saw it, in 64 bits."""
    V = x.shape[-1]
    # ln Z: at most V / 512 + 64 sums one after the other, 2^-24 each, 2^-22 of an
    # exponential; a value (x - m) / T has three roundings of itself.
    z = (V / 512 + 64) * 2.0 ** -24 + 2.0 ** -22
    lp, ent, rank = (t.cpu().numpy() for t in got[:3])
    for b in range(tokens.shape[0]):
        for t in range(tokens.shape[1]):
            token = int(tokens[b, t])
            if token == -1:
                assert lp[b, t] == 0 and ent[b, t] == 0 and rank[b, t] == -1
                if top:
                    assert bool((got.top_ids[b, t] == -1).all()) and not got.top_logprobs[b, t].any()
                continue
            row = x[b, t if rows is None else rows[b, t]]
            with np.errstate(divide="ignore"):
                wl, we, wr, ids, wt = ref.logprobs(row, token, T, top)
            lz = abs(wt[0]) if top else 0.0

            def near(g, w):
                if not np.isfinite(w):
                    return g == w
                return abs(g - w) <= z + (abs(w) + lz + np.log(V)) * 2.0 ** -21
            assert near(lp[b, t], wl), (b, t, lp[b, t], wl)
            assert abs(ent[b, t] - we) <= (2 + we) * (z + (we + np.log(V)) * 2.0 ** -21), (b, t, ent[b, t], we)
            assert rank[b, t] == wr, (b, t, rank[b, t], wr)
            if top:
                assert np.array_equal(got.top_ids[b, t].cpu().numpy(), ids), (b, t)
                for g, w in zip(got.top_logprobs[b, t].cpu().numpy(), wt):
                    assert near(g, w)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N,V,top,T", [
    (1, 1, 1, 1, 1.0), (1, 1, 7, 7, 1.0), (2, 3, 33, 32, 0.5), (3, 2, 255, 5, 1.0), (1, 2, 900, 32, 1.3), (2, 2, 1001, 20, 1.0),
    (1, 3, 2047, 0, 1.0), (2, 6, 32000, 20, 0.7), (1, 1, 32001, 5, 2.0), (1, 2, 128256, 32, 1.0), (40, 5, 5003, 3, 1.0),
    (300, 6, 1999, 8, 1.0), (1, 1, 700001, 32, 1.0)])
def test_rows(dtype, B, N, V, top, T):
    rng = np.random.default_rng([B, N, V, top])
    x = dev(-1.1 * np.log(1 + rng.permuted(np.tile(np.arange(V), (B, N, 1)), axis=-1)) + rng.normal(0, 1.5, (B, N, V)), dtype)
    tokens = rng.integers(-1, V, (B, N)).astype(np.int32)
    tokens[0, 0] = int(x[0, 0].float().argmax())
    ws = sv.new_workspace(sv.spec_verify_logprobs_workspace_size(), DEV)
    got = sv.logprobs(x, dev(tokens), temperature=T, top=top, workspace=ws)
    some = (np.arange(B) % max(1, B // 12) == 0)
    pick = lambda t: None if t is None else t[torch.from_numpy(some).to(DEV)]  # noqa: E731
    check(x.double().cpu().numpy()[some], tokens[some], None, T, top, sv.LogProbs(*map(pick, got)))
    assert sv.last_error(ws) == 0
    again = sv.logprobs(x, dev(tokens), temperature=T, top=top, workspace=ws)
    for a, b in zip(got, again):  # the same bits
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_paths(dtype):
    """Rows by an accepted path; pads and entries without a row of their own."""
    rng = np.random.default_rng(2)
    x = dev(rng.normal(size=(3, 21, 4097)), dtype)
    rows = np.array([[0, 3, 20, -1], [0, -1, -1, -1], [5, 5, 1, 0]], np.int32)
    tokens = np.where(rows >= 0, rng.integers(0, 4097, rows.shape), -1).astype(np.int32)
    got = sv.logprobs(x, dev(tokens), rows=dev(rows), top=4)
    check(x.double().cpu().numpy(), tokens, rows, 1.0, 4, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50, 3001, 40000])
def test_ties_and_masks(dtype, V):
    """Equal logits go by index; masked ones (-inf, or the type's lowest) come last."""
    rng = np.random.default_rng(V)
    low = torch.finfo(dtype).min
    rows = np.zeros((7, V))
    rows[1] = rng.integers(0, 3, V)                      # three values
    rows[2] = -np.inf
    rows[2, rng.choice(V, 5, replace=False)] = [1, 2, 2, 3, -1]
    rows[3] = np.where(np.arange(V) % 3 == 0, rng.normal(size=V), -np.inf)
    rows[4] = low
    rows[4, V // 2] = 0.5
    rows[5] = low                                        # all at the type's lowest
    rows[6] = np.where(rng.random(V) < 0.5, 0.0, -0.0)   # one value, two signs
    x = dev(rows[None], dtype)
    if dtype == torch.bfloat16:
        x[0, 4] = low
        x[0, 4, V // 2] = 0.5
        x[0, 5] = low
    ref_x = x.double().cpu().numpy()
    for tokens in (rng.integers(0, V, (1, 7)), np.zeros((1, 7), int), np.full((1, 7), V - 1)):
        tokens = tokens.astype(np.int32)
        check(ref_x, tokens, None, 1.0, 20, sv.logprobs(x, dev(tokens), top=20))


def test_sorted_rows():
    """Rising and falling rows: the most likely tokens in one thread's or one slice's vectors."""
    V = 20000
    up = np.arange(V) / 500.0
    x = dev(np.stack([up, up[::-1], np.roll(up, 777)])[None], torch.float32)
    tokens = np.array([[V - 1, 3, 777]], np.int32)
    check(x.double().cpu().numpy(), tokens, None, 1.0, 32, sv.logprobs(x, dev(tokens), top=32))


def test_data_errors():
    x = torch.randn((1, 5, 3000), device=DEV)
    x[0, 1, 2900] = float("nan")
    x[0, 2, 5] = float("inf")
    x[0, 3] = -float("inf")
    tokens = torch.tensor([[3, 4, 5, 6, 7]], dtype=torch.int32, device=DEV)
    ws = sv.new_workspace(sv.spec_verify_logprobs_workspace_size(), DEV)
    got = sv.logprobs(x, tokens, top=3, workspace=ws)
    for t, good in enumerate([True, False, False, False, True]):
        assert bool(torch.isfinite(got.logprob[0, t])) == good == bool(torch.isfinite(got.entropy[0, t]))
        assert (int(got.rank[0, t]) >= 0) == good and bool((got.top_ids[0, t] >= 0).all()) == good
        assert bool(torch.isnan(got.top_logprobs[0, t]).any()) != good
    assert sv.last_error(ws) == sv.SPEC_DATA_ROW_NONFINITE | sv.SPEC_DATA_ROW_ALL_NEG_INF
    bad = torch.tensor([[3000, -2, 5, 0, 0]], dtype=torch.int32, device=DEV)
    rows = torch.tensor([[0, 0, 5, -1, 4]], dtype=torch.int32, device=DEV)
    got = sv.logprobs(x, bad, rows=rows, top=3, workspace=ws)
    assert torch.isnan(got.logprob[0, :4]).all() and torch.isfinite(got.logprob[0, 4])
    assert sv.last_error(ws) == sv.SPEC_DATA_TOKEN_RANGE


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7])
def test_unaligned_rows(dtype, offset):
    """Rows on any element boundary; what lies beside the tensor does not count."""
    rng = np.random.default_rng(offset)
    V = 2999
    flat = dev(rng.normal(size=2 * V + 16), dtype)
    flat[:offset] = 1000.0
    flat[offset + 2 * V:] = 1000.0
    x = flat[offset:offset + 2 * V].view(1, 2, V)
    tokens = np.array([[0, V - 1]], np.int32)
    check(x.double().cpu().numpy(), tokens, None, 1.0, 6, sv.logprobs(x, dev(tokens), top=6))


def test_parts_and_refusals():
    x = torch.randn((2, 2, 100), device=DEV)
    tokens = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    all_of = sv.logprobs(x, tokens, top=2)
    some = sv.logprobs(x, tokens, entropy=False, rank=False)
    assert some.entropy is None and some.rank is None and some.top_ids is None
    # without candidates the kernel's code differs, its sums do not
    assert torch.equal(some.logprob, all_of.logprob)
    for bad in (dict(top=33), dict(temperature=0.0)):
        with pytest.raises(sv.SpecVerifyError):
            sv.logprobs(x, tokens, **bad)
    with pytest.raises(ValueError):
        sv.logprobs(x, tokens.long())
    with pytest.raises(TypeError):
        sv.logprobs(x.half(), tokens)
    empty = sv.logprobs(x[:0], tokens[:0], top=2)
    assert empty.logprob.shape == (0, 2)


def test_after_verification_and_captured():
    """With a verification's own workspace and outputs, captured and replayed on new logits."""
    g = torch.Generator(DEV)
    g.manual_seed(1)
    target, draft = (torch.randn((4, n, 3001), generator=g, device=DEV) for n in (4, 3))
    toks = torch.randint(3001, (4, 3), generator=g, device=DEV, dtype=torch.int32)
    uni = torch.rand((4, 4), generator=g, device=DEV)
    out, num, ws = sv.verify_sample(target, draft, toks, uni)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.logprobs(target, out, top=5, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.verify_sample(target, draft, toks, uni, out_tokens=out, out_num=num, workspace=ws)
        got = sv.logprobs(target, out, top=5, workspace=ws)
    target.copy_(torch.randn(target.shape, generator=g, device=DEV))
    graph.replay()
    check(target.double().cpu().numpy(), out.cpu().numpy(), None, 1.0, 5, got)
    assert bool((got.rank >= 0).sum(1).eq(num + 1).all())
    want, _, _ = sv.verify_sample(target, draft, toks, uni, workspace=ws)
    assert torch.equal(want, out) and sv.last_error(ws) == 0


def some_of(x, tokens, top, got, picked):
    """check() of the picked sequences."""
    at = torch.from_numpy(picked).to(DEV)
    part = sv.LogProbs(*(None if t is None else t[at] for t in got))
    check(x[at].double().cpu().numpy(), tokens[picked], None, 1.0, top, part)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", ["-inf", "lowest"])
def test_masked_rows_of_a_batch(dtype, low):
    """Rows that a mask leaves few tokens of, in calls of few and of many entries (one CTA or many a row)."""
    rng = np.random.default_rng(5)
    V = 50001
    low = -float("inf") if low == "-inf" else torch.finfo(dtype).min
    for B in (1, 500):
        x = torch.full((B, 1, V), low, dtype=dtype, device=DEV)
        keep = rng.choice(V, 12, replace=False)
        x[:, 0, torch.from_numpy(keep).to(DEV)] = torch.randn((B, 12), device=DEV).to(dtype)
        x[:, 0, 33:40] = 0.25  # equal ones among those left
        tokens = rng.integers(0, V, (B, 1)).astype(np.int32)
        tokens[:, 0] = np.where(np.arange(B) % 2 == 0, keep[0], tokens[:, 0])
        got = sv.logprobs(x, dev(tokens), top=32)
        some_of(x, tokens, 32, got, np.unique([0, B // 3, B - 1]))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_above_the_bar(dtype):
    """The largest logits in so few threads' vectors that the bar lies far below them."""
    V, E = 60000, 4 if dtype == torch.float32 else 8
    vec = torch.arange(V, device=DEV) // E % 256
    x = torch.randn((500, 1, V), device=DEV) + torch.where(vec < 124, 100.0, 0.0)
    x = x.to(dtype)
    tokens = np.full((500, 1), 17, np.int32)
    got = sv.logprobs(x, dev(tokens), top=32)
    some_of(x, tokens, 32, got, np.array([0, 499]))


def test_past_32_bits():
    """More than 2^31 logits, rows at both ends."""
    N, V = 16800, 128256
    x = torch.empty((1, N, V), dtype=torch.bfloat16, device=DEV)
    assert x.numel() > 2 ** 31
    rows = np.array([[0, N - 1, N - 2]], np.int32)
    x[0, rows[0].tolist()] = torch.randn((3, V), device=DEV).to(x.dtype)
    tokens = np.array([[5, V - 1, 77]], np.int32)
    got = sv.logprobs(x, dev(tokens), rows=dev(rows), top=6)
    few = x[:, rows[0].tolist()].double().cpu().numpy()
    check(few, tokens, np.arange(3)[None], 1.0, 6, got)
