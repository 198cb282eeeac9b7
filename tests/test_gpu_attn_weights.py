"""Softmax weights far below the largest one: one position holds most of the
weight, and thousands share the rest; values that are zero or tiny.  Over both
cache types the bound is the one of weights rounded to bf16, with no absolute
term: 2^-8 |out| + (2^-8 + 2^-13) sum p |v|, twice what the arithmetic gives.
(Over an e4m3 cache the query's two terms add less than the 2^-13 to it: they
lose under 2^-18 of its largest element.)
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

import speculative_decoding_verification_top_gb300 as sv  # noqa: E402
from test_gpu_attn_long import B, DEV, H, Batch  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    sv.build()


ROWS = [(1, 4), (6, 4), (12, 4), (25, 4), (64, 4)]


@pytest.mark.parametrize("value", [0.0, 2.0 ** -6, 1.0])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,G", ROWS)
def test_one_position_holds_most(N, G, D, e4m3, value):
    """Every query leans to u, and so does the key of position 17: its score is
    10 to 12 above the others, e^-10 to e^-12 of it their weights."""
    p = Batch(3, N, G, D, 64, e4m3)
    g = torch.Generator(DEV).manual_seed(5)
    u = torch.randint(0, 2, (D,), generator=g, device=DEV) * 2.0 - 1.0
    p.q = (p.q.float() + 4.0 * u).bfloat16()
    at = torch.full((B,), 17, dtype=torch.int32, device=DEV)
    key = (11.0 * 4.0 / D ** 0.5 * u).expand(B, 1, H, D).contiguous()
    v = value * torch.randn((B, 1, H, D), generator=g, device=DEV)
    sv.kv_append(p.cache, p.table, at, key, v)
    p.check(scale=D ** -0.5 / 16, floored=False)


@pytest.mark.parametrize("small", [2.0 ** -24, 2.0 ** -60, 2.0 ** 30])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("N,G,D", [(6, 4, 128), (12, 4, 64), (25, 4, 128), (64, 4, 64)])
def test_rows_of_zeros_between_values_of_any_size(N, G, D, e4m3, small):
    p = Batch(4, N, G, D, 64, e4m3, small=small)
    p.check(scale=D ** -0.5 / 16, floored=False)


@pytest.mark.parametrize("e4m3", [False, True])
def test_most_weight_in_a_shared_prefix(e4m3):
    p = Batch(6, 6, 4, 128, 64, e4m3, shared=4000, least=1, most=300)
    g = torch.Generator(DEV).manual_seed(7)
    u = torch.randint(0, 2, (128,), generator=g, device=DEV) * 2.0 - 1.0
    p.q = (p.q.float() + 4.0 * u).bfloat16()
    at = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    key = (11.0 * 4.0 / 128 ** 0.5 * u).expand(1, 1, H, 128).contiguous()
    sv.kv_append(p.cache, p.stable.view(1, -1), at, key, torch.zeros_like(key))
    p.check(scale=128 ** -0.5 / 16, floored=False)
