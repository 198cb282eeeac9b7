"""Attention and cache reads at the ends of what their arguments may hold."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

import speculative_decoding_verification_top_gb300 as sv  # noqa: E402

DEV = "cuda:0"


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
