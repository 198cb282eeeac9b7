"""The tests' own plain forms, pinned: the e4m3 format against torch's, and
the attention against a direct softmax."""
import numpy as np
import torch

import attn_reference as ref


def test_e4m3_table():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.e4m3_table(), want)


def test_quantise_rounds_to_nearest_even():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=(64, 64)), rng.normal(size=(64, 64)) * 2.0 ** rng.integers(-30, 30, (64, 1))])
    x = np.float64(np.float32(x))
    y, e = ref.quantise(x)
    scaled = torch.tensor(x * 2.0 ** -e[:, None].astype(float)).float()
    np.testing.assert_array_equal(y, scaled.to(torch.float8_e4m3fn).double().numpy())
    top = np.abs(x).max(1)
    assert np.all(top <= 448 * 2.0 ** e) and np.all(top > 448 * 2.0 ** (e - 1))


def test_quantise_edges():
    y, e = ref.quantise(np.array([[0.0, 0.0], [448.0, 1.0], [449.0, 0.0], [np.nan, 2.0], [np.inf, 0.0]]))
    assert list(e) == [0, 0, 1, -7, 0]
    assert np.isnan(y[3, 0]) and y[3, 1] == 256 and np.isnan(y[4, 0])


def test_attention_is_softmax():
    rng = np.random.default_rng(1)
    q, K, V = rng.normal(size=(3, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    seen = rng.random((3, 9)) < 0.6
    seen[1] = False
    out, lse, _, _ = ref.attention(q, K, V, seen, scale=0.5)
    for h in range(4):
        s = torch.tensor(0.5 * q[:, h] @ K[:, h // 2].T).masked_fill(~torch.tensor(seen), -np.inf)
        p = torch.softmax(s, -1).nan_to_num(0.0)
        np.testing.assert_allclose(out[:, h], (p @ torch.tensor(V[:, h // 2])).numpy(), atol=1e-12)
    assert np.all(out[1] == 0) and np.all(lse[1] == -np.inf)
