"""The decoding example: candidate trees give plain greedy decoding's tokens,
through every cache and attention call and the tree verification."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "tree_decode.py")


@pytest.mark.parametrize("e4m3", [False, True])
def test_tree_decode(e4m3):
    spec = importlib.util.spec_from_file_location("tree_decode", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    r = module.run(steps=24, batch=3, e4m3=e4m3)
    assert r["passes"] < 24  # more than a token a pass
    assert r["alike"] >= r["tokens"] // 2
