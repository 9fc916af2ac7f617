"""The serving example end to end: chunks, compressed pages, an 8-bit cache, single tokens."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("prompt,chunk,fmt", [(700, 256, "int8"), (333, 333, "e4m3"), (40, 7, "int8")])
def test_serving_example(prompt, chunk, fmt):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("serve_paged_cache", os.path.join(ROOT, "examples", "serve_paged_cache.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(prompt, chunk, 5, fmt, say=lambda *_: None)
    assert got["same"]
    assert got["ratio"] < 0.9  # random normal values: about 0.77
    # half a code step of a vector's largest value (about 3.3 sigma for 128 normal values), uniformly spread:
    # 3.3 / 127 / sqrt(12) = 0.0075 sigma on V (E4M3: a relative step of 2^-3 / sqrt(12) = 0.036, less where codes
    # are finer), as much again through the scores (|q . dk| / sqrt(128) of 128 such errors); twice that is the bound
    assert got["worst"] < (4 * 0.0075 if fmt == "int8" else 4 * 0.036)
