"""The example with drafted trees end to end."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("users,tokens,nodes,temperature", [(4, 48, 13, 0.7), (3, 20, 2, 0.0), (1, 30, 40, 0.5)])
def test_draft_trees(users, tokens, nodes, temperature):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("draft_trees", os.path.join(ROOT, "examples", "draft_trees.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(users, tokens, nodes, temperature, say=lambda *_: None)
    assert got["plain_steps"] == tokens and 1 <= got["steps"] <= tokens  # a step gives a token at least
    for answers in (got["answers"], got["plain"]):
        assert [len(a) for a in answers] == [tokens + 1] * users
        assert all(0 <= t < example.VOCAB for a in answers for t in a)
    assert [a[0] for a in got["answers"]] == [a[0] for a in got["plain"]]
