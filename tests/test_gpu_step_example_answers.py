"""The example with drafted trees at temperature 0: every token is the model's best
after those before it, to the rounding of its scores."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNIT = 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("draft_trees", os.path.join(ROOT, "examples", "draft_trees.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def scores64(ex, model, answer):
    """Scores of the vocabulary after each of the answer's tokens, in binary64, with the parts that they are added up
    from: the embedding's and attention's share of what meets the vocabulary."""
    H, G, D = ex.HEADS, ex.GROUP, ex.DIM
    x = model.embed[torch.tensor(answer, device="cuda")].double()
    q, k, v = (x @ model.qkv.double()).view(len(answer), -1, D).split([H * G, H, H], 1)
    at = torch.arange(len(answer), dtype=torch.float64, device="cuda")
    angle = (at[:, None] * 10000.0 ** (-2 * torch.arange(D // 2, device="cuda").double() / D))[:, None]

    def turned(y):
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)

    k, v = turned(k).repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    s = torch.einsum("ihd,jhd->hij", turned(q), k) * D ** -0.5
    s = s.masked_fill(torch.ones(s.shape[1:], dtype=torch.bool, device="cuda").triu(1), -float("inf"))
    attended = torch.einsum("hij,jhd->ihd", s.softmax(-1), v).flatten(1)
    jump, out = x @ model.jump.double(), attended @ model.out.double()
    return (jump + out) @ model.embed.double().T, jump, out


@pytest.mark.parametrize("users,tokens,nodes,seed", [(4, 48, 13, 0), (4, 48, 13, 1), (3, 20, 2, 2), (1, 30, 40, 3)])
def test_answers_are_the_models(example, users, tokens, nodes, seed):
    """With drafts and token by token.  The scores of the best token and of the chosen one are rounded to bf16 by the
    example, off by up to UNIT times the larger each; what meets the vocabulary is a sum of two rounded products,
    rounded, whose errors (uniform, UNIT / sqrt(3) of a value as their deviation at most, independent) reach the
    difference of two scores with their deviation: six of them, and as much again for attention's own roundings."""
    got = example.main(users, tokens, nodes, 0.0, seed, say=lambda *_: None)
    model = example.Toy(torch.Generator(device="cuda").manual_seed(seed))
    embed = model.embed.double()
    for answer in got["answers"] + got["plain"]:
        z, jump, out = scores64(example, model, answer[:-1])
        chosen = torch.tensor(answer[1:], device="cuda")
        best, which = z.max(-1)
        parts = (jump ** 2 + out ** 2 + (jump + out) ** 2) * (embed[which] - embed[chosen]) ** 2
        slack = 2 * UNIT * best.abs() + 2 * 6 * UNIT * (parts.sum(-1) / 3).sqrt()
        assert (best - z.gather(1, chosen[:, None])[:, 0] <= slack).all()
