"""Conversations continued with drafted trees of tokens, as a serving program
would run them on one GPU: a toy model (one layer of attention over the paged
cache, random weights) answers, and a draft of it, whose weights are a little
off, proposes a tree of tokens a step.  A step is one captured graph: tables and
masks from the lengths on the device, rotary positions while keys and values are
stored, attention over the tree, the target's probabilities, verification, and
the kept tokens' keys and values moved together.  Nothing of it waits for the
host, which only reads which tokens were kept.

    python examples/draft_trees.py [--users 4] [--tokens 48] [--nodes 13] [--temperature 0.7]

Prints how many tokens a step kept; with --temperature 0 the answers are the ones
that the model gives token by token, but where two of its bf16 scores are as good as
equal: products of another number of rows may round them the other way."""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import compression_coupled_collectives_gb300 as cc  # noqa: E402

HEADS, GROUP, DIM, PAGE, VOCAB, WIDTH = 2, 4, 64, 16, 512, 256


class Toy:
    """Embeds a token, attends, adds, and scores the vocabulary."""

    def __init__(self, gen: torch.Generator):
        def rand(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

        self.embed = rand(VOCAB, WIDTH, scale=1.0)
        self.qkv = rand(WIDTH, (HEADS * GROUP + 2 * HEADS) * DIM, scale=WIDTH ** -0.5)
        self.out = rand(HEADS * GROUP * DIM, WIDTH, scale=(HEADS * GROUP * DIM) ** -0.5)
        self.jump = rand(WIDTH, WIDTH, scale=2.0 * WIDTH ** -0.5)

    def project(self, tokens: torch.Tensor):
        x = self.embed[tokens.long()]
        return x, (x @ self.qkv).view(-1, HEADS * GROUP + 2 * HEADS, DIM).split([HEADS * GROUP, HEADS, HEADS], 1)

    def scores(self, x: torch.Tensor, attended: torch.Tensor) -> torch.Tensor:
        y = (x @ self.jump) + attended.flatten(1) @ self.out
        return (y @ self.embed.T).float() * (0.6 / WIDTH ** 0.5)


def probabilities(scores: torch.Tensor, temperature: float) -> torch.Tensor:
    if temperature > 0:
        return torch.softmax(scores / temperature, -1)
    return torch.nn.functional.one_hot(scores.argmax(-1), VOCAB).float()


def fan(nodes: int) -> list[int]:
    """The tree's parents: a trunk, and one more child beside each of its tokens."""
    parents, trunk = [-1], 0
    while len(parents) < nodes:
        parents.append(trunk)
        child = len(parents) - 1
        if len(parents) < nodes:
            parents.append(trunk)
        trunk = child
    return parents


class Server:
    """Users' caches, and one step for all of them."""

    def __init__(self, model: Toy, users: int, nodes: int, most: int, temperature: float, seed: int):
        self.model, self.users, self.nodes, self.temperature = model, users, nodes, temperature
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        rows = users * nodes
        pages = -(-most // PAGE) + 1
        self.cache = cc.KvCache.empty(users * pages, PAGE, HEADS, DIM)
        self.cache.k.zero_(), self.cache.v.zero_()
        self.tables = cc.StepTables.empty(users, pages, users * pages, PAGE)
        self.rotary = cc.StepRotary(DIM)
        zeros = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
        self.lens, self.new = zeros(users), torch.full((users,), nodes, dtype=torch.int32, device="cuda")
        self.parents = torch.tensor(fan(nodes) * users, dtype=torch.int32, device="cuda")
        self.tokens, self.uniform = zeros(rows), torch.zeros(rows, device="cuda")
        self.plan = {"cu_tokens": zeros(users + 1), "kv_lens": zeros(users), "positions": zeros(rows),
                     "mask": zeros(rows, -(-nodes // 32))}
        self.batch = cc.KvBatch(self.tables.page_table, self.plan["cu_tokens"], self.plan["kv_lens"], n_tokens=rows,
                                max_new=nodes, max_len=most)
        self.path, self.n_kept, self.next = zeros(rows), zeros(users), zeros(users)
        self.ws = cc.empty_kv_workspace(self.cache, self.batch, HEADS * GROUP)
        self.graph = None

    def enqueue(self) -> None:
        p = self.plan
        cc.cccl_step_plan(self.tables, self.lens, self.new, self.ws, parents=self.parents, **p)
        x, (q, k, v) = self.model.project(self.tokens)
        q, out = q.contiguous(), torch.empty(q.shape, dtype=q.dtype, device="cuda")
        cc.cccl_step_write(self.cache, self.batch, self.rotary, q, k, v, q, self.ws, positions=p["positions"])
        cc.cccl_step_attention(self.cache, self.batch, q, p["mask"], out, self.ws)
        target = probabilities(self.model.scores(x, out), self.temperature)
        cc.cccl_step_verify(target, None, self.tokens, self.parents, self.uniform, p["cu_tokens"], self.path, self.n_kept,
                            self.next, self.ws)
        cc.cccl_step_keep(self.cache, self.batch, self.path, self.n_kept, self.lens, self.ws)

    def step(self, tokens: torch.Tensor) -> list[list[int]]:
        """One step on every user's tree of tokens [users, nodes]; what each kept after its root, and the token after."""
        self.tokens.copy_(tokens.flatten())
        self.uniform.uniform_(generator=self.gen)
        if self.graph is None:  # the first step runs as it is, and is then captured
            self.enqueue()
            torch.cuda.synchronize()
            kept = self.answers()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.enqueue()
            return kept
        self.graph.replay()
        return self.answers()

    def answers(self) -> list[list[int]]:
        path, kept, following = self.path.view(self.users, -1).tolist(), self.n_kept.tolist(), self.next.tolist()
        tokens = self.tokens.view(self.users, -1).tolist()
        return [[tokens[u][i] for i in path[u][1:kept[u]]] + [following[u]] for u in range(self.users)]


def draft(model: Toy, roots: list[int], nodes: int, off: torch.Tensor) -> torch.Tensor:
    """A tree a user from the model's jump alone, a little off: no attention, two likeliest children a trunk token."""
    parents = fan(nodes)
    trees = torch.zeros(len(roots), nodes, dtype=torch.int64, device="cuda")
    trees[:, 0] = torch.tensor(roots, device="cuda")
    taken = [0] * nodes
    for i in range(1, nodes):
        x = model.embed[trees[:, parents[i]]]
        likely = ((x @ (model.jump + off)) @ model.embed.T).float().topk(2, -1).indices
        trees[:, i] = likely[:, taken[parents[i]]]
        taken[parents[i]] += 1
    return trees.to(torch.int32)


def main(users: int = 4, tokens: int = 48, nodes: int = 13, temperature: float = 0.7, seed: int = 0, say=print) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Toy(gen)
    off = (torch.randn(WIDTH, WIDTH, generator=gen, device="cuda") * 0.2 * WIDTH ** -0.5).to(torch.bfloat16)
    roots = torch.randint(VOCAB, (users,), generator=gen, device="cuda").tolist()
    got = {}
    for size in (nodes, 1):  # with drafts; token by token
        server = Server(model, users, size, tokens + 2 * nodes + 1, temperature, seed)
        answers, steps = [[r] for r in roots], 0
        while min(map(len, answers)) <= tokens:
            # users that have their tokens already go on with the others: their rows are only some more
            trees = draft(model, [a[-1] for a in answers], size, off)
            if max(map(len, answers)) > tokens + nodes:  # their pages are used up: from the front again
                full = torch.tensor([len(a) > tokens + nodes for a in answers], device="cuda")
                server.lens[full] = 0
                answers = [a[:tokens + 1] if len(a) > tokens + nodes else a for a in answers]
            for a, kept in zip(answers, server.step(trees)):
                a += kept
            steps += 1
        _, status = cc.cccl_get_result(server.ws)
        if status:
            raise cc.CcclError(status, "a step")
        got[size] = ([a[:tokens + 1] for a in answers], steps)
    kept = tokens / got[nodes][1]
    say("%d users, %d tokens each: %d steps with trees of %d, at least %.2f tokens a step; %d without" %
        (users, tokens, got[nodes][1], nodes, kept, got[1][1]))
    return {"answers": got[nodes][0], "plain": got[1][0], "steps": got[nodes][1], "plain_steps": got[1][1]}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--users", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--nodes", type=int, default=13)
    ap.add_argument("--temperature", type=float, default=0.7)
    a = ap.parse_args()
    main(a.users, a.tokens, a.nodes, a.temperature)
