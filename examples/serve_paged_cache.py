"""One conversation through the paged cache, as a serving program would run it
on one GPU: a prompt is read in chunks into a bf16 cache, its pages are
compressed where they lie and decompressed into another pool (what the prefill
side sends to the answering side), the cache is then held in 8 bits, and tokens
are appended and attended to one at a time, next to the 16-bit cache.

    python examples/serve_paged_cache.py [--prompt 2000] [--chunk 512] [--tokens 16] [--format int8|e4m3]

Keys, values and queries are random (there is no model here); a layer of 8 kv
heads and 32 query heads of 128."""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import compression_coupled_collectives_gb300 as cc  # noqa: E402

HEADS, Q_HEADS, DIM, PAGE = 8, 32, 128, 16


def int32(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def pool_cache(pages: int):
    """A pool whose blocks hold a page's K and V together (whole 4096-value chunks), and the cache on it."""
    pool = torch.empty(pages, 2, PAGE, HEADS, DIM, dtype=torch.bfloat16, device="cuda")
    return pool, cc.KvCache(pool[:, 0], pool[:, 1])


def batch_of(table: torch.Tensor, length: int, new: int) -> cc.KvBatch:
    """One sequence of `length` tokens, the last `new` of them this step's."""
    return cc.KvBatch(table[None], int32([0, new]), int32([length]), n_tokens=new, max_new=new, max_len=length)


def main(prompt: int = 2000, chunk: int = 512, tokens: int = 16, fmt: str = "int8", seed: int = 0, say=print) -> dict:
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(n, heads):
        return torch.randn(n, heads, DIM, generator=gen, device="cuda").to(torch.bfloat16)

    pages = -(-(prompt + tokens) // PAGE)
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    pool, cache = pool_cache(pages)
    sender = cache

    # the prompt, a chunk at a time: store its keys and values, then attend over all so far
    ws = cc.empty_kv_workspace(cache, batch_of(table, prompt, chunk), Q_HEADS)
    for at in range(0, prompt, chunk):
        n = min(chunk, prompt - at)
        step = batch_of(table, at + n, n)
        q, out = rand(n, Q_HEADS), torch.empty(n, Q_HEADS, DIM, dtype=torch.bfloat16, device="cuda")
        cc.cccl_kv_write(cache, step, rand(n, HEADS), rand(n, HEADS), ws)
        cc.cccl_kv_attention(cache, step, q, out, ws)
    if cc.cccl_get_result(ws)[1] != cc.CCCL_OK:
        raise RuntimeError("the prompt's calls reported a device error")

    # its pages, compressed and decompressed into other pages of another pool
    used = -(-prompt // PAGE)
    block = pool[0].numel()
    send = table[:used].contiguous()
    stream, cws = cc.empty_stream(used * block), cc.empty_workspace(used * block)
    cc.cccl_compress_paged(pool, block, send, stream, cws)
    size, status = cc.cccl_get_result(cws)
    assert status == cc.CCCL_OK
    there, other = pool_cache(pages)
    new_table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    cc.cccl_decompress_paged(stream[:size], there, block, new_table[:used].contiguous(), cws)
    assert cc.cccl_get_result(cws)[1] == cc.CCCL_OK
    say("prompt of %d tokens: %d pages, %d bytes, %d compressed (%.3f)"
        % (prompt, used, 2 * used * block, size, size / (2 * used * block)))

    # the answering side may hold the cache in 8 bits
    kind = {"int8": cc.CCCL_KV_INT8, "e4m3": cc.CCCL_KV_E4M3}[fmt]
    small = cc.KvCache.empty(pages, PAGE, HEADS, DIM, fmt=kind)
    k, v = cc.kv_read(other, batch_of(new_table, prompt, prompt))
    cc.kv_write(small, batch_of(new_table, prompt, prompt), k, v)

    # tokens, one at a time: the same on the sender's cache, the received one and the 8-bit one
    one = batch_of(table, prompt + tokens, 1)
    spaces = [cc.empty_kv_workspace(c, one, Q_HEADS) for c in (sender, other, small)]
    outs = [torch.empty(1, Q_HEADS, DIM, dtype=torch.bfloat16, device="cuda") for _ in spaces]
    same, worst = True, 0.0
    for i in range(tokens):
        k1, v1, q1 = rand(1, HEADS), rand(1, HEADS), rand(1, Q_HEADS)
        for c, t, out, w in zip((sender, other, small), (table, new_table, new_table), outs, spaces):
            step = batch_of(t, prompt + i + 1, 1)
            cc.cccl_kv_write(c, step, k1, v1, w)
            cc.cccl_kv_attention(c, step, q1, out, w)
        same &= torch.equal(outs[0], outs[1])
        off = (outs[2].float() - outs[0].float()).norm() / outs[0].float().norm()
        worst = max(worst, float(off))
    for w in spaces:
        assert cc.cccl_get_result(w)[1] == cc.CCCL_OK
    say("%d tokens: received cache %s, %s cache within %.4f of it"
        % (tokens, "the same bits" if same else "DIFFERS", fmt, worst))
    return {"ratio": size / (2 * used * block), "same": bool(same), "worst": worst}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompt", type=int, default=2000)
    ap.add_argument("--chunk", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--format", choices=("int8", "e4m3"), default="int8")
    args = ap.parse_args()
    main(args.prompt, args.chunk, args.tokens, args.format)
