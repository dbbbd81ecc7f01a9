"""Speculative decoding of a batch of requests with different LoRA adapters.

A small random transformer (attention layers only) whose q, k, v and o
projections carry LoRA adapters, one adapter per request.  Every step drafts a
tree of tokens per request, runs all trees through the layers in one batch,
keeps the tokens that the target distribution accepts, draws one more, and
moves the accepted tokens' keys and values to their places:

    sgmv_build_segments_device   group the rows by adapter, once per step
    sgmv_apply_multi             the adapters of q, k and v
    sgmv_rope                    rotary positions, k and v appended to the paged cache
    sgmv_tree_attention          every row over its context and its ancestors
    sgmv_apply                   the adapter of o
    sgmv_tree_verify             which drafted tokens are accepted
    sgmv_cache_commit            their keys and values, all layers at once

    python examples/speculative_decode.py [tokens]
"""
import os
import sys
from dataclasses import dataclass, field

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from rank_gemv_gb300 import sgmv  # noqa: E402

# The drafted tree: the last token, three guesses after it, two after each of those.
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 2, 3, 3]
DEPTH = [0, 1, 1, 1, 2, 2, 2, 2, 2, 2]
RANK = [0, 0, 1, 2, 0, 1, 0, 1, 0, 1]  # which of the draft's likeliest tokens


@dataclass
class Model:
    vocab: int = 512
    hidden: int = 512
    heads: int = 8
    layers: int = 2
    rank: int = 16
    adapters: int = 4
    seed: int = 0
    dtype: torch.dtype = torch.float16
    w: dict = field(default_factory=dict)

    def __post_init__(self):
        g = torch.Generator("cuda").manual_seed(self.seed)
        H, r, L = self.hidden, self.rank, self.adapters

        def rand(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(self.dtype)

        self.embed = rand(self.vocab, H, std=1.0)
        self.head = rand(H, self.vocab, std=4.0 * H ** -0.5)
        self.base = [[rand(H, H, std=H ** -0.5) for _ in range(4)] for _ in range(self.layers)]
        self.A = [[rand(L, H, r, std=H ** -0.5) for _ in range(4)] for _ in range(self.layers)]
        self.B = [[rand(L, r, H, std=r ** -0.5) for _ in range(4)] for _ in range(self.layers)]
        self.inv_freq = sgmv.sgmv_rope_frequencies(H // self.heads // 2)


class Requests:
    """Their paged cache, lengths, last tokens and adapters."""

    def __init__(self, model, batch, longest, block_size=16, seed=1):
        D = model.hidden // model.heads
        pages = -(-longest // block_size)
        g = torch.Generator().manual_seed(seed)
        self.bs = block_size
        self.table = torch.randperm(batch * pages, generator=g).to(torch.int32).view(batch, pages).cuda()
        shape = (model.layers, batch * pages, block_size, model.heads, D)
        self.k = torch.empty(shape, dtype=model.dtype, device="cuda")
        self.v = torch.empty_like(self.k)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.last = torch.randint(0, model.vocab, (batch,), generator=g).to(torch.int32).cuda()
        self.adapter = (torch.arange(batch) % model.adapters).to(torch.int32).cuda()
        self.random = torch.Generator("cuda").manual_seed(seed)


def logits_of(model, x):
    return (torch.nn.functional.layer_norm(x.float(), x.shape[-1:]).to(model.dtype) @ model.head).float()


def draft(model, last, parents):
    """Tokens [B, n] of a tree that grows from the last tokens: cheap guesses, the
    model's head on the embedding without its layers."""
    tokens = [last.long()]
    for i in range(1, len(parents)):
        guess = logits_of(model, model.embed[tokens[parents[i]]])
        tokens.append(guess.topk(RANK[i] + 1, -1).indices[:, -1])
    return torch.stack(tokens, 1).to(torch.int32)


def step(model, req, parents=PARENTS, depth=DEPTH, tokens=None, greedy=False):
    """One step of every request: (count [B], path [B, n], token [B], tokens [B, n])."""
    B, n = req.lens.numel(), len(parents)
    T, heads, H = B * n, model.heads, model.hidden
    D = H // heads
    if tokens is None:
        tokens = draft(model, req.last, parents)
    par = torch.tensor(parents, dtype=torch.int32, device="cuda").repeat(B)
    tree_ptr = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    positions = (req.lens[:, None] + torch.tensor(depth, dtype=torch.int32, device="cuda")).view(-1)
    place = req.lens[:, None] + torch.arange(n, dtype=torch.int32, device="cuda")
    slots = (req.table.gather(1, (place // req.bs).long()) * req.bs + place % req.bs).to(torch.int32).view(-1)
    perm, seg_ptr, idx, _ = sgmv.sgmv_build_segments_device(req.adapter.repeat_interleave(n), model.adapters)
    x = model.embed[tokens.view(-1).long()]
    for layer in range(model.layers):
        W, A, Bm = model.base[layer], model.A[layer], model.B[layer]
        h = torch.nn.functional.layer_norm(x.float(), (H,)).to(model.dtype)
        qkv = [h @ W[i] for i in range(3)]
        sgmv.sgmv_apply_multi(qkv, [h] * 3, A[:3], Bm[:3], seg_ptr, idx, 0.5, perm=perm)
        q, k, v = (t.view(T, heads, D) for t in qkv)
        sgmv.sgmv_rope(q, k, positions, model.inv_freq, v=v, k_cache=req.k[layer], v_cache=req.v[layer], slots=slots)
        attn = torch.empty_like(q)
        sgmv.sgmv_tree_attention(attn, q, req.k[layer], req.v[layer], req.table, req.lens, tree_ptr, par)
        attn = attn.view(T, H)
        y = attn @ W[3]
        sgmv.sgmv_apply(y, attn, A[3], Bm[3], seg_ptr, idx, 0.5, perm=perm)
        x = x + y
    logits = logits_of(model, x)
    if greedy:
        target = torch.zeros_like(logits).scatter_(1, logits.argmax(-1, keepdim=True), 1.0)
    else:
        target = torch.softmax(logits, -1)
    u = torch.rand(T + B, generator=req.random, device="cuda")
    count, path, token = sgmv.sgmv_tree_verify(target, None, tokens.view(-1), par, tree_ptr, u[:T], u[T:], n)
    sgmv.sgmv_cache_commit(req.k, req.v, req.table, req.lens, path, count)
    req.lens += count
    req.last = token
    return count, path, token, tokens


def generate(model, req, length, parents=PARENTS, depth=DEPTH, greedy=False, tokens=None):
    """At least `length` new tokens per request, as lists; and the steps it took.  Requests
    that run ahead of the slowest use up their pages sooner: then ValueError."""
    out = [[] for _ in range(req.lens.numel())]
    steps, held, room = 0, req.lens.tolist(), req.table.shape[1] * req.bs
    while min(map(len, out)) < length:
        if max(h + len(o) for h, o in zip(held, out)) + len(parents) > room:
            raise ValueError(f"a request's pages hold {room} tokens, too few for its next tree")
        count, path, token, drafted = step(model, req, parents, depth, tokens(out) if tokens else None, greedy)
        for b, (c, p, t) in enumerate(zip(count.tolist(), path.tolist(), token.tolist())):
            out[b] += [int(drafted[b, i]) for i in p[1:c]] + [t]
        steps += 1
    return out, steps


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 32
    model = Model()
    # a step adds up to three tokens to a request, and one at least to the slowest
    req = Requests(model, batch=8, longest=max(1024, (max(DEPTH) + 1) * steps + len(PARENTS)))
    out, took = generate(model, req, steps)
    assert sgmv.sgmv_get_device_error() == 0
    total = sum(map(len, out))
    print(f"{total} tokens of {len(out)} requests on {model.adapters} adapters in {took} steps "
          f"({total / len(out) / took:.2f} per request and step); the first: {out[0][:12]}")


if __name__ == "__main__":
    main()
