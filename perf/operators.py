"""The operators of one speculative decoding step over a paged KV cache, as cases to
measure: rotary positions with the append to the cache (rope), attention of a tree of
drafted tokens over the cache (attention), verification of the drafted tokens (verify)
and the move of the accepted tokens to their final places in the cache (commit).

Each case names its operator in "op".  With ``own`` false, run() computes the operator
from elementary torch operations in 32 bits; with ``own`` true it calls the package.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ONE = 1 << 38            # probability 1 in the fixed point of verify
UNIT = 1 << 24           # a uniform number's 24 bits


def _case(name, op, **kw):
    return {"name": name, "op": op, **kw}


def listed():
    return [
        # one new token of one request, a short context: pure latency
        _case("attn-decode-1", "attention", dtype="f16", B=1, n=1, ragged=False, hq=32, hkv=32,
              D=128, bs=16, longest=1500, pad=False),
        # the batch of the all-distinct decode workload (32 requests, 32 heads of 128), each with
        # a drafted tree of up to 16 tokens, contexts up to 4096
        _case("attn-tree-32", "attention", dtype="f16", B=32, n=16, ragged=True, hq=32, hkv=32,
              D=128, bs=16, longest=4096, pad=False),
        # grouped heads, long contexts and large trees: the most arithmetic per byte
        _case("attn-tree-gqa-long", "attention", dtype="bf16", B=8, n=64, ragged=True, hq=64,
              hkv=8, D=128, bs=64, longest=32768, pad=False),
        # a full decode batch (128 rows) padded to three tokens each, odd head size and page
        # size, some requests without any context yet
        _case("attn-decode-128-odd", "attention", dtype="bf16", B=128, n=3, ragged=True, hq=20,
              hkv=4, D=80, bs=24, longest=2100, pad=True),
        # the decode rows of one layer, rotated and appended to the cache
        _case("rope-append-128", "rope", dtype="f16", T=128, hq=32, hk=32, D=128, rd=128,
              interleaved=False, inverse=False, append=True, far=4096, factor=1.0),
        # a prefill of a long context, grouped heads, stretched frequencies, interleaved pairs
        _case("rope-prefill-8k", "rope", dtype="bf16", T=8192, hq=32, hk=8, D=128, rd=128,
              interleaved=True, inverse=False, append=True, far=131072, factor=8.0),
        # the gradient of a partial rotation
        _case("rope-grad-partial", "rope", dtype="bf16", T=2047, hq=40, hk=40, D=80, rd=32,
              interleaved=False, inverse=True, append=False, far=2048, factor=1.0),
        # one request's tree, drafted greedily (no draft distribution)
        _case("verify-1-greedy", "verify", B=1, n=16, V=32000, draft=False, sharp=4.0),
        # 32 requests with trees of up to 64 tokens drawn from a draft model
        _case("verify-32-tree", "verify", B=32, n=64, V=32000, draft=True, sharp=3.0),
        # a full batch with short chains and a large odd vocabulary
        _case("verify-128-large", "verify", B=128, n=4, V=100277, draft=True, sharp=3.0),
        # one request's accepted tokens, all layers
        _case("commit-1", "commit", dtype="f16", B=1, n=16, layers=32, hkv=32, D=128, bs=16),
        # a batch of 48 requests, grouped heads, an odd page size
        _case("commit-48", "commit", dtype="bf16", B=48, n=33, layers=32, hkv=8, D=128, bs=24),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "attention", "rope", "rope", "verify", "commit"))
    dtype = rng.choice(("f16", "bf16"))
    if op == "attention":
        hkv, group = rng.choice(((32, 1), (8, 8), (8, 4), (4, 5), (1, 16), (40, 1), (2, 7)))
        D = rng.choice((64, 80, 96, 128, 128))
        n = _log(rng, 1, 64)
        B = _log(rng, 1, 128)
        # no more tokens, and no more scores, than the largest listed cases hold
        most = min(4e8 / (2 * hkv * D * B), 1e9 / (B * hkv * group * n))
        return {"op": op, "dtype": dtype, "B": B, "n": n, "ragged": rng.random() < 0.7,
                "hq": hkv * group, "hkv": hkv, "D": D, "bs": rng.choice((1, 8, 16, 16, 24, 32, 64, 128)),
                "longest": _log(rng, 1, max(2, min(32768, most))), "pad": rng.random() < 0.3}
    if op == "rope":
        D = rng.choice((64, 80, 96, 128, 128, 256))
        rd = rng.choice((D, D, D // 2, 16))
        hk = rng.choice((1, 2, 8, 32))
        hq = hk * rng.choice((1, 4, 7))
        return {"op": op, "dtype": dtype, "T": _log(rng, 1, max(2, min(8192, 8192 * 40 * 128 // ((hq + 2 * hk) * D)))),
                "hq": hq, "hk": hk, "D": D, "rd": rd, "interleaved": rng.random() < 0.5,
                "inverse": rng.random() < 0.3, "append": rng.random() < 0.6,
                "far": _log(rng, 16, 131072), "factor": rng.choice((1.0, 1.0, 4.0, 32.0))}
    if op == "verify":
        V = rng.choice((_log(rng, 1000, 128000), 32000, 50257))
        n = _log(rng, 1, 64)
        return {"op": op, "B": _log(rng, 1, max(2, min(128, 2048 * 32000 // (V * n)))), "n": n,
                "V": V, "draft": rng.random() < 0.7, "sharp": rng.choice((1.0, 3.0, 6.0))}
    hkv = rng.choice((1, 4, 8, 32))
    return {"op": op, "dtype": dtype, "B": _log(rng, 1, 48 if hkv < 32 else 8), "n": _log(rng, 1, 64),
            "layers": rng.choice((1, 2, 32)), "hkv": hkv, "D": rng.choice((64, 80, 128)),
            "bs": rng.choice((1, 16, 24, 32, 64))}


# ---- the batch's shape, fixed by the case alone ------------------------------------------


def _trees(c):
    """Nodes and parents of every sequence: a root (-1), then nodes that continue one of the
    few nodes before them; with "pad", rows that hold no token (-2) up to n."""
    rng = random.Random(1000003 * c["B"] + c["n"])
    counts, parents = [], []
    for b in range(c["B"]):
        n = c["n"] if not c.get("ragged", True) or b == 0 else rng.randint(1, c["n"])
        p = [-1] + [rng.randint(max(0, i - 6), i - 1) for i in range(1, n)]
        if c.get("pad"):
            p += [-2] * (c["n"] - n)
        counts.append(len(p))
        parents += p
    return counts, parents


def _prefix(c):
    """Context lengths: the first is the longest, the others ragged, some of them zero."""
    rng = random.Random(7 * c["B"] + c["longest"])
    most = c["longest"]
    return [most if b == 0 else 0 if most < 3000 and rng.random() < 0.05 else rng.randint(max(1, most // 8), most)
            for b in range(c["B"])]


def _pages(c, lens, seed):
    """A block table of scattered pages that holds lens[b] tokens of every sequence."""
    need = [-(-x // c["bs"]) for x in lens]
    width = max(1, max(need))
    order = np.random.RandomState(seed % (1 << 32)).permutation(sum(need) + 3).astype(np.int32)
    table, at = np.zeros((c["B"], width), np.int32), 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table, sum(need) + 3


def _frequencies(c):
    """Inverse frequencies of the pairs; with a factor, the slow ones are stretched by it and
    the fast ones kept, with a linear ramp between."""
    out = []
    for i in range(c["rd"] // 2):
        f = 10000.0 ** (-2.0 * i / c["rd"])
        turns = 4096 * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
        out.append(f * keep + f / c["factor"] * (1.0 - keep))
    return out


def _attention_factor(c):
    return 1.0 if c["factor"] == 1.0 else 0.1 * math.log(c["factor"]) + 1.0


def _i32(values):
    return torch.tensor(np.asarray(values, np.int32), device="cuda")


# ---- inputs ------------------------------------------------------------------------------


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    host = np.random.RandomState((int(seed) * 2654435761 + 12345) % (1 << 32))
    s = {"c": c}

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[c["dtype"]])

    def cache(blocks, *lead):
        shape = (*lead, blocks, c["bs"], c["hkv"], c["D"])
        return torch.empty(shape, device="cuda", dtype=DTYPES[c["dtype"]]).normal_(generator=g)

    if c["op"] == "attention":
        counts, parents = _trees(c)
        prefix = _prefix(c)
        total = [p + n for p, n in zip(prefix, counts)]
        table, blocks = _pages(c, total, seed)
        s["k"], s["v"] = cache(blocks), cache(blocks)
        # slots that no token has been written to hold anything at all
        for b in range(c["B"]):
            last = total[b] % c["bs"]
            if last:
                s["k"][table[b, total[b] // c["bs"]], last:] = float("nan")
                s["v"][table[b, total[b] // c["bs"]], last:] = float("nan")
        T = sum(counts)
        s["q"] = randn(T, c["hq"], c["D"])
        s["table"], s["prefix"] = _i32(table), _i32(prefix)
        s["ptr"], s["parents"] = _i32(np.concatenate([[0], np.cumsum(counts)])), _i32(parents)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, c["hq"], device="cuda")
        s["nodes"] = max(counts)  # known to whoever built the batch
        s["length"] = max(total)
        if own:  # the workspace that a serving loop keeps
            from rank_gemv_gb300 import sgmv

            s["ws"] = torch.zeros(sgmv.sgmv_tree_attention_workspace_bytes(T, c["B"], c["hq"], c["hkv"], c["D"]),
                                  dtype=torch.uint8, device="cuda")
    elif c["op"] == "rope":
        T, hq, hk, D = c["T"], c["hq"], c["hk"], c["D"]
        qkv = randn(T, hq + 2 * hk, D)  # the fused projection's output; q, k and v are views of it
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["positions"] = _i32(host.randint(0, c["far"], T))
        s["inv_freq"] = torch.tensor(_frequencies(c), dtype=torch.float64)
        s["freq"] = s["inv_freq"].to(device="cuda", dtype=torch.float32)
        s["q_out"] = torch.empty(T, hq, D, device="cuda", dtype=qkv.dtype)
        if c["append"]:
            blocks = -(-T // 16) + 8
            slots = host.permutation(blocks * 16)[:T].astype(np.int32)
            if T > 2:
                slots[T // 3] = -1  # a padding row is not appended
            s["slots"] = _i32(slots)
            s["kc"] = torch.zeros(blocks, 16, hk, D, device="cuda", dtype=qkv.dtype)
            s["vc"] = torch.zeros_like(s["kc"])
        else:
            s["k_out"] = torch.empty(T, hk, D, device="cuda", dtype=qkv.dtype)
    elif c["op"] == "verify":
        counts, parents = _trees(c)
        T, V = sum(counts), c["V"]
        ptr = np.concatenate([[0], np.cumsum(counts)])
        first = np.repeat(ptr[:-1], counts)
        logits = torch.randn(T, V, generator=g, device="cuda") * c["sharp"]
        s["target"] = torch.softmax(logits, -1)
        # the draft model's opinion: near the target's
        logits += torch.randn(T, V, generator=g, device="cuda") * (0.25 * c["sharp"])
        s["draft"] = torch.softmax(logits, -1)
        rows = torch.tensor(np.where(np.asarray(parents) < 0, 0, parents) + first, device="cuda")
        if c["draft"]:
            # every node is its own draw from its parent's distribution
            tokens = (s["draft"][rows] / torch.empty_like(logits).exponential_(generator=g)).argmax(-1)
        else:  # the likeliest tokens, best first among siblings
            rank, seen = [], {}
            for p, f in zip(parents, first.tolist()):
                rank.append(seen.get((f, p), 0))
                seen[(f, p)] = rank[-1] + 1
            best = torch.topk(logits, max(rank) + 1, -1).indices
            tokens = best[rows, torch.tensor(rank, device="cuda")]
            s["draft"] = None
        del logits
        s["tokens"] = tokens.to(torch.int32)
        s["parents"], s["ptr"] = _i32(parents), _i32(ptr)
        s["accept"] = torch.rand(T, generator=g, device="cuda")
        s["sample"] = torch.rand(c["B"], generator=g, device="cuda")
        s["nodes"] = max(counts)
    else:
        rng = random.Random(31 * c["B"] + c["n"])
        path = np.full((c["B"], c["n"]), -1, np.int32)
        counts = []
        for b in range(c["B"]):  # a path through the drafted nodes: ascending, from the root
            k = rng.randint(1, min(c["n"], 8)) if b else min(c["n"], 6)
            path[b, :k] = [0] + sorted(rng.sample(range(1, c["n"]), k - 1))
            counts.append(k)
        prefix = [rng.randint(0, 200) for _ in range(c["B"])]
        table, blocks = _pages(c, [p + c["n"] for p in prefix], seed)
        s["k"], s["v"] = cache(blocks, c["layers"]), cache(blocks, c["layers"])
        s["table"], s["prefix"] = _i32(table), _i32(prefix)
        s["path"], s["counts"] = _i32(path), _i32(counts)
    return s


# ---- one pass ----------------------------------------------------------------------------


def run(s):
    return {"attention": _attention, "rope": _rope, "verify": _verify, "commit": _commit}[s["c"]["op"]](s)


def _attention(s):
    c = s["c"]
    if own:
        from rank_gemv_gb300 import sgmv

        sgmv.sgmv_tree_attention(s["out"], s["q"], s["k"], s["v"], s["table"], s["prefix"], s["ptr"],
                                 s["parents"], lse=s["lse"], workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    B, bs, hkv, D, n, L = c["B"], c["bs"], c["hkv"], c["D"], s["nodes"], s["length"]
    prefix, ptr = s["prefix"].long(), s["ptr"].long()
    count = ptr[1:] - ptr[:-1]
    node = torch.arange(n, device="cuda")
    live = node < count[:, None]                                        # [B, n]
    rows = torch.where(live, ptr[:-1, None] + node, 0)
    parent = torch.where(live, s["parents"].long()[rows], -2)
    live = parent > -2
    # who sees whom among the drafted tokens: itself and its ancestors
    sees = (parent[:, :, None] == node) | (torch.eye(n, device="cuda", dtype=torch.bool) & live[:, :, None])
    sees = sees.float()
    for _ in range(max(1, (n - 1).bit_length())):
        sees = ((sees @ sees) > 0).float()
    at = torch.arange(L, device="cuda")
    held = at < (prefix + count)[:, None]                               # [B, L]
    slot = torch.where(held, s["table"].long().gather(1, (at // bs).clamp(max=s["table"].shape[1] - 1).expand(B, L)) * bs + at % bs, 0)
    in_tree = (at - prefix[:, None]).clamp(0, n - 1)
    visible = torch.where((at < prefix[:, None])[:, None], live[:, :, None],
                          sees.gather(2, in_tree[:, None].expand(B, n, L)) > 0) & held[:, None]
    k = s["k"].reshape(-1, hkv, D)[slot].float()                        # [B, L, hkv, D]
    v = torch.where(held[:, :, None, None], s["v"].reshape(-1, hkv, D)[slot].float(), 0.0)
    q = s["q"].float()[rows].reshape(B, n, hkv, c["hq"] // hkv, D)
    scores = torch.einsum("bnhgd,blhd->bhgnl", q, k) * (1.0 / math.sqrt(D))
    scores = torch.where(visible[:, None, None], scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = (scores - top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgnl,blhd->bhgnd", e, v) / torch.where(total == 0, 1.0, total)
    lse = (total.log() + top)[..., 0]
    keep = node < count[:, None]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, n, c["hq"], D)[keep].to(s["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B, n, c["hq"])[keep]}


def _rope(s):
    c = s["c"]
    rd, scale = c["rd"], _attention_factor(c)
    if own:
        from rank_gemv_gb300 import sgmv

        if c["append"]:
            sgmv.sgmv_rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=c["interleaved"],
                           scale=scale, inverse=c["inverse"], q_out=s["q_out"], v=s["v"],
                           k_cache=s["kc"], v_cache=s["vc"], slots=s["slots"])
            return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}
        sgmv.sgmv_rope(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=c["interleaved"],
                       scale=scale, inverse=c["inverse"], q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    angle = s["positions"].float()[:, None] * s["freq"]
    cos, sin = (angle.cos() * scale)[:, None], (angle.sin() * scale)[:, None]
    if c["inverse"]:
        sin = -sin

    def rotate(x):
        x = x.float()
        a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if c["interleaved"] else (x[..., :rd // 2], x[..., rd // 2:rd])
        y, z = a * cos - b * sin, a * sin + b * cos
        y = torch.stack((y, z), -1).flatten(-2) if c["interleaved"] else torch.cat((y, z), -1)
        return torch.cat((y, x[..., rd:]), -1).to(s["q_out"].dtype)

    q, k = rotate(s["q"]), rotate(s["k"])
    if not c["append"]:
        return {"q": q, "k": k}
    live = s["slots"] >= 0
    to = s["slots"][live].long()
    s["kc"].reshape(-1, c["hk"], c["D"])[to] = k[live]
    s["vc"].reshape(-1, c["hk"], c["D"])[to] = s["v"][live]
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _verify(s):
    c = s["c"]
    if own:
        from rank_gemv_gb300 import sgmv

        count, path, token = sgmv.sgmv_tree_verify(s["target"], s["draft"], s["tokens"], s["parents"], s["ptr"],
                                                   s["accept"], s["sample"], s["nodes"])
        return {"count": count, "path": path, "token": token}
    # weights are whole numbers (2^38 is probability 1), so their sums have one value in any order
    B, n, V = c["B"], s["nodes"], c["V"]
    ptr = s["ptr"].long()
    every = torch.arange(B, device="cuda")

    def weights(p):
        return (p.clamp(0.0, 1.0) * float(ONE)).long()

    at = ptr[:-1].clone()                                   # row of the last accepted node
    w = weights(s["target"][at])
    total = torch.full((B,), ONE, device="cuda", dtype=torch.int64)
    count = torch.ones(B, device="cuda", dtype=torch.int64)
    path = torch.full((B, n + 1), -1, device="cuda", dtype=torch.int32)
    path[:, 0] = 0
    for i in range(1, n):
        row = torch.minimum(ptr[:-1] + i, ptr[1:] - 1)
        child = (ptr[:-1] + i < ptr[1:]) & (s["parents"][row] == at - ptr[:-1])
        token = s["tokens"][row].long()
        have = w[every, token].float()
        q = torch.ones_like(have) if s["draft"] is None else s["draft"][at, token].clamp(0.0, 1.0)
        yes = child & (s["accept"][row] * q * total.float() < have)
        no = child & ~yes
        if s["draft"] is None:
            less = w.scatter(1, token[:, None], 0)
        else:
            less = (w - (s["draft"][at].clamp(0.0, 1.0) * total.float()[:, None]).long()).clamp(min=0)
        w = torch.where(no[:, None], less, w)
        total = torch.where(no, less.sum(1), total)
        at = torch.where(yes, row, at)
        w = torch.where(yes[:, None], weights(s["target"][at]), w)
        total = torch.where(yes, ONE, total)
        path[every, torch.where(yes, count, n)] = i
        count += yes
    path[:, n] = -1
    run_sum = w.cumsum(1)
    plain = weights(s["target"][at]).cumsum(1)              # nothing left: the target's own
    run_sum = torch.where(run_sum[:, -1:] == 0, plain, run_sum)
    total = run_sum[:, -1]
    m = (s["sample"] * float(UNIT)).long().clamp(0, UNIT - 1)
    mark = (total >> 24) * m + (((total & (UNIT - 1)) * m) >> 24)
    token = torch.where(total > 0, (run_sum <= mark[:, None]).sum(1), -1)
    return {"count": count.int(), "path": path[:, :n].contiguous(), "token": token.int()}


def _commit(s):
    c = s["c"]
    if own:
        from rank_gemv_gb300 import sgmv

        sgmv.sgmv_cache_commit(s["k"], s["v"], s["table"], s["prefix"], s["path"], s["counts"])
        return {"k": s["k"], "v": s["v"]}
    step = torch.arange(c["n"], device="cuda")
    live = step < s["counts"][:, None]
    prefix = s["prefix"].long()[:, None]
    table = s["table"].long()

    def slots(position):
        position = torch.where(live, position, 0)
        return (table.gather(1, position // c["bs"]) * c["bs"] + position % c["bs"])[live]

    src, dst = slots(prefix + s["path"].long()), slots(prefix + step)
    for x in (s["k"], s["v"]):
        x = x.view(c["layers"], -1, c["hkv"], c["D"])
        x[:, dst] = x[:, src]
    return {"k": s["k"], "v": s["v"]}


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "attention":
        counts, parents = _trees(c)
        prefix = _prefix(c)
        T = sum(counts)
        tokens = sum(p + n for p, n in zip(prefix, counts))
        scores = sum(p * n for p, n in zip(prefix, counts)) * c["hq"]
        return {"bytes": 4 * tokens * c["hkv"] * c["D"] + 4 * T * c["hq"] * c["D"] + 4 * T * c["hq"],
                "flops": 4 * scores * c["D"]}
    if c["op"] == "rope":
        rows = c["T"] * c["D"] * (c["hq"] + c["hk"] * (2 if c["append"] else 1))
        return {"bytes": 4 * rows + 4 * c["T"], "flops": 3 * c["T"] * c["rd"] * (c["hq"] + c["hk"])}
    if c["op"] == "verify":
        # the distribution that the last token is sampled from, and the draft's beside it
        rows = c["B"] * (2 if c["draft"] else 1)
        return {"bytes": 4 * rows * c["V"] + 12 * c["B"] * c["n"], "flops": 4 * rows * c["V"]}
    rng = random.Random(31 * c["B"] + c["n"])
    moved = 0
    for b in range(c["B"]):
        k = rng.randint(1, min(c["n"], 8)) if b else min(c["n"], 6)
        nodes = [0] + sorted(rng.sample(range(1, c["n"]), k - 1))
        moved += sum(x != i for i, x in enumerate(nodes))
    return {"bytes": max(64, 8 * moved * c["layers"] * c["hkv"] * c["D"]), "flops": 0}


# ---- the definitions in 64 bits ----------------------------------------------------------


def exact(case, seed):
    c = dict(case)
    if c["op"] == "verify":
        return None  # whole numbers
    s = prepare(c, seed)
    if c["op"] == "attention":
        return _exact_attention(s)
    if c["op"] == "rope":
        return _exact_rope(s)
    table, prefix = s["table"].cpu().numpy(), s["prefix"].cpu().numpy()
    path, counts = s["path"].cpu().numpy(), s["counts"].cpu().numpy()
    bs = c["bs"]
    for x in (s["k"], s["v"]):
        old = x.clone()
        for b in range(c["B"]):
            for d in range(counts[b]):
                i, j = prefix[b] + d, prefix[b] + path[b, d]
                x[:, table[b, i // bs], i % bs] = old[:, table[b, j // bs], j % bs]
    return {"k": s["k"], "v": s["v"]}


def _exact_attention(s):
    c = s["c"]
    hq, hkv, D, bs = c["hq"], c["hkv"], c["D"], c["bs"]
    prefix, ptr = s["prefix"].tolist(), s["ptr"].tolist()
    parents = s["parents"].tolist()
    out = torch.zeros(ptr[-1], hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((ptr[-1], hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n, P = ptr[b + 1] - ptr[b], prefix[b]
        see = np.zeros((n, P + n), bool)
        for i in range(n):
            j = i
            see[i, :P] = parents[ptr[b] + i] != -2
            while j >= 0 and parents[ptr[b] + j] != -2:
                see[i, P + j] = True
                j = parents[ptr[b] + j]
        see = torch.tensor(see, device="cuda")
        pages = s["table"][b, :-(-(P + n) // bs)].long()
        k = s["k"][pages].reshape(-1, hkv, D)[:P + n].double()
        v = s["v"][pages].reshape(-1, hkv, D)[:P + n].double()
        some = see.any(1)
        for h in range(hq):
            e = s["q"][ptr[b]:ptr[b + 1], h].double() @ k[:, h // (hq // hkv)].T / math.sqrt(D)
            e = e.masked_fill(~see, float("-inf"))
            l = torch.logsumexp(e, 1)
            p = torch.where(some[:, None], torch.exp(e - torch.where(some, l, 0.0)[:, None]), 0.0)
            out[ptr[b]:ptr[b + 1], h] = p @ v[:, h // (hq // hkv)]
            lse[ptr[b]:ptr[b + 1], h] = l
    return {"out": out, "lse": lse}


def _exact_rope(s):
    c = s["c"]
    rd, half = c["rd"], c["rd"] // 2
    angle = s["positions"].double().cpu()[:, None] * s["inv_freq"]
    turn = torch.polar(torch.full_like(angle, _attention_factor(c)), -angle if c["inverse"] else angle).cuda()

    def rotate(x):
        y = x.double().clone()
        first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
        second = first + (1 if c["interleaved"] else half)
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = rotate(s["q"]), rotate(s["k"])
    if not c["append"]:
        return {"q": q, "k": k}
    kc, vc = s["kc"].double(), s["vc"].double()
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            kc[slot // 16, slot % 16] = k[t]
            vc[slot // 16, slot % 16] = s["v"][t].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}
