"""Operators of a decoding step of models with normalised heads and an 8-bit cache, as cases to
measure: norms of queries and keys with the rotary positions and the append to the cache (norm),
their gradient (grad), attention of drafted trees over the 8-bit cache (attention), and sampling
with temperature, top-k, top-p and min-p from given random numbers (sample).

Each case names its operator in "op".  With ``own`` false, run() computes the operator
from elementary torch operations in 32 bits, or 64; with ``own`` true it calls the package.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
TOP = 448.0              # the largest e4m3 value
ONE = 1 << 38            # the largest weight of a distribution
UNIT = 1 << 24           # a uniform number's 24 bits
EPS = 1e-6


def _case(name, op, **kw):
    return {"name": name, "op": op, **kw}


def listed():
    return [
        # the decode rows of one layer: norms, rotation, append to the 8-bit cache; latency
        _case("norm-append8-128", "norm", dtype="f16", T=128, hq=32, hk=8, D=128, rd=128,
              interleaved=False, cache="e4m3", far=4096, factor=1.0),
        # a prefill of a long context with stretched frequencies, interleaved pairs
        _case("norm-append8-8k", "norm", dtype="bf16", T=8192, hq=32, hk=8, D=128, rd=128,
              interleaved=True, cache="e4m3", far=131072, factor=8.0),
        # odd heads, a partial rotation, the 16-bit cache
        _case("norm-append16-odd", "norm", dtype="bf16", T=2047, hq=40, hk=40, D=80, rd=32,
              interleaved=False, cache="same", far=2048, factor=1.0),
        # the gradient over a batch of 8192 tokens, grouped heads
        _case("grad-8k", "grad", dtype="bf16", T=8192, hq=32, hk=8, D=128, rd=128,
              interleaved=False, far=4096, factor=1.0),
        # the gradient of a short odd batch
        _case("grad-partial", "grad", dtype="f16", T=131, hq=20, hk=4, D=80, rd=32,
              interleaved=True, far=2048, factor=1.0),
        # one new token of one request, a short context: pure latency
        _case("attn8-decode-1", "attention", dtype="f16", B=1, n=1, ragged=False, hq=32, hkv=32,
              D=128, bs=16, longest=1500, pad=False),
        # 32 requests, each with a drafted tree of up to 16 tokens, contexts up to 4096
        _case("attn8-tree-32", "attention", dtype="f16", B=32, n=16, ragged=True, hq=32, hkv=32,
              D=128, bs=16, longest=4096, pad=False),
        # grouped heads, long contexts, large trees: the most arithmetic per byte
        _case("attn8-tree-gqa-long", "attention", dtype="bf16", B=8, n=64, ragged=True, hq=64,
              hkv=8, D=128, bs=64, longest=32768, pad=False),
        # a full decode batch padded to three tokens each, odd head and page sizes
        _case("attn8-decode-128-odd", "attention", dtype="bf16", B=128, n=3, ragged=True, hq=20,
              hkv=4, D=80, bs=24, longest=2100, pad=True),
        # one request's next token
        _case("sample-1", "sample", dtype="f32", T=1, V=32000, sharp=3.0, filters="p", probs=False),
        # a full batch with every filter and a large odd vocabulary
        _case("sample-128-large", "sample", dtype="f32", T=128, V=100277, sharp=3.0, filters="kpm", probs=False),
        # the target distributions of 32 trees of 16 tokens, for their verification
        _case("sample-512-probs", "sample", dtype="bf16", T=512, V=32000, sharp=3.0, filters="kp", probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "grad", "attention", "attention", "attention", "sample", "sample"))
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
    if op == "sample":
        V = rng.choice((_log(rng, 1000, 128000), 32000, 50257))
        probs = rng.random() < 0.4
        return {"op": op, "dtype": rng.choice(("f32", "f16", "bf16")), "V": V,
                "T": _log(rng, 1, max(2, min(512, 128 * 100277 // V))), "sharp": rng.choice((1.0, 3.0, 6.0)),
                "filters": rng.choice(("", "k", "p", "m", "kp", "kpm")), "probs": probs}
    D = rng.choice((64, 80, 96, 128, 128, 256))
    hk = rng.choice((1, 2, 8, 32))
    hq = hk * rng.choice((1, 4, 7))
    c = {"op": op, "dtype": dtype, "T": _log(rng, 1, max(2, min(8192, 8192 * 40 * 128 // ((hq + 2 * hk) * D)))),
         "hq": hq, "hk": hk, "D": D, "rd": rng.choice((D, D, D // 2, 16)), "interleaved": rng.random() < 0.5,
         "far": _log(rng, 16, 131072), "factor": rng.choice((1.0, 1.0, 4.0, 32.0))}
    if op == "norm":
        c["cache"] = rng.choice(("e4m3", "e4m3", "same"))
    return c


# ---- the batch's shape, fixed by the case alone ------------------------------------------


def _trees(c):
    """Nodes and parents of every sequence: a root (-1), then nodes that continue one of the
    few nodes before them; with "pad", rows that hold no token (-2) up to n."""
    rng = random.Random(1000003 * c["B"] + c["n"])
    counts, parents = [], []
    for b in range(c["B"]):
        n = c["n"] if not c["ragged"] or b == 0 else rng.randint(1, c["n"])
        p = [-1] + [rng.randint(max(0, i - 6), i - 1) for i in range(1, n)]
        if c["pad"]:
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


def _frequencies(c):
    """Inverse frequencies of the pairs; with a factor, the slow ones are stretched by it and
    the fast ones kept, with a linear ramp between."""
    out = []
    for i in range(c["rd"] // 2):
        f = 10000.0 ** (-2.0 * i / c["rd"])
        keep = min(1.0, max(0.0, (4096 * f / (2 * math.pi) - 1.0) / 31.0))
        out.append(f * keep + f / c["factor"] * (1.0 - keep))
    return out


def _magnitude(c):
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
        return torch.randn(shape, generator=g, device="cuda").to(DTYPES[c["dtype"]])

    def scales(n):  # as calibrated: some six deviations of unit data reach the largest value
        return (torch.rand(n, generator=g, device="cuda") + 0.5) * (6.0 / TOP)

    if c["op"] == "attention":
        B, bs, hkv, D = c["B"], c["bs"], c["hkv"], c["D"]
        counts, parents = _trees(c)
        prefix = _prefix(c)
        total = [p + n for p, n in zip(prefix, counts)]
        need = [-(-x // bs) for x in total]
        order = host.permutation(sum(need) + 3).astype(np.int32)  # scattered pages
        table, at = np.zeros((B, max(need)), np.int32), 0
        for b, k in enumerate(need):
            table[b, :k] = order[at:at + k]
            at += k

        def cache():
            x = torch.empty(sum(need) + 3, bs, hkv, D, device="cuda", dtype=DTYPES["e4m3"])
            flat = x.view(-1)
            for a in range(0, flat.numel(), 1 << 26):
                part = flat[a:a + (1 << 26)]
                part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(75.0).clamp_(-TOP, TOP))
            raw = x.view(torch.uint8)
            for b in range(B):  # slots that no token has been written to hold anything at all
                if total[b] % bs:
                    raw[table[b, total[b] // bs], total[b] % bs:] = 0x7F  # no number
            return x

        s["k"], s["v"], s["ks"], s["vs"] = cache(), cache(), scales(hkv), scales(hkv)
        T = sum(counts)
        s["q"] = randn(T, c["hq"], D)
        s["table"], s["prefix"] = _i32(table), _i32(prefix)
        s["ptr"], s["parents"] = _i32(np.concatenate([[0], np.cumsum(counts)])), _i32(parents)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, c["hq"], device="cuda")
        s["nodes"], s["length"] = max(counts), max(total)  # known to whoever built the batch
        if own:  # the workspace that a serving loop keeps
            from rank_gemv_gb300 import sgmv

            s["ws"] = torch.zeros(sgmv.sgmv_quant_attention_workspace_bytes(T, B, c["hq"], hkv, D),
                                  dtype=torch.uint8, device="cuda")
        return s
    T = c["T"]
    if c["op"] == "sample":
        V = c["V"]
        s["logits"] = (torch.randn(T, V, generator=g, device="cuda") * c["sharp"]).to(DTYPES[c["dtype"]])
        s["u"] = torch.rand(T, generator=g, device="cuda")
        # every request has its own settings; some want the likeliest token
        tau = host.choice([0.6, 0.8, 1.0, 1.0, 1.3], T)
        if T > 4:
            tau[T // 3] = 0.0
        f = c["filters"]
        k = host.choice([1, 20, 50, 50, 1000, 0], T) if "k" in f else np.zeros(T, int)
        p = host.choice([0.5, 0.9, 0.95, 0.99, 1.0], T) if "p" in f else np.ones(T)
        m = host.choice([0.0, 0.02, 0.05, 0.1], T) if "m" in f else np.zeros(T)
        s["tau"], s["p"], s["m"] = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (tau, p, m))
        s["k"] = _i32(k)
        s["token"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["probs"] = torch.empty(T, V, device="cuda") if c["probs"] else None
        return s
    hq, hk, D = c["hq"], c["hk"], c["D"]
    qkv = randn(T, hq + 2 * hk, D)  # the fused projection's output; q, k and v are views of it
    s["q"], s["kk"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    s["wq"], s["wk"] = (1.0 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).to(qkv.dtype)
    s["positions"] = _i32(host.randint(0, c["far"], T))
    s["inv_freq"] = torch.tensor(_frequencies(c), dtype=torch.float64)
    s["freq"] = s["inv_freq"].cuda()
    if c["op"] == "grad":
        s["dq_out"], s["dk_out"] = randn(T, hq, D), randn(T, hk, D)
        s["dq"], s["dk"] = torch.empty_like(s["dq_out"]), torch.empty_like(s["dk_out"])
        if own:  # the workspace that a training loop keeps
            from rank_gemv_gb300 import sgmv

            s["ws"] = torch.zeros(sgmv.sgmv_norm_rope_grad_workspace_bytes(D), dtype=torch.uint8, device="cuda")
        return s
    s["q_out"] = torch.empty(T, hq, D, device="cuda", dtype=qkv.dtype)
    blocks = -(-T // 16) + 8
    slots = host.permutation(blocks * 16)[:T].astype(np.int32)
    if T > 2:
        slots[T // 3] = -1  # a padding row is not appended
    s["slots"] = _i32(slots)
    kind = DTYPES["e4m3"] if c["cache"] == "e4m3" else qkv.dtype
    s["kc"], s["vc"] = (torch.zeros(blocks, 16, hk, D, device="cuda").to(kind) for _ in range(2))
    s["ks"], s["vs"] = (scales(hk), scales(hk)) if c["cache"] == "e4m3" else (None, None)
    return s


# ---- one pass ----------------------------------------------------------------------------


def run(s):
    return {"norm": _norm, "grad": _grad, "attention": _attention, "sample": _sample}[s["c"]["op"]](s)


def _turns(s):
    """Cosines and sines of the rows' angles (in 64 bits until there), magnitude included."""
    angle = s["positions"].double()[:, None] * s["freq"]
    scale = _magnitude(s["c"])
    return (angle.cos() * scale).float()[:, None], (angle.sin() * scale).float()[:, None]


def _rotate(c, x, cos, sin):
    rd = c["rd"]
    a, b = (x[..., 0:rd:2], x[..., 1:rd:2]) if c["interleaved"] else (x[..., :rd // 2], x[..., rd // 2:rd])
    y, z = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((y, z), -1).flatten(-2) if c["interleaved"] else torch.cat((y, z), -1)
    return torch.cat((y, x[..., rd:]), -1)


def _norm(s):
    c = s["c"]
    if own:
        from rank_gemv_gb300 import sgmv

        sgmv.sgmv_norm_rope(s["q"], s["kk"], s["positions"], s["inv_freq"], s["wq"], s["wk"], eps=EPS,
                            interleaved=c["interleaved"], scale=_magnitude(c), q_out=s["q_out"], v=s["v"],
                            k_cache=s["kc"], v_cache=s["vc"], slots=s["slots"], k_scale=s["ks"], v_scale=s["vs"])
        return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}
    cos, sin = _turns(s)

    def normed(x, w):
        x = x.float()
        return _rotate(c, x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float(), cos, sin)

    q, k, v = normed(s["q"], s["wq"]).to(s["q_out"].dtype), normed(s["kk"], s["wk"]), s["v"].float()
    if s["ks"] is not None:
        k = (k / s["ks"][:, None]).clamp(-TOP, TOP)
        v = (v / s["vs"][:, None]).clamp(-TOP, TOP)
    live = s["slots"] >= 0
    to = s["slots"][live].long()
    word = torch.uint8 if s["ks"] is not None else torch.int16
    for cache, x in ((s["kc"], k), (s["vc"], v)):
        cache.view(word).view(-1, c["hk"], c["D"])[to] = x.to(cache.dtype).view(word)[live]
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _grad(s):
    c = s["c"]
    if own:
        from rank_gemv_gb300 import sgmv

        dq, dk, dwq, dwk = sgmv.sgmv_norm_rope_grad(
            s["dq_out"], s["dk_out"], s["q"], s["kk"], s["positions"], s["inv_freq"], s["wq"], s["wk"], eps=EPS,
            interleaved=c["interleaved"], scale=_magnitude(c), dq=s["dq"], dk=s["dk"], workspace=s["ws"])
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    cos, sin = _turns(s)

    def back(dy, x, w):
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        g, xh = _rotate(c, dy.float(), cos, -sin), x * r
        h = g * w.float()
        dx = r * (h - xh * (h * xh).mean(-1, keepdim=True))
        return dx.to(s["dq"].dtype), (g * xh).sum((0, 1), dtype=torch.float64).float()

    dq, dwq = back(s["dq_out"], s["q"], s["wq"])
    dk, dwk = back(s["dk_out"], s["kk"], s["wk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _attention(s):
    c = s["c"]
    if own:
        from rank_gemv_gb300 import sgmv

        sgmv.sgmv_quant_attention(s["out"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["prefix"],
                                  s["ptr"], s["parents"], lse=s["lse"], workspace=s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    B, bs, hkv, D, n, L = c["B"], c["bs"], c["hkv"], c["D"], s["nodes"], s["length"]
    prefix, ptr = s["prefix"].long(), s["ptr"].long()
    count = ptr[1:] - ptr[:-1]
    node = torch.arange(n, device="cuda")
    there = node < count[:, None]                                       # [B, n]
    rows = torch.where(there, ptr[:-1, None] + node, 0)
    parent = torch.where(there, s["parents"].long()[rows], -2)
    live = parent > -2
    # who sees whom among the drafted tokens: itself and its ancestors
    sees = ((parent[:, :, None] == node) | (torch.eye(n, device="cuda", dtype=torch.bool) & live[:, :, None])).float()
    for _ in range(max(1, (n - 1).bit_length())):
        sees = ((sees @ sees) > 0).float()
    at = torch.arange(L, device="cuda")
    held = at < (prefix + count)[:, None]                               # [B, L]
    page = s["table"].long().gather(1, (at // bs).clamp(max=s["table"].shape[1] - 1).expand(B, L))
    slot = torch.where(held, page * bs + at % bs, 0)
    in_tree = (at - prefix[:, None]).clamp(0, n - 1)
    visible = torch.where((at < prefix[:, None])[:, None], live[:, :, None],
                          sees.gather(2, in_tree[:, None].expand(B, n, L)) > 0) & held[:, None]

    def read(cache, scale):
        x = cache.view(torch.uint8).view(-1, hkv, D)[slot].view(cache.dtype).float()  # [B, L, hkv, D]
        return torch.where(held[:, :, None, None], x * scale[:, None], 0.0)

    q = s["q"].float()[rows].reshape(B, n, hkv, c["hq"] // hkv, D)
    scores = torch.einsum("bnhgd,blhd->bhgnl", q, read(s["k"], s["ks"])) * (1.0 / math.sqrt(D))
    scores = torch.where(visible[:, None, None], scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    e = (scores - top).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgnl,blhd->bhgnd", e, read(s["v"], s["vs"])) / torch.where(total == 0, 1.0, total)
    lse = (total.log() + top)[..., 0]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, n, c["hq"], D)[there].to(s["q"].dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B, n, c["hq"])[there]}


def _sample(s):
    if own:
        from rank_gemv_gb300 import sgmv

        sgmv.sgmv_sample(s["logits"], s["u"], temperature=s["tau"], top_k=s["k"], top_p=s["p"], min_p=s["m"],
                         token=s["token"], probs=s["probs"])
        return {"token": s["token"]} if s["probs"] is None else {"token": s["token"], "probs": s["probs"]}
    # weights are whole numbers (2^38 is the likeliest token's), so their sums have one value in any order
    x = s["logits"].float() + 0.0                                       # one zero
    V = x.shape[1]
    rank = torch.arange(V, device="cuda")
    ranked, order = x.sort(dim=-1, descending=True, stable=True)  # ties: the lowest index first
    tau = s["tau"].double()[:, None]
    w = (((ranked.double() - ranked[:, :1].double()) / tau).exp() * float(ONE)).floor()
    w = torch.where(tau > 0, w, torch.where(rank == 0, float(ONE), 0.0)).long()
    k = torch.where(s["k"] > 0, s["k"].clamp(max=V), V)[:, None]
    w = torch.where(rank < k, w, 0)
    before = w.cumsum(-1) - w

    def part(total, fraction):  # of a total, by a fraction of 24 bits
        f = (fraction * float(UNIT)).long()
        return (total >> 24) * f + (((total & (UNIT - 1)) * f) >> 24)

    all_k = w.sum(-1)
    keep = (before < part(all_k, s["p"].clamp(0.0, 1.0))[:, None]) | (rank == 0)
    keep &= w >= (s["m"].clamp(0.0, 1.0) * float(ONE)).long()[:, None]
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0))
    run_sum = kept.cumsum(-1)
    total = run_sum[:, -1]
    mark = part(total, s["u"].clamp(0.0, 1.0 - 1.0 / UNIT))
    token = (run_sum <= mark[:, None]).sum(-1).int()
    if s["probs"] is None:
        return {"token": token}
    return {"token": token, "probs": (kept.double() / total.double()[:, None]).float()}


# ---- what a pass cannot do without -------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "attention":
        counts, _ = _trees(c)
        prefix = _prefix(c)
        T = sum(counts)
        tokens = sum(p + n for p, n in zip(prefix, counts))
        scores = sum(p * n for p, n in zip(prefix, counts)) * c["hq"]
        return {"bytes": 2 * tokens * c["hkv"] * c["D"] + 4 * T * c["hq"] * c["D"] + 4 * T * c["hq"],
                "flops": 4 * scores * c["D"]}
    if c["op"] == "sample":
        each = (4 if c["dtype"] == "f32" else 2) + (4 if c["probs"] else 0)
        return {"bytes": each * c["T"] * c["V"], "flops": 8 * c["T"] * c["V"]}
    rows, T, D = c["T"] * c["D"], c["T"], c["D"]
    if c["op"] == "grad":
        return {"bytes": 6 * rows * (c["hq"] + c["hk"]) + 4 * T + 12 * D, "flops": 16 * rows * (c["hq"] + c["hk"])}
    stored = 1 if c["cache"] == "e4m3" else 2
    return {"bytes": rows * (4 * c["hq"] + 2 * (2 + stored) * c["hk"]) + 8 * T + 4 * D,
            "flops": 8 * rows * (c["hq"] + c["hk"])}


# ---- the definitions in 64 bits ----------------------------------------------------------


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"norm": _exact_norm, "grad": _exact_grad, "attention": _exact_attention, "sample": _exact_sample}[c["op"]](s)


def _matrices(s):
    """Row t's rotation as a complex factor per pair, and the pairs' columns."""
    c = s["c"]
    half = c["rd"] // 2
    angle = s["positions"].double().cpu()[:, None] * s["inv_freq"]
    turn = torch.polar(torch.full_like(angle, _magnitude(c)), angle).cuda()[:, None]
    first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    return turn, first, first + (1 if c["interleaved"] else half)


def _turn(x, turn, first, second):
    y = x.clone()
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_norm(s):
    c = s["c"]

    def normed(x, w):
        x = x.double()
        length = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        return _turn(w.double() * x / torch.sqrt(length ** 2 / c["D"] + EPS), *_matrices(s))

    q, k, v = normed(s["q"], s["wq"]), normed(s["kk"], s["wk"]), s["v"].double()
    if s["ks"] is not None:
        k, v = ((x / scale.double()[:, None]).clamp(-TOP, TOP) for x, scale in ((k, s["ks"]), (v, s["vs"])))
    kc, vc = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (s["kc"], s["vc"]))
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            kc[slot // 16, slot % 16], vc[slot // 16, slot % 16] = k[t], v[t]
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_grad(s):
    turn, first, second = _matrices(s)
    out = {}
    for name, dy, x, w in (("q", s["dq_out"], s["q"], s["wq"]), ("k", s["dk_out"], s["kk"], s["wk"])):
        # the derivative by differentiation of the definition, in pieces that fit
        wd, dw, dx = w.double().requires_grad_(), 0.0, []
        for a in range(0, x.shape[0], 2048):
            xd = x[a:a + 2048].double().requires_grad_()
            xh = xd * (xd.square().mean(-1, keepdim=True) + EPS) ** -0.5
            y = xh * wd
            # <dy, R y> = <R^T dy, y>
            back = _turn(dy[a:a + 2048].double(), turn[a:a + 2048].conj(), first, second)
            gx, gw = torch.autograd.grad((back * y).sum(), (xd, wd))
            dx.append(gx)
            dw = dw + gw
        out["d" + name], out["dw" + name] = torch.cat(dx), dw
    return out


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
        k, v = (x.view(torch.uint8)[pages].view(x.dtype).reshape(-1, hkv, D)[:P + n].double() for x in (s["k"], s["v"]))
        some = see.any(1)
        for h in range(hq):
            kv = h // (hq // hkv)
            e = s["q"][ptr[b]:ptr[b + 1], h].double() @ (k[:, kv].T * (s["ks"][kv].double() / math.sqrt(D)))
            e = e.masked_fill(~see, float("-inf"))
            l = torch.logsumexp(e, 1)
            p = torch.where(some[:, None], torch.exp(e - torch.where(some, l, 0.0)[:, None]), 0.0)
            out[ptr[b]:ptr[b + 1], h] = p @ v[:, kv] * s["vs"][kv].double()
            lse[ptr[b]:ptr[b + 1], h] = l
    return {"out": out, "lse": lse}


def _exact_sample(s):
    if s["probs"] is None:
        return None  # whole numbers
    logits = s["logits"].double().cpu().numpy()
    tau, k, p, m = (s[x].cpu().numpy() for x in ("tau", "k", "p", "m"))
    out = np.zeros(logits.shape)
    for t, x in enumerate(logits):
        order = np.lexsort((np.arange(x.size), -x))
        if tau[t] <= 0:
            out[t, order[0]] = 1.0
            continue
        w = np.floor(np.exp((x[order] - x[order[0]]) / float(tau[t])) * ONE)
        w = w[:k[t]] if k[t] > 0 else w
        reach = np.concatenate([[0.0], np.cumsum(w)])
        if p[t] < 1:
            w = w[reach[:-1] < float(p[t]) * reach[-1]]
        w = w[w >= float(m[t]) * ONE]
        out[t, order[:w.size]] = w / w.sum()
    return {"token": None, "probs": torch.from_numpy(out)}
