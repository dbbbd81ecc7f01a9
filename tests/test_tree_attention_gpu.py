"""sgmv_tree_attention against the softmax in 64 bits: head layouts and sizes,
page sizes, contexts and trees of any length, rows that see nothing, slots and
branches that hold NaN, strides, streams, long caches, bad metadata."""
import numpy as np
import pytest
import torch

from tests import spec_reference as ref
from tests.gpu_helpers import check_error_word

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


class Batch:
    """A random batch; parents: per sequence a list of parents, or None (chains)."""

    def __init__(self, prefix, nodes, Hq, Hkv, D, bs, dtype, seed=0, parents="random", order="pth", blocks=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator("cuda").manual_seed(seed)
        counts = [len(p) for p in parents] if isinstance(parents, list) else list(nodes)
        trees = parents if isinstance(parents, list) else [ref.random_tree(rng, n) for n in counts]
        self.total = [p + n for p, n in zip(prefix, counts)]
        self.table, used = ref.paged(rng, self.total, bs)
        blocks = blocks or used
        shape = (blocks, bs, Hkv, D)

        def rand(*s):
            return torch.randn(s, generator=g, device="cuda").to(dtype)

        if order == "pht":    # pages of [heads, tokens, D]
            self.k, self.v = (rand(blocks, Hkv, bs, D).transpose(1, 2) for _ in range(2))
        elif order == "kv":   # k and v of a page side by side
            self.k, self.v = rand(blocks, 2, bs, Hkv, D).unbind(1)
        else:
            self.k, self.v = rand(*shape), rand(*shape)
        self.prefix, self.ptr, self.bs = list(prefix), ref.ptr_of(counts), bs
        self.parents = None if parents is None else [p for t in trees for p in t]
        self.T, self.B, self.dtype, self.scale = int(self.ptr[-1]), len(prefix), dtype, D ** -0.5
        self.q = rand(self.T, Hq, D)
        self.out = torch.full_like(self.q, 7.0)
        self.lse = torch.full((self.T, Hq), 7.0, device="cuda")

    def dirty(self):
        """NaN and infinities in every slot that holds no token."""
        blocks, Hkv, D = self.k.shape[0], self.k.shape[2], self.k.shape[3]
        free = np.ones(blocks * self.bs, bool)
        for b in range(self.B):
            free[ref.slots_of(self.table, b, range(self.total[b]), self.bs)] = False
        at = torch.tensor(np.flatnonzero(free), device="cuda")
        for x, bad in ((self.k, float("nan")), (self.v, float("inf"))):
            x[at // self.bs, at % self.bs] = bad
        return self

    def meta(self):
        def i32(x):
            return torch.tensor(np.asarray(x, np.int32), device="cuda")

        return (i32(self.table), i32(self.prefix), i32(self.ptr),
                None if self.parents is None else i32(self.parents))

    def run(self, sgmv, **kw):
        table, prefix, ptr, parents = self.meta()
        sgmv.sgmv_tree_attention(self.out, self.q, self.k, self.v, table, prefix, ptr, parents,
                                 scale=self.scale, lse=self.lse, **kw)
        return self

    def check(self, rows=slice(None)):
        out, lse, tol, ltol = ref.attention(self.q, self.k, self.v, self.table, self.prefix, self.ptr,
                                            self.parents, self.scale, self.dtype)
        got, glse = ref.f64(self.out)[rows], ref.f64(self.lse)[rows]
        err = np.abs(got - out[rows])
        assert (err <= tol[rows]).all(), (np.nanmax(err), np.nanmax(err / tol[rows]))
        none = np.isneginf(lse[rows])
        assert np.array_equal(np.isneginf(glse), none)
        assert (np.abs(np.where(none, 0, glse) - np.where(none, 0, lse[rows])) <= ltol[rows]).all()


HEADS = [(4, 4), (8, 2), (5, 1), (16, 1), (14, 2)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("D", [8, 64, 80, 128, 136, 256])
def test_heads(sgmv, dtype, Hq, Hkv, D):
    b = Batch([37, 0, 260, 128], [5, 3, 1, 9], Hq, Hkv, D, 16, dtype, seed=Hq * D).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bs", [1, 5, 8, 16, 24, 32, 64, 128, 200])
def test_page_sizes(sgmv, dtype, bs):
    b = Batch([700, 63, 1, 129, 0], [4, 1, 17, 2, 40], 6, 3, 96, bs, dtype, seed=bs).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [0, 1, 15, 127, 128, 129, 255, 256, 1000, 5000])
@pytest.mark.parametrize("n", [1, 2, 64, 65, 130, 256])
def test_lengths(sgmv, dtype, prefix, n):
    b = Batch([prefix], [n], 3, 1, 64, 16, dtype, seed=prefix + n).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 2, 7, 16, 32])
@pytest.mark.parametrize("n", [1, 8, 50])
def test_groups(sgmv, dtype, group, n):
    b = Batch([300, 40], [n, 3], group * 2, 2, 128, 16, dtype, seed=group + n).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
def test_many_ragged_sequences(sgmv, dtype):
    rng = np.random.default_rng(1)
    prefix = [int(x) for x in rng.integers(0, 400, 300)]
    nodes = [int(x) for x in rng.integers(0, 6, 300)]  # some sequences have no rows at all
    b = Batch(prefix, nodes, 4, 2, 64, 16, dtype, seed=2).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("group,n,Hkv,prefix,B", [(1, 9, 32, 1000, 40), (1, 1, 40, 500, 64), (8, 4, 8, 2000, 60),
                                                  (8, 8, 8, 4000, 40), (8, 20, 8, 9000, 17), (4, 3, 2, 60000, 5)])
@pytest.mark.parametrize("bs", [16, 24])
def test_much_work(sgmv, group, n, Hkv, prefix, B, bs):
    """Every SM busy with several items, their ends cut and joined."""
    rng = np.random.default_rng(B)
    lens = [prefix] + [int(x) for x in rng.integers(prefix // 3, prefix, B - 1)]
    nodes = [n] + [int(x) for x in rng.integers(1, n + 1, B - 1)]
    b = Batch(lens, nodes, group * Hkv, Hkv, 64, bs, torch.bfloat16, seed=B + n).dirty()
    ws = torch.zeros(sgmv.sgmv_tree_attention_workspace_bytes(b.T, B, group * Hkv, Hkv, 64), dtype=torch.uint8,
                     device="cuda")
    b.run(sgmv, workspace=ws)
    check_error_word(0)
    first = b.out.clone()
    for _ in range(3):
        b.out.zero_()
        b.run(sgmv, workspace=ws)
        assert torch.equal(b.out, first)
    check_error_word(0)
    # a sample of the sequences against the reference
    few = sorted({0, B // 2, B - 1})
    rows = np.concatenate([np.arange(b.ptr[s], b.ptr[s + 1]) for s in few])
    b.total, b.table, b.prefix = [b.total[s] for s in few], b.table[few], [b.prefix[s] for s in few]
    b.parents = [b.parents[r] for r in rows]
    b.q, b.out, b.lse, b.ptr = b.q[rows], b.out[rows], b.lse[rows], ref.ptr_of([nodes[s] for s in few])
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group,Hkv,D", [(1, 4, 128), (2, 2, 64), (3, 2, 80), (5, 1, 128), (8, 2, 96), (9, 1, 64)])
@pytest.mark.parametrize("nodes", ["one", "uneven", "padded"])
@pytest.mark.parametrize("bs", [16, 24, 5])
def test_a_token_per_sequence(sgmv, dtype, group, Hkv, D, nodes, bs):
    """Decoding without drafts; and as many rows in all, but with sequences that
    have none or several of them, or rows that are padding.  Short and long contexts, scores
    that grow along one of them (its running maximum moves)."""
    prefix = [0, 1, 127, 128, 4000, 16, 300, 1100]
    counts = {"one": [1] * 8, "uneven": [0, 9, 1, 0, 1, 3, 0, 2], "padded": [1] * 8}[nodes]
    trees = None
    if nodes == "padded":
        trees = [[-2] if s in (1, 4) else [-1] for s in range(8)]
    b = Batch(prefix, counts, group * Hkv, Hkv, D, bs, dtype, seed=group + bs, parents=trees or "random")
    at = torch.tensor(ref.slots_of(b.table, 7, range(b.total[7]), bs), device="cuda")
    grow = torch.linspace(0, 4.0, len(at), device="cuda")[:, None, None].to(dtype)
    b.k.view(-1, Hkv, D)[at] *= grow
    b.dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group,tree", [(1, [-1]), (4, [-1, 0, -2, 0, 1]), (16, [-1, 0, 1, 2, 3, 4, 5, 6, 7])])
@pytest.mark.parametrize("prefix", [1100, 20000])
def test_one_sequence_in_many_parts(sgmv, dtype, group, tree, prefix):
    """A single sequence and KV head, cut into as many parts as there are, with
    scores that grow (parts differ in their maxima) and a row that sees nothing."""
    b = Batch([prefix], None, group, 1, 64, 16, dtype, seed=group, parents=[tree])
    at = torch.tensor(ref.slots_of(b.table, 0, range(b.total[0]), 16), device="cuda")
    b.k.view(-1, 1, 64)[at] *= torch.linspace(0, 3.0, len(at), device="cuda")[:, None, None].to(dtype)
    b.dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 4, 31, 200])
def test_chains_without_parents(sgmv, dtype, n):
    b = Batch([150, 0, 3], [n, n, 1], 4, 1, 64, 32, dtype, seed=n, parents=None).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [0, 70])
def test_rows_that_see_nothing(sgmv, dtype, prefix):
    trees = [[-1, 0, -2, 1, -2], [-2, -2], [-1], [-1, -2, 0, -1, 3, -1]]
    b = Batch([prefix] * 4, None, 6, 2, 80, 16, dtype, seed=3, parents=trees).dirty().run(sgmv)
    check_error_word(0)
    b.check()
    pad = np.flatnonzero(np.asarray(b.parents) == -2)
    assert (b.out[torch.tensor(pad)] == 0).all() and torch.isneginf(b.lse[torch.tensor(pad)]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 8, 32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_branch_with_bad_values_stays_alone(sgmv, dtype, group, bad):
    """Node 2's k and v are not finite: rows that do not see node 2 keep their
    values, rows that see it get what the formula gives (never finite here)."""
    tree = [-1, 0, 0, 1, 2, 3, 4, 1]
    b = Batch([130, 20], None, group * 2, 2, 64, 16, dtype, seed=4, parents=[tree, tree])
    s = ref.slots_of(b.table, 0, [130 + 2], 16)[0]
    b.dirty()
    b.v[s // 16, s % 16, :, ::3] = bad
    b.run(sgmv)
    check_error_word(0)
    sees = ref.ancestors(tree)[:, 2]
    got = ref.f64(b.out)
    hit = got[:8][sees]
    assert not np.isfinite(hit[..., ::3]).any()
    if np.isinf(bad):
        assert (hit[..., ::3] == bad).all()
    clean = np.concatenate([~sees, np.ones(8, bool)])
    b.v[s // 16, s % 16] = 0
    b.check(np.flatnonzero(clean))
    # a bad key: whoever sees it is lost, the others are not touched
    b.k[s // 16, s % 16] = float("nan")
    b.run(sgmv)
    assert np.isnan(ref.f64(b.out)[:8][sees]).all()
    b.k[s // 16, s % 16] = 0
    b.check(np.flatnonzero(clean))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 4, 32])
def test_growing_scores(sgmv, dtype, group):
    """Scores that keep growing along the context (the running maximum moves in
    every tile), and one outlier at its very start."""
    b = Batch([1500, 1500], [3, 3], group, 1, 64, 16, dtype, seed=5)
    for s, order in ((0, 1.0), (1, -1.0)):
        at = torch.tensor(ref.slots_of(b.table, s, range(1503), 16), device="cuda")
        ramp = torch.linspace(0, 6.0 * order, 1503, device="cuda")[:, None, None]
        b.k.view(-1, 1, 64)[at] = (ramp * 0.5 + 0.1 * b.k.view(-1, 1, 64)[at].float()).to(dtype)
    b.q = (b.q.float().abs() + 0.5).to(dtype)
    b.dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["pth", "pht", "kv"])
def test_strides(sgmv, dtype, order):
    b = Batch([200, 31], [9, 2], 8, 2, 80, 24, dtype, seed=6, order=order).dirty()
    wide = torch.randn(b.T, 12, 160, device="cuda").to(dtype)
    wide[:, 2:10, :80] = b.q
    b.q = wide[:, 2:10, :80]
    out = torch.full((b.T, 16, 96), 3.0, device="cuda", dtype=dtype)
    b.out = out[:, ::2, 8:88]
    b.run(sgmv)
    check_error_word(0)
    b.check()
    assert (out[:, 1::2] == 3).all() and (out[:, :, :8] == 3).all() and (out[:, :, 88:] == 3).all()


@pytest.mark.parametrize("Hq,D,n", [(4, 64, 3), (32, 128, 9), (2, 256, 2)])
def test_results_repeat_whatever_the_workspace_holds(sgmv, Hq, D, n):
    b = Batch([3000, 700, 10], [n, 1, 2], Hq, 2, D, 16, torch.bfloat16, seed=7).dirty()
    size = sgmv.sgmv_tree_attention_workspace_bytes(b.T, b.B, Hq, 2, D)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    b.run(sgmv, workspace=ws)
    first, lse = b.out.clone(), b.lse.clone()
    b.check()
    for fill in (None, 0, 0x7f):  # as the last call left it, and other contents
        if fill is not None:
            ws.fill_(fill)
        b.out.zero_()
        b.run(sgmv, workspace=ws)
        assert torch.equal(b.out, first) and torch.equal(b.lse, lse)
    other = Batch([40], [2], Hq, 2, D, 16, torch.bfloat16, seed=8).dirty().run(sgmv, workspace=ws)
    other.check()


def test_other_stream_and_graph(sgmv):
    b = Batch([900, 33], [6, 4], 8, 2, 128, 16, torch.float16, seed=9).dirty()
    b.run(sgmv)
    want = b.out.clone()
    ws = torch.zeros(sgmv.sgmv_tree_attention_workspace_bytes(b.T, b.B, 8, 2, 128), dtype=torch.uint8, device="cuda")
    table, prefix, ptr, parents = b.meta()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(b.q)
    with torch.cuda.stream(side):
        q = b.q * 2
        for _ in range(2):
            sgmv.sgmv_tree_attention(out, q, b.k, b.v, table, prefix, ptr, parents, scale=b.scale / 2, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgmv.sgmv_tree_attention(out, b.q, b.k, b.v, table, prefix, ptr, parents, scale=b.scale, workspace=ws)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_a_cache_beyond_32_bit_offsets(sgmv):
    """Pages above 2^31 elements, and above 2^32 bytes, from the cache's start."""
    blocks, bs, Hkv, D = 140_000, 16, 8, 128  # 2.3e9 elements
    b = Batch([200, 77], [4, 1], 16, Hkv, D, bs, torch.float16, seed=10)
    k = torch.empty(blocks, bs, Hkv, D, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    far = np.where(b.table >= 0, blocks - 1 - b.table, b.table)
    for s in range(b.B):
        for x in b.table[s][b.table[s] >= 0]:
            k[blocks - 1 - int(x)], v[blocks - 1 - int(x)] = b.k[int(x)], b.v[int(x)]
    b.k, b.v, b.table = k, v, far
    b.run(sgmv)
    check_error_word(0)
    b.check()


def test_rows_of_no_sequence_are_not_written(sgmv):
    b = Batch([60, 5], [4, 3], 4, 2, 64, 16, torch.float16, seed=11).dirty()
    b.q = torch.cat([b.q, b.q, b.q])
    b.out, b.lse = torch.full_like(b.q, 7.0), torch.full(b.q.shape[:2], 7.0, device="cuda")
    b.parents, b.T = [-1] * 5 + b.parents + [-1] * 9, 21
    b.ptr = b.ptr + 5
    b.run(sgmv)
    check_error_word(0)
    b.check(slice(5, 12))
    for x in (b.out, b.lse):
        assert (x[:5] == 7).all() and (x[12:] == 7).all()
    empty = Batch([9], [0], 4, 2, 64, 16, torch.float16, seed=12)
    empty.run(sgmv)  # no rows: nothing to do


@pytest.mark.parametrize("Hq,D", [(4, 64), (4, 256)])
def test_bad_metadata_is_reported_and_left_out(sgmv, Hq, D):
    def batch():
        return Batch([60, 5, 200], [4, 3, 2], Hq, 2, D, 16, torch.float16, seed=13).dirty()

    good = batch().run(sgmv)
    check_error_word(0)
    for change, status in (("length", 8), ("negative", 8), ("decreasing", 8), ("page", 4), ("parent", 4)):
        b = batch()
        if change == "length":
            b.prefix[1] = 16 * b.table.shape[1]
        elif change == "negative":
            b.prefix[1] = -1
        elif change == "decreasing":
            b.ptr = np.array([0, 4, 7, 6], np.int32)
        elif change == "page":
            b.table[1, 0] = b.k.shape[0]
        else:
            b.parents[5] = 1  # node 1 of sequence 1: its own parent
        b.run(sgmv)
        check_error_word(status)
        rows = np.r_[0:7] if change == "decreasing" else np.r_[0:4, 7:9]
        assert torch.equal(b.out[rows], good.out[rows])
