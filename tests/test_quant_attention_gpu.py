"""sgmv_quant_attention against the softmax in 64 bits over the values that its e4m3 caches
stand for, and against the f16 attention over the same values, bit for bit: head layouts
and sizes, page sizes, contexts and trees of any length, rows that see nothing, values that
are no numbers, strides, streams, long caches, bad metadata, waits that run out."""
import numpy as np
import pytest
import torch

from tests import decode_reference as dref
from tests import spec_reference as ref
from tests.gpu_helpers import check_error_word
from tests.test_tree_attention_gpu import Batch

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


class Quant(Batch):
    """A batch whose caches k8 and v8 hold e4m3 values; k and v are what these stand for."""

    def __init__(self, prefix, nodes, Hq, Hkv, D, bs, dtype, seed=0, parents="random", order="pth", ones=False):
        super().__init__(prefix, nodes, Hq, Hkv, D, bs, dtype, seed, parents)
        g = torch.Generator("cuda").manual_seed(seed + 1)
        scales = torch.ones(2, Hkv, device="cuda") if ones else 0.004 + 0.02 * torch.rand(2, Hkv, generator=g, device="cuda")
        self.ks, self.vs = scales
        blocks = self.k.shape[0]
        self.spread = 1.0 if ones else 75.0
        parts = []
        for x in (self.k, self.v):
            x8 = (x.float() * self.spread).clamp(-dref.TOP, dref.TOP).to(dref.E4M3).view(torch.uint8)
            parts.append(x8)
        if order == "pht":
            self.k8, self.v8 = (x.transpose(1, 2).contiguous().view(dref.E4M3).transpose(1, 2) for x in parts)
        elif order == "kv":
            self.k8, self.v8 = torch.stack(parts, 1).view(dref.E4M3).unbind(1)
        else:
            self.k8, self.v8 = (x.view(dref.E4M3) for x in parts)
        assert self.k8.shape == (blocks, bs, Hkv, D)
        self.stand()

    def stand(self):
        self.k, self.v = (x.double() * s.double()[:, None] for x, s in ((self.k8, self.ks), (self.v8, self.vs)))

    def dirty(self):
        """No numbers, and large ones, in every slot that holds no token."""
        free = np.ones(self.k8.shape[0] * self.bs, bool)
        for b in range(self.B):
            free[ref.slots_of(self.table, b, range(self.total[b]), self.bs)] = False
        at = torch.tensor(np.flatnonzero(free), device="cuda")
        for x, bad in ((self.k8, 0x7F), (self.v8, 0xFF)):
            x.view(torch.uint8)[at // self.bs, at % self.bs] = bad
        return self

    def run(self, sgmv, **kw):
        table, prefix, ptr, parents = self.meta()
        sgmv.sgmv_quant_attention(self.out, self.q, self.k8, self.v8, self.ks, self.vs, table, prefix, ptr, parents,
                                  scale=self.scale, lse=self.lse, **kw)
        return self


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (5, 1), (16, 1), (14, 2)])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
def test_heads(sgmv, dtype, Hq, Hkv, D):
    b = Quant([37, 0, 260, 128], [5, 3, 1, 9], Hq, Hkv, D, 16, dtype, seed=Hq * D).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bs", [1, 5, 8, 16, 24, 32, 40, 64, 128, 200])
@pytest.mark.parametrize("D", [64, 80])
def test_page_sizes(sgmv, dtype, bs, D):
    b = Quant([700, 63, 1, 129, 0], [4, 1, 17, 2, 40], 6, 3, D, bs, dtype, seed=bs).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [0, 1, 15, 127, 128, 129, 255, 256, 1000, 5000])
@pytest.mark.parametrize("n", [1, 2, 64, 130, 256])
def test_lengths(sgmv, dtype, prefix, n):
    b = Quant([prefix], [n], 3, 1, 64, 16, dtype, seed=prefix + n).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 2, 7, 16, 32])
@pytest.mark.parametrize("n", [1, 8, 50])
@pytest.mark.parametrize("bs", [16, 5])
def test_groups(sgmv, dtype, group, n, bs):
    b = Quant([300, 40], [n, 3], group * 2, 2, 128, bs, dtype, seed=group + n).dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", [torch.float16])
@pytest.mark.parametrize("group,n,D", [(1, 1, 128), (4, 1, 64), (3, 6, 80), (8, 4, 128), (8, 8, 96), (16, 9, 128)])
@pytest.mark.parametrize("bs", [16, 24, 3])
def test_the_same_bits_as_16_bit_caches(sgmv, dtype, group, n, D, bs):
    """e4m3 values are f16 values too: with scales of 1 only the way in differs."""
    b = Quant([3000, 130, 0, 500, 77, 1], [n] * 6, group * 2, 2, D, bs, dtype, seed=n, ones=True).dirty().run(sgmv)
    check_error_word(0)
    table, prefix, ptr, parents = b.meta()
    out, lse = torch.empty_like(b.out), torch.empty_like(b.lse)
    sgmv.sgmv_tree_attention(out, b.q, b.k8.float().to(dtype), b.v8.float().to(dtype), table, prefix, ptr, parents,
                             scale=b.scale, lse=lse)
    check_error_word(0)
    assert torch.equal(out, b.out) and torch.equal(lse, b.lse)


@pytest.mark.parametrize("dtype", TYPES)
def test_every_value_of_the_type(sgmv, dtype):
    """All 254 numbers of e4m3, subnormal ones and both zeros among them, come back as V."""
    numbers = torch.tensor([x for x in range(256) if x & 0x7F != 0x7F], dtype=torch.uint8, device="cuda")
    n = len(numbers)
    k = torch.zeros(n, 1, 1, 64, dtype=torch.uint8, device="cuda").view(dref.E4M3)
    v = numbers[:, None, None, None].expand(n, 1, 1, 64).contiguous().view(dref.E4M3)
    one = torch.ones(1, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    q, out = torch.zeros(1, 1, 64, dtype=dtype, device="cuda"), torch.empty(1, 1, 64, dtype=dtype, device="cuda")
    for i in range(n):  # a context of one token
        sgmv.sgmv_quant_attention(out, q, k, v, one, one, torch.full((1, 1), i, **i32), torch.zeros(1, **i32),
                                  torch.tensor([0, 1], **i32))
        assert (out.float() == v[i].float()).all(), i
    check_error_word(0)


@pytest.mark.parametrize("group,n", [(1, 1), (2, 6), (4, 7), (8, 8), (16, 9)])
@pytest.mark.parametrize("D", [80, 128])
def test_queries_of_any_size(sgmv, group, n, D):
    """bf16 queries are converted row by row: rows and columns of very different sizes, beyond
    f16's range on both sides, with scores that stay moderate."""
    b = Quant([400, 33], [n, n], group * 2, 2, D, 16, torch.bfloat16, seed=n).dirty()
    size = torch.logspace(-30, 30, b.T * group * 2, base=10, device="cuda").view(b.T, group * 2, 1)
    q = b.q.double() * size
    q[..., 1::3] *= 2.0 ** -20
    b.q = q.to(torch.bfloat16)
    # each row's own scale of k is not to be had: the call's goes by the largest, in parts
    for t in range(0, b.T * group * 2, 7):
        row, head = divmod(t, group * 2)
        c = Quant([400, 33], [n, n], group * 2, 2, D, 16, torch.bfloat16, seed=n).dirty()
        c.q, c.scale = b.q, float(D ** -0.5 / size[row, head, 0])
        c.run(sgmv)
        check_error_word(0)
        out, _, tol, _ = ref.attention(c.q[row:row + 1, head:head + 1].expand(1, group * 2, D).double()
                                       .repeat(c.T, 1, 1), c.k, c.v, c.table, c.prefix, c.ptr, c.parents, c.scale, c.dtype)
        # (every row of the reference has this row's query: its own place is looked at)
        err = np.abs(ref.f64(c.out)[row, head] - out[row, head])
        assert (err <= tol[row, head]).all(), (row, head, err.max())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_queries_that_are_no_numbers_stay_in_their_row(sgmv, bad):
    b = Quant([400, 33], [5, 3], 8, 2, 64, 16, torch.bfloat16, seed=30).dirty().run(sgmv)
    want = b.out.clone()
    b.q[3, 5, 7] = bad
    b.run(sgmv)
    check_error_word(0)
    assert not torch.isfinite(b.out[3, 5].float()).all() or np.isinf(bad)
    same = torch.ones(b.T, 8, dtype=torch.bool, device="cuda")
    same[3, 5] = False
    assert torch.equal(b.out[same], want[same])


@pytest.mark.parametrize("group,n,Hkv,prefix,B", [(1, 9, 32, 1000, 40), (1, 1, 40, 500, 64), (8, 8, 8, 4000, 40),
                                                  (8, 20, 8, 9000, 17), (4, 3, 2, 60000, 5)])
@pytest.mark.parametrize("bs", [16, 24, 5])
def test_much_work(sgmv, group, n, Hkv, prefix, B, bs):
    """Every SM busy with several items, their ends cut and joined; the same in every run."""
    rng = np.random.default_rng(B)
    lens = [prefix] + [int(x) for x in rng.integers(prefix // 3, prefix, B - 1)]
    nodes = [n] + [int(x) for x in rng.integers(0, n + 1, B - 1)]
    b = Quant(lens, nodes, group * Hkv, Hkv, 64, bs, torch.bfloat16, seed=B + n).dirty()
    ws = torch.full((sgmv.sgmv_quant_attention_workspace_bytes(b.T, B, group * Hkv, Hkv, 64),), 0xff,
                    dtype=torch.uint8, device="cuda")
    b.run(sgmv, workspace=ws)
    check_error_word(0)
    first = b.out.clone()
    for _ in range(3):
        b.out.zero_()
        b.run(sgmv, workspace=ws)
        assert torch.equal(b.out, first)
    check_error_word(0)
    few = sorted({0, B // 2, B - 1})
    rows = np.concatenate([np.arange(b.ptr[s], b.ptr[s + 1]) for s in few])
    b.total, b.table, b.prefix = [b.total[s] for s in few], b.table[few], [b.prefix[s] for s in few]
    b.parents = [b.parents[r] for r in rows]
    b.q, b.out, b.lse, b.ptr = b.q[rows], b.out[rows], b.lse[rows], ref.ptr_of([nodes[s] for s in few])
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [0, 70])
def test_rows_that_see_nothing(sgmv, dtype, prefix):
    trees = [[-1, 0, -2, 1, -2], [-2, -2], [-1], [-1, -2, 0, -1, 3, -1]]
    b = Quant([prefix] * 4, None, 6, 2, 80, 16, dtype, seed=3, parents=trees).dirty().run(sgmv)
    check_error_word(0)
    b.check()
    pad = torch.tensor(np.flatnonzero(np.asarray(b.parents) == -2))
    assert (b.out[pad] == 0).all() and torch.isneginf(b.lse[pad]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 8, 32])
@pytest.mark.parametrize("byte", [0x7F, 0xFF])
def test_a_branch_that_holds_no_numbers_stays_alone(sgmv, dtype, group, byte):
    """Node 2's k or v are NaN: rows that do not see it keep their values, the others are lost."""
    tree = [-1, 0, 0, 1, 2, 3, 4, 1]
    b = Quant([130, 20], None, group * 2, 2, 64, 16, dtype, seed=4, parents=[tree, tree]).dirty()
    s = ref.slots_of(b.table, 0, [132], 16)[0]
    sees = ref.ancestors(tree)[:, 2]
    clean = np.flatnonzero(np.concatenate([~sees, np.ones(8, bool)]))
    b.v8.view(torch.uint8)[s // 16, s % 16, :, ::3] = byte
    b.run(sgmv)
    check_error_word(0)
    hit = ref.f64(b.out)[:8][sees]
    assert np.isnan(hit[..., ::3]).all() and np.isfinite(hit[..., 1::3]).all()
    b.check(clean)
    b.k8.view(torch.uint8)[s // 16, s % 16] = byte
    b.run(sgmv)
    assert np.isnan(ref.f64(b.out)[:8][sees]).all()
    b.check(clean)
    # and in the context, where every row sees it
    c = Quant([300], [2], group, 1, 64, 16, dtype, seed=5)
    s = ref.slots_of(c.table, 0, [17], 16)[0]
    c.v8.view(torch.uint8)[s // 16, s % 16, :, 5] = byte
    got = ref.f64(c.run(sgmv).out)
    assert np.isnan(got[..., 5]).all() and np.isfinite(np.delete(got, 5, -1)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [1, 4, 32])
def test_growing_scores(sgmv, dtype, group):
    """Scores that keep growing along the context (the running maximum moves), and a large scale."""
    b = Quant([1500, 1500], [3, 3], group, 1, 64, 16, dtype, seed=5)
    for s, order in ((0, 1.0), (1, -1.0)):
        at = torch.tensor(ref.slots_of(b.table, s, range(1503), 16), device="cuda")
        ramp = torch.linspace(0, 200.0 * order, 1503, device="cuda")[:, None, None].expand(-1, 1, 64)
        b.k8.view(torch.uint8).view(-1, 1, 64)[at] = ramp.to(dref.E4M3).view(torch.uint8)
    b.q = (b.q.float().abs() + 0.5).to(dtype)
    b.ks = b.ks * 2
    b.stand()
    b.dirty().run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["pth", "pht", "kv"])
@pytest.mark.parametrize("bs", [24, 7])
def test_strides(sgmv, dtype, order, bs):
    b = Quant([200, 31], [9, 2], 8, 2, 80, bs, dtype, seed=6, order=order).dirty()
    wide = torch.randn(b.T, 12, 160, device="cuda").to(dtype)
    wide[:, 2:10, :80] = b.q
    b.q = wide[:, 2:10, :80]
    out = torch.full((b.T, 16, 96), 3.0, device="cuda", dtype=dtype)
    b.out = out[:, ::2, 8:88]
    b.run(sgmv)
    check_error_word(0)
    b.check()
    assert (out[:, 1::2] == 3).all() and (out[:, :, :8] == 3).all() and (out[:, :, 88:] == 3).all()


def test_a_cache_beyond_32_bit_offsets(sgmv):
    blocks, bs, Hkv, D = 290_000, 16, 8, 128  # 4.75e9 bytes
    for pages in (16, 15):
        b = Quant([200, 77], [4, 1], 16, Hkv, D, pages, torch.float16, seed=10)
        k, v = (torch.empty(blocks, pages, Hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        far = np.where(b.table >= 0, blocks - 1 - b.table, b.table)
        for x in b.table[b.table >= 0]:
            k[blocks - 1 - int(x)], v[blocks - 1 - int(x)] = (y.view(torch.uint8)[int(x)] for y in (b.k8, b.v8))
        near = b.table
        b.k8, b.v8, b.table = k.view(dref.E4M3), v.view(dref.E4M3), far
        b.run(sgmv)
        check_error_word(0)
        b.table = near
        b.check()


def test_other_stream_and_graphs(sgmv):
    """Two graphs with a workspace each, and a call on another stream."""
    b = Quant([900, 33], [6, 4], 8, 2, 128, 16, torch.float16, seed=9).dirty().run(sgmv)
    want = b.out.clone()
    table, prefix, ptr, parents = b.meta()
    size = sgmv.sgmv_quant_attention_workspace_bytes(b.T, b.B, 8, 2, 128)
    ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(b.q) for _ in range(2)]

    def call(i, q, scale):
        sgmv.sgmv_quant_attention(outs[i], q, b.k8, b.v8, b.ks, b.vs, table, prefix, ptr, parents, scale=scale,
                                  workspace=ws[i])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(0, b.q * 2, b.scale / 2)
    side.synchronize()
    assert torch.equal(outs[0], want)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            call(i, b.q, b.scale)
    for _ in range(3):
        for i, graph in enumerate(graphs):
            outs[i].zero_()
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_rows_of_no_sequence_are_not_written(sgmv):
    b = Quant([60, 5], [4, 3], 4, 2, 64, 16, torch.float16, seed=11).dirty()
    b.q = torch.cat([b.q, b.q, b.q])
    b.out, b.lse = torch.full_like(b.q, 7.0), torch.full(b.q.shape[:2], 7.0, device="cuda")
    b.parents, b.T = [-1] * 5 + b.parents + [-1] * 9, 21
    b.ptr = b.ptr + 5
    b.run(sgmv)
    check_error_word(0)
    b.check(slice(5, 12))
    for x in (b.out, b.lse):
        assert (x[:5] == 7).all() and (x[12:] == 7).all()
    Quant([9], [0], 4, 2, 64, 16, torch.float16, seed=12).run(sgmv)  # no rows: nothing to do


@pytest.mark.parametrize("bs", [16, 5])
def test_bad_metadata_is_reported_and_left_out(sgmv, bs):
    def batch():
        return Quant([60, 5, 200], [4, 3, 2], 4, 2, 64, bs, torch.float16, seed=13).dirty()

    good = batch().run(sgmv)
    check_error_word(0)
    for change, status in (("length", 8), ("negative", 8), ("page", 4), ("parent", 4)):
        b = batch()
        if change == "length":
            b.prefix[1] = bs * b.table.shape[1]
        elif change == "negative":
            b.prefix[1] = -1
        elif change == "page":
            b.table[1, 0] = b.k8.shape[0]
        else:
            b.parents[5] = 1  # node 1 of sequence 1: its own parent
        b.run(sgmv)
        check_error_word(status)
        rows = np.r_[0:4, 7:9]
        assert torch.equal(b.out[rows], good.out[rows])


# (query heads per KV head, rows per sequence): row tiles of 8, 16, 32, 64 and 128
@pytest.mark.parametrize("group,n", [(4, 1), (2, 6), (4, 7), (8, 8), (16, 9)])
@pytest.mark.parametrize("bs", [16, 24, 5])
@pytest.mark.parametrize("role", [1, 2, 3, 4])
def test_waits_that_run_out(sgmv, group, n, bs, role):
    """Each role gives up as if a wait had run out: reported, nothing written, the next call right."""
    b = Quant([9000, 130, 0, 500, 77], [n] * 5, group * 2, 2, 64, bs, torch.float16, seed=n).dirty()
    ws = torch.zeros(sgmv.sgmv_quant_attention_workspace_bytes(b.T, b.B, group * 2, 2, 64), dtype=torch.uint8,
                     device="cuda")
    b.run(sgmv, workspace=ws)
    check_error_word(0)
    b.check()
    out, lse = b.out.clone(), b.lse.clone()
    b.out.fill_(7.0)
    b.lse.fill_(7.0)
    sgmv.sgmv_debug_inject_wait_timeout(role)
    try:
        b.run(sgmv, workspace=ws)
    finally:
        sgmv.sgmv_debug_inject_wait_timeout(0)
    assert sgmv.sgmv_get_device_error() == 7
    assert (b.out == 7).all() and (b.lse == 7).all()
    b.run(sgmv, workspace=ws)
    check_error_word(0)
    assert torch.equal(b.out, out) and torch.equal(b.lse, lse)


# ---- the commit, and a step of everything together -----------------------------------------


@pytest.mark.parametrize("n,bs,layers,Hkv,D,order", [(16, 16, 3, 4, 128, "pth"), (40, 24, 1, 5, 80, "pht"),
                                                     (9, 1, 0, 2, 16, "pth"), (256, 64, 2, 1, 256, "pht")])
def test_commit_of_an_e4m3_cache(sgmv, n, bs, layers, Hkv, D, order):
    from tests.test_cache_commit_gpu import i32, paths

    rng = np.random.default_rng(n)
    prefix = rng.integers(0, 100, 5)
    table, blocks = ref.paged(rng, [int(p) + n for p in prefix], bs)
    path, count = paths(rng, 5, n, n)
    lead = (layers,) if layers else ()
    shape = (*lead, blocks, bs, Hkv, D) if order == "pth" else (*lead, blocks, Hkv, bs, D)
    raw = [torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = (x if order == "pth" else x.transpose(-3, -2) for x in raw)
    want = []
    for x in (k, v):
        x = x.cpu().numpy()
        want.append(ref.commit(x if layers else x[None], table, prefix, path, count))
    sgmv.sgmv_cache_commit(k.view(dref.E4M3), v.view(dref.E4M3), i32(table), i32(prefix), i32(path), i32(count))
    check_error_word(0)
    for x, w in zip((k, v), want):
        x = x.cpu().numpy()
        assert np.array_equal(x if layers else x[None], w)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_step_of_everything(sgmv, dtype):
    """Drafted trees of a model with head norms over an 8-bit cache: norms, rotation and append,
    attention, the filtered distributions, verification and commit, each against its reference
    on what the one before it left."""
    Hq, Hkv, D, bs, V = 8, 2, 64, 16, 700
    b = Quant([100, 0, 37], [9, 4, 1], Hq, Hkv, D, bs, dtype, seed=20).dirty()
    T, g = b.T, torch.Generator("cuda").manual_seed(21)
    table, prefix, ptr, parents = b.meta()
    counts = np.diff(b.ptr)
    place = np.concatenate([p + np.arange(n) for p, n in zip(b.prefix, counts)])
    slots = torch.tensor(np.concatenate([ref.slots_of(b.table, s, b.prefix[s] + np.arange(counts[s]), bs)
                                         for s in range(3)]), dtype=torch.int32, device="cuda")
    pos = torch.tensor(place, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
    wq, wk = (1 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).to(dtype)
    f = sgmv.sgmv_rope_frequencies(D // 2)
    b.ks, b.vs = (torch.full((Hkv,), 0.015, device="cuda") for _ in range(2))
    sgmv.sgmv_norm_rope(q, k, pos, f, wq, wk, q_out=b.q, v=v, k_cache=b.k8, v_cache=b.v8, slots=slots, k_scale=b.ks,
                        v_scale=b.vs)
    y, m = dref.norm_rope(k, wk, 1e-6, place, f.numpy(), False, 1.0)
    t, off = np.clip(y / 0.015, -dref.TOP, dref.TOP), dref.norm_rope_bound(y, m, D, None) / 0.015
    got = b.k8.float()[slots.long() // bs, slots.long() % bs]
    assert (np.abs(ref.f64(got) - t) <= dref.e4m3_bound(np.abs(t) + off) + off + 2.0 ** -22 * np.abs(t)).all()
    b.stand()
    b.run(sgmv)
    check_error_word(0)
    b.check()
    logits = (b.out.float().reshape(T, Hq * D) @ torch.randn(Hq * D, V, generator=g, device="cuda"))
    target = torch.empty(T, V, device="cuda")
    sgmv.sgmv_sample(logits, None, 0.8, 50, 0.95, 0.01, probs=target)
    rows = dref.canonical(logits)
    for r in range(T):
        _, w = dref.sample(rows[r], 0.8, 50, 0.95, 0.01, 0.0)
        assert np.abs(ref.f64(target[r]) - w / w.sum()).max() <= 2.0 ** -21
    tokens = target.argmax(1).roll(1).to(torch.int32)
    u = torch.rand(T + 3, generator=g, device="cuda")
    count, path, token = sgmv.sgmv_tree_verify(target, None, tokens, parents, ptr, u[:T], u[T:], 9)
    want = ref.verify(target.cpu().numpy(), None, tokens.cpu().numpy(), b.parents, b.ptr, u[:T].cpu().numpy(),
                      u[T:].cpu().numpy(), 9)
    for a, w in zip((count, path, token), want):
        assert np.array_equal(a.cpu().numpy(), w)
    k0, v0 = (x.view(torch.uint8).cpu().numpy()[None] for x in (b.k8, b.v8))
    sgmv.sgmv_cache_commit(b.k8, b.v8, table, prefix, path, count)
    check_error_word(0)
    for x, old in ((b.k8, k0), (b.v8, v0)):
        assert np.array_equal(x.view(torch.uint8).cpu().numpy()[None], ref.commit(old, b.table, b.prefix, want[1], want[0]))
