"""sgmv_norm_rope and its gradient against the formulas in 64 bits: pair layouts, partial
heads, strides, caches of 16 bits and of e4m3, differences, repeats, graphs, streams."""
import numpy as np
import pytest
import torch

from tests import decode_reference as dref
from tests import spec_reference as ref
from tests.gpu_helpers import check_error_word

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]
EPS = 1e-5
# T, Hq, Hk, D, pairs: lanes of 4 to 32 per head, idle lanes, pairs of any number, few and many rows
SHAPES = [(1, 32, 8, 128, 64), (7, 8, 2, 128, 32), (33, 3, 1, 80, 16), (5, 4, 4, 64, 5), (3, 1, 1, 16, 8),
          (4, 2, 2, 256, 128), (2, 5, 5, 96, 0), (300, 2, 1, 64, 13), (1000, 40, 8, 32, 16), (9, 1, 7, 48, 24),
          (40, 1, 1, 240, 8), (65, 7, 3, 112, 55), (6, 2, 1, 8, 4), (11, 3, 2, 24, 8)]


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def rand(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def frequencies(sgmv, pairs):
    return sgmv.sgmv_rope_frequencies(pairs) if pairs else torch.empty(0, dtype=torch.float64)


class Rows:
    def __init__(self, sgmv, T, Hq, Hk, D, pairs, dtype, seed=0, far=5000):
        g = torch.Generator("cuda").manual_seed(seed + T + D)
        self.qkv = rand(g, T, Hq + 2 * Hk, D, dtype=dtype)
        self.qkv *= torch.logspace(-2, 1, T, device="cuda")[:, None, None].to(dtype)  # rows of any size
        self.q, self.k, self.v = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hk], self.qkv[:, Hq + Hk:]
        self.wq, self.wk = (1 + 0.3 * rand(g, 2, D, dtype=torch.float32)).to(dtype)
        self.pos = torch.randint(0, far, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.f = frequencies(sgmv, pairs)
        self.dy = rand(g, T, Hq + Hk, D, dtype=dtype)
        self.slots = torch.randperm(T + 40, generator=g, device="cuda").to(torch.int32)[:T]
        self.shape, self.dtype, self.g = (T, Hq, Hk, D, pairs), dtype, g

    def want(self, x, w, interleaved, scale):
        return dref.norm_rope(x, w, EPS, self.pos.cpu().numpy(), self.f.numpy(), interleaved, scale)


def close(got, y, bound):
    err = np.abs(ref.f64(got) - y)
    assert (err <= bound).all(), (err.max(), (err / bound).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_layouts_and_sizes(sgmv, dtype, interleaved, shape):
    r = Rows(sgmv, *shape, dtype)
    T, Hq, Hk, D, _ = shape
    q_out, k_out = torch.empty(T, Hq, D, device="cuda", dtype=dtype), torch.empty(T, Hk, D, device="cuda", dtype=dtype)
    before = r.qkv.clone()
    sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, EPS, interleaved, 1.25, q_out=q_out, k_out=k_out)
    assert sgmv.sgmv_last_launch_count() == 1
    check_error_word(0)
    assert torch.equal(r.qkv, before)
    for got, x, w in ((q_out, r.q, r.wq), (k_out, r.k, r.wk)):
        y, m = r.want(x, w, interleaved, 1.25)
        close(got, y, dref.norm_rope_bound(y, m, D, dtype))
    # in place, on strided views, one of the two alone: the same bits
    sgmv.sgmv_norm_rope(r.q, None, r.pos, r.f, r.wq, None, EPS, interleaved, 1.25)
    sgmv.sgmv_norm_rope(None, r.k, r.pos, r.f, None, r.wk, EPS, interleaved, 1.25)
    assert torch.equal(r.q, q_out) and torch.equal(r.k, k_out)
    assert torch.equal(r.v, before[:, Hq + Hk:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] % 16 == 0])
@pytest.mark.parametrize("order", ["pth", "pht"])
def test_append_to_an_e4m3_cache(sgmv, dtype, interleaved, shape, order):
    T, Hq, Hk, D, _ = shape
    r = Rows(sgmv, *shape, dtype, seed=1)
    blocks, bs = (T + 40 + 7) // 8 + 2, 8
    raw = torch.full((2, blocks, bs, Hk, D) if order == "pth" else (2, blocks, Hk, bs, D), 0x11, dtype=torch.uint8,
                     device="cuda")
    kc, vc = raw.view(dref.E4M3) if order == "pth" else raw.view(dref.E4M3).transpose(2, 3)
    ks, vs = (0.002 + 0.1 * torch.rand(2, Hk, generator=r.g, device="cuda"))
    slots = r.slots.clone()
    if T > 2:
        slots[T // 2] = -1
    k_out = torch.empty(T, Hk, D, device="cuda", dtype=dtype)
    sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, EPS, interleaved, q_out=torch.empty_like(r.q), k_out=k_out,
                        v=r.v, k_cache=kc, v_cache=vc, slots=slots, k_scale=ks, v_scale=vs)
    check_error_word(0)
    y, m = r.want(r.k, r.wk, interleaved, 1.0)
    close(k_out, y, dref.norm_rope_bound(y, m, D, dtype))
    live = slots >= 0
    at = slots[live].long()
    fp32 = dref.norm_rope_bound(y, m, D, None)
    for cache, x, off, scale in ((kc, y, fp32, ks), (vc, ref.f64(r.v), 0.0, vs)):
        scale = ref.f64(scale)[:, None]
        t = np.clip(x / scale, -dref.TOP, dref.TOP)[live.cpu().numpy()]
        off = (off / scale + 2.0 ** -22 * np.abs(x / scale))[live.cpu().numpy()]  # and of the division
        close(cache.float()[at // bs, at % bs], t, dref.e4m3_bound(np.abs(t) + off) + off)
    untouched = torch.ones(blocks * bs, dtype=torch.bool, device="cuda")
    untouched[at] = False
    for x in (raw if order == "pth" else raw.transpose(2, 3)):
        assert (x.reshape(blocks * bs, Hk, D)[untouched] == 0x11).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_to_a_16_bit_cache(sgmv, dtype, interleaved):
    r = Rows(sgmv, 37, 6, 2, 80, 20, dtype, seed=2)
    kc, vc = torch.zeros(2, 10, 8, 2, 80, device="cuda", dtype=dtype)
    k_out = torch.empty(37, 2, 80, device="cuda", dtype=dtype)
    args = (r.q, r.k, r.pos, r.f, r.wq, r.wk, EPS, interleaved)
    kw = dict(q_out=torch.empty_like(r.q), v=r.v, k_cache=kc, v_cache=vc, slots=r.slots)
    sgmv.sgmv_norm_rope(*args, k_out=k_out, **kw)
    at = r.slots.long()
    assert torch.equal(kc[at // 8, at % 8], k_out) and torch.equal(vc[at // 8, at % 8], r.v)
    # a slot out of range is left out and reported, the others are written
    kc.zero_()
    bad = r.slots.clone()
    bad[3], bad[5] = 80, -2
    sgmv.sgmv_norm_rope(*args, **{**kw, "slots": bad})
    check_error_word(4)
    good = torch.tensor([t not in (3, 5) for t in range(37)], device="cuda")
    assert torch.equal(kc[at[good] // 8, at[good] % 8], k_out[good])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_without_weights_it_is_the_rotation(sgmv, dtype, interleaved):
    r = Rows(sgmv, 50, 5, 3, 96, 24, dtype, seed=3)
    want = sgmv.sgmv_rope(r.q, r.k, r.pos, r.f, interleaved, 0.7, q_out=torch.empty_like(r.q),
                          k_out=torch.empty_like(r.k))
    got = sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, None, None, EPS, interleaved, 0.7, q_out=torch.empty_like(r.q),
                              k_out=torch.empty_like(r.k))
    for a, b, x in zip(got, want, (r.q, r.k)):
        y, m = r.want(x, None, interleaved, 0.7)
        close(a, y, ref.rope_bound(y, m, dtype))
        close(b, y, ref.rope_bound(y, m, dtype))


def test_values_that_are_no_numbers_stay_in_their_head(sgmv):
    r = Rows(sgmv, 6, 4, 2, 64, 32, torch.float16, seed=4)
    kc, vc = torch.zeros(2, 1, 8, 2, 64, device="cuda").to(dref.E4M3)
    ones = torch.ones(2, device="cuda")
    clean = sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, q_out=torch.empty_like(r.q),
                                k_out=torch.empty_like(r.k))
    r.q[1, 2, 7], r.k[3, 1, 0], r.v[2, 0, 5], r.v[2, 0, 6] = float("nan"), float("nan"), float("nan"), float("inf")
    slots = torch.arange(6, device="cuda", dtype=torch.int32)
    q, k = sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, q_out=torch.empty_like(r.q),
                               k_out=torch.empty_like(r.k), v=r.v, k_cache=kc, v_cache=vc, slots=slots, k_scale=ones,
                               v_scale=ones)
    assert q[1, 2].isnan().all() and k[3, 1].isnan().all() and kc.float()[0, 3, 1].isnan().all()
    q[1, 2], k[3, 1] = clean[0][1, 2], clean[1][3, 1]
    assert torch.equal(q, clean[0]) and torch.equal(k, clean[1])
    v = vc.float()[0, :6]
    assert v[2, 0, 5].isnan() and v[2, 0, 6] == dref.TOP and v.isnan().sum() == 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("weights", ["both", "q", "none"])
def test_gradient(sgmv, dtype, interleaved, shape, weights):
    T, Hq, Hk, D, _ = shape
    r = Rows(sgmv, *shape, dtype, seed=5)
    wq, wk = r.wq if weights != "none" else None, r.wk if weights == "both" else None
    dy = r.dy.clone()
    dq_out, dk_out = r.dy[:, :Hq], r.dy[:, Hq:]
    got = sgmv.sgmv_norm_rope_grad(dq_out, dk_out, r.q, r.k, r.pos, r.f, wq, wk, EPS, interleaved, 1.25)
    check_error_word(0)
    assert torch.equal(r.dy, dy)
    for dx, dw, y, x, w in ((got[0], got[2], dq_out, r.q, wq), (got[1], got[3], dk_out, r.k, wk)):
        a, b, am, bm = dref.norm_rope_grad(y, x, w, EPS, r.pos.cpu().numpy(), r.f.numpy(), interleaved, 1.25)
        # fp32 as in the forward pass, twice over; one rounding to the type
        close(dx, a, ref.ROUNDOFF[dtype] * np.abs(a) + 2 * (D / 8 + 32) * 2.0 ** -24 * am + 2.0 ** -25)
        assert (dw is None) == (w is None)
        if w is not None:
            # each term as above, and sums of at most all rows of a lane, then of 8 warps
            close(dw, b, (D / 8 + 32 + T * (Hq + Hk) / 64 + 16) * 2.0 ** -24 * bm + 1e-30)
    again = sgmv.sgmv_norm_rope_grad(dq_out, dk_out, r.q, r.k, r.pos, r.f, wq, wk, EPS, interleaved, 1.25)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))
    # q alone, k alone: the same values
    alone = sgmv.sgmv_norm_rope_grad(dq_out, None, r.q, None, r.pos, r.f, wq, None, EPS, interleaved, 1.25)
    assert torch.equal(alone[0], got[0]) and alone[1] is None and alone[3] is None
    alone = sgmv.sgmv_norm_rope_grad(None, dk_out, None, r.k, r.pos, r.f, None, wk, EPS, interleaved, 1.25)
    assert torch.equal(alone[1], got[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(sgmv, interleaved):
    """<dy, y(x + h d) - y(x - h d)> / 2h = <dx, d>, and so for the weights, in 64 bits."""
    r = Rows(sgmv, 5, 3, 2, 64, 20, torch.float16, seed=6)
    pos, f = r.pos.cpu().numpy(), r.f.numpy()
    dq, dk, dwq, dwk = sgmv.sgmv_norm_rope_grad(r.dy[:, :3], r.dy[:, 3:], r.q, r.k, r.pos, r.f, r.wq, r.wk, EPS,
                                                interleaved)
    rng, h = np.random.default_rng(0), 1e-6

    def y(x, w):
        return dref.norm_rope(torch.from_numpy(x), torch.from_numpy(w), EPS, pos, f, interleaved, 1.0)[0]

    for x, w, dy, dx, dw in ((r.q, r.wq, r.dy[:, :3], dq, dwq), (r.k, r.wk, r.dy[:, 3:], dk, dwk)):
        x, w, dy = ref.f64(x), ref.f64(w), ref.f64(dy)
        d, e = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        step = np.abs(x).mean(-1, keepdims=True)  # rows differ in size
        num = (dy * (y(x + h * d * step, w) - y(x - h * d * step, w))).sum() / (2 * h)
        ana = (ref.f64(dx) * d * step).sum()
        assert abs(num - ana) <= 2.0 ** -11 * (np.abs(ref.f64(dx) * d * step)).sum() + 1e-6
        num = (dy * (y(x, w + h * e) - y(x, w - h * e))).sum() / (2 * h)
        assert abs(num - (ref.f64(dw) * e).sum()) <= 1e-5 * np.abs(ref.f64(dw) * e).sum() + 1e-6


def test_no_rows(sgmv):
    z = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    pos, f, w = torch.empty(0, dtype=torch.int32, device="cuda"), frequencies(sgmv, 32), torch.ones(64, device="cuda").half()
    sgmv.sgmv_norm_rope(z, z[:, :2], pos, f, w, w)
    dw = torch.full((64,), 7.0, device="cuda")
    out = sgmv.sgmv_norm_rope_grad(z, z[:, :2], z, z[:, :2], pos, f, w, w, dq_weight=dw)
    assert (dw == 0).all() and (out[3] == 0).all() and out[0].shape == z.shape
    check_error_word(0)


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(sgmv, dtype):
    """Outputs inside wider tensors: what lies around them is not touched."""
    r = Rows(sgmv, 19, 4, 2, 64, 32, dtype, seed=7)
    want = sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, q_out=torch.empty_like(r.q),
                               k_out=torch.empty_like(r.k))
    wide = torch.full((19, 12, 96), 3.0, device="cuda", dtype=dtype)
    got = sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, q_out=wide[:, 0:8:2, 8:72], k_out=wide[:, 9:11, 8:72])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g0 = sgmv.sgmv_norm_rope_grad(r.dy[:, :4], r.dy[:, 4:], r.q, r.k, r.pos, r.f, r.wq, r.wk)
    sgmv.sgmv_norm_rope_grad(r.dy[:, :4], r.dy[:, 4:], r.q, r.k, r.pos, r.f, r.wq, r.wk, dq=wide[:, 0:8:2, 8:72],
                             dk=wide[:, 9:11, 8:72])
    assert torch.equal(wide[:, 0:8:2, 8:72], g0[0]) and torch.equal(wide[:, 9:11, 8:72], g0[1])
    assert (wide[:, :, :8] == 3).all() and (wide[:, :, 72:] == 3).all() and (wide[:, 1:8:2] == 3).all()


def test_a_cache_beyond_32_bit_offsets(sgmv):
    r = Rows(sgmv, 3, 2, 8, 128, 64, torch.float16, seed=8)
    blocks = 290_000  # of 16 tokens, 8 heads of 128: 4.75e9 bytes
    kc, vc = (torch.empty(blocks, 16, 8, 128, dtype=dref.E4M3, device="cuda") for _ in range(2))
    small = torch.zeros(2, 1, 16, 8, 128, device="cuda").to(dref.E4M3)
    scale = torch.full((8,), 0.01, device="cuda")
    kw = dict(q_out=torch.empty_like(r.q), v=r.v, k_scale=scale, v_scale=scale)
    for caches, first in (((kc, vc), (blocks - 1) * 16), (small, 0)):
        slots = torch.arange(first, first + 3, device="cuda", dtype=torch.int32)
        sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, k_cache=caches[0], v_cache=caches[1], slots=slots, **kw)
    check_error_word(0)
    for a, b in zip((kc, vc), small):
        assert torch.equal(a[-1, :3].view(torch.uint8), b[0, :3].view(torch.uint8))


def test_streams_and_graphs(sgmv):
    r = Rows(sgmv, 90, 8, 2, 128, 64, torch.bfloat16, seed=9)
    dq_out, dk_out = r.dy[:, :8], r.dy[:, 8:]
    want = sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, q_out=torch.empty_like(r.q),
                               k_out=torch.empty_like(r.k))
    grads = sgmv.sgmv_norm_rope_grad(dq_out, dk_out, r.q, r.k, r.pos, r.f, r.wq, r.wk)
    ws = [torch.full((sgmv.sgmv_norm_rope_grad_workspace_bytes(128),), 0xff, dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    q, k = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    outs = [[torch.zeros_like(t) for t in grads] for _ in range(2)]

    def both(i):
        sgmv.sgmv_norm_rope(r.q, r.k, r.pos, r.f, r.wq, r.wk, q_out=q, k_out=k)
        sgmv.sgmv_norm_rope_grad(dq_out, dk_out, r.q, r.k, r.pos, r.f, r.wq, r.wk, dq=outs[i][0], dk=outs[i][1],
                                 dq_weight=outs[i][2], dk_weight=outs[i][3], workspace=ws[i])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(0)
    side.synchronize()
    assert torch.equal(q, want[0]) and all(torch.equal(a, b) for a, b in zip(outs[0], grads))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            both(i)
    for _ in range(2):
        for t in (q, k, *outs[0], *outs[1]):
            t.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert all(torch.equal(a, b) for o in outs for a, b in zip(o, grads))
