"""sgmv_sample against the definition in whole numbers: filters alone and together, ties,
values that are no numbers, vocabularies from one token to more than shared memory holds,
unaligned rows, the distribution it hands on, streams and graphs."""
import numpy as np
import pytest
import torch

from tests import decode_reference as dref
from tests.gpu_helpers import check_error_word

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def rows_of(kind, T, V, g):
    x = torch.randn(T, V, generator=g, device="cuda")
    return {"normal": lambda: 3 * x, "flat": lambda: 1e-3 * x, "equal": lambda: torch.full_like(x, -1.5),
            "two": lambda: torch.where(x > 0, 1.0, 0.5), "whole": lambda: torch.round(2 * x),
            "peak": lambda: x + 40 * (torch.arange(V, device="cuda") == V // 2),
            "masked": lambda: torch.where(x < 0.3, float("-inf"), x)}[kind]()


def check(sgmv, x, tau, k, p, m, u, probs=True):
    T, V = x.shape

    def f32(v):
        return torch.tensor(np.broadcast_to(np.asarray(v, np.float32), T).copy(), device="cuda")

    ks = torch.tensor(np.broadcast_to(np.asarray(k, np.int32), T).copy(), device="cuda")
    out = torch.full((T, V), 7.0, device="cuda") if probs else None
    token = sgmv.sgmv_sample(x, f32(u), f32(tau), ks, f32(p), f32(m), probs=out)
    check_error_word(0)
    rows = dref.canonical(x)
    token = token.cpu().numpy()
    got = None if out is None else out.double().cpu().numpy()
    for t in range(T):
        def of(v):
            return np.broadcast_to(np.asarray(v), T)[t]

        want, w = dref.sample(rows[t], of(tau), int(of(k)), of(p), of(m), of(u))
        assert token[t] == want, (t, token[t], want, of(tau), of(k), of(p), of(m), of(u))
        if got is not None:
            total = max(1, int(w.sum()))
            # weights are off by a few units of 2^-38 of the largest, the quotient by three roundings
            assert (np.abs(got[t] - w / total) <= 4 * 2.0 ** -24 * w / total + 8.0 / total).all()
            # (a weight of a unit or two may be there or not)
            assert ((got[t] > 0) == (w > 0))[(w == 0) | (w > 2)].all() or (w[(got[t] > 0) != (w > 0)] <= 2).all()
    return token


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 255, 257, 1000, 4097, 32000, 100277])
@pytest.mark.parametrize("kind", ["normal", "flat", "whole", "peak", "masked"])
def test_filters_together(sgmv, dtype, V, kind):
    g = torch.Generator("cuda").manual_seed(V)
    x = rows_of(kind, 9, V, g).to(dtype)
    rng = np.random.default_rng(V)
    check(sgmv, x, tau=rng.choice([0.3, 0.8, 1.0, 2.0], 9), k=rng.choice([0, 1, 5, 50, 600, V], 9),
          p=rng.choice([0.1, 0.9, 0.97, 1.0], 9), m=rng.choice([0.0, 0.01, 0.2], 9), u=rng.random(9, np.float32))


@pytest.mark.parametrize("V", [300, 5000, 128256])
@pytest.mark.parametrize("kind", ["normal", "flat", "equal", "two", "whole"])
@pytest.mark.parametrize("what", ["k", "p", "m", "none"])
def test_one_filter(sgmv, V, kind, what):
    """Cuts that fall into few tokens, into many, and into one value held by thousands."""
    g = torch.Generator("cuda").manual_seed(V + len(kind))
    x = rows_of(kind, 8, V, g)
    k = [1, 2, 33, 255, 256, 257, V // 2, V - 1] if what == "k" else 0
    p = [0.0, 1e-7, 0.2, 0.5, 0.9, 0.99, 0.9999, 1.0] if what == "p" else 1.0
    m = [0.0, 1e-9, 0.003, 0.05, 0.3, 0.9, 1.0, 2.0] if what == "m" else 0.0
    for tau in (1.0, 0.25):
        check(sgmv, x, tau, k, p, m, np.linspace(0, 1 - 2 ** -24, 8, dtype=np.float32))


@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_no_numbers(sgmv, dtype):
    x = torch.randn(8, 700, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(dtype)
    x[0, 5] = float("nan")
    x[1] = float("nan")
    x[2] = float("-inf")
    x[3, 100] = float("inf")
    x[4, [7, 300]] = float("inf")
    x[5, :699] = float("-inf")
    x[6, ::2] = -0.0
    x[6, 1::2] = 0.0
    x[7, 3] = torch.finfo(dtype).min
    u = np.full(8, 0.7, np.float32)
    got = check(sgmv, x, 1.0, 0, 1.0, 0.0, u)
    assert got[1] == got[2] == -1 and got[3] == 100 and got[4] == 300 and got[5] == 699
    check(sgmv, x, 0.5, 40, 0.9, 0.0, u)
    check(sgmv, x, [0.0, 0.0, 0.0, -1.0, np.nan, 0.0, 0.0, 0.0], 0, 1.0, 0.0, u)  # the likeliest
    check(sgmv, x, 1.0, 3, 1.0, 0.0, u)


def test_settings_that_are_no_numbers_or_out_of_range(sgmv):
    x = torch.randn(8, 500, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    check(sgmv, x, [np.inf, 1e30, 1e-30, 1e-45, -0.0, 1e3, 1, 1], [-5, 2 ** 31 - 1, 0, 0, 0, 0, -1, 500],
          [1, 1, 1, 1, 1, 2.0, -1.0, np.nan], [0, 0, 0, 0, 0, -1.0, 0, np.nan],
          np.array([0.5, 0.999, 0.1, 0.2, 0.3, 1.0, 2.0, -1.0], np.float32))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 33, 1001, 32000])
@pytest.mark.parametrize("skew", [0, 1, 2, 3, 5])
def test_rows_anywhere_in_memory(sgmv, dtype, V, skew):
    """Rows of odd lengths and starts, and what lies between them is not read or written."""
    g = torch.Generator("cuda").manual_seed(V + skew)
    wide = torch.full((5, V + 11), float("nan"), device="cuda", dtype=dtype)
    wide[:, skew:skew + V] = (3 * torch.randn(5, V, generator=g, device="cuda")).to(dtype)
    x = wide[:, skew:skew + V]
    check(sgmv, x, 0.9, [0, 20, 0, 3, 0], [0.9, 1.0, 1.0, 0.5, 0.99], 0.0, np.linspace(0.05, 0.95, 5, dtype=np.float32))
    out = torch.full((5, V + 11), 7.0, device="cuda")
    sgmv.sgmv_sample(x, None, 0.9, 20, 0.95, probs=out[:, skew:skew + V])
    assert (out[:, :skew] == 7).all() and (out[:, skew + V:] == 7).all()
    assert (out[:, skew:skew + V].sum(1) - 1).abs().max() < 1e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_vocabulary_larger_than_shared_memory(sgmv, dtype):
    g = torch.Generator("cuda").manual_seed(3)
    x = rows_of("normal", 6, 500_003, g).to(dtype)
    check(sgmv, x, [1.0, 1.0, 0.0, 1.0, 0.5, 1.0], [0, 50, 0, 5000, 0, 0], [1.0, 1.0, 1.0, 0.9, 0.95, 0.5],
          [0.0, 0.0, 0.0, 0.0, 0.0, 0.1], np.linspace(0.05, 0.95, 6, dtype=np.float32))


@pytest.mark.parametrize("T", [1, 2, 19, 40, 77, 160, 700])
def test_many_rows(sgmv, T):
    """Every number of CTAs per row."""
    g = torch.Generator("cuda").manual_seed(T)
    x = rows_of("normal", T, 20011, g)
    rng = np.random.default_rng(T)
    check(sgmv, x, rng.choice([0.0, 0.7, 1.0], T), rng.choice([0, 10, 400], T), rng.choice([0.9, 1.0], T), 0.0,
          rng.random(T, np.float32), probs=T < 100)


def test_tokens_follow_the_distribution(sgmv):
    """Evenly spread random numbers draw every token as often as its probability says."""
    x = torch.randn(1, 50, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    n = 1 << 14
    probs = torch.empty(1, 50, device="cuda")
    sgmv.sgmv_sample(x, None, 0.8, 20, 0.9, probs=probs)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    got = torch.bincount(sgmv.sgmv_sample(x.expand(n, 50).contiguous(), u, 0.8, 20, 0.9).long(), minlength=50)
    assert (got / n - probs[0]).abs().max() <= 2 / n


def test_numbers_and_tensors_are_the_same_settings(sgmv):
    g = torch.Generator("cuda").manual_seed(5)
    x, u = rows_of("normal", 30, 9000, g), torch.rand(30, generator=g, device="cuda")

    def each(v, dtype=torch.float32):
        return torch.full((30,), v, dtype=dtype, device="cuda")

    a = sgmv.sgmv_sample(x, u, 0.7, 40, 0.9, 0.02)
    b = sgmv.sgmv_sample(x, u, each(0.7), each(40, torch.int32), each(0.9), each(0.02))
    assert torch.equal(a, b)
    out = torch.empty(30, dtype=torch.int32, device="cuda")
    assert sgmv.sgmv_sample(x, u, 0.7, 40, 0.9, 0.02, token=out) is out and torch.equal(out, a)


def test_no_rows(sgmv):
    x = torch.empty(0, 100, device="cuda")
    assert sgmv.sgmv_sample(x, torch.empty(0, device="cuda")).shape == (0,)


def test_streams_and_graphs(sgmv):
    g = torch.Generator("cuda").manual_seed(6)
    x, u = rows_of("normal", 12, 50257, g), torch.rand(12, generator=g, device="cuda")
    p0 = torch.empty_like(x)
    want = sgmv.sgmv_sample(x, u, 1.0, 0, 0.95, probs=p0)
    token, probs = torch.zeros_like(want), torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = x * 2
        sgmv.sgmv_sample(y, u, 2.0, 0, 0.95, token=token, probs=probs)
    side.synchronize()
    assert torch.equal(token, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sgmv.sgmv_sample(x, u, 1.0, 0, 0.95, token=token, probs=probs)
    for _ in range(3):
        token.zero_()
        probs.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(token, want) and torch.equal(probs, p0)
