"""sgmv_cache_commit against the moves done one by one: bit for bit."""
import numpy as np
import pytest
import torch

from tests import spec_reference as ref
from tests.gpu_helpers import check_error_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def paths(rng, B, n, width):
    path, count = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        count[b] = rng.integers(0, min(n, width) + 1)
        path[b, :count[b]] = np.sort(rng.choice(n, count[b], replace=False))
    return path, count


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def bits(x):
    return x.view(torch.int16).cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,n,width,bs,layers,Hkv,D", [
    (1, 1, 1, 16, 1, 1, 8), (1, 16, 16, 16, 3, 4, 128), (5, 64, 20, 1, 2, 2, 64), (9, 40, 40, 24, 1, 5, 80),
    (3, 256, 256, 64, 1, 1, 256), (70, 5, 8, 32, 2, 3, 96), (2, 30, 30, 16, 0, 2, 64)])
@pytest.mark.parametrize("order", ["pth", "pht"])
def test_moves(sgmv, dtype, B, n, width, bs, layers, Hkv, D, order):
    """layers = 0: caches without a layer dimension.  NaN patterns are moved like any other bits."""
    rng = np.random.default_rng(B + n)
    prefix = rng.integers(0, 100, B)
    table, blocks = ref.paged(rng, [int(p) + n for p in prefix], bs)
    path, count = paths(rng, B, n, width)
    lead = (layers,) if layers else ()
    shape = (*lead, blocks, bs, Hkv, D) if order == "pth" else (*lead, blocks, Hkv, bs, D)
    k, v = (torch.randint(-2 ** 15, 2 ** 15, shape, dtype=torch.int16, device="cuda").view(dtype) for _ in range(2))
    if order == "pht":
        k, v = k.transpose(-3, -2), v.transpose(-3, -2)
    want = [ref.commit(bits(x) if layers else bits(x)[None], table, prefix, path, count) for x in (k, v)]
    sgmv.sgmv_cache_commit(k, v, i32(table), i32(prefix), i32(path), i32(count))
    check_error_word(0)
    for x, w in zip((k, v), want):
        assert np.array_equal(bits(x) if layers else bits(x)[None], w)


def test_long_cache(sgmv):
    """A page beyond 2^31 elements from the cache's start."""
    blocks = 140_000
    k = torch.empty(blocks, 16, 8, 128, dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    k[-1], v[-1] = torch.randn_like(k[-1]), torch.randn_like(v[-1])
    a, b = k[-1, 9].clone(), v[-1, 9].clone()
    sgmv.sgmv_cache_commit(k, v, i32([[blocks - 1]]), i32([3]), i32([[0, 6]]), i32([2]))
    check_error_word(0)
    assert torch.equal(k[-1, 4], a) and torch.equal(v[-1, 4], b)


def test_bad_metadata_is_reported_and_left_out(sgmv):
    rng = np.random.default_rng(0)
    k, v = (torch.randn(12, 16, 2, 64, device="cuda").half() for _ in range(2))
    table = i32([[0, 1], [2, 3], [4, 5]])
    prefix, path, count = [3, 4, 5], [[0, 4, 6], [1, 3, 9], [0, 2, 5]], [3, 3, 3]
    good = [x.clone() for x in (k, v)]
    sgmv.sgmv_cache_commit(*good, table, i32(prefix), i32(path), i32(count))
    check_error_word(0)
    for change in ("count", "order", "page", "length", "prefix"):
        t, p, a, c = table.clone(), list(prefix), [list(x) for x in path], list(count)
        if change == "count":
            c[1] = 4
        elif change == "order":
            a[1] = [3, 1, 9]
        elif change == "page":
            t[1, 0] = 12
        elif change == "length":
            a[1] = [1, 3, 40]
        else:
            p[1] = -5
        x, y = k.clone(), v.clone()
        sgmv.sgmv_cache_commit(x, y, t, i32(p), i32(a), i32(c))
        check_error_word(4)
        for got, want in ((x, good[0]), (y, good[1])):
            for page in (0, 1, 4, 5, 6, 7, 8, 9, 10, 11):  # the other sequences, and pages of none
                assert torch.equal(got[page], want[page])
