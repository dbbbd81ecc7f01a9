"""The stride of a dimension of one entry is never used, so any value of it is taken:
one row, one head, one page, one layer."""
import numpy as np
import pytest
import torch

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


def restride(x, *dims, stride=13):
    """The same elements, with another stride in dimensions of one entry."""
    s = list(x.stride())
    for d in dims:
        assert x.shape[d] == 1
        s[d] = stride
    return x.as_strided(x.shape, s)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq", [1, 4])
@pytest.mark.parametrize("D,bs", [(64, 16), (80, 24), (64, 5), (64, 1), (256, 16)])
def test_attention(sgmv, dtype, Hq, D, bs):
    b = Batch([0 if bs == 1 else 3], [1], Hq, 1, D, bs, dtype, seed=D + bs).dirty()
    if bs > 1:  # one page
        pages = int(b.table[0, 0])
        b.k, b.v, b.table = b.k[pages:pages + 1], b.v[pages:pages + 1], np.zeros((1, 1), np.int32)
        b.k, b.v = restride(b.k, 0, 2), restride(b.v, 0, 2, stride=7)
    else:
        b.k, b.v = restride(b.k, 1, 2), restride(b.v, 2)
    b.q = restride(b.q, *((0, 1) if Hq == 1 else (0,)))
    b.out = restride(b.out, *((0, 1) if Hq == 1 else (0,)), stride=3)
    b.run(sgmv)
    check_error_word(0)
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H", [1, 3])
def test_rope(sgmv, dtype, H):
    g = torch.Generator("cuda").manual_seed(H)
    dims = (0, 1) if H == 1 else (0,)
    plain = [torch.randn(1, H, 64, generator=g, device="cuda").to(dtype) for _ in range(3)]
    q, k, v = (restride(x.clone(), *dims) for x in plain)
    kc, vc = (torch.zeros(1, 1, H, 64, device="cuda", dtype=dtype) for _ in range(2))
    pos, f = torch.tensor([77], dtype=torch.int32, device="cuda"), sgmv.sgmv_rope_frequencies(32)
    want, wk = sgmv.sgmv_rope(plain[0], plain[1], pos, f, q_out=torch.empty_like(plain[0]),
                              k_out=torch.empty_like(plain[1]))
    cdims = (0, 1, 2) if H == 1 else (0, 1)
    out = restride(torch.empty_like(plain[0]), *dims, stride=5)
    sgmv.sgmv_rope(q, k, pos, f, q_out=out, v=v, k_cache=restride(kc, *cdims), v_cache=restride(vc, *cdims, stride=9),
                   slots=torch.zeros(1, dtype=torch.int32, device="cuda"))
    check_error_word(0)
    assert torch.equal(out, want) and torch.equal(kc[0], wk) and torch.equal(vc[0], plain[2])


@pytest.mark.parametrize("layers", [None, 1])
def test_commit(sgmv, layers):
    g = torch.Generator("cuda").manual_seed(1)
    shape = (1, 16, 1, 64) if layers is None else (1, 1, 16, 1, 64)
    k, v = (torch.randn(shape, generator=g, device="cuda").half() for _ in range(2))
    dims = (0, 2) if layers is None else (0, 1, 3)

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    path = np.array([[0, 2, 5]], np.int32)
    want = [ref.commit(x.view(1, 1, 16, 1, 64).cpu().numpy(), np.zeros((1, 1), np.int32), [4], path, [3])
            for x in (k, v)]
    sgmv.sgmv_cache_commit(restride(k, *dims), restride(v, *dims, stride=3), i32(0).view(1, 1), i32(4),
                           torch.tensor(path, device="cuda"), i32(3))
    check_error_word(0)
    for x, w in zip((k, v), want):
        assert np.array_equal(x.view(1, 1, 16, 1, 64).cpu().numpy(), w)
