"""Columns that do not turn are copied bit by bit, whatever stands beside them:
infinities, NaN and negative zeros, in heads whose last pair ends inside a vector."""
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


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,pairs", [(64, 1), (64, 5), (16, 6), (80, 13), (64, 15), (256, 125), (64, 8), (64, 0)])
def test_copied_columns_keep_their_bits(sgmv, dtype, interleaved, D, pairs):
    T, H = 9, 3
    g = torch.Generator("cuda").manual_seed(D + pairs)
    q = torch.randn(T, H, D, generator=g, device="cuda").to(dtype)
    clean = q.clone()
    kept = slice(2 * pairs, D)
    odd = torch.tensor([float("inf"), -0.0, float("nan"), float("-inf"), 0.0], device="cuda", dtype=dtype)
    n = D - 2 * pairs
    for t in range(T):  # every value beside every other
        q[t, :, kept] = odd[(torch.arange(n, device="cuda") * (1 + t % 3) + t) % 5]
    positions = torch.arange(T, dtype=torch.int32, device="cuda") * 31 + 1
    f = sgmv.sgmv_rope_frequencies(pairs) if pairs else torch.empty(0, dtype=torch.float64)
    kc, vc = (torch.zeros(T, 1, H, D, device="cuda", dtype=dtype) for _ in range(2))
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    out, _ = sgmv.sgmv_rope(q, q, positions, f, interleaved, scale=1.5, q_out=torch.empty_like(q), v=q, k_cache=kc,
                            v_cache=vc, slots=slots)
    check_error_word(0)
    for x in (out, kc[:, 0], vc[:, 0]):
        assert torch.equal(x[..., kept].view(torch.int16), q[..., kept].view(torch.int16))
    # and the columns that turn do not see them
    y, m = ref.rope(clean, positions.cpu().numpy(), f.numpy(), interleaved, 1.5, False)
    turn = slice(0, 2 * pairs)
    assert (np.abs(ref.f64(out) - y)[..., turn] <= ref.rope_bound(y, m, dtype)[..., turn]).all()
