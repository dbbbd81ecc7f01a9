"""Probabilities that are no numbers count as zero in every pass of the verification,
also in the passes after most of the distribution is gone."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import check_error_word
from tests.test_tree_verify_gpu import same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


@pytest.mark.parametrize("V", [7, 64, 3001])
@pytest.mark.parametrize("children", [1, 2, 5])
@pytest.mark.parametrize("bad", [float("nan"), -1.0, float("-inf")])
def test_a_draft_that_is_no_number(sgmv, V, children, bad):
    """One token holds nearly everything in target and draft and is rejected again and
    again; the others' draft probabilities are bad, so their weights stay."""
    n = children + 1
    target, draft = np.full((n, V), 0.004 / (V - 1), np.float32), np.full((n, V), bad, np.float32)
    target[:, 3], draft[:, 3] = 0.99, 0.995
    draft[:, 5] = 0.001 / V
    tokens = np.full(n, 3, np.int32)
    parents = np.array([-1] + [0] * children, np.int32)
    accept = np.full(n, np.float32(1 - 2.0 ** -24))
    for u in (0.0, 0.3, 0.7, float(np.float32(1 - 2.0 ** -24))):
        data = (torch.tensor(target), torch.tensor(draft), tokens, parents, np.array([0, n], np.int32), accept,
                np.array([u], np.float32))
        count, path, token = same(sgmv, data, n)
        check_error_word(0)
        assert count[0] == 1 and token[0] != 3


@pytest.mark.parametrize("draft", [True, False])
def test_scattered_bad_numbers(sgmv, draft):
    rng = np.random.default_rng(5)
    B, n, V = 6, 5, 2051
    T = B * n
    x = rng.standard_normal((T, V)).astype(np.float32) * 3
    target = torch.softmax(torch.tensor(x), -1)
    q = torch.softmax(torch.tensor(x + rng.standard_normal((T, V)).astype(np.float32)), -1)
    for k, p in enumerate((target, q)):
        for e, bad in enumerate((float("nan"), float("inf"), float("-inf"), -0.5, 2.0)):
            at = torch.tensor(rng.random((T, V)) < 2e-3)
            p[at] = bad
    # every node's children all propose the likeliest finite token
    best = torch.where(target < 1, target, torch.zeros(())).argmax(-1).numpy().astype(np.int32)
    parents = np.array([-1, 0, 0, 1, 1] * B, np.int32)
    ptr = np.arange(0, T + 1, n, dtype=np.int32)
    tokens = best[np.repeat(ptr[:-1], n) + np.maximum(parents, 0)]
    for seed in range(4):
        u = np.random.default_rng(seed)
        accept = np.maximum(u.random(T, np.float32), np.float32(0.9) if seed % 2 else np.float32(0))
        same(sgmv, (target, q if draft else None, tokens, parents, ptr, accept, u.random(B, np.float32)), n)
        check_error_word(0)
