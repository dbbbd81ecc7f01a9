"""The tree attention's workspace, sized once for the largest batch, serves every smaller one."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import check_error_word


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


@pytest.mark.parametrize("Hkv,group", [(8, 1), (8, 2), (4, 4), (2, 7), (8, 8), (1, 9), (1, 16), (1, 200)])
@pytest.mark.parametrize("D", [64, 256])
def test_no_smaller_batch_needs_more(sgmv, Hkv, group, D):
    sizes = [1, 2, 3, 4, 8, 15, 16, 17, 31, 33, 64, 65, 128, 129, 400, 2048]
    need = np.array([[sgmv.sgmv_tree_attention_workspace_bytes(T, B, Hkv * group, Hkv, D) for B in sizes]
                     for T in sizes], np.int64)
    assert (need > 0).all()
    most = np.maximum.accumulate(np.maximum.accumulate(need, 0), 1)
    assert (need == most).all()


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,group", [(4, 1), (2, 4), (1, 16)])
def test_one_workspace_for_a_loop(sgmv, Hkv, group):
    """Requests finish and trees grow: each batch is no larger than the workspace's, and the row
    tile goes through all that there are."""
    from tests.test_tree_attention_gpu import Batch

    Hq, D, T = Hkv * group, 64, 200
    ws = torch.empty(sgmv.sgmv_tree_attention_workspace_bytes(T, 50, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    for B, n in ((50, 1), (50, 4), (20, 10), (9, 20), (5, 40), (2, 100), (1, 200), (1, 1), (50, 1)):
        b = Batch([300 + 7 * i for i in range(B)], [n] * B, Hq, Hkv, D, 16, torch.float16, seed=n).dirty()
        b.run(sgmv, workspace=ws)
        check_error_word(0)
        b.check()
