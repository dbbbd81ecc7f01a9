"""A wait of the tree attention that runs out, in each of its roles: the status is
reported, nothing is written, and the next call on the same context is right.

As with the streaming kernel, the timeout is injected: the role gives up as if one of
its waits had run out, and everything after that is what a real one runs.  The other
roles' waits then end, the copies in flight land, tensor memory is returned and the join
leaves the items with lost parts alone."""
import pytest
import torch

from tests.gpu_helpers import check_error_word
from tests.test_tree_attention_gpu import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


# (query heads per KV head, rows per sequence): row tiles of 8, 16, 32, 64 and 128
@pytest.mark.parametrize("group,n", [(4, 1), (2, 6), (4, 7), (8, 8), (16, 9)])
@pytest.mark.parametrize("bs", [16, 24, 5])
@pytest.mark.parametrize("role", [1, 2, 3, 4])
def test_each_role(sgmv, group, n, bs, role):
    """Items that one CTA does whole and items that are cut."""
    b = Batch([9000, 130, 0, 500, 77], [n] * 5, group * 2, 2, 64, bs, torch.float16, seed=n).dirty()
    ws = torch.zeros(sgmv.sgmv_tree_attention_workspace_bytes(b.T, b.B, group * 2, 2, 64), dtype=torch.uint8,
                     device="cuda")
    check_error_word(0)
    b.run(sgmv, workspace=ws)  # leaves good parts behind that must not be taken for this call's
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
    assert sgmv.sgmv_get_device_error() == 7  # SGMV_ERR_TIMEOUT, and the word is cleared
    assert (b.out == 7).all() and (b.lse == 7).all()
    b.run(sgmv, workspace=ws)
    check_error_word(0)
    assert torch.equal(b.out, out) and torch.equal(b.lse, lse)
