"""NaN and infinities in what a row does see reach its output, in every kernel of the
tree attention: heads narrow and wide, pages copied by boxes and by rows."""
import numpy as np
import pytest
import torch

from tests import spec_reference as ref
from tests.gpu_helpers import check_error_word
from tests.test_tree_attention_gpu import Batch

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]
SHAPES = [(64, 16), (64, 5), (128, 24), (136, 16), (256, 16), (256, 5)]  # head size, page size


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,bs", SHAPES)
@pytest.mark.parametrize("prefix", [0, 2, 300])
def test_a_nan_query(sgmv, dtype, D, bs, prefix):
    b = Batch([prefix, 20], None, 4, 2, D, bs, dtype, seed=D, parents=[[-1, 0, 0, 1], [-1]]).dirty()
    good = b.q.clone()
    b.q[1, 2, D // 2] = float("nan")
    b.run(sgmv)
    check_error_word(0)
    assert np.isnan(ref.f64(b.out)[1, 2]).all() and np.isnan(ref.f64(b.lse)[1, 2])
    b.q, got, lse = good, b.out.clone(), b.lse.clone()
    b.run(sgmv)
    got[1, 2], lse[1, 2] = b.out[1, 2], b.lse[1, 2]
    assert torch.equal(got, b.out) and torch.equal(lse, b.lse)  # nobody else's changed
    b.check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,bs", SHAPES)
@pytest.mark.parametrize("prefix", [1, 2, 3, 5, 140])
@pytest.mark.parametrize("at", [0, -1])
def test_a_nan_key_of_the_context(sgmv, dtype, D, bs, prefix, at):
    """The first or last token of the context: every row of its sequence is lost, and
    only those, however few tokens there are besides."""
    b = Batch([prefix, 20], None, 4, 2, D, bs, dtype, seed=D, parents=[[-1, 0, 0, 1], [-1, 0]]).dirty()
    s = ref.slots_of(b.table, 0, range(prefix), bs)[at]
    b.k[s // bs, s % bs, :, 0] = float("nan")
    b.run(sgmv)
    check_error_word(0)
    assert np.isnan(ref.f64(b.out)[:4]).all() and np.isnan(ref.f64(b.lse)[:4]).all()
    b.k[s // bs, s % bs] = 0
    b.check(slice(4, 6))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,bs", SHAPES)
@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_branch_with_bad_values(sgmv, dtype, D, bs, group, bad):
    """Node 2's k and v are not finite: the rows that see it get what the formula gives,
    the others keep their values."""
    tree = [-1, 0, 0, 1, 2, 3, 4, 1]
    b = Batch([130, 20], None, group * 2, 2, D, bs, dtype, seed=4, parents=[tree, tree])
    s = ref.slots_of(b.table, 0, [130 + 2], bs)[0]
    b.dirty()
    b.v[s // bs, s % bs, :, ::3] = bad
    b.run(sgmv)
    check_error_word(0)
    sees = ref.ancestors(tree)[:, 2]
    hit = ref.f64(b.out)[:8][sees][..., ::3]
    assert (np.isnan(hit) if np.isnan(bad) else hit == bad).all()
    clean = np.flatnonzero(np.concatenate([~sees, np.ones(8, bool)]))
    b.v[s // bs, s % bs] = 0
    b.check(clean)
    b.k[s // bs, s % bs] = float("nan")
    b.run(sgmv)
    assert np.isnan(ref.f64(b.out)[:8][sees]).all()
    b.k[s // bs, s % bs] = 0
    b.check(clean)
