"""Queries with an infinity over an e4m3 cache: what the affected row gives, by the definition
in 64 bits.  Its scores are infinite, of the sign of the key's column, or no numbers where that
is zero (zero times infinity).  With +inf or NaN among them the softmax is NaN; with -inf alone
the sum of the weights is zero: output 0 and lse -inf, as for a row that sees nothing.  The same
as sgmv_tree_attention over the same values in 16 bits."""
import numpy as np
import pytest
import torch

from tests import spec_reference as ref
from tests.gpu_helpers import check_error_word
from tests.test_quant_attention_gpu import Quant

pytestmark = pytest.mark.gpu
ROW, HEAD, COLUMN = 3, 5, 7


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def signs(b, kind, seen):
    """The keys' column: of one sign for all, of both, or with one zero."""
    x = b.k8.view(torch.uint8)
    column = x[..., COLUMN] & 0x7F
    column = torch.where((column == 0) | (column == 0x7F), 0x30, column)  # a number other than zero
    if kind == "negative":
        column |= 0x80
    at = torch.tensor(seen, device="cuda")
    if kind == "both":
        column[at[::2] // b.bs, at[::2] % b.bs] |= 0x80
    if kind == "zero":
        column |= 0x80
        column[at[-1] // b.bs, at[-1] % b.bs] = 0
    x[..., COLUMN] = column
    b.stand()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("kind", ["positive", "negative", "both", "zero"])
@pytest.mark.parametrize("prefix", [0, 400, 6000])
def test_a_row_with_an_infinity(sgmv, dtype, bad, kind, prefix):
    b = Quant([prefix, 33], [5, 3], 8, 2, 64, 16, dtype, seed=31)
    sees = np.flatnonzero(ref.ancestors(list(b.parents[:5]))[ROW])
    seen = ref.slots_of(b.table, 0, [*range(prefix), *(prefix + sees)], b.bs)
    signs(b, kind, seen)
    b.run(sgmv)
    b.check()
    want, lse = b.out.clone(), b.lse.clone()
    b.q[ROW, HEAD, COLUMN] = bad
    b.run(sgmv)
    check_error_word(0)
    # the definition
    at = torch.tensor(seen, device="cuda")
    with np.errstate(invalid="ignore"):
        s = b.scale * (ref.f64(b.k)[at.cpu() // b.bs, at.cpu() % b.bs, HEAD // 4] * ref.f64(b.q)[ROW, HEAD]).sum(-1)
    assert not np.isfinite(s).any()
    got, got_lse = ref.f64(b.out)[ROW, HEAD], ref.f64(b.lse)[ROW, HEAD]
    if np.isneginf(s).all():
        assert (got == 0).all() and np.isneginf(got_lse)
    else:
        assert np.isnan(got).all() and not np.isfinite(got_lse) and not np.isneginf(got_lse)
    # the others' are untouched
    others = torch.ones(b.T, 8, dtype=torch.bool, device="cuda")
    others[ROW, HEAD] = False
    assert torch.equal(b.out[others], want[others]) and torch.equal(b.lse[others], lse[others])
    # and the 16-bit operator agrees (each head's keys are the stored ones, the scale in the scores)
    out, lse = torch.empty_like(b.out), torch.empty_like(b.lse)
    table, where, ptr, parents = b.meta()
    sgmv.sgmv_tree_attention(out, b.q, b.k8.float().to(dtype), b.v8.float().to(dtype), table, where, ptr, parents,
                             scale=b.scale, lse=lse)
    check_error_word(0)
    same = ref.f64(out)[ROW, HEAD]
    assert np.array_equal(np.isnan(same), np.isnan(got)) and (np.isnan(got) | (same == got)).all()
    assert np.array_equal(np.isneginf(ref.f64(lse)), np.isneginf(ref.f64(b.lse)))
