"""Where sgmv_sample's top-p cuts, token by token: rows of one large logit over a long tail of
weights of a few units, as a sure model's are, whose cut is deep in the tail.

The weights are the call's own: without filters its probabilities are the whole-number weights
over their sum, and with one weight of 2^38 exactly the others, up to 2^20, come back from the
quotients (three roundings of 2^-24: 0.19 of a unit at most).  The definition in whole numbers on
these is exact."""
import numpy as np
import pytest
import torch

from tests import decode_reference as dref
from tests.gpu_helpers import check_error_word

pytestmark = pytest.mark.gpu
TOP_P = [0.999, 0.9999, 0.99999, 0.999999, 0.9999995, 0.9999998, 1 - 2.0 ** -23, 1 - 2.0 ** -24]


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def whole_weights(sgmv, x, tau):
    """The weights of the rows of x, of which each has one of 2^38."""
    probs = torch.empty(x.shape, device="cuda")
    sgmv.sgmv_sample(x, None, tau, probs=probs)
    probs = probs.double().cpu().numpy()
    raw = probs / probs.max(1, keepdims=True) * dref.ONE
    w = np.round(raw)
    w[probs == probs.max(1, keepdims=True)] = dref.ONE
    tail = np.sort(w, 1)[:, :-1]
    assert tail.max() < 1 << 20 and (w.max(1) == dref.ONE).all()
    assert np.abs(raw - w).max() < 0.25
    # the definition's, to what fp32 exponents cost (the difference, its product and sum, of up to
    # 39 octaves: 98 units of 2^-24, and 2^-22 of the power) and the rounding down
    rows = dref.canonical(x)
    exact = np.exp((rows - rows.max(1, keepdims=True)) / tau) * dref.ONE
    assert (np.abs(w - np.floor(exact)) <= 1 + exact * (98 * 0.7 + 4) * 2.0 ** -24).all()
    return rows, w.astype(np.int64)


def check_cut(sgmv, x, tau, k, top_p, u):
    T, V = x.shape
    rows, w = whole_weights(sgmv, x, tau)
    p = torch.tensor(np.asarray(top_p, np.float32), device="cuda")
    probs = torch.full((T, V), 7.0, device="cuda")
    token = sgmv.sgmv_sample(x, torch.tensor(u, device="cuda"), tau, k, p, probs=probs)
    check_error_word(0)
    got, token = probs.cpu().numpy() > 0, token.cpu().numpy()
    for t in range(T):
        order = np.lexsort((np.arange(V), -rows[t]))
        ranked = w[t][order]
        if 0 < k < V:
            ranked[k:] = 0
        target = dref.part(int(ranked.sum()), top_p[t])
        before = np.concatenate([[0], np.cumsum(ranked)[:-1]])
        ranked[(before >= target) & (np.arange(V) > 0)] = 0
        kept = np.zeros(V, np.int64)
        kept[order] = ranked
        reached = int(w[t][got[t]].sum())
        assert reached >= target, (t, top_p[t], "the kept weights do not reach top_p", target - reached)
        last = order[np.flatnonzero(got[t][order])[-1]]
        assert reached - int(w[t][last]) < target, (t, top_p[t], "one token too many")
        assert (got[t] == (kept > 0)).all(), (t, top_p[t], int(got[t].sum()), int((kept > 0).sum()))
        run = np.cumsum(kept)
        assert token[t] == np.searchsorted(run, dref.part(int(run[-1]), u[t]), side="right"), (t, top_p[t])


def tail_rows(V, at, spread, tau, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x = at + spread * torch.randn(V, generator=g, device="cuda")
    x[V // 3] = 0
    return (tau * x).to(dtype).expand(len(TOP_P), V).contiguous()


@pytest.mark.parametrize("V", [5000, 100277, 262144])
@pytest.mark.parametrize("at,spread", [(-26.0, 0.2), (-25.9, 0.2), (-24.0, 0.5), (-23.0, 0.3), (-20.2, 0.5), (-16.0, 0.1),
                                       (-26.5, 0.3), (-22.0, 1.5)])
def test_a_cut_deep_in_the_tail(sgmv, V, at, spread):
    x = tail_rows(V, at, spread, 1.0, torch.float32, V)
    u = np.linspace(0, 1 - 2.0 ** -24, len(TOP_P), dtype=np.float32)
    check_cut(sgmv, x, 1.0, 0, TOP_P, u)
    check_cut(sgmv, x, 1.0, V // 2, TOP_P, u[::-1].copy())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("at,spread", [(-26.0, 0.2), (-23.0, 0.3), (-22.0, 1.5)])
@pytest.mark.parametrize("tau", [1.0, 0.25, 4.0])
def test_a_cut_among_tails_of_few_values(sgmv, dtype, at, spread, tau):
    x = tail_rows(100277, at, spread, tau, dtype, 7)
    u = np.linspace(1 - 2.0 ** -24, 0, len(TOP_P), dtype=np.float32)
    check_cut(sgmv, x, tau, 0, TOP_P, u)


def test_a_tail_in_a_vocabulary_larger_than_shared_memory(sgmv):
    x = tail_rows(500_003, -25.9, 0.2, 1.0, torch.float32, 9)
    check_cut(sgmv, x, 1.0, 0, TOP_P, np.full(len(TOP_P), 0.999, np.float32))


@pytest.mark.parametrize("V", [300, 5000, 100277])
@pytest.mark.parametrize("kind", ["normal", "flat", "whole", "masked"])
def test_what_is_kept_and_what_is_dropped(sgmv, V, kind):
    """Every token but those whose running weight is within the weights' own error of the
    target (six units for each token ranked before it, and for the total): kept and dropped
    ones, each held to the definition."""
    from tests.test_sample_gpu import rows_of

    x = rows_of(kind, 8, V, torch.Generator("cuda").manual_seed(V))
    probs = torch.empty(8, V, device="cuda")
    p = torch.tensor([0.1, 0.5, 0.8, 0.9, 0.95, 0.99, 0.999, 0.9999], device="cuda")
    sgmv.sgmv_sample(x, None, 1.0, 0, p, probs=probs)
    check_error_word(0)
    got, rows = probs.cpu().numpy() > 0, dref.canonical(x)
    for t in range(8):
        _, w = dref.sample(rows[t], 1.0, 0, 1.0, 0.0, 0.0)
        order = np.lexsort((np.arange(V), -rows[t]))
        before = np.concatenate([[0], np.cumsum(w[order])[:-1]])
        target, off, kept = dref.part(int(w.sum()), float(p[t])), 12 * V, got[t][order]
        assert kept[(before < target - off) & (w[order] > 6)].all() and kept[0]
        assert not kept[(before >= target + off) & (np.arange(V) > 0)].any()
