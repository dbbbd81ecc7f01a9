"""sgmv_tree_verify against the walk in whole numbers, number for number, and
the distribution of what it returns against the target's."""
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


def batch(counts, V, draft, seed, sharp=3.0, chains=False):
    rng = np.random.default_rng(seed)
    T = sum(counts)
    x = rng.standard_normal((T, V)) * sharp
    target = torch.softmax(torch.tensor(x), -1).float()
    q = torch.softmax(torch.tensor(x + rng.standard_normal((T, V)) * sharp * 0.4), -1).float()
    parents = [p for n in counts for p in ref.random_tree(rng, n, reach=3)]
    if chains:
        parents = [p for n in counts for p in ref.chain(n)]
    ptr = ref.ptr_of(counts)
    tokens = np.zeros(T, np.int32)
    for b, n in enumerate(counts):
        for i in range(1, n):
            t = int(ptr[b]) + i
            p = q[ptr[b] + parents[t]].double().numpy()
            tokens[t] = rng.choice(V, p=p / p.sum())
    return (target, q if draft else None, tokens, np.asarray(parents, np.int32), ptr,
            rng.random(T, np.float32), rng.random(len(counts), np.float32))


def run(sgmv, target, draft, tokens, parents, ptr, accept, sample, width, **kw):
    def dev(x):
        return None if x is None else torch.as_tensor(x).cuda()

    got = sgmv.sgmv_tree_verify(dev(target), dev(draft), dev(tokens), dev(parents), dev(ptr), dev(accept),
                                dev(sample), width, **kw)
    return [x.cpu().numpy() for x in got]


def same(sgmv, data, width):
    got = run(sgmv, *data, width)
    target, draft, *rest = data
    want = ref.verify(target.numpy(), None if draft is None else draft.numpy(), *rest, width)
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    return got


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 32000, 100277])
def test_vocabularies(sgmv, draft, V):
    same(sgmv, batch([9, 1, 0, 16, 5], V, draft, V), 16)
    check_error_word(0)


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("counts", [[1], [64] * 7, [256], list(range(0, 40)), [3] * 200])
@pytest.mark.parametrize("sharp", [0.3, 6.0])
def test_trees(sgmv, draft, counts, sharp):
    data = batch(counts, 517, draft, sum(counts), sharp)
    same(sgmv, data, max(counts))
    same(sgmv, data, 2)  # the walk stops when the path is full
    check_error_word(0)


@pytest.mark.parametrize("draft", [True, False])
def test_long_accepted_paths(sgmv, draft):
    """Drafts as good as the target: paths go deep."""
    data = list(batch([64] * 5 + [200], 517, draft, 8, sharp=6.0))
    data[0][:] = torch.softmax(data[0].log() * 40, -1)
    if draft:
        data[1][:] = data[0]
    for b in range(6):
        t0, n = data[4][b], data[4][b + 1] - data[4][b]
        for i in range(1, n):
            data[2][t0 + i] = int(data[0][t0 + data[3][t0 + i]].argmax())
    count, _, _ = same(sgmv, data, 200)
    assert count.max() > 8
    check_error_word(0)



@pytest.mark.parametrize("draft", [True, False])
def test_chains_without_parents(sgmv, draft):
    data = list(batch([6, 3, 1, 8], 700, draft, 5, chains=True))
    want = same(sgmv, data, 8)
    data[3] = None
    for g, w in zip(same(sgmv, data, 8), want):
        assert np.array_equal(g, w)


def test_extremes(sgmv):
    """Uniform numbers at their ends, point masses, all-zero, NaN, negative and
    too large probabilities, equal and repeated tokens."""
    for seed in range(6):
        for draft in (True, False):
            data = list(batch([5, 5, 5, 5, 5, 5], 97, draft, seed))
            target, q, tokens, parents, ptr, accept, sample = data
            accept[:10] = 0.0
            accept[10:20] = np.float32(1 - 2.0 ** -24)
            sample[:2], sample[2:4] = 0.0, np.float32(1 - 2.0 ** -24)
            target[5:10] = 0
            target[5:10, 3] = 1           # a point mass
            target[10:15] = 0             # nothing at all
            target[15, 7:20] = float("nan")
            target[16, 7:20] = -1.0
            target[17, 7:20] = 4.0
            if draft:
                q[20:25] = target[20:25]  # the draft is the target: everything is accepted
                q[0, :] = float("nan")
            tokens[ptr[5] + 1:ptr[5] + 5] = tokens[ptr[5] + 1]
            parents[ptr[5] + 1:ptr[5] + 5] = 0
            same(sgmv, data, 5)
            check_error_word(0)


def test_rows_with_strides_and_given_outputs(sgmv):
    target, q, *rest = batch([7, 4], 130, True, 3)
    wide = torch.rand(11, 2, 133).cuda()
    wide[:, 0, 1:131], wide[:, 1, 2:132] = target.cuda(), q.cuda()
    out = tuple(torch.full(s, 9, dtype=torch.int32, device="cuda") for s in ((2,), (2, 7), (2,)))
    got = run(sgmv, wide[:, 0, 1:131], wide[:, 1, 2:132], *rest, 7, out=out)
    for g, w in zip(got, ref.verify(target.numpy(), q.numpy(), *rest, 7)):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("draft", [True, False])
def test_the_target_distribution_is_kept(sgmv, draft):
    """First token after the root (accepted child or drawn): over many
    sequences with the same distributions its frequencies follow the
    target's.  Chi-squared with 11 degrees of freedom: below 45 but for 5e-6."""
    V, n, B = 12, 4, 20000
    rng = np.random.default_rng(17)
    p = rng.dirichlet(np.ones(V)).astype(np.float32)
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    T = B * n
    tokens = rng.choice(V, size=T, p=q.astype(np.float64) / q.astype(np.float64).sum()).astype(np.int32)
    if not draft:  # proposals that do not depend on the numbers drawn later
        tokens = np.tile(np.array([0, 3, 5, 3], np.int32), B)
    parents = np.tile(np.array([-1, 0, 0, 0], np.int32), B)
    target = torch.tensor(p).expand(T, V).contiguous()
    count, path, token = run(sgmv, target, torch.tensor(q).expand(T, V).contiguous() if draft else None, tokens,
                             parents, ref.ptr_of([n] * B), rng.random(T, np.float32), rng.random(B, np.float32), n)
    first = np.where(count > 1, tokens[np.arange(B) * n + np.maximum(path[:, 1], 0)], token)
    seen = np.bincount(first, minlength=V)
    expect = B * p.astype(np.float64) / p.astype(np.float64).sum()
    assert ((seen - expect) ** 2 / expect).sum() < 45
    assert 0 < (count > 1).mean() < 1


def test_bad_metadata_is_reported_and_left_out(sgmv):
    data = batch([4, 4, 4], 50, True, 1)
    good = run(sgmv, *data, 4)
    check_error_word(0)
    for what, status in (("token", 4), ("parent", 4), ("ptr", 8)):
        target, q, tokens, parents, ptr, accept, sample = [None if x is None else x.copy() if isinstance(x, np.ndarray)
                                                           else x for x in data]
        if what == "token":
            tokens[5] = 50
            parents[5] = 0
        elif what == "parent":
            parents[5] = 1
        else:
            ptr[2:] = [3, 12]
        got = run(sgmv, target, q, tokens, parents, ptr, accept, sample, 4)
        check_error_word(status)
        for g, w in zip(got, good):
            assert np.array_equal(g[0], w[0])
            if what != "ptr":
                assert np.array_equal(g[2], w[2])
        if what == "ptr":
            assert got[0][1] == 0 and got[2][1] == -1 and (got[1][1] == -1).all()
