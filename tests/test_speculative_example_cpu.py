"""The example stops with an error before a request outgrows its pages (its block table
would be indexed past the end on the GPU)."""
from types import SimpleNamespace

import pytest
import torch

from examples import speculative_decode as ex


def requests(pages, bs, lens):
    return SimpleNamespace(table=torch.zeros(len(lens), pages, dtype=torch.int32), bs=bs,
                           lens=torch.tensor(lens, dtype=torch.int32))


def fake_step(grown):
    """A step that accepts grown[b] tokens of request b and checks the places it would use."""
    def step(model, req, parents, depth, tokens, greedy):
        place = req.lens[:, None] + torch.arange(len(parents))
        assert int(place.max()) // req.bs < req.table.shape[1]
        count = torch.tensor(grown, dtype=torch.int32)
        req.lens += count
        B, n = len(grown), len(parents)
        return count, torch.zeros(B, n, dtype=torch.int32), torch.zeros(B, dtype=torch.int32), torch.zeros(B, n)

    return step


@pytest.mark.parametrize("lens", [[0, 0, 0], [5, 100, 0]])
@pytest.mark.parametrize("grown", [[1, 1, 1], [3, 1, 2]])
def test_a_request_that_outgrows_its_pages(monkeypatch, lens, grown):
    monkeypatch.setattr(ex, "step", fake_step(grown))
    with pytest.raises(ValueError, match="pages"):
        ex.generate(None, requests(16, 16, lens), 10_000)


def test_what_fits_runs_to_its_end(monkeypatch):
    monkeypatch.setattr(ex, "step", fake_step([1, 2]))
    n = len(ex.PARENTS)
    req = requests(16, 16, [0, 3])
    fits = (256 - 3 - n) // 2 + 1  # the faster request's last tree ends at the last slot
    out, steps = ex.generate(None, req, fits)
    assert steps == fits and [len(o) for o in out] == [fits, 2 * fits]
    with pytest.raises(ValueError, match="pages"):
        ex.generate(None, requests(16, 16, [0, 3]), fits + 1)
