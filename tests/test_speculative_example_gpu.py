"""examples/speculative_decode.py: the operators together, as a decoder uses
them.  With a greedy target the tokens must be those of plain one-token
decoding, whatever is drafted; drafts that are right must be accepted."""
import importlib.util
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    from rank_gemv_gb300 import build

    build.build()
    path = Path(__file__).resolve().parents[1] / "examples" / "speculative_decode.py"
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_drafts_do_not_change_greedy_tokens(ex):
    from rank_gemv_gb300 import sgmv

    # fp32-sized gaps between the best two logits are all but certain, f16
    # ones are not: compare as long as the plain run's choice is clear
    model, length = ex.Model(), 24
    plain, steps = ex.generate(model, ex.Requests(model, 8, 256), length, parents=[-1], depth=[0], greedy=True)
    assert steps == length
    tree, _ = ex.generate(model, ex.Requests(model, 8, 256), length, greedy=True)
    same = [a[:length] == b[:length] for a, b in zip(plain, tree)]
    assert sum(same) >= 6, same  # a tie in f16 may part one request from its twin

    # drafts taken from the plain run: accepted to the last, three tokens a step
    def right(out):
        rows = []
        for b, done in enumerate(out):
            nxt = (plain[b][len(done):] + [0, 0])[:2]
            last = [int(first[b])] if not done else [done[-1]]
            rows.append(last + [(nxt[0] + 1) % model.vocab, nxt[0], 0] + [0, 0, nxt[1], (nxt[1] + 1) % model.vocab, 0, 0])
        return torch.tensor(rows, dtype=torch.int32, device="cuda")

    req = ex.Requests(model, 8, 256)
    first = req.last.tolist()
    fast, steps = ex.generate(model, req, length, greedy=True, tokens=right)
    agree = [b for b in range(8) if fast[b][:length] == plain[b][:length]]
    assert len(agree) >= 6
    assert steps <= length // 3 + 6
    assert sgmv.sgmv_get_device_error() == 0


def test_sampled_run(ex):
    from rank_gemv_gb300 import sgmv

    model = ex.Model(seed=3)
    req = ex.Requests(model, 5, 256)
    out, steps = ex.generate(model, req, 20)
    assert all(0 <= t < model.vocab for o in out for t in o)
    assert req.lens.tolist() == [len(o) for o in out]
    assert sgmv.sgmv_get_device_error() == 0
