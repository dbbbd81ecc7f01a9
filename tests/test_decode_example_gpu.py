"""examples/speculative_decode.py with head norms and an 8-bit cache: drafts do not change
greedy tokens, and sampled runs draw from the filtered distribution."""
import pytest
import torch

from tests.test_speculative_example_gpu import ex  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norms", [False, True])
def test_drafts_do_not_change_greedy_tokens(ex, norms):  # noqa: F811
    from rank_gemv_gb300 import sgmv

    model, length = ex.Model(head_norms=norms, e4m3=True), 24
    plain, steps = ex.generate(model, ex.Requests(model, 8, 256), length, parents=[-1], depth=[0], greedy=True)
    assert steps == length
    tree, _ = ex.generate(model, ex.Requests(model, 8, 256), length, greedy=True)
    # (rounding to 8 bits can part a request from its twin where a logit or a key is on an edge)
    assert sum(a[:length] == b[:length] for a, b in zip(plain, tree)) >= 6
    assert sgmv.sgmv_get_device_error() == 0


def test_sampled_run_keeps_to_the_filters(ex, monkeypatch):  # noqa: F811
    from rank_gemv_gb300 import sgmv

    model = ex.Model(seed=3, head_norms=True, e4m3=True, temperature=0.8, top_k=20, top_p=0.9)
    seen, real = [], sgmv.sgmv_tree_verify

    def verify(target, *args):
        got = real(target, *args)
        seen.append(((target > 0).sum(1).max().item(), (target.sum(1) - 1).abs().max().item()))
        return got

    monkeypatch.setattr(sgmv, "sgmv_tree_verify", verify)
    req = ex.Requests(model, 5, 256)
    out, _ = ex.generate(model, req, 20)
    assert all(0 <= t < model.vocab for o in out for t in o)
    assert req.lens.tolist() == [len(o) for o in out]
    assert all(n <= 20 and off <= 1e-5 for n, off in seen)
    assert req.k.dtype == torch.float8_e4m3fn
    assert sgmv.sgmv_get_device_error() == 0
