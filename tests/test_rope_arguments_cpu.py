"""Combinations of sgmv_rope's tensors that belong together are refused as a whole, with a
ValueError that says so, before anything is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def test_what_belongs_together(sgmv):
    h = torch.float16
    q, k, c = torch.zeros(2, 4, 64, dtype=h), torch.zeros(2, 2, 64, dtype=h), torch.zeros(3, 16, 2, 64, dtype=h)
    pos, f = torch.zeros(2, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    whole = dict(v=k, k_cache=c, v_cache=c, slots=pos)
    for args, kw in (((None, None), {}), ((q, None), whole), ((q, None), dict(k_out=k)), ((None, k), dict(q_out=q)),
                     *(((q, k), {n: t for n, t in whole.items() if n != gone}) for gone in whole),
                     ((q, k), dict(v_cache=c)), ((q, k), dict(slots=pos)), ((q, k), dict(v_cache=c, v=k))):
        with pytest.raises(ValueError) as e:
            sgmv.sgmv_rope(*args, pos, f, **kw)
        assert "cuda device" not in str(e.value), (kw.keys(), e.value)
