"""sgmv_norm_rope_grad refuses an output at the address of any of its inputs, of the other
side too, and of the other output; what a call does not use may be anywhere."""
import pytest
import torch

from tests.test_decode_args_cpu import GRAD
from tests.test_spec_args_cpu import A16, INVALID, caller

FREQ = torch.ones(64, dtype=torch.float64)


@pytest.fixture(scope="module")
def grad():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    tensors = "dq dk dq_out dk_out q k q_weight k_weight dq_weight dk_weight positions workspace".split()
    base = dict({f: 64 for f in GRAD if f.endswith(("_token", "_head"))},
                **{name: A16 + 65536 * i for i, name in enumerate(tensors)}, inv_freq=FREQ.data_ptr(),
                workspace_bytes=sgmv.sgmv_norm_rope_grad_workspace_bytes(64), T=4, Hq=2, Hk=2, D=64, pairs=32,
                scale=1.0, eps=1e-6)
    return base, caller(sgmv, "sgmv_norm_rope_grad", sgmv._NORM_GRAD_ARGS, GRAD, base)


@pytest.mark.parametrize("out", ["dq", "dk"])
@pytest.mark.parametrize("other", ["dq_out", "dk_out", "q", "k"])
def test_outputs_at_an_inputs_address(grad, out, other):
    base, call = grad
    assert call(**{out: base[other]}) == INVALID


def test_outputs_at_each_others_address(grad):
    base, call = grad
    assert call(dq=base["dk"]) == INVALID
    assert call(dq_weight=base["dk_weight"]) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are no memory")
def test_what_is_not_used_may_be_anywhere(grad):
    """(Without a GPU a call that is not refused ends with a CUDA error.)"""
    base, call = grad
    plain = dict(q_weight=0, dq_weight=0)
    assert call(**plain, q=base["dq"]) != INVALID  # not read without its weight
    assert call(**plain, q=base["dk"]) != INVALID
    only_q = dict(Hk=0, k_weight=0, dk_weight=0, dk=0)
    assert call(**only_q, dk_out=base["dq"], k=base["dq"]) != INVALID
