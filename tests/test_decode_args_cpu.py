"""The calls of head norms, e4m3 caches and sampling refuse bad arguments on the host,
before anything is launched: the C ABI by status, the binding by exception."""
import subprocess
from pathlib import Path

import pytest
import torch

from tests.test_spec_args_cpu import (A16, ALIGNMENT, ATTENTION, COMMIT, INVALID, MIS, OK, ROPE, UNSUPPORTED, WORKSPACE,
                                      caller)

H, I, E4M3 = torch.float16, torch.int32, torch.float8_e4m3fn
GRAD = ("dq dk dq_out dk_out q k q_weight k_weight dq_weight dk_weight positions inv_freq workspace workspace_bytes "
        "dq_token dq_head dk_token dk_head dq_out_token dq_out_head dk_out_token dk_out_head q_token q_head k_token "
        "k_head T Hq Hk D pairs dtype interleaved scale eps").split()
SAMPLE = ("logits u temperature top_k top_p min_p token probs logits_row probs_row T V dtype top_k_all "
          "temperature_all top_p_all min_p_all").split()


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


@pytest.fixture(scope="module")
def freq():
    return torch.ones(64, dtype=torch.float64)


class Two:
    """A struct that begins with another."""

    def __init__(self, first, rest, n):
        self.first, self.rest, self.n = first, rest, n

    def pack(self, *values):
        return self.first.pack(*values[:self.n]) + self.rest.pack(*values[self.n:])


def test_norm_rope_refusals(sgmv, freq):
    fields = ROPE + "q_weight k_weight k_scale v_scale eps".split()
    base = dict({f: 64 for f in ROPE if f.endswith(("_token", "_head", "_block"))}, q_out=A16, q=A16, k_out=A16, k=A16,
                v=A16, k_cache=A16, v_cache=A16, positions=A16, slots=A16, inv_freq=freq.data_ptr(), T=4, Hq=2, Hk=2,
                D=64, pairs=32, num_blocks=3, block_size=16, scale=1.0, q_weight=A16, k_weight=A16, k_scale=A16,
                v_scale=A16, eps=1e-6)
    call = caller(sgmv, "sgmv_norm_rope", Two(sgmv._ROPE_ARGS, sgmv._NORM_ARGS, len(ROPE)), fields, base)
    for bad in (dict(T=-1), dict(Hq=-1), dict(dtype=2), dict(dtype=3), dict(D=0), dict(pairs=33), dict(inv_freq=0),
                dict(q=0), dict(q_out=0), dict(k=0), dict(v=0), dict(slots=0), dict(positions=0), dict(eps=0.0),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(inverse=1), dict(k_scale=0),
                dict(v_scale=0), dict(k_cache=0, v_cache=0, slots=0), dict(block_size=0), dict(num_blocks=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=60), dict(D=56, pairs=28), dict(q=MIS), dict(k_cache=MIS), dict(cache_token=72),
                dict(cache_head=8), dict(cache_block=24), dict(q_weight=MIS), dict(k_weight=MIS), dict(v_token=4)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(D=272, pairs=4) == UNSUPPORTED
    assert call(T=1 << 29) == UNSUPPORTED
    assert call(T=0) == OK
    assert sgmv.load_library().sgmv_norm_rope(None, None) == INVALID
    bad = torch.full((64,), float("nan"), dtype=torch.float64)
    assert call(inv_freq=bad.data_ptr()) == INVALID


def test_norm_rope_grad_refusals(sgmv, freq):
    size = sgmv.sgmv_norm_rope_grad_workspace_bytes(64)
    base = dict({f: 64 for f in GRAD if f.endswith(("_token", "_head"))}, dq=A16, dk=A16, dq_out=A16, dk_out=A16, q=A16,
                k=A16, q_weight=A16, k_weight=A16, dq_weight=A16, dk_weight=A16, positions=A16,
                inv_freq=freq.data_ptr(), workspace=A16, workspace_bytes=size, T=4, Hq=2, Hk=2, D=64, pairs=32,
                scale=1.0, eps=1e-6)
    call = caller(sgmv, "sgmv_norm_rope_grad", sgmv._NORM_GRAD_ARGS, GRAD, base)
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hk=-1), dict(dtype=2), dict(D=0), dict(pairs=-1), dict(pairs=33),
                dict(inv_freq=0), dict(dq=0), dict(dk=0), dict(dq_out=0), dict(dk_out=0), dict(q=0), dict(k=0),
                dict(q_weight=0), dict(dk_weight=0), dict(positions=0), dict(eps=0.0), dict(eps=float("nan")),
                dict(Hq=0), dict(Hk=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=60), dict(q=MIS), dict(dq=MIS), dict(dk_out=MIS), dict(k_head=4), dict(dq_out_token=9),
                dict(q_weight=MIS), dict(dk_weight=A16 + 2), dict(workspace=MIS)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(D=264) == UNSUPPORTED and call(T=1 << 30) == UNSUPPORTED
    assert call(workspace_bytes=size - 1) == WORKSPACE and call(workspace=0) == WORKSPACE
    assert call(T=0, q_weight=0, dq_weight=0, k_weight=0, dk_weight=0) == OK
    assert sgmv.load_library().sgmv_norm_rope_grad(None, None) == INVALID
    assert sgmv.sgmv_norm_rope_grad_workspace_bytes(0) == 0 == sgmv.sgmv_norm_rope_grad_workspace_bytes(264)


def test_quant_attention_refusals(sgmv):
    size = sgmv.sgmv_quant_attention_workspace_bytes(4, 2, 4, 2, 64)
    base = dict({f: 64 for f in ATTENTION if f.endswith(("_token", "_head", "_block"))}, out=A16, q=A16, k_cache=A16,
                v_cache=A16, block_table=A16, prefix_lens=A16, tree_ptr=A16, workspace=A16, workspace_bytes=size,
                table_row=8, T=4, B=2, Hq=4, Hkv=2, D=64, num_blocks=3, block_size=16, max_blocks=8, scale=0.125,
                k_scale=A16, v_scale=A16)
    call = caller(sgmv, "sgmv_quant_attention", Two(sgmv._ATTENTION_ARGS, sgmv._SCALE_ARGS, len(ATTENTION)),
                  ATTENTION + ["k_scale", "v_scale"], base)
    for bad in (dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(dtype=2), dict(dtype=3), dict(D=0),
                dict(out=0), dict(q=0), dict(k_cache=0), dict(v_cache=0), dict(block_table=0), dict(prefix_lens=0),
                dict(tree_ptr=0), dict(num_blocks=0), dict(block_size=0), dict(max_blocks=0), dict(table_row=-1),
                dict(scale=float("nan")), dict(k_scale=0), dict(v_scale=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=60), dict(D=72), dict(q=MIS), dict(out=MIS), dict(k_cache=MIS), dict(v_cache=MIS),
                dict(q_token=7), dict(cache_block=8), dict(cache_token=24), dict(cache_head=4),
                dict(workspace=A16 + 16)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(D=144) == UNSUPPORTED and call(D=264) == UNSUPPORTED
    assert call(max_blocks=1 << 30) == UNSUPPORTED
    assert call(workspace_bytes=size - 1) == WORKSPACE and call(workspace=0) == WORKSPACE
    assert call(T=0) == OK and call(B=0) == OK
    assert sgmv.load_library().sgmv_quant_attention(None, None) == INVALID
    assert sgmv.sgmv_quant_attention_workspace_bytes(0, 1, 1, 1, 64) == 0
    assert sgmv.sgmv_quant_attention_workspace_bytes(1, 1, 1, 1, 144) == 0


def test_commit_refusals_of_e4m3(sgmv):
    base = dict(k_cache=A16, v_cache=A16, block_table=A16, prefix_lens=A16, path=A16, count=A16, cache_layer=640,
                cache_block=64, cache_token=64, cache_head=64, table_row=4, layers=2, B=2, Hkv=2, D=64, num_blocks=3,
                block_size=16, max_blocks=4, max_path=4, dtype=3)
    call = caller(sgmv, "sgmv_cache_commit", sgmv._COMMIT_ARGS, COMMIT, base)
    for bad in (dict(D=72), dict(k_cache=MIS), dict(cache_layer=8), dict(cache_block=24), dict(cache_token=8),
                dict(cache_head=40)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(dtype=4) == INVALID and call(D=272) == UNSUPPORTED and call(B=0) == OK


def test_sample_refusals(sgmv):
    base = dict(logits=A16, u=A16, token=A16, probs=A16, logits_row=50, probs_row=50, T=4, V=50, dtype=2,
                temperature_all=1.0, top_p_all=1.0)
    call = caller(sgmv, "sgmv_sample", sgmv._SAMPLE_ARGS, SAMPLE, base)
    for bad in (dict(T=-1), dict(V=0), dict(dtype=3), dict(dtype=9), dict(logits=0), dict(u=0), dict(token=0)):
        assert call(**bad) == INVALID, bad
    assert call(logits=A16 + 2) == ALIGNMENT and call(logits=A16 + 1, dtype=0) == ALIGNMENT
    assert call(probs=A16 + 2) == ALIGNMENT
    assert call(V=(1 << 24) + 1) == UNSUPPORTED and call(T=(1 << 27) + 1) == UNSUPPORTED
    assert call(T=0) == OK and call(u=0, token=0, probs=0) == OK
    assert sgmv.load_library().sgmv_sample(None, None) == INVALID


def test_gradient_and_sampling_are_not_in_place(sgmv, freq):
    size = sgmv.sgmv_norm_rope_grad_workspace_bytes(64)
    apart = dict(zip(("dq", "dk", "dq_out", "dk_out", "q", "k"), range(A16, A16 + 6 * 4096, 4096)))
    base = dict({f: 64 for f in GRAD if f.endswith(("_token", "_head"))}, **apart, q_weight=A16, k_weight=A16,
                dq_weight=A16, dk_weight=A16, positions=A16, inv_freq=freq.data_ptr(), workspace=A16,
                workspace_bytes=size, T=4, Hq=2, Hk=2, D=64, pairs=32, scale=1.0, eps=1e-6)
    call = caller(sgmv, "sgmv_norm_rope_grad", sgmv._NORM_GRAD_ARGS, GRAD, base)
    for side in "qk":
        for other in (f"d{side}_out", side):
            assert call(**{f"d{side}": base[other]}) == INVALID, other
    base = dict(logits=A16, u=A16, token=A16, probs=A16, logits_row=50, probs_row=50, T=4, V=50, dtype=2,
                temperature_all=1.0, top_p_all=1.0)
    assert caller(sgmv, "sgmv_sample", sgmv._SAMPLE_ARGS, SAMPLE, base)() == INVALID


def i32(*x):
    return torch.tensor(x, dtype=I)


def calls(sgmv):
    """(function, its tensors by name, other arguments) of every call."""
    q, k = torch.zeros(2, 4, 64, dtype=H), torch.zeros(2, 2, 64, dtype=H)
    c, w, s = torch.zeros(3, 16, 2, 64).to(E4M3), torch.ones(64, dtype=H), torch.ones(2)
    f = dict(inv_freq=torch.ones(32, dtype=torch.float64))
    norm = dict(q=q, k=k, positions=i32(0, 1), q_weight=w, k_weight=w.clone(), q_out=q.clone(), k_out=k.clone(),
                v=k.clone(), k_cache=c, v_cache=c.clone(), slots=i32(0, 1), k_scale=s, v_scale=s.clone())
    grad = dict(dq_out=q, dk_out=k, q=q.clone(), k=k.clone(), positions=i32(0, 1), q_weight=w, k_weight=w.clone(),
                dq=q.clone(), dk=k.clone(), dq_weight=torch.zeros(64), dk_weight=torch.zeros(64),
                workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    attention = dict(out=q.clone(), q=q, k_cache=c, v_cache=c.clone(), k_scale=s, v_scale=s.clone(),
                     block_table=i32(0, 1, 2).view(1, 3), prefix_lens=i32(0), tree_ptr=i32(0, 2), parents=i32(-1, 0),
                     lse=torch.zeros(2, 4), workspace=torch.zeros(1 << 25, dtype=torch.uint8))
    sample = dict(logits=torch.zeros(2, 9), u=torch.zeros(2), temperature=torch.ones(2), top_k=i32(1, 2),
                  top_p=torch.ones(2), min_p=torch.zeros(2), token=i32(0, 0), probs=torch.zeros(2, 9))
    return ((sgmv.sgmv_norm_rope, norm, f), (sgmv.sgmv_norm_rope_grad, grad, f),
            (sgmv.sgmv_quant_attention, attention, {}), (sgmv.sgmv_sample, sample, {}))


def test_each_tensor_must_be_on_the_gpu(sgmv):
    class Said(torch.Tensor):
        is_cuda = property(lambda self: True)

    for fn, tensors, rest in calls(sgmv):
        with pytest.raises(ValueError, match="cuda device"):
            fn(**tensors, **rest)
        for name in tensors:
            args = {n: t if n == name else t.as_subclass(Said) for n, t in tensors.items()}
            with pytest.raises(ValueError, match="cuda device"):
                fn(**args, **rest)


def test_binding_refusals(sgmv):
    """Shapes, types and layouts that the C ABI cannot see."""
    (norm, nt, f), (grad, gt, _), (attention, at, _), (sample, st, _) = calls(sgmv)
    q, c, w, s = nt["q"], nt["k_cache"], nt["q_weight"], nt["k_scale"]
    for change, error in ((dict(q_weight=w.float()), TypeError), (dict(k_weight=w[:32]), ValueError),
                          (dict(k_cache=c.half(), v_cache=c.half()), TypeError), (dict(k_scale=None), ValueError),
                          (dict(k_scale=None, v_scale=None), TypeError), (dict(k_scale=s.double()), TypeError),
                          (dict(v_scale=torch.ones(3)), ValueError), (dict(v=None), ValueError),
                          (dict(q=None, q_out=None), ValueError), (dict(q=q.float()), TypeError),
                          (dict(k_cache=None, v_cache=None, slots=None), ValueError),
                          (dict(k=None, k_out=None, k_cache=None, v_cache=None, slots=None, k_scale=None, v_scale=None),
                           ValueError), (dict(positions=i32(0)), ValueError)):
        with pytest.raises(error):
            norm(**{**nt, **change}, **f)
    for change, error in ((dict(dq_out=None), ValueError), (dict(dq_out=None, dk_out=None), ValueError),
                          (dict(q=None), ValueError), (dict(q_weight=None), ValueError),
                          (dict(q_weight=w.float()), TypeError), (dict(dq_weight=torch.zeros(32)), ValueError),
                          (dict(dk_weight=torch.zeros(64).half()), TypeError), (dict(k=q), ValueError),
                          (dict(dq=q.float()), TypeError), (dict(dk_out=nt["k"].bfloat16()), TypeError),
                          (dict(dq_out=q[0]), TypeError), (dict(positions=torch.zeros(2)), TypeError)):
        with pytest.raises(error):
            grad(**{**gt, **change}, **f)
    with pytest.raises(TypeError):
        grad(**gt, inv_freq=f["inv_freq"].float())
    for change, error in ((dict(k_cache=c.half(), v_cache=c.half()), TypeError), (dict(k_scale=s.half()), TypeError),
                          (dict(v_scale=torch.ones(1)), ValueError), (dict(out=q[:, :2]), ValueError),
                          (dict(q=q.double(), out=q.double()), TypeError), (dict(lse=torch.zeros(2, 3)), TypeError)):
        with pytest.raises(error):
            attention(**{**at, **change})
    x = st["logits"]
    for change, error in ((dict(logits=x.double()), TypeError), (dict(logits=x[0]), TypeError),
                          (dict(logits=torch.zeros(9, 2).T), TypeError), (dict(u=torch.zeros(3)), ValueError),
                          (dict(u=None), ValueError), (dict(u=None, token=None, probs=None), ValueError),
                          (dict(temperature=torch.ones(2).half()), TypeError), (dict(top_k=torch.ones(2)), TypeError),
                          (dict(top_p=torch.ones(1)), ValueError), (dict(token=torch.zeros(2)), TypeError),
                          (dict(probs=torch.zeros(2, 8)), TypeError), (dict(probs=x.half()), TypeError)):
        with pytest.raises(error):
            sample(**{**st, **change})


def test_argument_structs_match_the_header(sgmv, tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "sgmv.h"\nint main(void) { printf("%zu %zu %zu %zu", '
                   "sizeof(sgmv_norm_rope_args), sizeof(sgmv_norm_rope_grad_args), sizeof(sgmv_quant_attention_args), "
                   "sizeof(sgmv_sample_args)); return 0; }\n")
    inc = Path(__file__).resolve().parents[1] / "include"
    subprocess.run(["gcc", f"-I{inc}", str(src), "-o", str(tmp_path / "s")], check=True)
    sizes = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in sizes] == [sgmv._ROPE_ARGS.size + sgmv._NORM_ARGS.size, sgmv._NORM_GRAD_ARGS.size,
                                       sgmv._ATTENTION_ARGS.size + sgmv._SCALE_ARGS.size, sgmv._SAMPLE_ARGS.size]


@pytest.mark.parametrize("Hkv,group", [(8, 1), (4, 4), (8, 8), (1, 16), (1, 200)])
def test_no_smaller_batch_needs_a_larger_workspace(sgmv, Hkv, group):
    sizes = [1, 2, 4, 8, 15, 16, 17, 33, 64, 65, 129, 400, 2048]
    need = [[sgmv.sgmv_quant_attention_workspace_bytes(T, B, Hkv * group, Hkv, 64) for B in sizes] for T in sizes]
    for i in range(len(sizes)):
        for j in range(len(sizes)):
            assert need[i][j] == max(need[a][b] for a in range(i + 1) for b in range(j + 1)) > 0
