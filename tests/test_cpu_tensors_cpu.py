"""Tensors that are not on the GPU are refused by the binding of every operator before
anything is launched: a kernel could not use their addresses."""
import pytest
import torch

H, I = torch.float16, torch.int32


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def i32(*x):
    return torch.tensor(x, dtype=I)


def lora():
    """y, x, A, B, seg_ptr, idx of one segment of two rows."""
    return (torch.zeros(2, 64), torch.zeros(2, 64, dtype=H), torch.zeros(1, 64, 8, dtype=H),
            torch.zeros(1, 8, 64, dtype=H), i32(0, 2), i32(0))


def test_lora_operators(sgmv):
    y, x, A, B, seg_ptr, idx = lora()
    v, rows = torch.zeros(2, 8), i32(0, 0)
    for call in (lambda: sgmv.sgmv_apply(y, x, A, B, seg_ptr, idx),
                 lambda: sgmv.sgmv_apply_noalloc(y, x, A, B, seg_ptr, idx),
                 lambda: sgmv.sgmv_apply_multi([y], [x], [A], [B], seg_ptr, idx),
                 lambda: sgmv.sgmv_apply_rows(y, x, A, B, rows),
                 lambda: sgmv.sgmv_shrink(v, x, A, seg_ptr, idx),
                 lambda: sgmv.sgmv_expand(y, v, B, seg_ptr, idx),
                 lambda: sgmv.sgmv_fused_linear_lora(y, x, torch.zeros(64, 64, dtype=H), A, B, seg_ptr, idx),
                 lambda: sgmv.sgmv_build_segments_device(rows, 1)):
        with pytest.raises(ValueError, match="cuda device"):
            call()


def decoding(sgmv):
    """Every operator's call, as (function, its tensors by name, other arguments)."""
    q, k, c = torch.zeros(2, 4, 64, dtype=H), torch.zeros(2, 2, 64, dtype=H), torch.zeros(3, 16, 2, 64, dtype=H)
    rope = dict(q=q, k=k, positions=i32(0, 1), q_out=q.clone(), k_out=k.clone(), v=k.clone(), k_cache=c,
                v_cache=c.clone(), slots=i32(0, 1))
    attention = dict(out=q.clone(), q=q, k_cache=c, v_cache=c.clone(), block_table=i32(0, 1, 2).view(1, 3),
                     prefix_lens=i32(0), tree_ptr=i32(0, 2), parents=i32(-1, 0), lse=torch.zeros(2, 4),
                     workspace=torch.zeros(1 << 25, dtype=torch.uint8))
    p = torch.zeros(2, 9)
    verify = dict(target=p, draft=p.clone(), tokens=i32(0, 1), parents=i32(-1, 0), tree_ptr=i32(0, 2),
                  u_accept=torch.zeros(2), u_sample=torch.zeros(1))
    commit = dict(k_cache=c, v_cache=c.clone(), block_table=i32(0, 1, 2).view(1, 3), prefix_lens=i32(0),
                  path=i32(0, 1).view(1, 2), count=i32(2))
    f = torch.ones(32, dtype=torch.float64)
    return ((sgmv.sgmv_rope, rope, dict(inv_freq=f)), (sgmv.sgmv_tree_attention, attention, {}),
            (sgmv.sgmv_tree_verify, verify, dict(max_path=2)), (sgmv.sgmv_cache_commit, commit, {}))


def test_decoding_operators(sgmv):
    for fn, tensors, rest in decoding(sgmv):
        with pytest.raises(ValueError, match="cuda device"):
            fn(**tensors, **rest)


def test_each_tensor_is_looked_at(sgmv, monkeypatch):
    """One tensor of a call on the CPU, the others elsewhere (here: said to be)."""
    for fn, tensors, rest in decoding(sgmv):
        for name in tensors:
            class Said(torch.Tensor):
                is_cuda = property(lambda self: True)

            args = {n: t if n == name else t.as_subclass(Said) for n, t in tensors.items()}
            with pytest.raises(ValueError, match="cuda device"):
                fn(**args, **rest)
    _, tensors, rest = decoding(sgmv)[2]
    out = [torch.zeros(1, dtype=I), torch.zeros(1, 2, dtype=I), torch.zeros(1, dtype=I)]
    for i in range(3):
        with pytest.raises(ValueError, match="cuda device"):
            sgmv.sgmv_tree_verify(**{n: t.as_subclass(Said) for n, t in tensors.items()}, **rest,
                                  out=[t if j == i else t.as_subclass(Said) for j, t in enumerate(out)])
