"""The speculative decoding calls refuse bad arguments on the host, before
anything is launched: the C ABI by status, the binding by exception."""
import struct

import pytest
import torch

A16, MIS = 0x10000, 0x10008  # aligned and misaligned addresses that nothing reads
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 6


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


ROPE = ("q_out q k_out k v k_cache v_cache positions slots inv_freq q_out_token q_out_head q_token q_head k_out_token "
        "k_out_head k_token k_head v_token v_head cache_block cache_token cache_head T Hq Hk D pairs num_blocks "
        "block_size dtype interleaved inverse scale").split()
ATTENTION = ("out q k_cache v_cache lse block_table prefix_lens tree_ptr parents workspace workspace_bytes out_token "
             "out_head q_token q_head cache_block cache_token cache_head table_row T B Hq Hkv D num_blocks block_size "
             "max_blocks dtype scale").split()
VERIFY = ("target draft tokens parents tree_ptr u_accept u_sample count path token target_row draft_row T B V "
          "max_path").split()
COMMIT = ("k_cache v_cache block_table prefix_lens path count cache_layer cache_block cache_token cache_head "
          "table_row layers B Hkv D num_blocks block_size max_blocks max_path dtype").split()


def caller(sgmv, name, layout, fields, base):
    fn = getattr(sgmv.load_library(), name)

    def call(**change):
        values = {f: base.get(f, 0) for f in fields}
        assert set(change) <= set(values)
        values.update(change)
        return fn(layout.pack(*(values[f] for f in fields)), None)

    return call


@pytest.fixture(scope="module")
def freq():
    return torch.ones(64, dtype=torch.float64)


def test_rope_refusals(sgmv, freq):
    strides = {f: 64 for f in ROPE if f.endswith(("_token", "_head", "_block"))}
    base = dict(strides, q_out=A16, q=A16, k_out=A16, k=A16, v=A16, k_cache=A16, v_cache=A16, positions=A16,
                slots=A16, inv_freq=freq.data_ptr(), T=4, Hq=2, Hk=2, D=64, pairs=32, num_blocks=3, block_size=16,
                scale=1.0)
    call = caller(sgmv, "sgmv_rope", sgmv._ROPE_ARGS, ROPE, base)
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hk=-1), dict(dtype=2), dict(dtype=9), dict(D=0), dict(pairs=-1),
                dict(pairs=33), dict(inv_freq=0), dict(q=0), dict(q_out=0), dict(k=0), dict(positions=0), dict(v=0),
                dict(slots=0), dict(k_cache=0), dict(v_cache=0), dict(num_blocks=0), dict(block_size=0), dict(Hk=0),
                dict(k_out=0, k_cache=0, v_cache=0, slots=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=60), dict(q=MIS), dict(q_out=MIS), dict(k=MIS), dict(k_out=MIS), dict(v=MIS), dict(k_cache=MIS),
                dict(v_cache=MIS), dict(q_token=65), dict(k_head=4), dict(v_token=1), dict(cache_block=4),
                dict(cache_token=12), dict(cache_head=2), dict(q_out_head=33), dict(k_out_token=9)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(D=264, pairs=4) == UNSUPPORTED
    assert call(T=0) == OK
    bad = torch.full((64,), float("nan"), dtype=torch.float64)
    assert call(inv_freq=bad.data_ptr()) == INVALID
    assert sgmv.load_library().sgmv_rope(None, None) == INVALID


def test_frequency_refusals(sgmv):
    for kw in (dict(pairs=0), dict(pairs=4, base=0.0), dict(pairs=4, factor=0.0), dict(pairs=4, factor=-1.0),
               dict(pairs=4, factor=2.0, fast=3.0, slow=1.0), dict(pairs=4, factor=2.0, trained=9.0, fast=1.0, slow=1.0)):
        with pytest.raises(sgmv.SgmvError) as e:
            sgmv.sgmv_rope_frequencies(**kw)
        assert e.value.status == INVALID


def test_attention_refusals(sgmv):
    strides = {f: 64 for f in ATTENTION if f.endswith(("_token", "_head", "_block"))}
    size = sgmv.sgmv_tree_attention_workspace_bytes(4, 2, 4, 2, 64)
    base = dict(strides, out=A16, q=A16, k_cache=A16, v_cache=A16, block_table=A16, prefix_lens=A16, tree_ptr=A16,
                workspace=A16, workspace_bytes=size, table_row=8, T=4, B=2, Hq=4, Hkv=2, D=64, num_blocks=3,
                block_size=16, max_blocks=8, scale=0.125)
    call = caller(sgmv, "sgmv_tree_attention", sgmv._ATTENTION_ARGS, ATTENTION, base)
    for bad in (dict(T=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(dtype=2), dict(D=0), dict(out=0),
                dict(q=0), dict(k_cache=0), dict(v_cache=0), dict(block_table=0), dict(prefix_lens=0),
                dict(tree_ptr=0), dict(num_blocks=0), dict(block_size=0), dict(max_blocks=0), dict(table_row=-1),
                dict(scale=float("nan"))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=60), dict(q=MIS), dict(out=MIS), dict(k_cache=MIS), dict(v_cache=MIS), dict(q_token=7),
                dict(out_head=4), dict(cache_block=4), dict(cache_token=2), dict(cache_head=1),
                dict(workspace=A16 + 16)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(D=264) == UNSUPPORTED
    assert call(workspace_bytes=size - 1) == WORKSPACE
    assert call(workspace=0) == WORKSPACE
    assert call(T=0) == OK and call(B=0) == OK
    assert sgmv.load_library().sgmv_tree_attention(None, None) == INVALID
    assert sgmv.sgmv_tree_attention_workspace_bytes(0, 1, 1, 1, 64) == 0


def test_verify_refusals(sgmv):
    base = dict(target=A16, draft=A16, tokens=A16, tree_ptr=A16, u_accept=A16, u_sample=A16, count=A16, path=A16,
                token=A16, target_row=50, draft_row=50, T=4, B=2, V=50, max_path=4)
    call = caller(sgmv, "sgmv_tree_verify", sgmv._VERIFY_ARGS, VERIFY, base)
    for bad in (dict(T=-1), dict(B=-1), dict(V=0), dict(max_path=0), dict(target=0), dict(tokens=0), dict(tree_ptr=0),
                dict(u_accept=0), dict(u_sample=0), dict(count=0), dict(path=0), dict(token=0)):
        assert call(**bad) == INVALID, bad
    assert call(target=A16 + 2) == ALIGNMENT and call(draft=A16 + 1) == ALIGNMENT
    assert call(V=(1 << 24) + 1) == UNSUPPORTED
    assert call(B=0) == OK
    assert sgmv.load_library().sgmv_tree_verify(None, None) == INVALID


def test_commit_refusals(sgmv):
    base = dict(k_cache=A16, v_cache=A16, block_table=A16, prefix_lens=A16, path=A16, count=A16, cache_layer=640,
                cache_block=64, cache_token=64, cache_head=64, table_row=4, layers=2, B=2, Hkv=2, D=64, num_blocks=3,
                block_size=16, max_blocks=4, max_path=4)
    call = caller(sgmv, "sgmv_cache_commit", sgmv._COMMIT_ARGS, COMMIT, base)
    for bad in (dict(layers=-1), dict(B=-1), dict(Hkv=0), dict(max_path=-1), dict(dtype=2), dict(D=0), dict(k_cache=0),
                dict(v_cache=0), dict(block_table=0), dict(prefix_lens=0), dict(path=0), dict(count=0),
                dict(num_blocks=0), dict(block_size=0), dict(max_blocks=0), dict(table_row=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(D=60), dict(k_cache=MIS), dict(v_cache=MIS), dict(cache_layer=4), dict(cache_block=2),
                dict(cache_token=4), dict(cache_head=7)):
        assert call(**bad) == ALIGNMENT, bad
    assert call(D=264) == UNSUPPORTED and call(layers=40000) == UNSUPPORTED
    assert call(layers=0) == OK and call(B=0) == OK and call(max_path=0) == OK
    assert sgmv.load_library().sgmv_cache_commit(None, None) == INVALID


def test_binding_refusals(sgmv):
    """Shapes, types and layouts that the C ABI cannot see."""
    h, f = torch.float16, torch.ones(32, dtype=torch.float64)
    q, k = torch.zeros(4, 4, 64, dtype=h), torch.zeros(4, 2, 64, dtype=h)
    pos, c = torch.zeros(4, dtype=torch.int32), torch.zeros(3, 16, 2, 64, dtype=h)
    for args, kw, error in (
            ((q, k, pos.long(), f), {}, TypeError), ((q, k, pos[:3], f), {}, ValueError),
            ((q, k.bfloat16(), pos, f), {}, TypeError), ((q, k[:3], pos, f), {}, ValueError),
            ((q, k[..., :32], pos, f), {}, ValueError), ((q, k, pos, f.float()), {}, TypeError),
            ((q, k, pos, f), dict(q_out=q[:, :3]), ValueError), ((q.transpose(1, 2), None, pos, f), {}, TypeError),
            ((q, k, pos, f), dict(v=k, k_cache=c, v_cache=c[:2], slots=pos), ValueError),
            ((q, k, pos, f), dict(v=k, k_cache=c, v_cache=c.bfloat16(), slots=pos), TypeError),
            ((q, q, pos, f), dict(v=q, k_cache=c, v_cache=c, slots=pos), ValueError)):
        with pytest.raises(error):
            sgmv.sgmv_rope(*args, **kw)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    table, lens, ptr = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), pos[:2]
    good = dict(out=q, q=q, k_cache=c, v_cache=c, block_table=table, prefix_lens=lens, tree_ptr=ptr, workspace=ws)
    for change, error in ((dict(out=q.float()), TypeError), (dict(k_cache=c.float()), TypeError),
                          (dict(block_table=table.long()), TypeError), (dict(tree_ptr=pos), ValueError),
                          (dict(parents=pos[:2]), ValueError), (dict(lse=q[..., 0].float().T), TypeError),
                          (dict(out=q[:, :2]), ValueError), (dict(q=q[..., :32], out=q[..., :32]), ValueError),
                          (dict(block_table=table.T), TypeError)):
        with pytest.raises(error):
            sgmv.sgmv_tree_attention(**{**good, **change})
    p, u = torch.zeros(4, 9), torch.zeros(4)
    good = dict(target=p, draft=p, tokens=pos, parents=pos, tree_ptr=ptr, u_accept=u, u_sample=u[:1], max_path=4)
    for change, error in ((dict(target=p.double()), TypeError), (dict(draft=p[:3]), TypeError),
                          (dict(tokens=pos[:3]), ValueError), (dict(u_accept=u.double()), TypeError),
                          (dict(target=torch.zeros(9, 4).T), TypeError)):
        with pytest.raises(error):
            sgmv.sgmv_tree_verify(**{**good, **change})
    with pytest.raises(ValueError):
        sgmv.sgmv_cache_commit(c, c, table, lens, pos.view(1, 4), pos)


def test_argument_structs_match_the_header(sgmv, tmp_path):
    """The packed layouts have the sizes that a C compiler gives the structs."""
    import subprocess
    from pathlib import Path

    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "sgmv.h"\nint main(void) { printf("%zu %zu %zu %zu", '
                   "sizeof(sgmv_rope_args), sizeof(sgmv_tree_attention_args), sizeof(sgmv_tree_verify_args), "
                   "sizeof(sgmv_cache_commit_args)); return 0; }\n")
    inc = Path(__file__).resolve().parents[1] / "include"
    subprocess.run(["gcc", f"-I{inc}", str(src), "-o", str(tmp_path / "s")], check=True)
    sizes = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    layouts = (sgmv._ROPE_ARGS, sgmv._ATTENTION_ARGS, sgmv._VERIFY_ARGS, sgmv._COMMIT_ARGS)
    assert [int(x) for x in sizes] == [s.size for s in layouts]
    assert struct.calcsize("P") == 8
