"""Arrays of 32-bit words at addresses that are no multiples of 4 are refused on the host by
every decoding call: on the device they would be misaligned loads and stores."""
import pytest
import torch

from tests.test_decode_args_cpu import GRAD, SAMPLE, Two
from tests.test_spec_args_cpu import A16, ALIGNMENT, ATTENTION, COMMIT, ROPE, VERIFY, caller

FREQ = torch.ones(64, dtype=torch.float64)


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def struct_of(sgmv, call):
    rope, attention = (sgmv._ROPE_ARGS, ROPE), (sgmv._ATTENTION_ARGS, ATTENTION)
    return {"sgmv_rope": rope, "sgmv_tree_attention": attention,
            "sgmv_tree_verify": (sgmv._VERIFY_ARGS, VERIFY), "sgmv_cache_commit": (sgmv._COMMIT_ARGS, COMMIT),
            "sgmv_norm_rope": (Two(*[rope[0], sgmv._NORM_ARGS, len(ROPE)]),
                               ROPE + "q_weight k_weight k_scale v_scale eps".split()),
            "sgmv_norm_rope_grad": (sgmv._NORM_GRAD_ARGS, GRAD),
            "sgmv_quant_attention": (Two(attention[0], sgmv._SCALE_ARGS, len(ATTENTION)), ATTENTION + ["k_scale", "v_scale"]),
            "sgmv_sample": (sgmv._SAMPLE_ARGS, SAMPLE)}[call]


POINTERS = ("q_out q k_out k v k_cache v_cache positions slots q_weight k_weight k_scale v_scale out lse block_table "
            "prefix_lens tree_ptr parents target draft tokens u_accept u_sample count path token logits u temperature "
            "top_k top_p min_p probs dq dk dq_out dk_out dq_weight dk_weight workspace").split()
SIZES = dict(T=4, B=2, Hq=4, Hk=2, Hkv=2, D=64, pairs=32, num_blocks=3, block_size=16, max_blocks=8, table_row=8,
             layers=2, max_path=4, V=50, scale=1.0, eps=1e-6, workspace_bytes=1 << 25, inv_freq=FREQ.data_ptr())


@pytest.mark.parametrize("call,words", [
    ("sgmv_rope", "positions slots"),
    ("sgmv_tree_attention", "lse block_table prefix_lens tree_ptr parents"),
    ("sgmv_tree_verify", "target draft tokens parents tree_ptr u_accept u_sample count path token"),
    ("sgmv_cache_commit", "block_table prefix_lens path count"),
    ("sgmv_norm_rope", "positions slots k_scale v_scale"),
    ("sgmv_norm_rope_grad", "positions dq_weight dk_weight"),
    ("sgmv_quant_attention", "lse block_table prefix_lens tree_ptr parents k_scale v_scale"),
    ("sgmv_sample", "u temperature top_k top_p min_p token probs")])
def test_misaligned_words(sgmv, call, words):
    layout, fields = struct_of(sgmv, call)
    base = {f: 64 for f in fields if f.endswith(("_token", "_head", "_block", "_layer", "_row"))}
    base.update({f: A16 + 4096 * i for i, f in enumerate(POINTERS) if f in fields})
    base.update({f: v for f, v in SIZES.items() if f in fields})
    refuse = caller(sgmv, call, layout, fields, base)
    for name in words.split():
        for off in (1, 2, 3):
            assert refuse(**{name: base[name] + off}) == ALIGNMENT, (name, off)
