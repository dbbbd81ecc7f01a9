"""Lengths whose work the tree attention cannot count are refused, also where tiles are
small: 8 rows, and pages of 72 tokens that fill a tile by themselves."""
import pytest

A16 = 0x10000  # an address that nothing reads
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (64, 64), (8, 1)])
@pytest.mark.parametrize("block_size,tile", [(72, 72), (16, 128), (5, 128), (24, 120), (88, 88)])
def test_a_count_of_32_bits_is_never_passed(sgmv, Hq, Hkv, block_size, tile):
    """T <= B gives tiles of 8 rows, yet one sequence may have all 256 nodes: the shortest
    length whose items times tiles pass 2^32 must be refused."""
    items = Hkv * (256 * (Hq // Hkv) // 8)
    pages = ((1 << 32) // items * tile + tile) // block_size
    if pages * block_size > 2 ** 31:
        return  # no such length
    size = sgmv.sgmv_tree_attention_workspace_bytes(256, 256, Hq, Hkv, 64)
    args = sgmv._ATTENTION_ARGS.pack(A16, A16, A16, A16, 0, A16, A16, A16, 0, A16, size, *[64] * 7, pages, 256, 256, Hq,
                                     Hkv, 64, 3, block_size, pages, 0, 0.125)
    assert sgmv.load_library().sgmv_tree_attention(args, None) == UNSUPPORTED


def test_long_contexts_are_not(sgmv):
    """A context of 16 million tokens, 64 heads: past this check, to the next one (no workspace)."""
    args = sgmv._ATTENTION_ARGS.pack(A16, A16, A16, A16, 0, A16, A16, A16, 0, 0, 0, *[64] * 7, 1 << 20, 256, 256, 64, 8,
                                     64, 3, 16, 1 << 20, 0, 0.125)
    assert sgmv.load_library().sgmv_tree_attention(args, None) == 6
