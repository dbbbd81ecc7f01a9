"""Streaming kernel: the B chunks of a launch that end inside a chunk of 1024
(512, 256) columns, with H2 a multiple of 256 and one- and several-CTA
clusters.  The tensor map of such a launch has the rank of its copies: a copy
of another rank than its map's is an illegal instruction."""
import pytest
import torch

import oracle
from rank_gemv_gb300 import workloads as wl
from tests.gpu_helpers import assert_close, check_error_word

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [20, 80, 130])
@pytest.mark.parametrize("H2", [256, 512, 1024, 1280, 2048, 2816])
@pytest.mark.parametrize("r", [16, 32])
def test_partial_chunks(T, H2, r):
    from rank_gemv_gb300 import build, sgmv

    build.build()
    L = 5
    g = torch.Generator().manual_seed(T + H2)
    ids = torch.randint(-1, L, (T,), generator=g, dtype=torch.int32)
    ws = [wl.draw(T, L, 512, H2, r, ids, y0="randn", seed=k) for k in range(2)]
    perm, seg_ptr, idx, _ = sgmv.sgmv_build_segments_device(ids.cuda(), L)
    ys = [w.Y0.cuda() for w in ws]
    sgmv.sgmv_apply_multi(ys, [w.X.cuda() for w in ws], [w.A.cuda() for w in ws], [w.B.cuda() for w in ws], seg_ptr,
                          idx, 0.5, perm=perm, S=sgmv.sgmv_max_segments(T, L))
    check_error_word(0)
    o = oracle.build_segments(ids, L)
    for w, y in zip(ws, ys):
        assert_close(y, oracle.sgmv_apply(w.Y0, w.X, w.A, w.B, o[1], o[2], 0.5, perm=o[0]), f"H2 = {H2}")
