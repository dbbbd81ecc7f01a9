"""sgmv_rope against the rotation in 64 bits: pair layouts, partial heads,
strides, positions of any size, the append to the cache, the gradient."""
import numpy as np
import pytest
import torch

from tests import spec_reference as ref
from tests.gpu_helpers import check_error_word

pytestmark = pytest.mark.gpu
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def sgmv():
    from rank_gemv_gb300 import build, sgmv

    build.build()
    return sgmv


def close(got, x, positions, inv_freq, interleaved, scale=1.0, inverse=False):
    y, m = ref.rope(x, positions, inv_freq, interleaved, scale, inverse)
    err = np.abs(ref.f64(got) - y)
    assert (err <= ref.rope_bound(y, m, got.dtype)).all(), err.max()


def rand(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,pairs", [(1, 32, 32, 128, 64), (7, 8, 2, 128, 32), (33, 3, 1, 80, 16),
                                             (5, 4, 4, 64, 5), (3, 1, 1, 8, 4), (4, 2, 2, 256, 128),
                                             (2, 5, 5, 96, 0), (300, 2, 1, 64, 13)])
def test_layouts_and_sizes(sgmv, dtype, interleaved, T, Hq, Hk, D, pairs):
    g = torch.Generator("cuda").manual_seed(T + D)
    qkv = rand(g, T, Hq + 2 * Hk, D, dtype=dtype)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    positions = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = sgmv.sgmv_rope_frequencies(pairs) if pairs else torch.empty(0, dtype=torch.float64)
    q_out, k_out = torch.empty(T, Hq, D, device="cuda", dtype=dtype), torch.empty(T, Hk, D, device="cuda", dtype=dtype)
    before = qkv.clone()
    sgmv.sgmv_rope(q, k, positions, f, interleaved, scale=1.25, q_out=q_out, k_out=k_out)
    assert sgmv.sgmv_last_launch_count() == 1
    check_error_word(0)
    assert torch.equal(qkv, before)
    pos = positions.cpu().numpy()
    close(q_out, q, pos, f.numpy(), interleaved, 1.25)
    close(k_out, k, pos, f.numpy(), interleaved, 1.25)
    # in place, on strided views, one of the two alone: the same bits
    sgmv.sgmv_rope(q, None, positions, f, interleaved, scale=1.25)
    sgmv.sgmv_rope(None, k, positions, f, interleaved, scale=1.25)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


@pytest.mark.parametrize("dtype", TYPES)
def test_positions_of_any_size(sgmv, dtype):
    pos = [0, 1, -1, 65535, 131071, 10 ** 6 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -(2 ** 31)]
    g = torch.Generator("cuda").manual_seed(3)
    q = rand(g, len(pos), 2, 64, dtype=dtype)
    f = sgmv.sgmv_rope_frequencies(32, base=5e5, factor=8.0, trained=8192, slow=1.0, fast=4.0)
    # the reference angle in twice the digits: position and frequency are
    # doubles, their product modulo a turn is taken in whole numbers
    from fractions import Fraction

    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    turns = np.array([[float(Fraction(p) * Fraction(x) / two_pi % 1) for x in f.tolist()] for p in pos])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    x = ref.f64(q)
    y = np.concatenate([x[..., :32] * c - x[..., 32:] * s, x[..., :32] * s + x[..., 32:] * c], -1)
    m = np.tile(np.abs(x[..., :32]) + np.abs(x[..., 32:]), 2)
    out = torch.empty_like(q)
    sgmv.sgmv_rope(q, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), f, q_out=out)
    # the frequency in turns is a double: 2^31 * 2^-53 turns of a pair off
    bound = ref.rope_bound(y, m, dtype) + 2 * np.pi * 2.0 ** -21 * m
    assert (np.abs(ref.f64(out) - y) <= bound).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("order", ["pages-tokens-heads", "pages-heads-tokens", "k-and-v-in-one"])
@pytest.mark.parametrize("bs", [1, 16, 24])
def test_append(sgmv, dtype, order, bs):
    g = torch.Generator("cuda").manual_seed(bs)
    T, Hq, Hk, D, blocks = 41, 6, 3, 80, 60
    qkv = rand(g, T, Hq + 2 * Hk, D, dtype=dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    if order == "pages-heads-tokens":
        kc, vc = (rand(g, blocks, Hk, bs, D, dtype=dtype).transpose(1, 2) for _ in range(2))
    elif order == "k-and-v-in-one":
        kc, vc = rand(g, blocks, 2, bs, Hk, D, dtype=dtype).unbind(1)
    else:
        kc, vc = (rand(g, blocks, bs, Hk, D, dtype=dtype) for _ in range(2))
    slots = torch.randperm(blocks * bs, generator=torch.Generator().manual_seed(1))[:T].to(torch.int32)
    slots[::7] = -1
    positions = torch.arange(T, dtype=torch.int32, device="cuda") * 17
    f = sgmv.sgmv_rope_frequencies(20)
    want_k, want_v = kc.clone(), vc.clone()
    _, rot = sgmv.sgmv_rope(None, k, positions, f, k_out=torch.empty(T, Hk, D, dtype=dtype, device="cuda"))
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // bs, s % bs], want_v[s // bs, s % bs] = rot[t], v[t]
    before = k.clone()
    q_out = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    sgmv.sgmv_rope(q, k, positions, f, q_out=q_out, v=v, k_cache=kc, v_cache=vc, slots=slots.cuda())
    check_error_word(0)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v) and torch.equal(k, before)
    close(q_out, q, positions.cpu().numpy(), f.numpy(), False)
    # a slot outside the cache is reported and left out
    slots[3] = blocks * bs
    sgmv.sgmv_rope(None, k, positions, f, v=v, k_cache=kc, v_cache=vc, slots=slots.cuda())
    check_error_word(4)
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(sgmv, interleaved):
    """d sum(g . rope(x)) / dx is rope(g, inverse): by the formula, and by
    differences of the forward pass (which is linear, so a step of 1 is as good
    as a small one) of every coordinate of one head."""
    dtype, T, D, pairs, scale = torch.float16, 3, 16, 6, 1.5
    gen = torch.Generator("cuda").manual_seed(9)
    x, g = rand(gen, T, 1, D, dtype=dtype), rand(gen, T, 1, D, dtype=dtype)
    positions = torch.tensor([1, 77, 4000], dtype=torch.int32, device="cuda")
    f = sgmv.sgmv_rope_frequencies(pairs)
    grad, _ = sgmv.sgmv_rope(g, None, positions, f, interleaved, scale=scale, inverse=True, q_out=torch.empty_like(g))
    close(grad, g, positions.cpu().numpy(), f.numpy(), interleaved, scale, inverse=True)

    def loss(x):
        y, _ = sgmv.sgmv_rope(x, None, positions, f, interleaved, scale=scale, q_out=torch.empty_like(x))
        return (ref.f64(y) * ref.f64(g)).sum(-1), np.abs(ref.f64(y) * ref.f64(g)).sum(-1)

    for d in range(D):
        step = torch.zeros_like(x)
        step[..., d] = 1.0
        (up, a), (down, b) = loss(x + step), loss(x - step)
        # x +- 1 and the outputs are rounded to f16, the gradient itself too
        slack = 2.0 ** -11 * (a + b + 2 * scale * np.abs(ref.f64(g)).sum(-1) * (np.abs(ref.f64(x)[..., d]) + 1)
                            + np.abs(ref.f64(grad)[..., d])) + 1e-4
        assert (np.abs((up - down) / 2 - ref.f64(grad)[..., d]) <= slack).all()


def test_frequencies(sgmv):
    i = np.arange(64)
    base = 10000.0 ** (-i / 64)
    assert np.allclose(sgmv.sgmv_rope_frequencies(64).numpy(), base, rtol=1e-14)
    assert np.allclose(sgmv.sgmv_rope_frequencies(64, factor=4.0).numpy(), base / 4, rtol=1e-14)
    got = sgmv.sgmv_rope_frequencies(64, factor=4.0, trained=4096, slow=1.0, fast=32.0).numpy()
    turns = 4096 * base / (2 * np.pi)
    assert np.allclose(got[turns > 32], base[turns > 32], rtol=1e-14)
    assert np.allclose(got[turns < 1], base[turns < 1] / 4, rtol=1e-14)
    keep = np.clip((turns - 1) / 31, 0, 1)
    assert np.allclose(got, base * keep + base / 4 * (1 - keep), rtol=1e-13)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,pairs", [(1300, 32, 8, 128, 64), (2500, 7, 7, 80, 16), (4100, 1, 1, 64, 32),
                                             (1217, 40, 40, 128, 32), (1999, 3, 2, 96, 20), (5000, 2, 2, 8, 4)])
def test_many_rows(sgmv, dtype, interleaved, T, Hq, Hk, D, pairs):
    """Several rows per CTA: against the reference, append and in-place included."""
    g = torch.Generator("cuda").manual_seed(T)
    qkv = rand(g, T, Hq + 2 * Hk, D, dtype=dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    positions = torch.randint(0, 100000, (T,), generator=g, device="cuda", dtype=torch.int32)
    f = sgmv.sgmv_rope_frequencies(pairs)
    slots = torch.randperm(T + 5, generator=g, device="cuda")[:T].to(torch.int32)
    slots[7::50] = -1
    kc, vc = rand(g, T + 5, 1, Hk, D, dtype=dtype), rand(g, T + 5, 1, Hk, D, dtype=dtype)
    want_k, want_v = kc.clone(), vc.clone()
    q_out, k_out = torch.empty(T, Hq, D, device="cuda", dtype=dtype), torch.empty(T, Hk, D, device="cuda", dtype=dtype)
    before = qkv.clone()
    sgmv.sgmv_rope(q, k, positions, f, interleaved, q_out=q_out, k_out=k_out, v=v, k_cache=kc, v_cache=vc, slots=slots)
    check_error_word(0)
    assert torch.equal(qkv, before)
    pos = positions.cpu().numpy()
    close(q_out, q, pos, f.numpy(), interleaved)
    close(k_out, k, pos, f.numpy(), interleaved)
    live = slots >= 0
    want_k[slots[live].long(), 0], want_v[slots[live].long(), 0] = k_out[live], v[live]
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)
    sgmv.sgmv_rope(q, k, positions, f, interleaved)
    assert torch.equal(q, q_out) and torch.equal(k, k_out) and torch.equal(v, before[:, Hq + Hk:])


def test_other_stream(sgmv):
    g = torch.Generator("cuda").manual_seed(5)
    q = rand(g, 64, 8, 128, dtype=torch.bfloat16)
    f, positions = sgmv.sgmv_rope_frequencies(64), torch.arange(64, dtype=torch.int32, device="cuda")
    want, _ = sgmv.sgmv_rope(q, None, positions, f, q_out=torch.empty_like(q))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = q * 2  # the call is ordered after its own stream's work
        got, _ = sgmv.sgmv_rope(x, None, positions, f, scale=0.5, q_out=torch.empty_like(q))
    side.synchronize()
    assert torch.equal(got, want)
