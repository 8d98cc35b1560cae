"""Norms of query and key heads with their rotation on the GPU against a plain 64-bit reference."""
import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


def run(M, heads, q, k, D, rot, inter=0, layout="heads", gains="both", pos="random", pos0=0, in_place=False, pad=0, seed=0,
        eps=1e-6, x=None, **kw):
    rng = np.random.default_rng(seed)
    freq, scale = fq.fq_rope_freqs(rot, **kw) if rot else (None, 1.0)
    ld = heads * D + pad
    if x is None:
        x = ref.bf16(rng, M, ld, scale=3.0)
    p = rng.integers(-2 ** 31, 2 ** 31, M).astype(np.int32) if pos == "random" else (pos0 + np.arange(M)).astype(np.int32)
    gq = rng.uniform(0.5, 1.5, D).astype(np.float32) if gains in ("both", "q") else None
    gk = rng.uniform(0.5, 1.5, D).astype(np.float32) if gains in ("both", "k") else None
    xd = dev(x)
    if in_place:
        y, yt, yh = xd, ld, D
    elif layout == "heads":
        y, yt, yh = dev(np.full((heads, M + 1, D), 0x1234, np.uint16)), D, (M + 1) * D
    else:
        y, yt, yh = dev(np.full((M, ld), 0x1234, np.uint16)), ld, D
    up = lambda a: None if a is None else dev(a)  # noqa: E731
    fq.fq_qk_norm_rope(xd, ld, D, M, heads, q, k, D, up(gq), up(gk), eps, rot, inter, None if freq is None else dev(freq.view(np.int64)),
                       scale, up(p) if pos == "random" else None, pos0, y, yt, yh)
    got = host(y, np.uint16)
    if layout == "heads" and not in_place:
        assert np.all(got[:, M] == 0x1234), "wrote past the last token"
        got = got[:, :M]
    else:
        if pad:
            assert np.array_equal(got[:, heads * D:], x[:, heads * D:] if in_place else np.full((M, pad), 0x1234)), "pad"
        got = got[:, :heads * D].reshape(M, heads, D).transpose(1, 0, 2)
    xb = x[:, :heads * D].reshape(M, heads, D).transpose(1, 0, 2)
    n = q + k
    assert np.array_equal(got[n:], xb[n:]), "value heads are copied"
    if n:
        y64, mag = attnref.qk_norm(bf16_to_f64(xb), q, k, gq, gk, eps, rot, inter, p, freq, scale)
        # sums of up to 256 squares in float32 (2^-20 of themselves at most, half of it in the root), cos and sin
        # within 2^-22, and a handful of float32 roundings
        ref.assert_bf16(got[:n], y64[:n], mag[:n], f"{M}x{heads}x{D} rot={rot}", ulps=2.0 ** -19)


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (80, 32), (80, 80), (96, 24), (128, 16), (128, 2), (64, 20),
                                   (16, 16), (48, 14), (32, 0), (112, 112), (192, 48), (240, 240), (256, 0), (256, 250), (16, 8)])
def test_heads_and_parts(D, rot, inter):
    run(5, 7, 3, 2, D, rot, inter, seed=D + rot)


@pytest.mark.parametrize("M,heads,q,k", [(1, 1, 1, 0), (1, 12, 8, 2), (2, 3, 0, 0), (3, 3, 0, 2), (67, 9, 9, 0), (300, 36, 28, 4),
                                         (1, 300, 200, 99), (1, 1, 0, 1)])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("layout", ["heads", "rows", "in place"])
def test_tokens_and_layouts(M, heads, q, k, inter, layout):
    run(M, heads, q, k, 64, 64, inter, layout="rows" if layout == "in place" else layout, pad=24, in_place=layout == "in place", seed=M)


@pytest.mark.parametrize("M,heads,q,k,D,rot,inter", [(40000, 7, 4, 2, 64, 64, 0), (33000, 6, 3, 3, 96, 32, 1), (17000, 5, 2, 2, 256, 256, 0),
                                                    (70000, 3, 1, 1, 16, 8, 1)])
def test_many_tokens(M, heads, q, k, D, rot, inter):
    """A thread takes all heads of its token, queries and keys."""
    run(M, heads, q, k, D, rot, inter, seed=M)


@pytest.mark.parametrize("gains", ["both", "q", "k", "none"])
@pytest.mark.parametrize("rot", [64, 20])
def test_gains_may_be_left_out(gains, rot):
    run(9, 6, 2, 2, 64, rot, gains=gains)


@pytest.mark.parametrize("pos0", [0, 4095, 2 ** 31 - 33, -5])
@pytest.mark.parametrize("inter,rot", [(0, 128), (1, 128), (0, 10)])
def test_counted_positions(pos0, inter, rot):
    run(33, 3, 1, 1, 128, rot, inter, pos="count", pos0=pos0)


@pytest.mark.parametrize("rot", [64, 20])
def test_zero_heads_and_large_values(rot):
    rng = np.random.default_rng(1)
    x = ref.bf16(rng, 8, 4 * 64)
    x[:, :64] = 0              # a head of zeros stays zero
    x[:, 64:128] = ref.bf16(rng, 8, 64, scale=2.0 ** 55)  # squares up to 2^115
    x[:, 128:192] = ref.bf16(rng, 8, 64, scale=2.0 ** -60)  # below eps: the root of eps divides
    run(8, 4, 2, 1, 64, rot, x=x)


def test_matches_the_rotation_of_the_normed_heads():
    """Unit gains and rows of equal squares: the norm is a division by a power of two, so the result is fq_rope's."""
    rng = np.random.default_rng(2)
    M, H, D = 70, 4, 64
    x = np.where(rng.random((M, H * D)) < 0.5, -4.0, 4.0).astype(np.float32)
    xd = torch.from_numpy(x).to(torch.bfloat16).cuda()
    freq, s = fq.fq_rope_freqs(D)
    fd = dev(freq.view(np.int64))
    y, want = torch.empty_like(xd), torch.empty_like(xd)
    fq.fq_qk_norm_rope(xd, H * D, D, M, H, 3, 1, D, None, None, 0.0, D, 0, fd, s, None, 11, y, H * D, D)
    fq.fq_rope(xd / 4, H * D, D, M, H, H, D, D, 0, fd, s, None, 11, 0, want, H * D, D)
    assert torch.equal(y, want)
