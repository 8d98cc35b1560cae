"""Extreme values through the FP8 sites: groups at the edge of the code range, tokens that are not finite."""
import numpy as np
import pytest

import blockref as ref
import synth
import w4a4_integer_gemm_amd as fq
from fp8checks import assert_full_range
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


def test_every_bf16_maximum_of_a_group():
    """All finite bf16 magnitudes as a group's largest value: codes and scales of the definition, none NaN."""
    bits = np.arange(0x7F80, dtype=np.uint16)  # 0 .. the largest finite value
    M, K = 255, 128 * 128
    assert bits.size == M * 128
    rng = np.random.default_rng(0)
    x = np.zeros((M, 128, 128), np.uint16)
    top = bits.reshape(M, 128)
    # the other values: any magnitude up to the largest, either sign
    x[:] = np.minimum(rng.integers(0, 0x7F80, x.shape), top[..., None]).astype(np.uint16) | (rng.integers(0, 2, x.shape) << 15).astype(np.uint16)
    at = rng.integers(0, 128, top.shape)
    np.put_along_axis(x, at[..., None], (top | (rng.integers(0, 2, top.shape) << 15).astype(np.uint16))[..., None], -1)
    x = x.reshape(M, K)
    codes, scales = dev(np.zeros((M, K), np.uint8)), dev(np.zeros((K // 128, 256), np.float32))
    fq.fq_fp8_prologue(dev(x), M, K, K, None, 0.0, codes, scales)
    q, s = host(codes), host(scales)[:, :M]
    assert_full_range(q, s)
    v = synth.bf16_bits_to_f32(x).reshape(M, 128, 128)
    want = np.abs(v).max(-1) / np.float32(448)
    assert np.array_equal(s, want.T)
    quot = np.divide(v, want[..., None], out=np.zeros_like(v), where=want[..., None] > 0)  # float32 division
    assert np.array_equal(ref.TABLE[q], ref.TABLE[ref.e4m3_round(quot.astype(np.float64)).reshape(M, K)])


@pytest.mark.parametrize("M,K", [(1, 3584), (1, 16384), (3, 2048), (16, 256), (40, 1152), (1200, 3584), (3, 33024)])
@pytest.mark.parametrize("norm", [False, True])
def test_codes_of_the_sites_use_the_full_range(M, K, norm):
    """fq_fp8_prologue, and fq_fp8_linear with the codes that it leaves in its workspace."""
    rng = np.random.default_rng(M + K)
    site = fq.Fp8Site((rng.standard_normal((8, K)) * 0.02).astype(np.float32),
                      gamma=rng.uniform(0.5, 1.5, K).astype(np.float32) if norm else None)
    x = dev(ref.bf16(rng, M, K))
    for q, s in (site.prologue(x), (site.linear(x), site.workspace_codes(M))[1]):
        assert_full_range(host(q), host(s)[:, :M], f"{M}x{K} norm={norm}")


@pytest.mark.parametrize("M,K", [(1, 2048), (5, 1152), (300, 3584), (1200, 3584), (2, 33024)])
@pytest.mark.parametrize("f32", [0, 1])
def test_codes_of_the_block_norm_use_the_full_range(M, K, f32):
    rng = np.random.default_rng(M + K + f32)
    x, r = ref.bf16(rng, M, K), rng.standard_normal((M, K)).astype(np.float32) * 3
    r = dev(r if f32 else synth.f32_to_bf16_bits(r))
    cond = dev(ref.bf16(rng, M, 2 * K, scale=0.4))
    q, s = dev(np.zeros((M, K), np.uint8)), dev(np.zeros((K // 128, -(-M // 4) * 4), np.float32))
    fq.fq_block_norm(M, K, dev(x), K, None, 0.0, None, 0, 0.5, r, K, r, K, f32, dev(rng.uniform(0.5, 1.5, K).astype(np.float32)),
                     1e-6, cond, cond[:, K:], 2 * K, 1, None, 0, q, s)
    assert_full_range(host(q), host(s)[:, :M], f"{M}x{K}")


# one launch (one token, a few, two pieces and more), the GEMV, tiles, K in parts
NON_FINITE = [(1, 512, 72), (1, 3584, 4112), (1, 8320, 40), (1, 18944, 136), (2, 256, 512), (4, 1024, 4104), (4, 3584, 264),
              (16, 256, 512), (20, 2048, 2056), (33, 384, 264), (130, 1024, 392), (40, 8192, 520), (300, 640, 1032)]


@pytest.mark.parametrize("M,K,N", NON_FINITE)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("bits", [0x7FC0, 0xFFC1, 0x7F80, 0xFF80])
def test_a_token_that_is_not_finite_stays_alone(M, K, N, norm, bits):
    """NaN and infinity of either sign in one token: its outputs are not finite, the others are as without it."""
    rng = np.random.default_rng(M + K + N)
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32), bias=rng.standard_normal(N).astype(np.float32),
                      gamma=rng.uniform(0.5, 1.5, K).astype(np.float32) if norm else None)
    x, residual = ref.bf16(rng, M, K), dev(ref.bf16(rng, M, N))
    clean = host(site.linear(dev(x), residual=residual), np.uint16)
    clean_codes, clean_scales = site.prologue(dev(x))
    row, others = M // 2, np.arange(M) != M // 2
    x[row, K - 5] = bits
    xd = dev(x)
    codes, scales = site.prologue(xd)
    for y in (site.linear(xd, residual=residual), site.gemm(codes, scales, M, residual=residual)):
        assert not np.any(np.isfinite(bf16_to_f64(host(y, np.uint16)[row])))
    assert np.array_equal(host(site.linear(xd, residual=residual), np.uint16)[others], clean[others])
    assert np.array_equal(host(codes)[others], host(clean_codes)[others])
    assert np.array_equal(host(scales)[:, :M][:, others], host(clean_scales)[:, :M][:, others])


@pytest.mark.parametrize("M,K,N", NON_FINITE)
def test_a_token_of_nan_alone_and_of_zeros(M, K, N):
    """A token whose every value is NaN, and one of zeros: not finite, and the bias and residual exactly."""
    rng = np.random.default_rng(M + K + N)
    bias = rng.standard_normal(N).astype(np.float32)
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32), bias=bias)
    x, residual = ref.bf16(rng, M, K), ref.bf16(rng, M, N)
    for fill in (0x7FC0, 0xFFC0, 0x0000, 0x8000):
        x[M // 2] = fill
        y = host(site.linear(dev(x), residual=dev(residual)), np.uint16)[M // 2]
        if fill & 0x7FFF:
            assert not np.any(np.isfinite(bf16_to_f64(y)))
        else:
            want = bias + synth.bf16_bits_to_f32(residual[M // 2])  # (one float32 add)
            assert np.array_equal(y, synth.f32_to_bf16_bits(want))
