"""Rows, weights and heads that lie beyond 2^32 bytes of their base: strides wide enough, or matrices large enough,
that a 32-bit offset would wrap, on sampled outputs."""
import numpy as np
import pytest
import torch

import blockref as ref
import synth
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu

FAR = 1 << 30  # elements between rows: the third row is past 2^32 bytes of bf16, the second of float32


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def far_rows(bits, ld=FAR):
    """Rows of `bits` at a stride of ld elements (what lies between is not initialised)."""
    t = torch.empty((bits.shape[0] - 1) * ld + bits.shape[1], dtype=torch.int16 if bits.dtype == np.uint16 else torch.float32,
                    device="cuda")
    v = t.as_strided(bits.shape, (ld, 1))
    v.copy_(dev(bits))
    return v


@pytest.mark.parametrize("f32", [0, 1])
def test_block_norm_rows(f32):
    rng = np.random.default_rng(f32)
    M, K = 4, 264
    x = ref.bf16(rng, M, K)
    r = rng.standard_normal((M, K)).astype(np.float32)
    rb = r if f32 else synth.f32_to_bf16_bits(r)
    r64 = (r if f32 else synth.bf16_bits_to_f32(rb)).astype(np.float64)
    gain = rng.uniform(0.5, 1.5, K).astype(np.float32)
    xd, rd = far_rows(x), far_rows(rb)
    h = far_rows(np.zeros((M, K), np.uint16))
    fq.fq_block_norm(M, K, xd, FAR, dev(gain), 1e-6, None, 0, 0.5, rd, FAR, rd, FAR, f32, dev(gain), 1e-6, None, None, 0,
                     1, h, FAR)
    want, mag = ref.block_norm(bf16_to_f64(x), gain, 1e-6, None, 0.5, r64, 1)
    got = host(rd.contiguous())
    if f32:
        stored = got.astype(np.float64)
        assert np.all(np.abs(stored - want) <= mag * 2.0 ** -20)
    else:
        ref.assert_bf16(got.view(np.uint16), want, mag, "stream")
        stored = bf16_to_f64(got.view(np.uint16))
    hw, hm = ref.pre_norm(stored, gain, 1e-6, None, None, 1)
    ref.assert_bf16(host(h.contiguous(), np.uint16), hw, hm, "h")


@pytest.mark.parametrize("M", [1, 4, 40])
def test_fp8_rows_residual_and_outputs(M):
    """x, the residual and y at wide strides (M = 40 with a smaller one: 40 rows past 2^32 bytes)."""
    rng = np.random.default_rng(M)
    K, N = 384, 72
    ld = FAR if M <= 4 else 1 << 26
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32))
    x, residual = ref.bf16(rng, M, K), ref.bf16(rng, M, N)
    y = far_rows(np.zeros((M, N), np.uint16), ld)
    site.linear(far_rows(x, ld), residual=far_rows(residual, ld), y=y)
    codes, scales = (host(t) for t in site.workspace_codes(M))
    ref.assert_codes8(codes, scales, *ref.quant_rows(bf16_to_f64(x)), what=f"M={M}")
    want, tol = ref.fp8_gemm(codes, scales, host(site.codes), host(site.wscale), None, residual)
    ref.assert_gemm(host(y.contiguous(), np.uint16), want, tol, f"M={M}")


@pytest.mark.parametrize("M", [1, 7, 40])
def test_fp8_weights_past_32_bits(M):
    """N x K = 70 000 x 65 536 codes (4.6 GB), the last blocks of rows among those checked; without a norm one token
    of this K takes the two launches, and few tiles of it K in parts (the last 64 rows as a layer of their own)."""
    N, K = 70000, 65536
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.randint(0, 256, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x30
    wscale = torch.rand((-(-N // 128), K // 128), generator=g, device="cuda") * 0.01 + 0.001
    rng = np.random.default_rng(M)
    x = dev(ref.bf16(rng, M, K))
    site = fq.Fp8Site(codes=codes, wscale=wscale)
    y = host(site.linear(x), np.uint16)
    qa, sa = (host(t) for t in site.workspace_codes(M))
    blocks = np.array([0, 300, N // 128])  # (65 536 rows of this K begin past 2^32 bytes; the last block is short)
    for b in blocks:
        rows = slice(128 * b, min(128 * b + 16, N))
        want, tol = ref.fp8_gemm(qa, sa, host(codes[rows]), host(wscale[b:b + 1]))
        ref.assert_gemm(y[:, rows], want, tol, f"M={M} block {b}")
    tail = fq.Fp8Site(codes=codes[N - 112:N - 48], wscale=wscale[-1:].contiguous())
    want, tol = ref.fp8_gemm(qa, sa, host(tail.codes), host(tail.wscale))
    ref.assert_gemm(host(tail.linear(x), np.uint16), want, tol, f"M={M} K in parts")


def test_rope_heads_and_tokens():
    rng = np.random.default_rng(0)
    M, H, D = 3, 2, 64
    bits = ref.bf16(rng, H, M, D)
    t = torch.empty((M - 1) * FAR + H * D, dtype=torch.int16, device="cuda")  # tokens far apart
    v = t.as_strided((H, M, D), (D, FAR, 1))
    v.copy_(dev(bits))
    o = torch.empty((H - 1) * 3 * FAR + M * D, dtype=torch.int16, device="cuda")  # heads far apart
    w = o.as_strided((H, M, D), (3 * FAR, D, 1))
    freq, att = fq.fq_rope_freqs(D)
    fq.fq_rope(v, FAR, D, M, H, H, D, D, 0, dev(freq.view(np.int64)), att, None, 5, 0, w, D, 3 * FAR)
    want, mag = ref.rope(bf16_to_f64(bits), np.arange(5, 5 + M), freq, att, H, D, 0, False)
    ref.assert_bf16(host(w.contiguous(), np.uint16), want, mag, "rope")


def test_more_rows_than_a_launch_takes_along_x():
    """8.4 million short rows without a norm: sampled codes and scales, the last rows among them."""
    M, K = (1 << 23) + 77, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-2 ** 15, 2 ** 15, (M, K), generator=g, device="cuda", dtype=torch.int16)
    x = torch.where((x & 0x7F80) == 0x7F80, torch.full_like(x, 0x3F80), x)  # finite
    codes = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    scales = torch.empty((1, -(-M // 4) * 4), dtype=torch.float32, device="cuda")
    fq.fq_fp8_prologue(x, M, K, K, None, 0.0, codes, scales)
    rows = torch.tensor([0, 1, 12345, (1 << 23) - 1, 1 << 23, M - 1], device="cuda")
    v = synth.bf16_bits_to_f32(host(x[rows], np.uint16))
    s = (np.abs(v).max(-1) / np.float32(448)).astype(np.float32)
    assert np.array_equal(host(scales[0, rows]), s)
    q = ref.e4m3_round((v / s[:, None]).astype(np.float64))
    assert np.array_equal(ref.TABLE[host(codes[rows])], ref.TABLE[q])
