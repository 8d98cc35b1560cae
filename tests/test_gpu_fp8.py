"""FP8 sites with block scales on the GPU against plain 64-bit references."""
import numpy as np
import pytest
import torch

import blockref as ref
import synth
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


def rand_site(rng, M, N, K, spread=True):
    """Codes over the whole table (no NaN) with uneven scales, as numpy."""
    pick = np.array([p for p in range(256) if (p & 0x7F) != 0x7F], np.uint8)
    qa, qw = pick[rng.integers(0, pick.size, (M, K))], pick[rng.integers(0, pick.size, (N, K))]
    sa = np.exp(rng.uniform(-4, 2, (K // 128, M)) if spread else np.zeros((K // 128, M))).astype(np.float32)
    sw = np.exp(rng.uniform(-8, -4, (-(-N // 128), K // 128))).astype(np.float32)
    return qa, sa, qw, sw


def dev_scales(sa):
    """[K / 128][M] scales in the kernel's stride, the pad filled with NaN (never used)."""
    g, M = sa.shape
    full = np.full((g, -(-M // 4) * 4), np.nan, np.float32)
    full[:, :M] = sa
    return dev(full)


def run_gemm(qa, sa, qw, sw, bias=None, residual=None, head_dim=0, ldy=None):
    M, K = qa.shape
    N = qw.shape[0]
    guard = np.uint16(0xABCD)
    if head_dim:
        y = np.full((N // head_dim, M, head_dim), guard, np.uint16)
    else:
        ldy = ldy or N
        y = np.full((M + 1, ldy), guard, np.uint16)  # a row behind the last stays as it was
    yd = dev(y)
    res = None if residual is None else dev(residual)
    fq.fq_fp8_gemm(dev(qa), dev_scales(sa), M, dev(qw), dev(sw), N, K, None if bias is None else dev(bias), res,
                   0 if residual is None else residual.shape[1], head_dim, yd, ldy or 0)
    out = host(yd, np.uint16)
    if head_dim:
        return out.transpose(1, 0, 2).reshape(M, N)
    assert np.all(out[M:] == guard) and np.all(out[:, N:] == guard), "wrote outside its rows"
    return out[:M, :N]


SHAPES = [(1, 8, 128), (1, 4096, 1024), (2, 24, 256), (7, 136, 640), (16, 512, 256), (17, 264, 384), (32, 1000, 2048),
          (33, 8, 128), (40, 128, 128), (64, 264, 512), (127, 128, 256), (128, 136, 384), (129, 520, 640), (200, 1032, 1280),
          (256, 256, 896), (300, 512, 1152), (31, 72, 16384), (257, 72, 8192)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_matches_reference(M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    y, tol = ref.fp8_gemm(qa, sa, qw, sw)
    ref.assert_gemm(run_gemm(qa, sa, qw, sw), y, tol, f"gemm {M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 9, 20, 70, 130])
@pytest.mark.parametrize("head_dim", [0, 8, 40, 120])
def test_gemm_bias_residual_strides_and_heads(M, head_dim):
    N, K = 360, 512
    rng = np.random.default_rng(M + head_dim)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    bias = rng.standard_normal(N).astype(np.float32)
    residual = ref.bf16(rng, M, N + 24)
    y, tol = ref.fp8_gemm(qa, sa, qw, sw, bias, residual[:, :N])
    got = run_gemm(qa, sa, qw, sw, bias, residual, head_dim, None if head_dim else N + 40)
    ref.assert_gemm(got, y, tol, f"M={M} head_dim={head_dim}")


@pytest.mark.parametrize("M", [3, 29, 65, 140])
def test_gemm_codes_of_one_value_are_exact(M):
    """Codes +-1 and power-of-two scales: every sum is exact, so the bf16 result is the rounding of the true one."""
    N, K = 200, 1024
    rng = np.random.default_rng(M)
    qa = rng.choice(np.array([0x38, 0xB8], np.uint8), (M, K))
    qw = rng.choice(np.array([0x38, 0xB8], np.uint8), (N, K))
    sa = 2.0 ** rng.integers(-2, 3, (K // 128, M)).astype(np.float32)
    sw = 2.0 ** rng.integers(-2, 3, (2, K // 128)).astype(np.float32)
    y, _ = ref.fp8_gemm(qa, sa, qw, sw)
    got = run_gemm(qa, sa, qw, sw)
    assert np.array_equal(got, synth.f32_to_bf16_bits(y.astype(np.float32)))


def test_gemm_largest_codes():
    """+-448 everywhere: sums of the largest products stay finite and right."""
    M, N, K = 48, 128, 4096
    rng = np.random.default_rng(0)
    qa = np.full((M, K), 0x7E, np.uint8)
    qw = np.where(rng.random((N, K)) < 0.25, 0xFE, 0x7E).astype(np.uint8)
    sa, sw = np.full((K // 128, M), 0.37, np.float32), np.full((1, K // 128), 1.9, np.float32)
    y, tol = ref.fp8_gemm(qa, sa, qw, sw)
    ref.assert_gemm(run_gemm(qa, sa, qw, sw), y, tol, "largest codes")


@pytest.mark.parametrize("M", [4, 100])
def test_gemm_nan_stays_with_its_token(M):
    N, K = 136, 384
    rng = np.random.default_rng(M)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    clean = run_gemm(qa, sa, qw, sw)
    qa[2, 200] = 0x7F
    sa[1, 3] = np.inf
    got = bf16_to_f64(run_gemm(qa, sa, qw, sw))
    assert np.all(~np.isfinite(got[2])) and np.all(~np.isfinite(got[3]))
    keep = [m for m in range(M) if m not in (2, 3)]
    assert np.array_equal(got[keep], bf16_to_f64(clean)[keep])


@pytest.mark.parametrize("M,K", [(1, 128), (1, 4096), (3, 2176), (5, 8192), (2, 8320), (4, 18944), (3, 33024), (130, 384)])
@pytest.mark.parametrize("norm", [False, True])
def test_prologue_matches_reference(M, K, norm):
    rng = np.random.default_rng(M + K + norm)
    x = ref.bf16(rng, M, K + 16)
    x[:, 3] = synth.f32_to_bf16_bits(np.full(M, 25.0, np.float32))
    x[0, :128] = 0  # (without the norm: scale 0, codes 0)
    gamma = rng.uniform(0.5, 1.5, K).astype(np.float32) if norm else None
    codes, scales = dev(np.full((M + 1, K), 0x55, np.uint8)), dev(np.full((K // 128, -(-M // 4) * 4), -1, np.float32))
    fq.fq_fp8_prologue(dev(x), M, K, K + 16, None if gamma is None else dev(gamma), 1e-6, codes, scales)
    h = bf16_to_f64(x[:, :K])
    if norm:
        h = ref.rms(h, 1e-6) * gamma
    q, s = ref.quant_rows(h)
    got, gs = host(codes), host(scales)
    assert np.all(got[M] == 0x55) and np.all(gs[:, M:] == -1), "wrote past the last token"
    ref.assert_codes8(got[:M], gs[:, :M], q, s, f"prologue {M}x{K} norm={norm}")
    assert np.all(got[0, :128] & 0x7F == 0) and gs[0, 0] == 0


def test_prologue_exact_without_norm():
    """No norm: quotients are single IEEE divisions, so codes and scales are the reference's bit for bit,
    at every magnitude a bf16 input can have."""
    rng = np.random.default_rng(5)
    M, K = 64, 1024
    x = ref.bf16(rng, M, K)
    for m in range(M):  # tokens from 2^-126 up to 2^126
        x[m] = synth.f32_to_bf16_bits(synth.bf16_bits_to_f32(x[m]) * np.float32(2.0) ** np.float32(-126 + 4 * (m % 63)))
    codes, scales = dev(np.zeros((M, K), np.uint8)), dev(np.zeros((K // 128, M), np.float32))
    fq.fq_fp8_prologue(dev(x), M, K, K, None, 0.0, codes, scales)
    v = synth.bf16_bits_to_f32(x).reshape(M, K // 128, 128)
    s = (np.abs(v).max(-1) / np.float32(448)).astype(np.float32)
    quot = np.divide(v, s[..., None], out=np.zeros_like(v), where=s[..., None] > 0)  # float32 division
    q = ref.e4m3_round(quot.astype(np.float64)).reshape(M, K)
    assert np.array_equal(host(scales), s.T)
    assert np.array_equal(ref.TABLE[host(codes)], ref.TABLE[q])


LINEAR = [(1, 128, 8), (1, 2048, 4104), (1, 3584, 1000), (1, 4224, 264), (1, 18944, 136), (2, 256, 512), (16, 256, 512),
          (23, 2048, 264), (32, 1152, 72), (33, 384, 264), (130, 1024, 392), (300, 640, 1032)]


@pytest.mark.parametrize("M,K,N", LINEAR)
@pytest.mark.parametrize("norm,extras", [(True, False), (False, True)])
def test_linear_matches_its_own_codes(M, K, N, norm, extras):
    """fq_fp8_linear's codes against the prologue's reference, its outputs against those codes."""
    rng = np.random.default_rng(M + K + N)
    x = ref.bf16(rng, M, K)
    x[:, K // 2] = synth.f32_to_bf16_bits(np.full(M, -30.0, np.float32))
    gamma = rng.uniform(0.5, 1.5, K).astype(np.float32) if norm else None
    bias = rng.standard_normal(N).astype(np.float32) if extras else None
    residual = ref.bf16(rng, M, N) if extras else None
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32), gamma=gamma, bias=bias)
    y = host(site.linear(dev(x), residual=None if residual is None else dev(residual)), np.uint16)
    codes, scales = site.workspace_codes(M)
    qa, sa = host(codes), host(scales)
    h = bf16_to_f64(x)
    if norm:
        h = ref.rms(h, 1e-6) * gamma
    ref.assert_codes8(qa, sa, *ref.quant_rows(h), what=f"linear {M}x{K}x{N}")
    want, tol = ref.fp8_gemm(qa, sa, host(site.codes), host(site.wscale), bias, residual)
    ref.assert_gemm(y, want, tol, "outputs")


def test_linear_uses_the_prologue_and_the_gemm():
    """One call equals the two calls: codes and scales bit for bit, outputs to the sum's order."""
    rng = np.random.default_rng(9)
    K, N = 2048, 520
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32), gamma=np.ones(K, np.float32))
    for M in (1, 5, 31, 33, 100):
        x = dev(ref.bf16(rng, M, K))
        y1 = host(site.linear(x, head_dim=40), np.uint16)
        c1, s1 = (host(t) for t in site.workspace_codes(M))
        codes, scales = site.prologue(x)
        assert np.array_equal(c1, host(codes)) and np.array_equal(s1, host(scales)[:, :M])
        y2 = host(site.gemm(codes, scales, M, head_dim=40), np.uint16)
        y, tol = ref.fp8_gemm(c1, s1, host(site.codes), host(site.wscale))
        for got in (y1, y2):
            ref.assert_gemm(got.transpose(1, 0, 2).reshape(M, N), y, tol, f"M={M}")


def test_linear_is_repeatable_and_leaves_its_inputs():
    rng = np.random.default_rng(11)
    K, N = 1024, 776
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32))
    for M in (1, 12, 200):
        xb = ref.bf16(rng, M, K)
        x = dev(xb)
        first = host(site.linear(x), np.uint16)
        for _ in range(3):
            assert np.array_equal(host(site.linear(x), np.uint16), first)
        assert np.array_equal(host(x, np.uint16), xb)


TILES = ["256x256", "256x128", "128x192", "128x160", "128x128", "128x96", "128x64", "64x128", "64x64"]


@pytest.mark.parametrize("tile", TILES)
def test_every_tile_shape(tile, hook):
    hook("fp8_tile=" + tile)
    rng = np.random.default_rng(len(tile))
    for M, N, K in ((33, 8, 128), (130, 264, 384), (257, 392, 256), (64, 520, 1152)):
        qa, sa, qw, sw = rand_site(rng, M, N, K)
        bias, residual = rng.standard_normal(N).astype(np.float32), ref.bf16(rng, M, N)
        y, tol = ref.fp8_gemm(qa, sa, qw, sw, bias, residual)
        ref.assert_gemm(run_gemm(qa, sa, qw, sw, bias, residual), y, tol, f"{tile} {M}x{N}x{K}")
        ref.assert_gemm(run_gemm(qa, sa, qw, sw, bias, residual, head_dim=8), y, tol, f"{tile} {M}x{N}x{K} heads")


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("K", [128, 256, 640])
def test_more_tiles_than_workgroups(tile, K, hook):
    """Each workgroup runs several tiles, its copies ahead into the next one; sampled outputs."""
    hook("fp8_tile=" + tile)
    M, N = (4101, 5000) if tile == "256x256" else (2053, 5000)
    rng = np.random.default_rng(K)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    got = run_gemm(qa, sa, qw, sw)
    rows = np.unique(np.concatenate([np.arange(0, M, 293), [M - 1]]))
    b = np.array([0, 1, 7, 20, 38])
    cols = (128 * b[:, None] + np.arange(128)).ravel()
    y, tol = ref.fp8_gemm(qa[rows], sa[:, rows], qw[cols], sw[b])
    ref.assert_gemm(got[np.ix_(rows, cols)], y, tol, f"{tile} K={K}")
    # every output of a workgroup's tiles: against a float32 product of the same codes, coarsely
    import torch
    tab = torch.from_numpy(ref.TABLE.astype(np.float32)).cuda()
    a = tab[torch.from_numpy(qa.astype(np.int64)).cuda()] * dev(sa).t().repeat_interleave(128, 1)
    w = tab[torch.from_numpy(qw.astype(np.int64)).cuda()] * dev(sw).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
    full = (a @ w.t()).cpu().numpy()
    g = bf16_to_f64(got)
    scale = np.sqrt(np.mean(full.astype(np.float64) ** 2))
    # the bf16 rounding (2^-8) and sums of products cut at 2^-13 of the largest of eight
    assert np.all(np.abs(g - full) <= 2.0 ** -7 * np.abs(full) + 2.0 ** -7 * scale)


def test_full_size_layers_sampled():
    """The gate+up decode layer, prefills of the qkv and down layers, on sampled outputs."""
    rng = np.random.default_rng(13)
    for M, K, N in ((1, 3584, 37888), (1024, 3584, 4608), (811, 16384, 2048)):
        qa, sa, qw, sw = rand_site(rng, M, N, K)
        got = run_gemm(qa, sa, qw, sw)
        rows = np.unique(np.concatenate([[0, M - 1], rng.integers(0, M, 6)]))
        b = np.unique(np.concatenate([[0, N // 128 - 1], rng.integers(0, N // 128, 2)]))  # whole blocks of rows
        cols = (128 * b[:, None] + np.arange(128)).ravel()
        y, tol = ref.fp8_gemm(qa[rows], sa[:, rows], qw[cols], sw[b])
        ref.assert_gemm(got[np.ix_(rows, cols)], y, tol, f"{M}x{K}x{N}")


@pytest.mark.parametrize("M,N,K", [(9, 16400, 256), (16, 12296, 1152), (32, 20008, 384), (1, 33000, 128)])
def test_few_tokens_and_wide_layers(M, N, K):
    """Up to 32 tokens where row groups outnumber CUs: both sides of the choice between the two products."""
    rng = np.random.default_rng(M + N + K)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    y, tol = ref.fp8_gemm(qa, sa, qw, sw)
    ref.assert_gemm(run_gemm(qa, sa, qw, sw), y, tol, f"gemm {M}x{N}x{K}")


@pytest.mark.parametrize("K,N", [(128, 16), (640, 4104), (1024, 4104), (1280, 4104), (3584, 4112), (4096, 40), (5120, 72),
                                 (8192, 4104), (8320, 40), (16512, 24), (32768, 16), (33024, 8)])
@pytest.mark.parametrize("norm", [False, True])
def test_one_token_linear(K, N, norm):
    """One token: the codes and scales are the prologue's bit for bit, the outputs those codes' products."""
    rng = np.random.default_rng(K + N + norm)
    gamma = rng.uniform(0.5, 1.5, K).astype(np.float32) if norm else None
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32), gamma=gamma,
                      bias=rng.standard_normal(N).astype(np.float32))
    x, residual = dev(ref.bf16(rng, 1, K)), ref.bf16(rng, 1, N)
    y = host(site.linear(x, residual=dev(residual)), np.uint16)
    codes, scales = (host(t) for t in site.workspace_codes(1))
    want_codes, want_scales = (host(t) for t in site.prologue(x))
    assert np.array_equal(codes, want_codes) and np.array_equal(scales, want_scales[:, :1])
    want, tol = ref.fp8_gemm(codes, scales, host(site.codes), host(site.wscale), host(site.bias), residual)
    ref.assert_gemm(y, want, tol, f"K={K} N={N} norm={norm}")


@pytest.mark.parametrize("tile", ["256x256", "64x64"])
def test_tiles_take_single_tokens_too(tile, hook):
    hook("fp8_tile=" + tile)
    rng = np.random.default_rng(17)
    for M, N, K in ((1, 264, 384), (5, 8, 128), (32, 72, 640)):
        qa, sa, qw, sw = rand_site(rng, M, N, K)
        y, tol = ref.fp8_gemm(qa, sa, qw, sw)
        ref.assert_gemm(run_gemm(qa, sa, qw, sw), y, tol, f"{tile} {M}x{N}x{K}")


@pytest.mark.parametrize("M,K,N", [(2, 128, 8), (3, 640, 4112), (5, 1408, 72), (8, 512, 4104), (7, 1024, 40), (4, 4096, 264),
                                   (2, 8192, 72), (16, 256, 512), (9, 896, 4104), (3, 5248, 24), (17, 384, 4120),
                                   (32, 512, 136), (32, 1024, 72), (5, 4096, 24), (2, 4096, 4104)])
@pytest.mark.parametrize("norm", [False, True])
def test_few_tokens_linear(M, K, N, norm):
    """A few tokens, strided, in one launch or two: codes and scales are the prologue's bit for bit."""
    rng = np.random.default_rng(M + K + N + norm)
    gamma = rng.uniform(0.5, 1.5, K).astype(np.float32) if norm else None
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32), gamma=gamma)
    x, residual = dev(ref.bf16(rng, M, K + 24)), ref.bf16(rng, M, N)
    x = x[:, :K]
    y = host(site.linear(x, residual=dev(residual)), np.uint16)
    codes, scales = (host(t) for t in site.workspace_codes(M))
    want_codes, want_scales = (host(t) for t in site.prologue(x))
    assert np.array_equal(codes, want_codes) and np.array_equal(scales, want_scales[:, :M])
    want, tol = ref.fp8_gemm(codes, scales, host(site.codes), host(site.wscale), None, residual)
    ref.assert_gemm(y, want, tol, f"M={M} K={K} N={N} norm={norm}")


@pytest.mark.parametrize("M", [17, 24, 32])
@pytest.mark.parametrize("N,K", [(2048, 384), (2056, 1152), (24, 2176), (4096, 128)])
def test_two_token_tiles_of_narrow_layers(M, N, K):
    """Either side of the choice to give the second tile of 16 tokens workgroups of its own."""
    rng = np.random.default_rng(M + N + K)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    residual = ref.bf16(rng, M, N)
    y, tol = ref.fp8_gemm(qa, sa, qw, sw, None, residual)
    ref.assert_gemm(run_gemm(qa, sa, qw, sw, None, residual), y, tol, f"gemm {M}x{N}x{K}")


@pytest.mark.parametrize("M,K,N", [(2, 4096, 64), (17, 16384, 136), (23, 18944, 72), (40, 4096, 1032), (64, 8192, 520), (65, 5120, 264),
                                   (130, 9728, 896), (200, 16384, 512), (33, 5248, 264), (1024, 8192, 64), (2050, 4096, 16), (3, 65536, 40)])
@pytest.mark.parametrize("head_dim", [0, 8])
def test_long_narrow_layers(M, K, N, head_dim):
    """Few tiles of long sums: K in parts that meet in the workspace."""
    rng = np.random.default_rng(M + K + N)
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32), gamma=rng.uniform(0.5, 1.5, K).astype(np.float32),
                      bias=rng.standard_normal(N).astype(np.float32))
    x, residual = dev(ref.bf16(rng, M, K)), ref.bf16(rng, M, N + 8)
    site.workspace(M).fill_(0xFF)  # (NaN patterns wherever a part is not written)
    y = torch.full((N // 8, M, 8) if head_dim else (M + 1, N + 16), 77, dtype=torch.int16, device="cuda")
    site.linear(x, residual=dev(residual), head_dim=head_dim, y=y[:M, :N] if not head_dim else y)
    codes, scales = (host(t) for t in site.workspace_codes(M))
    want, tol = ref.fp8_gemm(codes, scales, host(site.codes), host(site.wscale), host(site.bias), residual[:, :N])
    got = host(y, np.uint16)
    if head_dim:
        got = got.transpose(1, 0, 2).reshape(M, N)
    else:
        assert np.all(got[M:] == 77) and np.all(got[:, N:] == 77), "wrote outside its rows"
    ref.assert_gemm(got[:M, :N], want, tol, f"M={M} K={K} N={N}")


@pytest.mark.parametrize("M,K,N", [(1, 512, 264), (3, 640, 72), (20, 1152, 2056), (40, 512, 264), (140, 640, 520), (300, 256, 1032),
                                   (48, 8192, 136)])
def test_output_over_its_residual(M, K, N):
    """y = residual: each output replaces the value that it added."""
    rng = np.random.default_rng(M + K + N)
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32))
    x, residual = dev(ref.bf16(rng, M, K)), dev(ref.bf16(rng, M, N))
    want = host(site.linear(x, residual=residual))
    y = residual.clone()
    assert np.array_equal(host(site.linear(x, residual=y, y=y)), want)
    codes, scales = site.prologue(x)
    want = host(site.gemm(codes, scales, M, residual=residual))
    y = residual.clone()
    assert np.array_equal(host(site.gemm(codes, scales, M, residual=y, y=y)), want)


@pytest.mark.parametrize("M,N,K", [(33, 264, 384), (47, 1024, 640), (64, 2048, 256), (65, 512, 1152), (100, 1024, 384),
                                   (128, 512, 2176), (255, 256, 512), (300, 64, 128), (1000, 24, 384)])
def test_many_tokens_of_narrow_layers(M, N, K):
    """More than 32 tokens that the GEMV may take, in tiles of 16 or 32, the last one ragged."""
    rng = np.random.default_rng(M + N + K)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    bias, residual = rng.standard_normal(N).astype(np.float32), ref.bf16(rng, M, N)
    y, tol = ref.fp8_gemm(qa, sa, qw, sw, bias, residual)
    ref.assert_gemm(run_gemm(qa, sa, qw, sw, bias, residual), y, tol, f"gemm {M}x{N}x{K}")
    ref.assert_gemm(run_gemm(qa, sa, qw, sw, bias, residual, head_dim=8), y, tol, f"gemm {M}x{N}x{K} heads")


@pytest.mark.parametrize("M,N,K", [(1, 72, 4224), (1, 264, 8192), (2, 136, 5120), (3, 40, 5248), (1, 24, 16384), (2, 16, 8192),
                                   (1, 4104, 4352), (1, 8, 32768), (1, 8, 32896), (4, 24, 4224), (3, 16, 8192)])
def test_few_tokens_of_long_sums(M, N, K):
    """A few tokens' codes through LDS where K is long, and the calls beside that choice."""
    rng = np.random.default_rng(M + N + K)
    qa, sa, qw, sw = rand_site(rng, M, N, K)
    bias, residual = rng.standard_normal(N).astype(np.float32), ref.bf16(rng, M, N)
    y, tol = ref.fp8_gemm(qa, sa, qw, sw, bias, residual)
    ref.assert_gemm(run_gemm(qa, sa, qw, sw, bias, residual), y, tol, f"gemm {M}x{N}x{K}")
    ref.assert_gemm(run_gemm(qa, sa, qw, sw, bias, residual, head_dim=8), y, tol, f"gemm {M}x{N}x{K} heads")
