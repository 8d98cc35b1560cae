"""What a site refuses before it hands a pointer to the library: tensors of another type, shape, layout or device.
The sites are built on the CPU; calls that pass every check end at the binding, which takes GPU tensors only."""
import numpy as np
import pytest
import torch

import w4a4_integer_gemm_amd as fq

N, K, M = 264, 256, 5


@pytest.fixture(scope="module")
def site():
    return fq.Fp8Site(np.ones((N, K), np.float32), gamma=np.ones(K, np.float32), bias=np.zeros(N, np.float32), device="cpu")


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


GOOD_X = [bf16(M, K), bf16(M, K).view(torch.int16), bf16(M, K + 8)[:, :K], bf16(1, K)]


@pytest.mark.parametrize("x", GOOD_X)
@pytest.mark.parametrize("call", ["linear", "prologue"])
def test_good_rows_reach_the_binding(site, x, call):
    with pytest.raises(ValueError, match="GPU tensors"):
        getattr(site, call)(x)


def test_good_outputs_and_residuals_reach_the_binding(site):
    x = bf16(M, K)
    codes, scales = site.empty_codes(M)
    for kw in (dict(y=bf16(M, N)), dict(y=bf16(M + 1, N + 16)), dict(residual=bf16(M, N + 8)), dict(head_dim=8),
               dict(head_dim=8, y=bf16(N // 8, M, 8), residual=bf16(M, N)), dict(head_dim=8, y=bf16(M * N))):
        with pytest.raises(ValueError, match="GPU tensors"):
            site.linear(x, **kw)
        with pytest.raises(ValueError, match="GPU tensors"):
            site.gemm(codes, scales, M, **kw)
        with pytest.raises(ValueError, match="GPU tensors"):
            site.gemm(codes.view(torch.float8_e4m3fn), scales[:, :M], M, **kw)
        with pytest.raises(ValueError, match="GPU tensors"):
            site.gemm(codes.flatten(), scales.flatten(), M, **kw)


@pytest.mark.parametrize("x,match", [
    (torch.zeros(M, K), "x has dtype torch.float32"),
    (torch.zeros(M, K, dtype=torch.float16), "x has dtype torch.float16"),
    (bf16(M, K + 8), f"x is {M} x {K + 8}, not {M} x {K}"),
    (bf16(M, K - 128), f"x is {M} x {K - 128}"),
    (bf16(K), "x has 1 dimensions"),
    (bf16(1, M, K), "x has 3 dimensions"),
    (bf16(K, M).t(), f"x has stride {M} along its rows"),
    (bf16(M, K).to("meta"), "x is on meta, the site on cpu"),
])
@pytest.mark.parametrize("call", ["linear", "prologue"])
def test_rows_are_refused(site, x, match, call):
    with pytest.raises(ValueError, match=match):
        getattr(site, call)(x)


@pytest.mark.parametrize("kw,match", [
    (dict(residual=torch.zeros(M, N)), "residual has dtype torch.float32"),
    (dict(residual=bf16(M - 1, N)), f"residual is {M - 1} x {N}, not {M} x {N}"),
    (dict(residual=bf16(M, N - 8)), f"residual is {M} x {N - 8}"),
    (dict(residual=bf16(N, M).t()), "residual has stride"),
    (dict(y=torch.zeros(M, N)), "y has dtype torch.float32"),
    (dict(y=bf16(M - 1, N)), f"y is {M - 1} x {N}"),
    (dict(y=bf16(M, N - 8)), f"y is {M} x {N - 8}"),
    (dict(y=bf16(N // 8, M, 8)), "y has 3 dimensions"),
    (dict(y=bf16(M, N), head_dim=8), r"y is \(5, 264\)"),
    (dict(y=bf16(N // 8, M - 1, 8), head_dim=8), r"y is \(33, 4, 8\)"),
    (dict(y=bf16(N // 8, M, 16)[..., :8], head_dim=8), "contiguous"),
    (dict(y=bf16(M * N - 1), head_dim=8), r"y is \(1319,\)"),
    (dict(y=bf16(M, N).to("meta")), "y is on meta"),
    (dict(y=torch.zeros(N // 8, M, 8), head_dim=8), "y is torch.float32 on cpu"),
])
def test_outputs_and_residuals_are_refused(site, kw, match):
    with pytest.raises(ValueError, match=match):
        site.linear(bf16(M, K), **kw)
    codes, scales = site.empty_codes(M)
    with pytest.raises(ValueError, match=match):
        site.gemm(codes, scales, M, **kw)


@pytest.mark.parametrize("codes,scales,match", [
    (bf16(M, K), torch.zeros(2, 8), "codes are 5 x 256 bytes"),
    (torch.zeros(M, K - 128, dtype=torch.uint8), torch.zeros(2, 8), "codes are"),
    (torch.zeros(M, K + 128, dtype=torch.uint8)[:, :K], torch.zeros(2, 8), "codes are"),
    (torch.zeros(M, K, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.float64), "scales are float32 2 x 5 in rows of 8"),
    (torch.zeros(M, K, dtype=torch.uint8), torch.zeros(2, 5), "scales are"),
    (torch.zeros(M, K, dtype=torch.uint8), torch.zeros(1, 8), "scales are"),
    (torch.zeros(M, K, dtype=torch.uint8), torch.zeros(2, 8)[:, :4], "scales are"),
    (torch.zeros(M, K, dtype=torch.uint8), torch.zeros(15), "scales are"),
    (torch.zeros(M, K, dtype=torch.uint8), torch.zeros(32)[::2], "scales are"),
    (torch.zeros(M * K - 1, dtype=torch.uint8), torch.zeros(2, 8), "codes are"),
    (torch.zeros(M, K, dtype=torch.uint8), torch.zeros(2, 8, device="meta"), "the site on cpu"),
])
def test_codes_and_scales_are_refused(site, codes, scales, match):
    with pytest.raises(ValueError, match=match):
        site.gemm(codes, scales, M)
    with pytest.raises(ValueError, match=match):
        site.prologue(bf16(M, K), codes, scales)


def test_a_call_on_another_current_device_is_refused(site, monkeypatch):
    codes, scales = site.empty_codes(M)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    far = fq.Fp8Site(np.ones((N, K), np.float32), device="cpu")
    far.device = torch.device("cuda", 1)
    monkeypatch.setattr("w4a4_integer_gemm_amd.site._rows", lambda *a, **k: K)
    monkeypatch.setattr(far, "_check_codes", lambda *a: None)
    for call in (lambda: far.linear(bf16(M, K)), lambda: far.prologue(bf16(M, K)), lambda: far.gemm(codes, scales, M)):
        with pytest.raises(ValueError, match="the site is on cuda:1, the current device is 0"):
            call()


@pytest.mark.parametrize("kw,match", [
    (dict(W=np.ones((8, K), np.float32), gamma=np.ones(K - 128, np.float32)), "gamma has shape"),
    (dict(W=np.ones((8, K), np.float32), bias=np.ones(16, np.float32)), "bias has shape"),
    (dict(codes=np.zeros((8, K), np.uint8)), "come with wscale"),
    (dict(codes=np.zeros(K, np.uint8), wscale=np.zeros(2, np.float32)), "codes are a matrix"),
    (dict(codes=torch.zeros(8, K, dtype=torch.uint8), wscale=torch.zeros(1, 2, device="meta")), "wscale is on meta"),
])
def test_parameters_are_refused(kw, match):
    with pytest.raises(ValueError, match=match):
        fq.Fp8Site(device="cpu", **kw)


# ------------------------------------------------------------------ the integer sites
@pytest.fixture(scope="module", params=[(8, 8), (4, 4)])
def integer_site(request):
    wbits, abits = request.param
    return fq.DeviceSite(np.ones((N, K), np.float32), 64, wbits, abits, gamma=np.ones(K, np.float32), device="cpu")


@pytest.mark.parametrize("x", GOOD_X + [bf16(M, K + 8)])
def test_good_integer_calls_reach_the_binding(integer_site, x):
    s, m = integer_site, x.shape[0]
    codes, scales = s.empty_codes(m)
    y, res = bf16(m + 1, N + 16), bf16(m, N + 8)
    for call in (lambda: s.prologue(x), lambda: s.prologue(x, codes, scales), lambda: s.linear(x, residual=res, y=y),
                 lambda: s.linear_noalloc(x), lambda: s.linear_heads(x, 8, residual=res),
                 lambda: s.linear_heads(x, 8, y=bf16(N // 8, m, 8)), lambda: s.gemm(codes, scales, m, residual=res, y=y),
                 lambda: s.gemm(codes, scales, m, acc=torch.zeros(m, N, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()


@pytest.mark.parametrize("x,match", [
    (torch.zeros(M, K), "x has dtype torch.float32"),
    (bf16(M, K - 64), f"x is {M} x {K - 64}, not {M} x {K}"),
    (bf16(1, M, K), "x has 3 dimensions"),
    (bf16(K, M).t(), "x has stride"),
    (bf16(M, K).to("meta"), "x is on meta, the site on cpu"),
])
def test_integer_rows_are_refused(integer_site, x, match):
    s = integer_site
    for call in (s.linear, s.linear_noalloc, s.prologue, lambda v: s.linear_heads(v, 8)):
        with pytest.raises(ValueError, match=match):
            call(x)


@pytest.mark.parametrize("kw,match", [
    (dict(residual=torch.zeros(M, N)), "residual has dtype torch.float32"),
    (dict(residual=bf16(M - 1, N)), f"residual is {M - 1} x {N}, not {M} x {N}"),
    (dict(y=bf16(M - 1, N)), f"y is {M - 1} x {N}"),
    (dict(y=bf16(M, N - 8)), f"y is {M} x {N - 8}"),
])
def test_integer_outputs_and_residuals_are_refused(integer_site, kw, match):
    s, x = integer_site, bf16(M, K)
    codes, scales = s.empty_codes(M)
    for call in (lambda: s.linear(x, **kw), lambda: s.linear_noalloc(x, **kw), lambda: s.gemm(codes, scales, M, **kw)):
        with pytest.raises(ValueError, match=match):
            call()


def test_integer_codes_heads_and_sums_are_refused(integer_site):
    s, x = integer_site, bf16(M, K)
    codes, scales = s.empty_codes(M)
    for c, sc, match in ((codes[:-1], scales, "codes are"), (codes, scales[:-1], "scales are"),
                         (codes, scales.to(torch.float64), "scales are"), (codes, scales.to("meta"), "the site on cpu")):
        with pytest.raises(ValueError, match=match):
            s.prologue(x, c, sc)
        with pytest.raises(ValueError, match=match):
            s.gemm(c, sc, M)
    with pytest.raises(ValueError, match=f"acc is {M} x {N} int32"):
        s.gemm(codes, scales, M, acc=torch.zeros(M - 1, N, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        s.linear_heads(x, 8, y=bf16(N // 8, M, 16)[..., :8])
    with pytest.raises(ValueError, match=r"y is \(33, 4, 8\)"):
        s.linear_heads(x, 8, y=bf16(N // 8, M - 1, 8))


@pytest.mark.parametrize("kw", [dict(gamma=np.ones(K - 64, np.float32)), dict(bias=np.ones(N + 8, np.float32)),
                                dict(ascale=np.ones(K + 64, np.float32))])
def test_integer_parameters_are_refused(kw):
    with pytest.raises(ValueError, match=f"{next(iter(kw))} has shape"):
        fq.DeviceSite(np.ones((N, K), np.float32), 64, 8, 8, device="cpu", **kw)
