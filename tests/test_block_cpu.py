"""CPU checks of the operators around the integer sites: the FP8 packer and the
rotary plan against plain 64-bit references, buffer sizes, and the refusals of
every entry point (before any device work)."""
import re
from fractions import Fraction

import numpy as np
import pytest

import blockref as ref
import w4a4_integer_gemm_amd as fq

DEV, BAD = 0x10000, 0x10001  # aligned and misaligned "device pointers"; validation never reads them
WS = 0x100000


# ------------------------------------------------------------------ FP8 host parts
def test_e4m3_table_matches_torch():
    import torch
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(ref.TABLE, t, equal_nan=True)


@pytest.mark.parametrize("N,K", [(1, 128), (128, 128), (130, 384), (256, 256), (385, 640)])
def test_fp8_packer_matches_reference(N, K):
    rng = np.random.default_rng(N + K)
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    W[:, 5] *= 40
    W[N // 2, K // 2] = -3.0
    W[:, K - 128:][:128] = 0.0  # a block of zeros: scale 0, codes 0
    codes, s = fq.fq_fp8_pack_weights(W)
    assert s.shape == (-(-N // 128), K // 128) and fq.fq_fp8_wscale_count(N, K) == s.size
    for b in range(s.shape[0]):
        for g in range(s.shape[1]):
            blk = W[128 * b:128 * b + 128, 128 * g:128 * g + 128].astype(np.float64)
            sd = np.float32(np.abs(blk).max() / 448.0)
            assert s[b, g] == sd
            want = ref.e4m3_round(blk / np.float64(sd)) if sd > 0 else np.zeros(blk.shape, np.uint8)
            assert np.array_equal(codes[128 * b:128 * b + 128, 128 * g:128 * g + 128], want)
    back = fq.fq_fp8_dequant_rows(codes, s)
    full = ref.TABLE[codes] * np.repeat(np.repeat(s.astype(np.float64), 128, 0)[:N], 128, 1)
    assert np.array_equal(back, full.astype(np.float32))


def test_fp8_packer_rounds_ties_to_even_and_keeps_subnormals():
    W = np.zeros((1, 128), np.float32)
    W[0, 0] = 448.0  # scale 1
    v = np.concatenate([ref._MID[::2], -ref._MID[1::2]])
    W[0, 1:1 + v.size] = v
    codes, s = fq.fq_fp8_pack_weights(W)
    assert s[0, 0] == 1.0
    assert np.array_equal(codes[0], ref.e4m3_round(W[0].astype(np.float64)))
    assert np.all(codes[0, 1:1 + v.size] % 2 == 0)


@pytest.mark.parametrize("amax", [3e38, 1e-30, 1e-41, 1e-45])
def test_fp8_packer_extreme_scales(amax):
    W = np.zeros((2, 128), np.float32)
    W[0, :4] = np.array([1, -1, 0.5, 0.25]) * np.float32(amax)
    codes, s = fq.fq_fp8_pack_weights(W)
    sd = np.float32(np.float64(np.abs(W).max()) / 448.0)
    assert s[0, 0] == sd
    want = ref.e4m3_round(W.astype(np.float64) / np.float64(sd)) if sd > 0 else np.zeros_like(codes)
    assert np.array_equal(codes, want)
    assert not np.any((codes & 0x7F) == 0x7F)


def test_fp8_dequant_keeps_nan_codes():
    codes = np.full((1, 128), 0x7F, np.uint8)
    assert np.all(np.isnan(fq.fq_fp8_dequant_rows(codes, np.ones((1, 1), np.float32))))


def test_fp8_sizes():
    assert fq.fq_fp8_wscale_count(4608, 3584) == 36 * 28
    assert fq.fq_fp8_wscale_count(129, 128) == 2
    assert fq.fq_fp8_ascale_count(5, 256) == 2 * 8
    assert fq.fq_fp8_wscale_count(0, 128) == 0 and fq.fq_fp8_wscale_count(8, 100) == 0
    assert fq.fq_fp8_ascale_count(0, 128) == 0 and fq.fq_fp8_ascale_count(1, 131072) == 0
    assert fq.fq_fp8_linear_workspace_bytes(3, 256) == 768 + 256
    assert fq.fq_fp8_linear_workspace_bytes(70000, 65536) >= 70000 * 65536  # past 32 bits
    assert fq.fq_fp8_linear_workspace_bytes(3, 200) == 0
    assert fq.fq_fp8_ascale_count(2 ** 31 - 513, 128) == 2 ** 31 - 512 and fq.fq_fp8_ascale_count(2 ** 31 - 512, 128) == 0


def test_fp8_workspace_has_room_for_parts():
    """Long sums of two tokens and more: 256 tiles of 128 x 128 floats behind the codes and scales."""
    for M, K in ((2, 4096), (1024, 65536), (37, 5120)):
        codes = -(-M * K // 256) * 256
        scales = -(-4 * fq.fq_fp8_ascale_count(M, K) // 256) * 256
        assert fq.fq_fp8_linear_workspace_bytes(M, K) == codes + scales + (16 << 20)
    assert fq.fq_fp8_linear_workspace_bytes(1, 4096) == 4096 + 512
    assert fq.fq_fp8_linear_workspace_bytes(64, 3968) < 1 << 20
    sizes = [fq.fq_fp8_linear_workspace_bytes(M, K) for M in (1, 2, 3, 31, 32, 33, 64, 1024, 1025, 5000)
             for K in (128, 3968, 4096, 4224, 65536)]
    for at in range(5):  # a workspace for the most tokens and the longest K serves every call
        assert sizes[at::5] == sorted(sizes[at::5])
    for at in range(0, len(sizes), 5):
        assert sizes[at:at + 5] == sorted(sizes[at:at + 5])


def test_fp8_tile_hook_parses_and_rejects():
    names = ("256x256", "256x128", "128x192", "128x160", "128x128", "128x96", "128x64", "64x128", "64x64", "auto")
    for name in names:
        fq.fq_test_hook("fp8_tile=" + name)
    with pytest.raises(fq.FqError, match="unknown fp8_tile '32x32'"):
        fq.fq_test_hook("fp8_tile=32x32")
    fq.fq_test_hook("")


@pytest.mark.parametrize("W,match", [
    (np.full((2, 128), np.nan, np.float32), r"W\[\d\]\[\d+\] is not finite"),
    (np.full((2, 128), np.inf, np.float32), "is not finite"),
    (np.zeros((2, 100), np.float32), "K=100"),
    (np.zeros((2, 192), np.float32), r"K=192 is not a multiple of 128 \(192/128 = 1.50\)"),
])
def test_fp8_packer_refuses(W, match):
    with pytest.raises(fq.FqError, match=match):
        fq.fq_fp8_pack_weights(W)


def test_fp8_host_null_arguments():
    L = fq.lib()
    assert L.fq_fp8_pack_weights(None, 1, 128, DEV, DEV) == 1
    assert L.fq_fp8_dequant_rows(None, DEV, 1, 128, DEV) == 1
    with pytest.raises(ValueError, match="wscale has 1 values, not 2"):
        fq.fq_fp8_dequant_rows(np.zeros((129, 128), np.uint8), np.ones((1, 1), np.float32))


# ------------------------------------------------------------------ rotary plan
KINDS = [(fq.ROPE_PLAIN, {}), (fq.ROPE_LINEAR, dict(factor=4.0)), (fq.ROPE_BASE, dict(factor=8.0)),
         (fq.ROPE_BANDS, dict(factor=8.0, trained_len=8192, low=1.0, high=4.0)),
         (fq.ROPE_RAMP, dict(factor=16.0, trained_len=4096, low=1.0, high=32.0))]


@pytest.mark.parametrize("rot", [4, 20, 64, 128, 256])
@pytest.mark.parametrize("kind,kw", KINDS)
@pytest.mark.parametrize("base", [10000.0, 1e6])
def test_rope_plan_matches_definition(rot, kind, kw, base):
    freq, scale = fq.fq_rope_freqs(rot, base, kind, **kw)
    th, want = ref.rope_theta(rot, base, kind, kw.get("factor", 1.0), kw.get("trained_len", 1), kw.get("low", 1.0),
                              kw.get("high", 32.0))
    assert scale == np.float32(want)
    # the float64 reference is itself off by some 2^-50 relative (pow and log);
    # an entry is a multiple of 2^-64 turns, so it is off by up to half of that too
    turns = freq.astype(np.float64) / 2.0 ** 64
    assert np.all(np.abs(turns - th / (2 * np.pi)) <= 2.0 ** -46 * th + 2.0 ** -64)


def test_rope_plan_pair_factors_and_first_pair():
    pf = np.array([1.0, 2.0, 0.05, 8.0], np.float32)
    freq, scale = fq.fq_rope_freqs(8, 10000.0, fq.ROPE_PAIRS, pair_factors=pf)
    th, _ = ref.rope_theta(8, 10000.0, 5, pair=pf)
    assert scale == 1.0
    assert np.all(np.abs(freq.astype(np.float64) / 2.0 ** 64 - (th / (2 * np.pi)) % 1.0) < 2.0 ** -45)
    # pair 0 of the plain rule turns by exactly 1 radian: 1 / (2 pi) turns, to 2^-63
    inv_two_pi = Fraction(1) / (2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459"))
    freq, _ = fq.fq_rope_freqs(2)
    assert abs(Fraction(int(freq[0]), 2 ** 64) - inv_two_pi) < Fraction(1, 2 ** 63)


@pytest.mark.parametrize("kw,match", [
    (dict(rot_dim=7), "rot_dim=7 must be even"),
    (dict(rot_dim=0), "rot_dim=0"),
    (dict(base=1.0), "base=1"),
    (dict(base=float("inf")), "base=inf"),
    (dict(kind=9), "kind=9 is not a scaling rule"),
    (dict(kind=fq.ROPE_LINEAR, factor=0.5), "factor=0.5"),
    (dict(kind=fq.ROPE_BASE, rot_dim=2, factor=2.0), "rot_dim=2 must be at least 4"),
    (dict(kind=fq.ROPE_BANDS, factor=2.0, trained_len=0), "trained_len=0"),
    (dict(kind=fq.ROPE_RAMP, factor=2.0, low=4.0, high=4.0), "0 < low < high"),
    (dict(kind=fq.ROPE_PAIRS), "pair_factors is NULL"),
    (dict(kind=fq.ROPE_PAIRS, pair_factors=np.zeros(4, np.float32)), r"pair_factors\[0\]=0"),
])
def test_rope_plan_refuses(kw, match):
    a = dict(rot_dim=8)
    a.update(kw)
    with pytest.raises(fq.FqError, match=match):
        fq.fq_rope_freqs(**a)


def test_rope_plan_checks_the_factor_count():
    with pytest.raises(ValueError, match="pair_factors has 3 values, not 4"):
        fq.fq_rope_freqs(8, kind=fq.ROPE_PAIRS, pair_factors=np.ones(3, np.float32))


# ------------------------------------------------------------------ refusals of the device calls
def refused(name, rc, status, match):
    assert rc == status, (rc, fq.last_error())
    msg = fq.last_error()
    assert msg.startswith(name + ":") and re.search(match, msg), msg


@pytest.mark.parametrize("kw,status,match", [
    (dict(x=None), 1, "x_bf16 is NULL"),
    (dict(codes=None), 1, "act_codes is NULL"),
    (dict(scale=None), 1, "act_scale is NULL"),
    (dict(M=0), 2, "M=0"),
    (dict(M=2 ** 31 - 1), 2, "M=2147483647"),
    (dict(M=2 ** 27), 2, "too many for one launch"),
    (dict(K=160, ldx=160), 2, r"K=160 is not a multiple of 128 \(160/128 = 1.25\)"),
    (dict(K=131072, ldx=131072), 2, "K=131072 outside"),
    (dict(ldx=248), 2, "ldx=248 < 256"),
    (dict(ldx=260), 4, "ldx=260 is not a multiple of 8"),
    (dict(eps=-1.0), 1, "eps=-1"),
    (dict(eps=float("nan")), 1, "eps=nan"),
    (dict(x=BAD), 4, "x_bf16 is not 16-byte aligned"),
    (dict(gamma=BAD), 4, "gamma is not 16-byte aligned"),
    (dict(scale=BAD), 4, "act_scale is not 16-byte aligned"),
])
def test_fp8_prologue_refuses(kw, status, match):
    a = dict(x=DEV, M=16, K=256, ldx=256, gamma=DEV, eps=1e-6, codes=DEV, scale=DEV)
    a.update(kw)
    refused("fq_fp8_prologue", fq.lib().fq_fp8_prologue(a["x"], a["M"], a["K"], a["ldx"], a["gamma"], a["eps"],
                                                        a["codes"], a["scale"], None), status, match)


GEMM_CASES = [
    (dict(w=None), 1, "w_codes is NULL"),
    (dict(sw=None), 1, "wscale is NULL"),
    (dict(y=None), 1, "y_bf16 is NULL"),
    (dict(M=0), 2, "M=0"),
    (dict(N=0), 2, "N=0"),
    (dict(N=100, ldy=104), 2, r"N=100 is not a positive multiple of 8 \(100/8 = 12.500\)"),
    (dict(K=64), 2, "K=64 outside"),
    (dict(K=192), 2, r"K=192 is not a multiple of 128"),
    (dict(M=2 ** 23, N=2 ** 23, ldy=2 ** 23), 2, "too large for one launch"),
    (dict(ldy=64), 2, "ldy=64 < 128"),
    (dict(ldy=132), 4, "ldy=132 is not a multiple of 8"),
    (dict(res=DEV, ldr=64), 2, "ldr=64 < 128"),
    (dict(res=BAD, ldr=128), 4, "residual_bf16 is not 16-byte aligned"),
    (dict(hd=-8), 2, "head_dim=-8"),
    (dict(hd=12), 2, "head_dim=12 is not a multiple of 8"),
    (dict(hd=48), 2, r"N=128 is not a whole number of heads of head_dim=48 \(128/48 = 2.667\)"),
    (dict(w=BAD), 4, "w_codes is not 16-byte aligned"),
    (dict(sw=BAD), 4, "wscale is not 4-byte aligned"),
    (dict(bias=BAD), 4, "bias is not 16-byte aligned"),
    (dict(y=BAD), 4, "y_bf16 is not 16-byte aligned"),
]


@pytest.mark.parametrize("kw,status,match", GEMM_CASES + [
    (dict(act=None), 1, "act_codes is NULL"), (dict(sa=None), 1, "act_scale is NULL"),
    (dict(act=BAD), 4, "act_codes is not 16-byte aligned"), (dict(sa=BAD), 4, "act_scale is not 16-byte aligned")])
def test_fp8_gemm_refuses(kw, status, match):
    a = dict(act=DEV, sa=DEV, M=16, w=DEV, sw=DEV, N=128, K=256, bias=None, res=None, ldr=0, hd=0, y=DEV, ldy=128)
    a.update(kw)
    refused("fq_fp8_gemm", fq.lib().fq_fp8_gemm(a["act"], a["sa"], a["M"], a["w"], a["sw"], a["N"], a["K"], a["bias"],
                                                a["res"], a["ldr"], a["hd"], a["y"], a["ldy"], None), status, match)


@pytest.mark.parametrize("kw,status,match", [c for c in GEMM_CASES if "K" not in c[0] and c[0].get("M") != 2 ** 23] + [
    (dict(ws=None), 1, "workspace is NULL"),
    (dict(ws=WS + 16), 4, "workspace is not 256-byte aligned"),
    (dict(wsb=100), 1, "workspace_bytes=100 < 4352 needed for M=16 K=256"),
    (dict(K=192, ldx=192), 2, "K=192 is not a multiple of 128"),
    (dict(x=BAD), 4, "x_bf16 is not 16-byte aligned"),
    (dict(ldx=128), 2, "ldx=128 < 256")])
def test_fp8_linear_refuses(kw, status, match):
    a = dict(x=DEV, M=16, K=256, ldx=256, gamma=DEV, eps=1e-6, w=DEV, sw=DEV, N=128, bias=None, res=None, ldr=0, hd=0,
             y=DEV, ldy=128, ws=WS, wsb=1 << 20)
    a.update(kw)
    refused("fq_fp8_linear", fq.lib().fq_fp8_linear(a["x"], a["M"], a["K"], a["ldx"], a["gamma"], a["eps"], a["w"],
                                                    a["sw"], a["N"], a["bias"], a["res"], a["ldr"], a["hd"], a["y"],
                                                    a["ldy"], a["ws"], a["wsb"], None), status, match)


@pytest.mark.parametrize("kw,status,match", [
    (dict(M=0), 2, "M=0"),
    (dict(K=12), 2, r"K=12 is not a multiple of 8"),
    (dict(K=65544), 2, "K=65544 outside"),
    (dict(q=DEV, sq=DEV, K=136, ld=136), 2, "K=136 is not a multiple of 128"),
    (dict(M=2 ** 30), 2, "too many for one launch"),
    (dict(f32=2), 1, "stream_f32=2"),
    (dict(r=None), 1, "stream_in is NULL"),
    (dict(x=None), 1, "post_gamma, gate_bf16 and stream_out need x_bf16"),
    (dict(x=None, pg=None, gate=None, ro=None, h=None, g=None, ms=None, mt=None), 1, "nothing to write"),
    (dict(ro=None), 1, "stream_out is NULL"),
    (dict(q=DEV), 1, "act_codes and act_scale come together"),
    (dict(sq=DEV), 1, "act_codes and act_scale come together"),
    (dict(h=None), 1, "need h_bf16 or act_codes"),
    (dict(ld=132), 4, "ld_in=132 is not a multiple of 8"),
    (dict(ld=124, f32=1), 2, "ld_in=124 < 128"),
    (dict(ldx=120), 2, "ldx=120 < 128"),
    (dict(ro=DEV, ldo=136), 2, "in place needs ld_out=136 equal to ld_in=128"),
    (dict(c=float("nan")), 1, "res_scale=nan"),
    (dict(pe=-1.0), 1, "post_eps=-1"),
    (dict(e=float("inf")), 1, "pre_eps=inf"),
    (dict(per=0), 2, "rows_per_cond=0"),
    (dict(ldg=64), 2, "ld_gate=64 < 128"),
    (dict(ldm=132), 4, "ld_mod=132 is not a multiple of 8"),
    (dict(h=BAD), 4, "h_bf16 is not 16-byte aligned"),
    (dict(pg=BAD), 4, "post_gamma is not 16-byte aligned"),
    (dict(mt=BAD), 4, "mod_shift_bf16 is not 16-byte aligned"),
])
def test_block_norm_refuses(kw, status, match):
    a = dict(M=4, K=128, x=DEV, ldx=128, pg=DEV, pe=1e-6, gate=DEV, ldg=128, c=1.0, r=DEV, ld=128, ro=2 * DEV, ldo=128,
             f32=0, g=DEV, e=1e-6, ms=DEV, mt=DEV, ldm=128, per=2, h=DEV, ldh=128, q=None, sq=None)
    a.update(kw)
    refused("fq_block_norm", fq.lib().fq_block_norm(
        a["M"], a["K"], a["x"], a["ldx"], a["pg"], a["pe"], a["gate"], a["ldg"], a["c"], a["r"], a["ld"], a["ro"],
        a["ldo"], a["f32"], a["g"], a["e"], a["ms"], a["mt"], a["ldm"], a["per"], a["h"], a["ldh"], a["q"], a["sq"],
        None), status, match)


@pytest.mark.parametrize("kw,status,match", [
    (dict(x=None), 1, "x_bf16 is NULL"),
    (dict(freq=None), 1, "freq is NULL"),
    (dict(M=0), 2, "M=0"),
    (dict(heads=0), 2, "heads=0"),
    (dict(rh=5), 2, r"rot_heads=5 outside \[0, heads=4\]"),
    (dict(D=12), 2, "head_dim=12"),
    (dict(rot=7), 2, "rot_dim=7"),
    (dict(rot=72), 2, r"rot_dim=72 must be even and in \[2, head_dim=64\]"),
    (dict(inter=2), 1, "interleaved=2"),
    (dict(inv=-1), 1, "inverse=-1"),
    (dict(scale=float("nan")), 1, "attn_scale=nan"),
    (dict(pos=None, pos0=2 ** 31 - 4), 1, "passes the last position"),
    (dict(xh=32), 2, "x_head=32 < head_dim=64"),
    (dict(yt=260), 4, "y_token=260 is not a multiple of 8"),
    (dict(yt=64, yh=64), 2, "make 4 heads of 8 tokens overlap"),
    (dict(y=DEV, yt=64, yh=512), 2, "in place needs the strides"),
    (dict(y=BAD), 4, "y_bf16 is not 16-byte aligned"),
    (dict(freq=DEV + 8), 4, "freq is not 16-byte aligned"),
    (dict(M=2 ** 27), 2, "too large for one launch"),
])
def test_rope_refuses(kw, status, match):
    a = dict(x=DEV, xt=256, xh=64, M=8, heads=4, rh=3, D=64, rot=64, inter=0, freq=DEV, scale=1.0, pos=DEV, pos0=0,
             inv=0, y=2 * DEV, yt=256, yh=64)
    a.update(kw)
    refused("fq_rope", fq.lib().fq_rope(a["x"], a["xt"], a["xh"], a["M"], a["heads"], a["rh"], a["D"], a["rot"],
                                        a["inter"], a["freq"], a["scale"], a["pos"], a["pos0"], a["inv"], a["y"],
                                        a["yt"], a["yh"], None), status, match)
