"""Norms around a block on the GPU against a plain 64-bit reference."""
import itertools

import numpy as np
import pytest

import blockref as ref
import synth
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


def run(M, K, seed, post=True, gate=True, mod=True, x=True, f32=False, out="bf16", per=3, scale=0.7, pad=8, in_place=False,
        pre=True, blow=1.0):
    rng = np.random.default_rng(seed)
    guard = 0x5A5A
    xb = ref.bf16(rng, M, K + pad, scale=blow) if x else None
    r = rng.standard_normal((M, K + pad)).astype(np.float32) * 3
    rbits = synth.f32_to_bf16_bits(r)
    r64 = (r if f32 else synth.bf16_bits_to_f32(rbits)).astype(np.float64)[:, :K]
    conds = -(-M // per)
    pg = rng.uniform(0.5, 1.5, K).astype(np.float32) if post and x else None
    g = rng.uniform(0.5, 1.5, K).astype(np.float32) if pre else None
    cond = ref.bf16(rng, conds, 3 * K + pad, scale=0.4)
    cd = dev(cond)
    rd = dev(r if f32 else rbits)
    ro = None
    if x:
        ro = rd if in_place else dev(np.full((M + 1, K + pad), guard, np.float32 if f32 else np.uint16))
    h = dev(np.full((M + 1, K + pad), guard, np.uint16)) if out in ("bf16", "both") else None
    q = s = None
    if out in ("fp8", "both"):
        q, s = dev(np.full((M + 1, K), 0x55, np.uint8)), dev(np.full((K // 128, -(-M // 4) * 4), -1, np.float32))
    fq.fq_block_norm(M, K, None if xb is None else dev(xb), K + pad, None if pg is None else dev(pg), 1e-6,
                     cd[:, :K] if gate and x else None, 3 * K + pad, scale, rd, K + pad, ro, K + pad, int(f32),
                     None if g is None or out == "none" else dev(g), 1e-5, cd[:, K:] if mod and out != "none" else None,
                     cd[:, 2 * K:] if mod and out != "none" else None, 3 * K + pad, per, h, K + pad, q, s)
    c64 = bf16_to_f64(cond)
    want, mag = ref.block_norm(None if xb is None else bf16_to_f64(xb[:, :K]), pg, 1e-6, c64[:, :K] if gate and x else None,
                               scale, r64, per)
    what = f"{M}x{K} post={post} gate={gate} mod={mod} x={x} f32={f32} out={out}"
    stream = r64
    if x:
        got = host(ro) if f32 else host(ro, np.uint16)
        if not in_place:
            assert np.all(got[M:] == guard) and np.all(got[:, K:] == guard), "wrote outside its rows"
        if f32:
            err = np.abs(got[:M, :K].astype(np.float64) - want)
            assert np.all(err <= mag * 2.0 ** -20), what  # 16 float32 roundings of the terms
            stream = got[:M, :K].astype(np.float64)
        else:
            ref.assert_bf16(got[:M, :K], want, mag, what + " stream")
            stream = bf16_to_f64(got[:M, :K])
    if out == "none":
        return
    hw, hm = ref.pre_norm(stream, g, 1e-5, c64[:, K:2 * K] if mod else None, c64[:, 2 * K:3 * K] if mod else None, per)
    if h is not None:
        hb = host(h, np.uint16)
        assert np.all(hb[M:] == guard) and np.all(hb[:, K:] == guard), "wrote outside its rows"
        ref.assert_bf16(hb[:M, :K], hw, hm, what + " h")
    if q is not None:
        qh, sh = host(q), host(s)
        assert np.all(qh[M] == 0x55) and np.all(sh[:, M:] == -1), "wrote outside its rows"
        qr, sr = ref.quant_rows(hw)
        ref.assert_codes8(qh[:M], sh[:, :M], qr, sr, what)


@pytest.mark.parametrize("post,gate,mod,f32", list(itertools.product([False, True], repeat=4)))
@pytest.mark.parametrize("out", ["bf16", "fp8"])
def test_every_option(post, gate, mod, f32, out):
    run(5, 384, 1, post=post, gate=gate, mod=mod, f32=f32, out=out)


@pytest.mark.parametrize("M,K", [(1, 8), (1, 24), (2, 504), (1, 512), (3, 520), (1, 2048), (7, 3584), (2, 8192), (3, 8200),
                                 (2, 16384), (2, 16392), (1, 32768), (1, 32776), (1, 65536), (300, 136), (257, 2056), (256, 520),
                                 (258, 8200)])
@pytest.mark.parametrize("f32", [False, True])
def test_sizes(M, K, f32):
    run(M, K, M + K, f32=f32)


@pytest.mark.parametrize("M,K", [(1, 128), (5, 1152), (2, 8320), (1, 18944), (1, 33024), (131, 256), (300, 1152), (257, 8320)])
@pytest.mark.parametrize("f32", [False, True])
def test_code_sizes(M, K, f32):
    run(M, K, M + K, f32=f32, out="both")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("out", ["bf16", "fp8", "both"])
def test_norm_of_the_stream_alone(f32, out):
    run(6, 640, 2, x=False, f32=f32, out=out)
    run(6, 640, 3, x=False, f32=f32, out=out, mod=False, pre=False)


@pytest.mark.parametrize("f32", [False, True])
def test_update_alone_and_in_place(f32):
    run(6, 640, 4, f32=f32, out="none")
    run(6, 640, 5, f32=f32, in_place=True)
    run(33, 2048, 6, f32=f32, in_place=True, out="both", pad=0)


@pytest.mark.parametrize("per", [1, 2, 10, 1000])
def test_conditions(per):
    run(10, 256, per, per=per)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.25, 1e-3])
def test_residual_scale(scale):
    run(4, 264, 7, scale=scale)


@pytest.mark.parametrize("blow", [1e-18, 1e15])
def test_post_norm_of_small_and_large_outputs(blow):
    run(4, 512, 8, blow=blow, gate=False)


def test_rows_of_zeros_and_non_finite_rows():
    """A row of zeros stays finite (eps); a NaN or infinity stays in its row."""
    M, K = 6, 256
    rng = np.random.default_rng(0)
    x, r = ref.bf16(rng, M, K), ref.bf16(rng, M, K)
    g = dev(np.ones(K, np.float32))

    def go(x, r):
        ro, h = dev(np.zeros((M, K), np.uint16)), dev(np.zeros((M, K), np.uint16))
        q, s = dev(np.zeros((M, K), np.uint8)), dev(np.zeros((K // 128, 8), np.float32))
        fq.fq_block_norm(M, K, dev(x), K, g, 1e-6, None, 0, 1.0, dev(r), K, ro, K, 0, g, 1e-6, None, None, 0, 1, h, K, q, s)
        return host(ro, np.uint16), host(h, np.uint16), host(q), host(s)[:, :M]

    clean = go(x, r)
    x[1] = 0
    r[1] = 0
    x[3, 7] = 0x7FC0   # NaN
    r[4, 9] = 0x7F80   # infinity
    got = go(x, r)
    assert np.all(got[0][1] == 0) and np.all(got[1][1] == 0) and np.all(got[2][1] & 0x7F == 0) and np.all(got[3][:, 1] == 0)
    assert np.all(np.isnan(bf16_to_f64(got[0][3]))) and np.all(np.isnan(bf16_to_f64(got[1][3])))
    assert np.isinf(bf16_to_f64(got[0][4, 9])) and np.isnan(bf16_to_f64(got[1][4, 9]))
    keep = [0, 2, 5]
    for a, b in zip(got[:3], clean[:3]):
        assert np.array_equal(a[keep], b[keep])
    assert np.array_equal(got[3][:, keep], clean[3][:, keep])


@pytest.mark.parametrize("M,K,out,f32", [(4099, 1032, "bf16", True), (4101, 1024, "both", False), (1025, 4352, "fp8", False),
                                         (521, 8192, "both", True), (2055, 2056, "none", False)])
def test_many_rows(M, K, out, f32):
    """Calls large enough for two pieces per lane."""
    run(M, K, 8, out=out, f32=f32, per=64)
