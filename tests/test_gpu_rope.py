"""Rotary positions on the GPU against a plain 64-bit reference."""
import numpy as np
import pytest

import blockref as ref
import synth
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


def test_a_host_call_before_torch_leaves_the_device_usable():
    """A fresh process whose first call is the host plan (torch not imported yet), then a rotation."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import numpy as np, w4a4_integer_gemm_amd as fq\n"
            "f, s = fq.fq_rope_freqs(64)\n"
            "import torch\n"
            "x = torch.ones(2, 64, dtype=torch.bfloat16, device='cuda')\n"
            "y = torch.zeros_like(x)\n"
            "fq.fq_rope(x, 64, 64, 2, 1, 1, 64, 64, 0, torch.from_numpy(f.view('int64')).cuda(), s, None, 0, 0, y, 64, 64)\n"
            "assert torch.equal(y[0], x[0]) and not torch.equal(y[1], x[1])\n"
            "print('rotated')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "rotated" in r.stdout, r.stderr[-2000:]


def run(M, heads, rot_heads, D, rot, inter=0, inverse=0, layout="heads", kind=fq.ROPE_PLAIN, pos="random", pos0=0, seed=0,
        in_place=False, pad=0, **kw):
    rng = np.random.default_rng(seed)
    freq, scale = fq.fq_rope_freqs(rot, kind=kind, **kw)
    ld = heads * D + pad
    x = ref.bf16(rng, M, ld)
    if pos == "random":
        p = rng.integers(-2 ** 31, 2 ** 31, M).astype(np.int32)
        p[0] = 2 ** 31 - 1
    else:
        p = (pos0 + np.arange(M)).astype(np.int32)
    fd = dev(freq.view(np.int64))
    pd = dev(p) if pos == "random" else None
    xd = dev(x)
    if in_place:
        y, yt, yh = xd, ld, D
    elif layout == "heads":
        y, yt, yh = dev(np.full((heads, M + 1, D), 0x1234, np.uint16)), D, (M + 1) * D
    else:
        y, yt, yh = dev(np.full((M, ld), 0x1234, np.uint16)), ld, D
    fq.fq_rope(xd, ld, D, M, heads, rot_heads, D, rot, inter, fd, scale, pd, pos0, inverse, y, yt, yh)
    got = host(y, np.uint16)
    if layout == "heads" and not in_place:
        assert np.all(got[:, M] == 0x1234), "wrote past the last token"
        got = got[:, :M]
    else:
        if pad:
            assert np.array_equal(got[:, heads * D:], x[:, heads * D:] if in_place else np.full((M, pad), 0x1234)), "pad"
        got = got[:, :heads * D].reshape(M, heads, D).transpose(1, 0, 2)
    xb = x[:, :heads * D].reshape(M, heads, D).transpose(1, 0, 2)
    # elements that are copied are copied bit for bit
    assert np.array_equal(got[rot_heads:], xb[rot_heads:]) and np.array_equal(got[:, :, rot:], xb[:, :, rot:])
    if rot_heads:
        y64, mag = ref.rope(bf16_to_f64(xb), p, freq, scale, rot_heads, rot, inter, inverse)
        # cos and sin in float32: each within 2^-22 (series, angle and their roundings)
        ref.assert_bf16(got[:rot_heads], y64[:rot_heads], mag[:rot_heads], f"{M}x{heads}x{D} rot={rot}", ulps=2.0 ** -21)


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("inverse", [0, 1])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (80, 32), (80, 80), (96, 24), (128, 16), (128, 2), (64, 20),
                                   (8, 8), (40, 14), (24, 24), (72, 72), (192, 48)])
def test_heads_and_parts(D, rot, inter, inverse):
    run(5, 5, 4, D, rot, inter, inverse, seed=D + rot)


@pytest.mark.parametrize("M,heads,rot_heads", [(1, 1, 1), (1, 12, 10), (2, 3, 0), (67, 9, 9), (300, 36, 32), (1, 300, 299)])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("layout", ["heads", "rows"])
def test_tokens_and_layouts(M, heads, rot_heads, inter, layout):
    run(M, heads, rot_heads, 64, 64, inter, layout=layout, pad=24, seed=M)


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("inverse", [0, 1])
@pytest.mark.parametrize("M,heads,rot_heads,D,rot", [(700, 9, 7, 64, 64), (260, 33, 30, 128, 32), (900, 5, 5, 80, 48),
                                                     (150, 13, 11, 256, 16), (2000, 2, 1, 72, 72), (3001, 3, 3, 40, 16)])
@pytest.mark.parametrize("layout", ["heads", "rows", "in place"])
def test_many_tokens(M, heads, rot_heads, D, rot, inter, inverse, layout):
    """Above the size where a thread takes whole pieces of several heads."""
    assert M * heads * D // 2 > 128 * 1024
    run(M, heads, rot_heads, D, rot, inter, inverse, layout="rows" if layout == "in place" else layout, pad=16,
        in_place=layout == "in place", seed=M)


@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("D,rot", [(64, 64), (80, 20)])
def test_in_place(D, rot, inter):
    run(9, 4, 3, D, rot, inter, in_place=True, layout="rows", pad=8)


@pytest.mark.parametrize("pos0", [0, 1, 4095, 10 ** 6, 2 ** 31 - 33, -5])
@pytest.mark.parametrize("inter", [0, 1])
def test_counted_positions(pos0, inter):
    run(33, 3, 2, 128, 128, inter, pos="count", pos0=pos0)


@pytest.mark.parametrize("kind,kw", [(fq.ROPE_LINEAR, dict(factor=4.0)), (fq.ROPE_BASE, dict(factor=8.0)),
                                     (fq.ROPE_BANDS, dict(factor=8.0, trained_len=8192, low=1.0, high=4.0)),
                                     (fq.ROPE_RAMP, dict(factor=16.0, trained_len=4096)),
                                     (fq.ROPE_PAIRS, dict(pair_factors=np.linspace(0.3, 9, 32).astype(np.float32)))])
def test_scaling_rules(kind, kw):
    run(17, 4, 3, 64, 64, kind=kind, **kw)


def test_position_zero_is_the_identity():
    x = ref.bf16(np.random.default_rng(1), 3, 4 * 64)
    freq, _ = fq.fq_rope_freqs(64)
    for inter in (0, 1):
        y = dev(np.zeros_like(x))
        fq.fq_rope(dev(x), 256, 64, 3, 4, 4, 64, 64, inter, dev(freq.view(np.int64)), 1.0, dev(np.zeros(3, np.int32)), 0, 0,
                   y, 256, 64)
        assert np.array_equal(host(y, np.uint16), x)


def test_inverse_undoes_and_is_the_transpose():
    """R^T R = 1 to two bf16 roundings, and <R u, v> = <u, R^T v>."""
    rng = np.random.default_rng(2)
    M, H, D = 11, 3, 128
    freq, _ = fq.fq_rope_freqs(D)
    fd, pos = dev(freq.view(np.int64)), dev(rng.integers(0, 10 ** 6, M).astype(np.int32))

    def apply(bits, inverse):
        y = dev(np.zeros_like(bits))
        fq.fq_rope(dev(bits), H * D, D, M, H, H, D, D, 0, fd, 1.0, pos, 0, inverse, y, H * D, D)
        return host(y, np.uint16)

    u, v = ref.bf16(rng, M, H * D), ref.bf16(rng, M, H * D)
    back = bf16_to_f64(apply(apply(u, 0), 1))
    u64, v64 = bf16_to_f64(u), bf16_to_f64(v)
    pair = np.abs(u64).reshape(M, H, 2, D // 2).sum(2, keepdims=True).repeat(2, 2).reshape(M, H * D)
    assert np.all(np.abs(back - u64) <= pair * 2.0 ** -7)  # each pass: half a bf16 ulp (2^-9 .. 2^-8) of the pair
    ru, rv = bf16_to_f64(apply(u, 0)), bf16_to_f64(apply(v, 1))
    # both sides round their vectors once: 2^-8 of the products' magnitudes
    lhs, rhs = (ru * v64).reshape(M, H, D).sum(-1), (u64 * rv).reshape(M, H, D).sum(-1)
    mag = (np.abs(ru * v64) + np.abs(u64 * rv)).reshape(M, H, D).sum(-1)
    assert np.all(np.abs(lhs - rhs) <= mag * 2.0 ** -8)


def test_rotation_depends_on_the_distance_only():
    """<R_p q, R_r k> is a function of p - r, also far out."""
    rng = np.random.default_rng(3)
    D = 64
    q, k = ref.bf16(rng, 1, D), ref.bf16(rng, 1, D)
    freq, _ = fq.fq_rope_freqs(D)
    fd = dev(freq.view(np.int64))

    def at(bits, p):
        y = dev(np.zeros_like(bits))
        fq.fq_rope(dev(bits), D, D, 1, 1, 1, D, D, 0, fd, 1.0, None, p, 0, y, D, D)
        return bf16_to_f64(host(y, np.uint16))

    base = float((at(q, 17) * at(k, 5)).sum())
    mag = float((np.abs(bf16_to_f64(q)).sum() * np.abs(bf16_to_f64(k)).max()))
    for far in (1000, 10 ** 6, 2 * 10 ** 9):
        assert abs(float((at(q, far + 12) * at(k, far)).sum()) - base) <= mag * 2.0 ** -7
