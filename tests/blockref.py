"""Plain 64-bit references of the operators around the integer sites (FP8 block
scales, block norms, rotary positions), with tolerances from their arithmetic."""
from __future__ import annotations

import numpy as np

import synth
from fqtest import bf16_half_ulp, bf16_to_f64, log

G = 128  # values that share a scale


def e4m3_table():
    """Value of each of the 256 patterns, from the format's definition."""
    p = np.arange(256)
    e, m = (p >> 3) & 15, p & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(e == 15) & (m == 7)] = np.nan
    return np.where(p & 128, -v, v)


TABLE = e4m3_table()
_POS = TABLE[:127]                      # 0 .. 448, increasing; index = pattern
_MID = (_POS[1:] + _POS[:-1]) / 2       # exact in float64


def e4m3_round(v):
    """Nearest e4m3 pattern of |v| <= 448 (more is clamped), ties to the even pattern."""
    a = np.minimum(np.abs(v), 448.0)
    lo = np.searchsorted(_MID, a, side="left")    # a tie goes down ...
    up = np.searchsorted(_MID, a, side="right")   # ... or up
    i = np.where(lo % 2 == 0, lo, up)
    return (i + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quant_rows(h):
    """(codes [M][K], float32 scales [K / 128][M]) of float64 rows h.  The scale and
    the quotient are float32 values by definition (bf16 inputs meet rounding
    borders of e4m3 that a float64 quotient misses by 2^-25)."""
    M, K = h.shape
    v = h.reshape(M, K // G, G)
    s = (np.abs(v).max(-1) / 448.0).astype(np.float32)
    sd = s.astype(np.float64)[..., None]
    quot = np.divide(v, sd, out=np.zeros_like(v), where=sd > 0).astype(np.float32)
    q = e4m3_round(quot.astype(np.float64))
    return q.reshape(M, K), np.ascontiguousarray(s.T)


def rms(x, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def fp8_gemm(qa, sa, qw, sw, bias=None, residual=None):
    """(y float64 [M][N], its tolerance before the bf16 rounding), from codes.

    The matrix instruction adds the products of 8 consecutive k after aligning
    them to the largest exponent sum E among them and drops what lies below
    2^(E - 13).  Exponents are the codes' (subnormals and zero: -6); a product
    of two 4-bit significands has its last bit at 2^(e - 6), so only products
    with e < E - 7 lose anything: less than 2^(E - 13), and at most themselves.
    The sums of 8 and all that follows are float32: 16 adds and the scaled fma
    per group of 128, the scale product, up to 8 partial sums joined, bias and
    residual, each off by at most 2^-23 of the magnitudes summed."""
    M, K = qa.shape
    N, g = qw.shape[0], K // G
    sw_rows = np.repeat(sw.astype(np.float64), G, 0)[:N]           # [N][g]
    ta, tw = TABLE[qa], TABLE[qw]
    a = (ta.reshape(M, g, G) * sa.astype(np.float64).T[:, :, None]).reshape(M, K)
    w = tw * np.repeat(sw_rows, G, 1)
    y, S = a @ w.T, np.abs(a) @ np.abs(w).T
    expo = lambda q: (np.maximum((q >> 3) & 15, 1).astype(np.int16) - 7)  # noqa: E731
    ea, ew = expo(qa), expo(qw)
    lost = np.zeros((M, N))
    cols = max(1, (1 << 22) // K)
    aa, aw = np.abs(ta).astype(np.float32), np.abs(tw).astype(np.float32)
    for m in range(M):
        for n0 in range(0, N, cols):
            n1 = min(N, n0 + cols)
            e = (ea[m][None] + ew[n0:n1]).reshape(n1 - n0, K // 8, 8)
            E = e.max(-1, keepdims=True)
            p = (aa[m][None] * aw[n0:n1]).reshape(e.shape)
            d = np.where(e < E - 7, np.minimum(p, np.ldexp(np.float32(1), E - 13)), np.float32(0))
            per = d.reshape(n1 - n0, g, G).sum(-1, dtype=np.float64)
            lost[m, n0:n1] = (per * sw_rows[n0:n1]) @ sa[:, m].astype(np.float64)
    tol = lost + S * ((16 + 2 * g + 10) * 2.0 ** -23)
    for t in (None if bias is None else bias.astype(np.float64)[None, :],
              None if residual is None else bf16_to_f64(residual)):
        if t is not None:
            y = y + t
            tol = tol + (S + np.abs(t)) * 2.0 ** -23
    return y, tol


def assert_gemm(y_bits, y, tol, what=""):
    """Half a bf16 ulp plus the sums' tolerance."""
    bound = (bf16_half_ulp(np.abs(y) + tol)) * (1 + 1e-6) + tol
    err = np.abs(bf16_to_f64(y_bits) - y)
    log(f"  {what} max err/bound {np.max(err / np.maximum(bound, 1e-300)):.3f}")
    assert np.all(err <= bound), f"{what}: {np.count_nonzero(err > bound)} outputs outside the bound"


def assert_codes8(q, s, q_ref, s_ref, what=""):
    """Scales within 2^-20; codes equal but for at most 0.1 % that moved to a
    neighbour (a quotient next to a rounding border, moved by float32)."""
    rel = np.abs(s.astype(np.float64) - s_ref) / np.maximum(np.abs(s_ref), 1e-38)
    assert np.all(rel <= 2.0 ** -20), f"{what}: scales off by {rel.max():.3e}"
    order = lambda p: np.where(p & 128, -(p & 127).astype(int), p.astype(int))  # noqa: E731
    d = np.abs(order(q) - order(q_ref))
    log(f"  {what} codes: {np.count_nonzero(d)}/{d.size} differ, scales off by at most {rel.max():.1e}")
    assert d.max() <= 1 and np.count_nonzero(d) <= 1e-3 * d.size, f"{what}: codes differ"


def block_norm(x, post_gamma, post_eps, gate, res_scale, r, per):
    """(r' before rounding, magnitude of its terms)."""
    if x is None:
        return r, np.abs(r)
    p = x if post_gamma is None else rms(x, post_eps) * post_gamma.astype(np.float64)
    if gate is not None:
        p = p * gate[np.arange(x.shape[0]) // per]
    return r + res_scale * p, np.abs(r) + np.abs(res_scale * p)


def pre_norm(r, gamma, eps, scale, shift, per):
    """(h, magnitude of its terms) from the stored stream r."""
    h = rms(r, eps)
    if gamma is not None:
        h = h * gamma.astype(np.float64)
    mag = np.abs(h)
    at = np.arange(r.shape[0]) // per
    if scale is not None:
        mag = mag * (1 + np.abs(scale[at]))
        h = h * (1 + scale[at])
    if shift is not None:
        mag = mag + np.abs(shift[at])
        h = h + shift[at]
    return h, mag


def assert_bf16(bits, ref, mag, what="", ulps=2.0 ** -20):
    """Half a bf16 ulp plus 16 float32 roundings (2^-24 each) of the terms' magnitudes."""
    err = np.abs(bf16_to_f64(bits) - ref)
    bound = bf16_half_ulp(ref) * (1 + 1e-6) + mag * ulps
    log(f"  {what} max err/bound {np.max(err / np.maximum(bound, 1e-300)):.3f}")
    assert np.all(err <= bound), f"{what}: {np.count_nonzero(err > bound)} values outside the bound"


def rope_theta(rot, base=10000.0, kind=0, factor=1.0, trained=1, low=1.0, high=32.0, pair=None):
    """(radians per position, factor on cos and sin), float64, from the header's rules."""
    i = np.arange(rot // 2, dtype=np.float64)
    th = base ** (-2 * i / rot)
    if kind == 1:
        return th / factor, 1.0
    if kind == 2:
        return (base * factor ** (rot / (rot - 2.0))) ** (-2 * i / rot), 1.0
    if kind == 3:
        keep = np.clip((trained * th / (2 * np.pi) - low) / (high - low), 0, 1)
        return th * (keep + (1 - keep) / factor), 1.0
    if kind == 4:
        at = lambda n: rot * np.log(trained / (2 * np.pi * n)) / (2 * np.log(base))  # noqa: E731
        lo, hi = max(np.floor(at(high)), 0), min(np.ceil(at(low)), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0, 1)
        return th * (1 - ramp) + th / factor * ramp, 0.1 * np.log(factor) + 1
    if kind == 5:
        return th / pair.astype(np.float64), 1.0
    return th, 1.0


def rope(x, pos, turns, scale, rot_heads, rot, interleaved, inverse):
    """x float64 [heads][M][D]; turns: fraction of a turn per position of each pair
    (exact integers / 2^64).  Returns (y, |a| + |b| of each rotated element)."""
    # the fraction of a turn in integers modulo 2^64 (wrapping products), then one rounding
    frac = (np.asarray(turns, np.uint64)[None] * np.asarray(pos).astype(np.int64).astype(np.uint64)[:, None]) / 2.0 ** 64
    c, s = np.cos(2 * np.pi * frac) * scale, np.sin(2 * np.pi * frac) * scale * (-1 if inverse else 1)
    y, mag = x.copy(), np.zeros_like(x)
    i = np.arange(rot // 2)
    e0, e1 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[:rot_heads][:, :, e0], x[:rot_heads][:, :, e1]
    y[:rot_heads, :, e0] = a * c - b * s
    y[:rot_heads, :, e1] = b * c + a * s
    mag[:rot_heads, :, e0] = mag[:rot_heads, :, e1] = (np.abs(a) + np.abs(b)) * abs(scale)
    return y, mag


def bf16(rng, *shape, scale=1.0):
    return synth.f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))
