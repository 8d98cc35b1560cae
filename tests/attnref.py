"""Plain 64-bit references of the operators between the qkv site and the o site, with tolerances from their arithmetic."""
from __future__ import annotations

import numpy as np

import blockref as ref
from fqtest import bf16_half_ulp, bf16_to_f64, log


def attend(q, k, v, last, scale):
    """Rows q [n][D] over keys 0 .. last[i] of k, v [m][D], float64.  Returns (o, tolerance before the last rounding).

    p is rounded to bf16 before it is multiplied by v: 2^-8 of sum w|v|, w the softmax's weights.  (An 8-bit cache
    multiplies p by the value's scale first: one more rounding of float32.)  A score is off by its products' float32 sums
    (D + 8 of them, 2^-23 each of sum |q k| scale, the keys' scale among them) and by the rounding of its difference to
    the maximum; that moves its weight by as much, relative, twice with the sum below the fraction.  The sums over
    the keys are float32: 2^-23 for each of the keys."""
    n, D = q.shape
    m = k.shape[0]
    o, tol = np.zeros((n, D)), np.zeros((n, D))
    if m == 0:
        return o, tol
    s = (q @ k.T) * scale
    see = np.arange(m)[None] <= np.asarray(last)[:, None]
    s = np.where(see, s, -np.inf)
    some = see.any(1)
    top = np.where(some, s.max(1, initial=-np.inf), 0.0)
    w = np.where(see, np.exp(s - top[:, None]), 0.0)
    total = w.sum(1, keepdims=True)
    w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    o = w @ v
    mag = (np.abs(q) @ np.abs(k).T) * abs(scale)
    off = np.where(see, (D + 16) * 2.0 ** -23 * mag + np.abs(np.where(see, s, 0) - top[:, None]) * 2.0 ** -22, 0.0).max(1)
    A = w @ np.abs(v)
    return o, A * (2.0 ** -8 + 2 * off[:, None] + (m + 16) * 2.0 ** -23)


def assert_attn(bits, o, tol, what=""):
    """Half a bf16 step of the output plus the tolerance."""
    err = np.abs(bf16_to_f64(bits) - o)
    bound = bf16_half_ulp(np.abs(o) + tol) * (1 + 1e-6) + tol
    worst = np.max(err / np.maximum(bound, 1e-300)) if err.size else 0.0
    log(f"  {what} max err/bound {worst:.3f}")
    assert np.all(err <= bound), f"{what}: {np.count_nonzero(err > bound)} of {err.size} outputs outside the bound"


def prefill(q, k, v, cu_q, cu_k, scale, causal):
    """q [H][M][D], k, v [kv][M_k][D] float64; (o, tolerance) [H][M][D] of the rows inside a sequence, and which those are."""
    H, M, D = q.shape
    G = H // k.shape[0]
    o, tol, inside = np.zeros_like(q), np.zeros_like(q), np.zeros(M, bool)
    for s in range(len(cu_q) - 1):
        a, b, ka, kb = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        n, m = b - a, kb - ka
        inside[a:b] = True
        last = np.arange(n) + m - n if causal else np.full(n, m - 1)
        for h in range(H):
            o[h, a:b], tol[h, a:b] = attend(q[h, a:b], k[h // G, ka:kb], v[h // G, ka:kb], last, scale)
    return o, tol, inside


def quant_heads(x):
    """(codes, float32 scales) of float64 rows x [...][D], one scale for a row."""
    s = (np.abs(x).max(-1) / 448.0).astype(np.float32)
    sd = s.astype(np.float64)[..., None]
    quot = np.divide(x, sd, out=np.zeros_like(x), where=sd > 0).astype(np.float32)
    return ref.e4m3_round(quot.astype(np.float64)), s


def qk_norm(x, q_heads, k_heads, q_gamma, k_gamma, eps, rot, inter, pos, turns, scale):
    """x float64 [heads][M][D]; (y, magnitude of its terms)."""
    n = x.copy()
    for h in range(q_heads + k_heads):
        g = q_gamma if h < q_heads else k_gamma
        n[h] = ref.rms(x[h], eps) * (1.0 if g is None else g.astype(np.float64))
    if rot == 0:
        return n, np.abs(n)
    y, mag = ref.rope(n, pos, turns, scale, q_heads + k_heads, rot, inter, False)
    return y, np.maximum(mag, np.abs(n))
