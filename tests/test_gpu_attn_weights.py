"""The softmax's weights of decode and of prompts of few rows: what a matrix product's bf16 operand leaves of them is
multiplied too.  Against a plain 64-bit reference, with 2^-16 of the weights where one rounding to bf16 would take 2^-8."""
import numpy as np
import pytest

import attnref
import blockref as ref
from fqtest import bf16_to_f64
from test_gpu_attn_decode import Batch
from test_gpu_attn_prefill import call

pytestmark = pytest.mark.gpu


def attend(q, k, v, last, scale):
    """(o, tolerance before the last rounding) of rows q over keys 0 .. last[i].

    A weight is the sum of two bf16 values: the second is off by at most half a step, 2^-8, of a remainder of at most 2^-8
    of the weight.  Everything else is attnref.attend's float32 arithmetic: the scores' sums and differences (`off`), the
    products with the values and the sums over the keys."""
    n, D = q.shape
    m = k.shape[0]
    s = (q @ k.T) * scale
    see = np.arange(m)[None] <= np.asarray(last)[:, None]
    top = np.where(see, s, -np.inf).max(1, keepdims=True)
    w = np.where(see, np.exp(np.minimum(s - top, 0)), 0.0)
    w /= w.sum(1, keepdims=True)
    mag = (np.abs(q) @ np.abs(k).T) * abs(scale)
    off = np.where(see, (D + 16) * 2.0 ** -23 * mag + np.abs(s - top) * 2.0 ** -22, 0.0).max(1, keepdims=True)
    return w @ v, (w @ np.abs(v)) * (2.0 ** -16 + 2 * off + (m + 16) * 2.0 ** -23)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("D", [64, 80, 128, 256])
@pytest.mark.parametrize("lens", [[1, 2, 3, 5, 40], [700, 130], [9001]])
def test_decode(lens, D, bits):
    b = Batch(lens, 4, 2, D, 16, bits, seed=D + bits, q_scale=0.5)
    got = b.run()
    at, G = 0, b.H // b.kv
    for i, n in enumerate(lens):
        for h in range(b.kv):
            q = bf16_to_f64(b.q[i, h * G:(h + 1) * G])
            o, tol = attend(q, b.k64[h, at:at + n], b.v64[h, at:at + n], np.full(G, n - 1), D ** -0.5)
            attnref.assert_attn(got[i, h * G:(h + 1) * G], o, tol, f"sequence {i} of {n}")
        at += n


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("n,m", [(1, 2), (5, 5), (50, 866), (33, 300)])
def test_few_rows(n, m, D, causal, hook):
    hook("attn_prefill=rows")
    rng = np.random.default_rng(D + m)
    H, kv = 4, 1
    q, k, v = ref.bf16(rng, H, n, D, scale=0.5), ref.bf16(rng, kv, m, D), ref.bf16(rng, kv, m, D)
    got = call(q, k, v, [0, n], [0, m], D ** -0.5, causal)
    last = np.arange(n) + m - n if causal else np.full(n, m - 1)
    for h in range(H):
        o, tol = attend(*(bf16_to_f64(t) for t in (q[h], k[0], v[0])), last, D ** -0.5)
        attnref.assert_attn(got[h], o, tol, f"head {h}")
