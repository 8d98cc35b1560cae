"""Scales far from the usual one, with scores that are as far from it the other way: only their product counts."""
import numpy as np
import pytest

import attnref
import blockref as ref
from fqtest import bf16_to_f64
from test_gpu_attn_decode import Batch
from test_gpu_attn_prefill import call

pytestmark = pytest.mark.gpu

# scores of about scale * size^2 * sqrt(64): from 1 to 20 of them
SCALES = [(1e-33, 2.0 ** 53), (-3e-35, 2.0 ** 57), (1e-38, 2.0 ** 61), (2e-36, 2.0 ** 58), (1e12, 2.0 ** -21), (1e30, 2.0 ** -51)]


@pytest.mark.parametrize("kernel", ["auto", "rows", "64", "128", "small", "wide"])
@pytest.mark.parametrize("scale,size", SCALES)
@pytest.mark.parametrize("causal", [0, 1])
def test_prompts(scale, size, causal, kernel, hook):
    hook(f"attn_prefill={kernel}")
    rng = np.random.default_rng(1)
    H, kv, n, m, D = 2, 1, 100, 170, 64
    q, k, v = ref.bf16(rng, H, n, D, scale=size), ref.bf16(rng, kv, m, D, scale=size), ref.bf16(rng, kv, m, D)
    got = call(q, k, v, [0, 30, n], [0, 60, m], scale, causal)
    scale = float(np.float32(scale))
    o, tol, _ = attnref.prefill(*(bf16_to_f64(t) for t in (q, k, v)), [0, 30, n], [0, 60, m], scale, causal)
    attnref.assert_attn(got, o, tol, f"scale {scale}")


@pytest.mark.parametrize("kernel", ["auto", "rows", "64", "128", "small", "wide"])
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_prompts_of_scale_zero(scale, kernel, hook):
    """Every key that a row sees counts the same, however large the scores are."""
    hook(f"attn_prefill={kernel}")
    rng = np.random.default_rng(2)
    H, kv, n, D = 2, 1, 130, 64
    q, k, v = ref.bf16(rng, H, n, D, scale=2.0 ** 58), ref.bf16(rng, kv, n, D, scale=2.0 ** 58), ref.bf16(rng, kv, n, D)
    got = call(q, k, v, [0, n], None, scale, 1)
    o, tol, _ = attnref.prefill(*(bf16_to_f64(t) for t in (q, k, v)), [0, n], [0, n], 0.0, 1)
    attnref.assert_attn(got, o, tol, "scale 0")


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("scale,q_scale", [(1e-33, 2.0 ** 106), (1e-38, 2.0 ** 120), (1e12, 2.0 ** -41), (0.0, 2.0 ** 110)])
def test_tokens(scale, q_scale, bits):
    Batch([200, 1, 33], 4, 2, 64, 16, bits, q_scale=q_scale, seed=3).check(float(np.float32(scale)))
