"""Attention of many sequences: each finds its own among thousands."""
import numpy as np
import pytest

import attnref
import blockref as ref
from fqtest import bf16_to_f64
from test_gpu_attn_prefill import MARK, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kernel", ["auto", "rows", "64", "128", "small", "wide"])
@pytest.mark.parametrize("seqs", [65, 128, 4096, 4097, 9000])
def test_prompts(seqs, kernel, hook):
    """Lengths of 0 to 4 and a few long ones; NaN before the first sequence and behind the last."""
    hook(f"attn_prefill={kernel}")
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 5, seqs)
    lens[rng.integers(0, seqs, 3)] = [300, 150, 70]
    lead, tail, H, kv, D = 7, 9, 2, 1, 64
    cu = lead + np.concatenate([[0], np.cumsum(lens)])
    M = int(cu[-1]) + tail
    q, k, v = (ref.bf16(rng, n, M, D) for n in (H, kv, kv))
    for t in (q, k, v):
        t[:, :lead] = t[:, M - tail:] = 0x7FC0
    got = call(q, k, v, cu, None, 0.125, 1)
    with np.errstate(invalid="ignore"):
        o, tol, inside = attnref.prefill(*(bf16_to_f64(t) for t in (q, k, v)), cu, cu, 0.125, 1)
    assert np.all(got[:, ~inside] == MARK)
    attnref.assert_attn(got[:, inside], o[:, inside], tol[:, inside], f"{seqs} sequences")
