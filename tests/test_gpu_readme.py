"""README's example as it stands, run and checked against plain 64-bit references."""
import os
import re

import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("H,KV", [(4, 2), (3, 3), (8, 1)])
def test_example(H, KV):
    code = re.search(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S).group(1)
    rng = np.random.default_rng(H)
    K, D, page, lens = 256, 64, 64, [70, 1, 150]
    M, seqs = sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    need = [-(-n // page) for n in lens]
    pages = sum(need)
    table = np.full((seqs, max(need)), -1, np.int32)
    order, at = rng.permutation(pages), 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    slots = np.concatenate([table[s, np.arange(n) // page] * page + np.arange(n) % page for s, n in enumerate(lens)]).astype(np.int32)
    x, q = ref.bf16(rng, M, K), ref.bf16(rng, seqs, H, D)
    W = (rng.standard_normal(((H + 2 * KV) * D, K)) * K ** -0.5).astype(np.float32)
    gain = rng.uniform(0.5, 1.5, K).astype(np.float32)
    ns = dict(H=H, KV=KV, D=D, M=M, W=W, gain=gain, x=dev(x), positions=dev(pos), pages=pages, slots=dev(slots), cu=dev(cu), seqs=seqs,
              q=dev(q), page_table=dev(table), lens=dev(np.array(lens, np.int32)))
    exec(code, ns)
    torch.cuda.synchronize()
    got = host(ns["heads"], np.uint16)
    assert got.shape == (H + 2 * KV, M, D)
    # the site's heads again, rotated by the reference
    raw = bf16_to_f64(host(ns["qkv"].linear(ns["x"], head_dim=D), np.uint16))
    turns, grow = fq.fq_rope_freqs(D, 10000.0)
    y, mag = ref.rope(raw, pos, turns, grow, H + KV, D, False, False)
    ref.assert_bf16(got, y, np.maximum(mag, np.abs(y)), "heads")
    assert np.array_equal(got[H + KV:], host(ns["qkv"].linear(ns["x"], head_dim=D), np.uint16)[H + KV:])
    # the prompts
    h64 = bf16_to_f64(got)
    o, tol, _ = attnref.prefill(h64[:H], h64[H:H + KV], h64[H + KV:], cu, cu, D ** -0.5, 1)
    attnref.assert_attn(host(ns["o"].view(torch.int16), np.uint16).transpose(1, 0, 2), o, tol, "prompts")
    # a token of each over the 8-bit cache
    (kq, ks), (vq, vs) = (attnref.quant_heads(h64[a:a + KV]) for a in (H, H + KV))
    k64, v64, o1, G = ref.TABLE[kq] * ks[..., None], ref.TABLE[vq] * vs[..., None], host(ns["o1"], np.uint16), H // KV
    for s, n in enumerate(lens):
        for h in range(KV):
            mine = slice(h * G, (h + 1) * G)
            o, tol = attnref.attend(bf16_to_f64(q[s, mine]), k64[h, cu[s]:cu[s + 1]], v64[h, cu[s]:cu[s + 1]], np.full(G, n - 1), D ** -0.5)
            attnref.assert_attn(o1[s, mine], o, tol, f"token of sequence {s}")
