"""Attention of many sequences: each finds its own among thousands."""
import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host
from test_gpu_attn_decode import Batch
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


def tokens(rng, seqs):
    """Lengths: most of them short, some none, a few in many parts."""
    lens = rng.integers(-1, 60, seqs)
    lens[rng.integers(0, seqs, 4)] = [5000, 129, 700, 257]
    return [int(n) for n in lens]


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("H,kv", [(4, 2), (17, 1)])
@pytest.mark.parametrize("seqs", [65, 255, 256, 257, 320, 1023, 1024, 1025, 3000])
def test_tokens(seqs, H, kv, bits):
    b = Batch(tokens(np.random.default_rng(seqs), seqs), H, kv, 32, 16, bits, seed=seqs)
    nbytes, edge = fq.fq_attn_decode_workspace_bytes(seqs, H, kv, 32, b.width * 16), 1 << 16
    buf = torch.full((nbytes + 2 * edge,), 0xA5, dtype=torch.uint8, device="cuda")
    got = b.run(workspace=buf[edge:edge + nbytes])
    assert bool((buf[:edge] == 0xA5).all()) and bool((buf[edge + nbytes:] == 0xA5).all())
    b.check(got=got)


def test_batches_of_any_lengths_in_one_graph():
    """Captured once, replayed with other lengths; a small batch's graph on the same workspace in turns."""
    rng = np.random.default_rng(4)
    seqs, H, kv, D, page, pages = 700, 4, 2, 64, 16, 600
    c = fq.KVCache(pages, page, kv, D, 8)
    n = pages * page
    c.write(dev(ref.bf16(rng, n, kv, D)), dev(ref.bf16(rng, n, kv, D)), dev(np.arange(n, dtype=np.int32)))
    ws = torch.empty(fq.fq_attn_decode_workspace_bytes(seqs, H, kv, D, 300 * page), dtype=torch.uint8, device="cuda")
    graphs = []
    for m in (seqs, 5):
        q, table = dev(ref.bf16(rng, m, H, D)), dev(rng.integers(0, pages, (m, 300)).astype(np.int32))
        lens, o = torch.zeros(m, dtype=torch.int32, device="cuda"), torch.empty(m, H, D, dtype=torch.int16, device="cuda")
        c.attend(q, table, lens, o=o, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.attend(q, table, lens, o=o, workspace=ws)
        graphs.append((g, q, table, lens, o))
    for k in range(5):
        for g, q, table, lens, o in graphs:
            top = (60, 4800, 1, 300, 4800)[k]
            lens.copy_(dev(rng.integers(0, top + 1, len(lens)).astype(np.int32)))
            own = torch.empty(ws.numel(), dtype=torch.uint8, device="cuda").fill_(k)
            want = host(c.attend(q, table, lens, workspace=own)).copy()
            o.fill_(3)
            ws.fill_(0xFF)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(host(o), want)
            assert not np.any(want[host(lens) == 0])
