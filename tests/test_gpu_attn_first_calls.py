"""A process whose first calls between the qkv site and the o site are inside a graph capture, the cache's workspace and the
outputs among what the capture allocates; and rows of the cache read into outputs of any strides."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import dev, host, log

pytestmark = pytest.mark.gpu

SCRIPT = r"""
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
import torch
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import dev, host

H, KV, D, M, bits, seqs = {H}, {KV}, {D}, 150, {bits}, {seqs}
rng = np.random.default_rng(0)
N = H + 2 * KV
x = dev(ref.bf16(rng, N, M, D))
freq = dev(fq.fq_rope_freqs(D)[0].view(np.int64))
gain = dev(np.ones(D, np.float32))
cache = fq.KVCache(16, 16, KV, D, bits)
slots = dev(np.arange(M, dtype=np.int32))
cu = dev(np.array([0, 100, M], np.int32))
q = dev(ref.bf16(rng, seqs, H, D))
table = dev(np.tile(np.arange(16, dtype=np.int32), (seqs, 1)))
lens = dev(rng.integers(0, M + 1, seqs).astype(np.int32))
y = torch.empty(N, M, D, dtype=torch.int16, device="cuda")
o = torch.empty(M, H, D, dtype=torch.int16, device="cuda")
o1 = torch.empty(seqs, H, D, dtype=torch.int16, device="cuda")


def step(c):
    fq.fq_qk_norm_rope(x, D, M * D, M, N, H, KV, D, gain, gain, 1e-6, D, 0, freq, 1.0, None, 0, y, D, M * D)
    k, v = y[H:H + KV], y[H + KV:]
    c.write(k.transpose(0, 1), v.transpose(0, 1), slots)
    back = c.read(slots)
    fq.fq_attn_prefill(y, D, M * D, k, D, M * D, v, D, M * D, M, M, cu, None, 2, H, KV, D, D ** -0.5, 1, o, H * D, D)
    c.attend(q, table, lens, o=o1)
    return (y, o, o1, *back)


torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = step(cache)
twin = fq.KVCache(16, 16, KV, D, bits)
want = None
for k in range(3):
    for t in got:
        t.fill_(5)
    g.replay()
    torch.cuda.synchronize()
    have = [host(t.view(torch.int16)).copy() for t in got]
    if want is None:
        want = [host(t.view(torch.int16)).copy() for t in step(twin)]
        twin.attend(q, table, lens)
    assert all(np.array_equal(a, b) for a, b in zip(have, want)), k
    cache._ws.fill_(0xFF)
print("first-call capture ok")
"""


@pytest.mark.parametrize("H,KV,D,bits,seqs", [(4, 2, 64, 8, 3), (8, 1, 256, 16, 300)])
def test_first_calls_inside_a_capture(H, KV, D, bits, seqs):
    tests = os.path.dirname(os.path.abspath(__file__))
    code = SCRIPT.format(root=os.path.dirname(tests), tests=tests, H=H, KV=KV, D=D, bits=bits, seqs=seqs)
    p = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    log(p.stdout[-1000:] + p.stderr[-3000:])
    assert p.returncode == 0 and "first-call capture ok" in p.stdout


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("layout", ["heads", "rows"])
def test_read_into_other_strides(layout, bits):
    """Outputs in either layout with rows and values between them that have to stay."""
    rng = np.random.default_rng(3)
    M, KV, D = 37, 3, 80
    c = fq.KVCache(4, 16, KV, D, bits)
    slots = rng.permutation(64)[:M].astype(np.int32)
    c.write(dev(ref.bf16(rng, M, KV, D)), dev(ref.bf16(rng, M, KV, D)), dev(slots))
    slots[[3, 30]] = [-1, 64]
    want = [host(t.view(torch.int16)) for t in c.read(dev(slots))]
    outs = []
    for pad in (8, 24):  # keys and values of different strides
        if layout == "heads":
            buf = torch.full((KV, M + 2, D + pad), 77, dtype=torch.int16, device="cuda")
            outs.append((buf, buf[:, 1:M + 1, 8:8 + D].transpose(0, 1)))
        else:
            buf = torch.full((M + 2, KV * (D + pad)), 77, dtype=torch.int16, device="cuda")
            outs.append((buf, buf[1:M + 1].view(M, KV, D + pad)[:, :, 8:8 + D]))
    c.read(dev(slots), k=outs[0][1], v=outs[1][1])
    for (buf, view), w in zip(outs, want):
        assert np.array_equal(host(view.contiguous()), w)
        view.fill_(77)
        assert bool((buf == 77).all())
