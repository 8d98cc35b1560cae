"""Calls between the qkv site and the o site with stream=: they run behind what that stream has queued, whatever the
current stream is; and a decode call stays inside a workspace of the size that the library asks for."""
import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host
from test_gpu_attn_decode import Batch

pytestmark = pytest.mark.gpu

M, H, KV, D = 60, 4, 2, 64


class Late:
    """Buffers of zeros that the stream fills with their values some 20 ms from now."""

    def __init__(self):
        self.stream, self.other = torch.cuda.Stream(), torch.cuda.Stream()

    def fill(self, *values):
        bufs = [torch.zeros_like(v) for v in values]
        torch.cuda.synchronize()
        with torch.cuda.stream(self.stream):
            torch.cuda._sleep(40_000_000)
            for b, v in zip(bufs, values):
                b.copy_(v)
        return bufs

    def run(self, call):
        """call(stream), from another current stream; back when it is done."""
        with torch.cuda.stream(self.other):
            call(self.stream)
        self.stream.synchronize()


def test_prompt_attention():
    rng = np.random.default_rng(0)
    bits = [ref.bf16(rng, n, M, D) for n in (H, KV, KV)]
    late = Late()
    o, cu = torch.full((M, H, D), 7, dtype=torch.int16, device="cuda"), dev(np.array([0, M], np.int32))
    q, k, v = late.fill(*(dev(b) for b in bits))
    late.run(lambda s: fq.fq_attn_prefill(q, D, M * D, k, D, M * D, v, D, M * D, M, M, cu, None, 1, H, KV, D, 0.125, 1, o, H * D, D, s))
    want, tol, _ = attnref.prefill(*(bf16_to_f64(b) for b in bits), [0, M], [0, M], 0.125, 1)
    attnref.assert_attn(host(o, np.uint16).transpose(1, 0, 2), want, tol, "prompt")


@pytest.mark.parametrize("rot", [64, 20])
def test_head_norms(rot):
    rng = np.random.default_rng(1)
    x = ref.bf16(rng, H + 2 * KV, M, D, scale=3.0)
    freq, s = fq.fq_rope_freqs(rot)
    fd, g = dev(freq.view(np.int64)), dev(np.ones(D, np.float32))
    y = torch.full((H + 2 * KV, M, D), 7, dtype=torch.int16, device="cuda")
    late = Late()
    xd, = late.fill(dev(x))
    late.run(lambda st: fq.fq_qk_norm_rope(xd, D, M * D, M, H + 2 * KV, H, KV, D, g, g, 1e-6, rot, 0, fd, s, None, 5, y, D, M * D, st))
    want, mag = attnref.qk_norm(bf16_to_f64(x), H, KV, np.ones(D, np.float32), np.ones(D, np.float32), 1e-6, rot, 0, 5 + np.arange(M), freq, s)
    got = host(y, np.uint16)
    ref.assert_bf16(got[:H + KV], want[:H + KV], mag[:H + KV], "heads", ulps=2.0 ** -19)
    assert np.array_equal(got[H + KV:], x[H + KV:])


@pytest.mark.parametrize("bits", [8, 16])
def test_cache_write(bits):
    rng = np.random.default_rng(2)
    c = fq.KVCache(5, 16, KV, D, bits)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.view(torch.uint8).zero_()
    k, v = (ref.bf16(rng, M, KV, D) for _ in range(2))
    slots = dev(rng.permutation(80)[:M].astype(np.int32))
    late = Late()
    kd, vd = late.fill(dev(k), dev(v))
    late.run(lambda s: c.write(kd, vd, slots, stream=s))
    twin = fq.KVCache(5, 16, KV, D, bits)
    for t in (twin.k, twin.v, twin.k_scale, twin.v_scale):
        if t is not None:
            t.view(torch.uint8).zero_()
    twin.write(dev(k), dev(v), slots)
    torch.cuda.synchronize()
    assert bool(c.k.view(torch.uint8).any())
    for a, b in zip((c.k, c.v, c.k_scale, c.v_scale), (twin.k, twin.v, twin.k_scale, twin.v_scale)):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("lens,heads,kv,d,page,width", [
    ([5], 4, 2, 64, 16, None), ([100], 4, 2, 64, 16, 8), ([128, 1, 0], 8, 1, 256, 64, None), ([129], 3, 3, 80, 16, None),
    ([20011], 8, 2, 128, 64, None), ([20011], 5, 1, 16, 64, 400), ([3000] * 9 + [1, 0, 77], 28, 4, 128, 64, None), ([900] * 70, 40, 8, 112, 16, 100),
])
def test_decode_stays_inside_its_workspace(lens, heads, kv, d, page, width, bits):
    """Exactly the size that the library names, between guards; every part of every sequence writes into it."""
    b = Batch(lens, heads, kv, d, page, bits, seed=len(lens), width=width)
    want = b.run().copy()
    nbytes = fq.fq_attn_decode_workspace_bytes(len(lens), heads, kv, d, b.width * page)
    edge = 1 << 16
    buf = torch.full((nbytes + 2 * edge,), 0xA5, dtype=torch.uint8, device="cuda")
    got = b.run(workspace=buf[edge:edge + nbytes])
    assert bool((buf[:edge] == 0xA5).all()) and bool((buf[edge + nbytes:] == 0xA5).all())
    assert np.array_equal(got, want)
