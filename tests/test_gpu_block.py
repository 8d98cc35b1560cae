"""A transformer block of the operators together: norm to FP8 codes -> qkv site in the head layout -> rotary
positions in place -> o site -> norm, gate, residual scale and the next norm to codes -> gate+up site -> GeGLU
-> down site -> the closing norm into an integer site.  Every node is checked against its plain 64-bit form on
its own GPU inputs; the block is captured into graphs, run on another stream and run twice at once."""
import numpy as np
import pytest
import torch

import blockref as ref
import fq_block_chain as chain
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 7, 29, 40, 150])
@pytest.mark.parametrize("f32", [0, 1])
def test_every_node_of_a_block(M, f32):
    b = chain.Block(M, f32, seed=M + f32)
    r0 = host(b.stream).copy()
    b.run()
    torch.cuda.synchronize()
    s64 = lambda t: host(t).astype(np.float64) if f32 else bf16_to_f64(host(t, np.uint16))  # noqa: E731
    r0 = r0.astype(np.float64) if f32 else bf16_to_f64(r0.view(np.uint16))

    # the opening norm's codes and the qkv product
    h, _ = ref.pre_norm(r0, b.g1_host, b.eps, None, None, 1)
    qa, sa = host(b.codes1), host(b.scales1)[:, :M]
    ref.assert_codes8(qa, sa, *ref.quant_rows(h), what="norm 1")
    y, tol = ref.fp8_gemm(qa, sa, host(b.qkv.codes), host(b.qkv.wscale))
    got = host(b.qkv_out, np.uint16)  # [heads][M][D]
    ref.assert_gemm(got.transpose(1, 0, 2).reshape(M, -1), y, tol, "qkv")

    # rotary positions of the query and key heads
    want, mag = ref.rope(bf16_to_f64(got), host(b.pos), b.freq_host, 1.0, b.rot_heads, b.D, 0, False)
    rot = host(b.heads, np.uint16)
    assert np.array_equal(rot[b.rot_heads:], got[b.rot_heads:])
    ref.assert_bf16(rot[:b.rot_heads], want[:b.rot_heads], mag[:b.rot_heads], "rope")

    # the o site (its own prologue, no norm)
    o_in = bf16_to_f64(host(b.o_in, np.uint16))
    y, tol = ref.fp8_gemm(*ref.quant_rows(o_in), host(b.o.codes), host(b.o.wscale), host(b.o.bias))
    ref.assert_gemm(host(b.o_out, np.uint16), y, tol, "o")

    # gate, residual scale, stream update, modulated norm to codes
    cond = bf16_to_f64(host(b.cond, np.uint16))
    scale, shift, gate = (cond[:, i * b.K:(i + 1) * b.K] for i in range(3))
    r1, mag = ref.block_norm(bf16_to_f64(host(b.o_out, np.uint16)), b.g2_host, b.eps, gate, 0.5, r0, b.per)
    stored = s64(b.stream1)
    if f32:
        assert np.all(np.abs(stored - r1) <= mag * 2.0 ** -20)
    else:
        ref.assert_bf16(host(b.stream1, np.uint16), r1, mag, "stream")
    h, _ = ref.pre_norm(stored, None, b.eps, scale, shift, b.per)
    qa, sa = host(b.codes2), host(b.scales2)[:, :M]
    ref.assert_codes8(qa, sa, *ref.quant_rows(h), what="norm 2")
    y, tol = ref.fp8_gemm(qa, sa, host(b.up.codes), host(b.up.wscale))
    ref.assert_gemm(host(b.up_out, np.uint16), y, tol, "gate+up")

    # the down site and the closing norm, which updates the stream in place
    y, tol = ref.fp8_gemm(*ref.quant_rows(bf16_to_f64(host(b.mlp, np.uint16))), host(b.down.codes),
                          host(b.down.wscale))
    ref.assert_gemm(host(b.down_out, np.uint16), y, tol, "down")
    r2, mag = ref.block_norm(bf16_to_f64(host(b.down_out, np.uint16)), b.g3_host, b.eps, None, 1.0, stored, 1)
    final = s64(b.stream2)
    assert np.all(np.abs(final - r2) <= mag * 2.0 ** -20 + (0 if f32 else np.abs(r2) * 2.0 ** -8))
    h, mag = ref.pre_norm(final, b.g1_host, b.eps, None, None, 1)
    ref.assert_bf16(host(b.h, np.uint16), h, mag, "closing norm")


def test_integer_heads_take_the_rotation():
    """Rotary positions in place on the head layout that fq_linear_heads writes."""
    import synth
    M, D, H = 19, 32, 6
    wl = synth.random_workload(M, 256, H * D, 64, 8, 8, seed=3, norm=True)
    site = fq.DeviceSite(wl.W, wl.hblock, wl.wbits, wl.abits, gamma=wl.gamma, eps=wl.eps)
    y = torch.empty((H, M, D), dtype=torch.int16, device="cuda")
    ws = site.workspace(M)
    fq.fq_linear_heads(dev(wl.x), M, 256, 256, site.gamma, site.eps, None, 0, wl.hblock, wl.abits, site.codes,
                       site.wscale, site.N, wl.wbits, None, None, 0, D, y, ws, ws.numel())
    before = host(y, np.uint16).copy()
    freq, att = fq.fq_rope_freqs(D, 10000.0)
    fq.fq_rope(y, D, M * D, M, H, 4, D, D, 0, dev(freq.view(np.int64)), att, None, 100, 0, y, D, M * D)
    want, mag = ref.rope(bf16_to_f64(before), np.arange(100, 100 + M), freq, att, 4, D, 0, False)
    got = host(y, np.uint16)
    assert np.array_equal(got[4:], before[4:])
    ref.assert_bf16(got[:4], want[:4], mag[:4], "rope on integer heads")


@pytest.mark.parametrize("M", [1, 3, 23, 33, 140])
def test_graph_replays_match_eager(M):
    """Captured once, replayed on new inputs with eager work and synchronizations in between; two graphs of two
    blocks take turns, each with its own workspaces."""
    blocks = [chain.Block(M, 0, seed=5), chain.Block(M, 1, seed=6)]
    graphs = []
    for b in blocks:
        b.run()  # first calls outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.run()
        graphs.append(g)
    rng = np.random.default_rng(M)
    for rep in range(4):
        for b in blocks:
            b.new_inputs(rng)
        want = []
        for b in blocks:
            b.run()
            torch.cuda.synchronize()
            want.append([host(t).copy() for t in b.outputs()])
            b.poison()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b, w in zip(blocks, want):
            for got, one in zip(b.outputs(), w):
                assert np.array_equal(host(got), one), f"replay {rep}"


@pytest.mark.parametrize("M", [2, 64])
def test_on_another_stream_and_two_at_once(M):
    """Two blocks with buffers of their own on two streams at once give what each gives alone."""
    blocks = [chain.Block(M, 0, seed=i) for i in (1, 2)]
    want = []
    for b in blocks:
        b.run()
        torch.cuda.synchronize()
        want.append([host(t).copy() for t in b.outputs()])
        b.poison()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(8):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.run()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for got, one in zip(b.outputs(), w):
            assert np.array_equal(host(got), one)


def test_a_captured_site_keeps_its_workspace():
    """A graph of a small call replays right after a larger call made the site's workspace grow."""
    rng = np.random.default_rng(0)
    K, N = 512, 264
    site = fq.Fp8Site((rng.standard_normal((N, K)) * 0.02).astype(np.float32))
    x, y = dev(ref.bf16(rng, 40, K)), torch.empty((40, N), dtype=torch.int16, device="cuda")
    want = host(site.linear(x)).copy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        site.linear(x, y=y)
    big = dev(ref.bf16(rng, 3000, K))
    for _ in range(3):
        want_big = host(site.linear(big)).copy()
        filler = [torch.full((40 * K + 256,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(y), want)
        assert np.array_equal(host(site.linear(big)), want_big)
        assert all(bool((t == 255).all()) for t in filler)
        y.fill_(7)
