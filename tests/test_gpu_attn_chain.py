"""The way from the qkv site to the o site as a model goes it: prompts through the qkv site, norms and rotation, the cache,
attention, the o site; then token after token over the cache.  Every node is checked on its own GPU inputs; the steps
are captured and replayed, run on other streams and twice at once."""
import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu

K, H, KV, D, EPS = 256, 6, 2, 64, 1e-6


class Layer:
    """One layer's attention part over a cache of its own."""

    def __init__(self, bits, seed, seqs, page=16, pages=80, width=20, integer=False):
        rng = np.random.default_rng(seed)
        w = lambda n, k: (rng.standard_normal((n, k)) * k ** -0.5).astype(np.float32)  # noqa: E731
        self.rng, self.bits, self.seqs, self.page, self.width = rng, bits, seqs, page, width
        if integer:
            self.qkv = fq.DeviceSite(w((H + 2 * KV) * D, K), 64, 8, 8)
        else:
            self.qkv = fq.Fp8Site(w((H + 2 * KV) * D, K))
        self.o = fq.Fp8Site(w(K, H * D))
        self.gq, self.gk = (rng.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
        self.dgq, self.dgk = dev(self.gq), dev(self.gk)
        self.freq, _ = fq.fq_rope_freqs(D)
        self.dfreq = dev(self.freq.view(np.int64))
        self.cache = fq.KVCache(pages, page, KV, D, bits)
        self.table = np.sort(rng.permutation(pages)[:seqs * width].reshape(seqs, width)).astype(np.int32)
        self.table = rng.permuted(self.table, axis=1)
        self.dtable = dev(self.table)

    def slot(self, s, pos):
        return self.table[s, pos // self.page] * self.page + pos % self.page

    def heads_of(self, x, M):
        """[heads][M][D] of the qkv site."""
        if isinstance(self.qkv, fq.DeviceSite):
            return self.qkv.linear_heads(x, D)
        return self.qkv.linear(x, head_dim=D)

    def norm(self, heads, M, pos):
        fq.fq_qk_norm_rope(heads, D, M * D, M, H + 2 * KV, H, KV, D, self.dgq, self.dgk, EPS, D, 0, self.dfreq, 1.0, pos, 0, heads, D,
                           M * D)

    def prompt(self, x, lens, pos, slots, cu):
        """x [M][K] packed; (normed heads, attention's output [M][H][D], o site's output)."""
        M = x.shape[0]
        heads = self.heads_of(x, M)
        raw = heads.clone()
        self.norm(heads, M, pos)
        k, v = heads[H:H + KV], heads[H + KV:]
        self.cache.write(k.transpose(0, 1), v.transpose(0, 1), slots)
        att = torch.empty((M, H, D), dtype=torch.int16, device="cuda")
        fq.fq_attn_prefill(heads, D, M * D, k, D, M * D, v, D, M * D, M, M, cu, None, len(lens), H, KV, D, D ** -0.5, 1, att, H * D, D)
        return raw, heads, att, self.o.linear(att.view(M, H * D))

    def step(self, x, pos, slots, lens, out):
        """One token of each sequence; out: (heads, attention, o site's output) buffers."""
        M = self.seqs
        heads, att, y = out
        heads.copy_(self.heads_of(x, M))
        self.norm(heads, M, pos)
        self.cache.write(heads[H:H + KV].transpose(0, 1), heads[H + KV:].transpose(0, 1), slots)
        self.cache.attend(heads[:H].transpose(0, 1), self.dtable, lens, o=att)
        self.o.linear(att.view(M, H * D), y=y)

    def buffers(self):
        e = lambda *s: torch.empty(s, dtype=torch.int16, device="cuda")  # noqa: E731
        return e(H + 2 * KV, self.seqs, D), e(self.seqs, H, D), e(self.seqs, K)

    def token(self, at):
        """(x, positions, slots, lens) of sequences whose next tokens are at positions `at`; -1: an idle place."""
        at = np.asarray(at)
        slots = np.array([self.slot(s, p) if p >= 0 else -1 for s, p in enumerate(at)], np.int32)
        return dev(ref.bf16(self.rng, self.seqs, K)), dev(np.maximum(at, 0).astype(np.int32)), dev(slots), dev((at + 1).astype(np.int32))


def fill(layer, lens):
    """Prompts of the given lengths through the layer; what prompt() returns."""
    M = sum(lens)
    x = dev(ref.bf16(layer.rng, M, K))
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    slots = np.concatenate([[layer.slot(s, p) for p in range(n)] for s, n in enumerate(lens)]).astype(np.int32)
    return layer.prompt(x, lens, dev(pos), dev(slots), dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))), pos


def dequantised(layer, x):
    """What the cache holds of bf16 bits [..][D], float64."""
    x = bf16_to_f64(x)
    if layer.bits == 16:
        return x
    q, s = attnref.quant_heads(x)
    return ref.TABLE[q] * s[..., None]


@pytest.mark.parametrize("bits,integer", [(8, False), (16, False), (8, True)])
def test_every_node_of_prompts_and_tokens(bits, integer):
    lens = [70, 1, 190]
    layer = Layer(bits, seed=bits, seqs=len(lens), integer=integer)
    (raw, heads, att, y), pos = fill(layer, lens)
    torch.cuda.synchronize()
    # norms and rotation
    want, mag = attnref.qk_norm(bf16_to_f64(host(raw, np.uint16)), H, KV, layer.gq, layer.gk, EPS, D, 0, pos, layer.freq, 1.0)
    got = host(heads, np.uint16)
    assert np.array_equal(got[H + KV:], host(raw, np.uint16)[H + KV:])
    ref.assert_bf16(got[:H + KV], want[:H + KV], mag[:H + KV], "heads", ulps=2.0 ** -19)
    # attention of the prompts
    cu = np.concatenate([[0], np.cumsum(lens)])
    h64 = bf16_to_f64(got)
    o, tol, _ = attnref.prefill(h64[:H], h64[H:H + KV], h64[H + KV:], cu, cu, D ** -0.5, 1)
    attnref.assert_attn(host(att, np.uint16).transpose(1, 0, 2), o, tol, "prompts")
    # the o site
    yy, tol = ref.fp8_gemm(*ref.quant_rows(bf16_to_f64(host(att, np.uint16)).reshape(-1, H * D)), host(layer.o.codes),
                           host(layer.o.wscale))
    ref.assert_gemm(host(y, np.uint16), yy, tol, "o")
    # tokens: the cache holds what the prompts wrote, then each new token
    keys = [dequantised(layer, got[H:H + KV, cu[s]:cu[s + 1]]) for s in range(len(lens))]
    values = [dequantised(layer, got[H + KV:, cu[s]:cu[s + 1]]) for s in range(len(lens))]
    out = layer.buffers()
    for step in range(3):
        layer.step(*layer.token([n + step for n in lens]), out)
        new = host(out[0], np.uint16)
        att = host(out[1], np.uint16)
        for s in range(len(lens)):
            keys[s] = np.concatenate([keys[s], dequantised(layer, new[H:H + KV, s:s + 1])], 1)
            values[s] = np.concatenate([values[s], dequantised(layer, new[H + KV:, s:s + 1])], 1)
            for h in range(KV):
                q = bf16_to_f64(new[h * H // KV:(h + 1) * H // KV, s])
                o, tol = attnref.attend(q, keys[s][h], values[s][h], np.full(len(q), keys[s].shape[1] - 1), D ** -0.5)
                attnref.assert_attn(att[s, h * H // KV:(h + 1) * H // KV], o, tol, f"step {step} sequence {s}")
    # and read back as the prefix of a prompt that goes on: the keys are what attention used
    k, v = layer.cache.read(dev(np.array([layer.slot(2, p) for p in range(lens[2] + 3)], np.int32)))
    for t, want in ((k, keys[2]), (v, values[2])):
        err = np.abs(bf16_to_f64(host(t.view(torch.int16), np.uint16)).transpose(1, 0, 2) - want)
        assert np.all(err <= np.abs(want) * 2.0 ** -8)  # one rounding to bf16


def test_a_token_gives_what_its_prompt_gives():
    """With a bf16 cache a sequence's last row of a whole prompt and the same token decoded agree to the roundings of both."""
    n = 150
    layer = Layer(16, seed=5, seqs=1)
    (raw, heads, att, _), _ = fill(layer, [n])
    got = layer.cache.attend(heads[:H, n - 1:].transpose(0, 1), layer.dtable, dev(np.array([n], np.int32)))
    h64 = bf16_to_f64(host(heads, np.uint16))
    a, b = bf16_to_f64(host(att, np.uint16))[n - 1], bf16_to_f64(host(got, np.uint16))[0]
    for h in range(H):
        o, tol = attnref.attend(h64[h, n - 1:], h64[H + h // (H // KV)], h64[H + KV + h // (H // KV)], [n - 1], D ** -0.5)
        assert np.all(np.abs(a[h] - b[h]) <= 2 * (tol + np.abs(o) * 2.0 ** -8)[0])


def test_a_prompt_that_goes_on_behind_its_cached_prefix():
    """The second part's queries over the prefix read back from the cache and their own keys: the rows of the whole prompt."""
    n, first = 170, 100
    layer = Layer(16, seed=6, seqs=1)
    (raw, heads, att, _), _ = fill(layer, [n])
    k, v = layer.cache.read(dev(np.array([layer.slot(0, p) for p in range(n)], np.int32)))
    m = n - first
    q = heads[:H, first:].contiguous()
    out = torch.empty((m, H, D), dtype=torch.int16, device="cuda")
    fq.fq_attn_prefill(q, D, m * D, k, KV * D, D, v, KV * D, D, m, n, dev(np.array([0, m], np.int32)), dev(np.array([0, n], np.int32)), 1, H,
                       KV, D, D ** -0.5, 1, out, H * D, D)
    h64 = bf16_to_f64(host(heads, np.uint16))
    o, tol, _ = attnref.prefill(h64[:H, first:], h64[H:H + KV], h64[H + KV:], [0, m], [0, n], D ** -0.5, 1)
    attnref.assert_attn(host(out, np.uint16).transpose(1, 0, 2), o, tol, "second part")


@pytest.mark.parametrize("bits", [8, 16])
def test_a_captured_step_serves_any_batch(bits):
    """One graph of a step: replayed at other positions, lengths and idle places, with eager work in between; the lengths,
    the slots and the page table are read on the device."""
    seqs = 4
    layer, twin = (Layer(bits, seed=9, seqs=seqs) for _ in range(2))
    lens = [200, 3, 40, 1]
    fill(layer, lens), fill(twin, lens)
    x, pos, slots, n = layer.token([lens[0], lens[1], lens[2], lens[3]])
    out, want = layer.buffers(), twin.buffers()
    layer.cache.workspace(seqs, H, layer.width)
    layer.heads_of(x, seqs), layer.o.workspace(seqs)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.step(x, pos, slots, n, out)
    twin.rng = np.random.default_rng(1)
    for at in ([200, 3, 40, 1], [201, -1, 41, -1], [202, 4, -1, 2], [-1, -1, -1, -1], [203, 5, 42, 3]):
        new = twin.token(at)
        for dst, src in zip((x, pos, slots, n), new):
            dst.copy_(src)
        twin.step(*new, want)
        ok = np.array(at) >= 0
        for t in out:
            t.fill_(77)
        layer.cache._ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out[1:], want[1:]):
            assert np.array_equal(host(a)[ok], host(b)[ok])
        assert not np.any(host(out[1])[~ok])
        for a, b in zip((layer.cache.k, layer.cache.v), (twin.cache.k, twin.cache.v)):
            for s in range(seqs):
                for p in range(max(at[s], 0)):
                    page, place = divmod(int(layer.slot(s, p)), layer.page)
                    assert torch.equal(a.view(torch.uint8)[page, :, place], b.view(torch.uint8)[page, :, place])


def test_two_graphs_share_a_workspace():
    """Two captured calls of different sizes on one workspace, replayed in turns."""
    rng = np.random.default_rng(3)
    caches = [fq.KVCache(40, 16, KV, D, 8) for _ in range(2)]
    for c in caches:
        n = 40 * 16
        c.write(dev(ref.bf16(rng, n, KV, D)), dev(ref.bf16(rng, n, KV, D)), dev(np.arange(n, dtype=np.int32)))
    calls = []
    ws = torch.empty(fq.fq_attn_decode_workspace_bytes(3, H, KV, D, 40 * 16), dtype=torch.uint8, device="cuda")
    for c, lens in zip(caches, ([600], [300, 17, 0])):
        q = dev(ref.bf16(rng, len(lens), H, D))
        table = dev(np.stack([rng.permutation(40) for _ in lens]).astype(np.int32))
        n, o = dev(np.array(lens, np.int32)), torch.empty((len(lens), H, D), dtype=torch.int16, device="cuda")
        want = host(c.attend(q, table, n)).copy()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.attend(q, table, n, o=o, workspace=ws)
        calls.append((g, o, want, (q, table, n)))
    for _ in range(4):
        for g, o, want, _ in calls:
            o.fill_(9)
            g.replay()
        torch.cuda.synchronize()
        for _, o, want, _ in calls:
            assert np.array_equal(host(o), want)
        ws.fill_(0xFF)


def test_on_other_streams_and_two_at_once():
    """Calls with stream=, and two layers on two streams at once, give what each gives alone."""
    layers = [Layer(8, seed=i, seqs=2) for i in (1, 2)]
    want, args = [], []
    for l in layers:
        fill(l, [180, 33])
        args.append((*l.token([180, 33]), l.buffers()))
        l.step(*args[-1])
        torch.cuda.synchronize()
        want.append([host(t).copy() for t in args[-1][4]])
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(6):
        for l, a, s in zip(layers, args, streams):
            with torch.cuda.stream(s):
                for t in a[4]:
                    t.fill_(5)
                l.step(*a)
    torch.cuda.synchronize()
    for a, w in zip(args, want):
        for t, one in zip(a[4], w):
            assert np.array_equal(host(t), one)
    # stream=: new outputs belong to that stream
    l, a = layers[0], args[0]
    heads = a[4][0]
    s = streams[1]
    s.wait_stream(torch.cuda.current_stream())
    k, v = l.cache.read(a[2], stream=s)
    o = l.cache.attend(heads[:H].transpose(0, 1), l.dtable, a[3], stream=s)
    s.synchronize()
    assert np.array_equal(host(o), want[0][1])
    assert np.array_equal(host(k.view(torch.int16)), host(l.cache.read(a[2])[0].view(torch.int16)))


def test_prompts_captured_and_replayed():
    """Offsets are read on the device: one graph serves packed batches of other lengths."""
    rng = np.random.default_rng(11)
    M, seqs = 400, 4
    q, k, v = (torch.empty((n, M, D), dtype=torch.int16, device="cuda") for n in (H, KV, KV))
    cu, o = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda"), torch.empty((M, H, D), dtype=torch.int16, device="cuda")

    def call():
        fq.fq_attn_prefill(q, D, M * D, k, D, M * D, v, D, M * D, M, M, cu, None, seqs, H, KV, D, 0.125, 1, o, H * D, D)

    def inputs(lens):
        for t in (q, k, v):
            t.copy_(dev(ref.bf16(rng, *t.shape)))
        cu.copy_(dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)))

    inputs([100, 100, 100, 100])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([100] * 4, [400, 0, 0, 0], [1, 2, 3, 394], [0, 130, 0, 7], [0, 0, 0, 0]):
        inputs(lens)
        o.fill_(3)
        call()
        torch.cuda.synchronize()
        want = host(o).copy()
        o.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(o), want)
        assert np.all(host(o)[sum(lens):] == 3)
