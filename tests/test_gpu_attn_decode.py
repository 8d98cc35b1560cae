"""Attention of one token per sequence over the paged cache on the GPU against a plain 64-bit reference."""
import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


class Batch:
    """Sequences in pages of any order; every place that holds no token holds NaN (bf16, codes and scales)."""

    def __init__(self, lens, H, kv, D, page, bits, seed=0, width=None, spare=3, q_scale=2.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.kv, self.D, self.page, self.bits = lens, H, kv, D, page, bits
        need = [-(-max(n, 0) // page) for n in lens]
        pages = sum(need) + spare
        self.width = max(max(need), 1) if width is None else width
        self.cache = fq.KVCache(pages, page, kv, D, bits)
        for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale):
            if t is not None:
                t.view(torch.uint8).fill_(0xFF)
        order = rng.permutation(pages)
        self.table = rng.integers(-5, 2 * pages, (len(lens), self.width)).astype(np.int32)  # (behind the end: anything)
        at = 0
        for i, x in enumerate(need):
            self.table[i, :x] = order[at:at + x]
            at += x
        total = sum(max(n, 0) for n in lens)
        self.k, self.v = ref.bf16(rng, kv, max(total, 1), D), ref.bf16(rng, kv, max(total, 1), D)
        slots = np.concatenate([self.table[i, np.arange(max(n, 0)) // page] * page + np.arange(max(n, 0)) % page
                                for i, n in enumerate(lens)] + [np.zeros(0)]).astype(np.int32)
        if total:
            self.cache.write(dev(self.k).transpose(0, 1), dev(self.v).transpose(0, 1), dev(slots))
        if bits == 8:
            (kq, ks), (vq, vs) = (attnref.quant_heads(bf16_to_f64(t)) for t in (self.k, self.v))
            self.k64, self.v64 = ref.TABLE[kq] * ks[..., None], ref.TABLE[vq] * vs[..., None]
        else:
            self.k64, self.v64 = bf16_to_f64(self.k), bf16_to_f64(self.v)
        self.q = ref.bf16(rng, len(lens), H, D, scale=q_scale)
        self.dev_q, self.dev_table, self.dev_lens = dev(self.q), dev(self.table), dev(np.array(lens, np.int32))

    def run(self, scale=None, **kw):
        return host(self.cache.attend(self.dev_q, self.dev_table, self.dev_lens, scale, **kw), np.uint16)

    def check(self, scale=None, got=None, what=""):
        got = self.run(scale) if got is None else got
        scale = self.D ** -0.5 if scale is None else scale
        at, G = 0, self.H // self.kv
        for i, n in enumerate(self.lens):
            n = max(n, 0)
            for h in range(self.kv):
                q = bf16_to_f64(self.q[i, h * G:(h + 1) * G])
                o, tol = attnref.attend(q, self.k64[h, at:at + n], self.v64[h, at:at + n], np.full(G, n - 1), scale)
                attnref.assert_attn(got[i, h * G:(h + 1) * G], o, tol, f"{what} sequence {i} of {n}, key head {h}")
            at += n
        return got


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 224, 256])
def test_head_sizes(D, bits):
    Batch([1, 45, 300], 6, 2, D, 16, bits, seed=D).check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("H,kv", [(1, 1), (3, 3), (8, 1), (28, 4), (16, 1), (17, 1), (40, 1), (64, 2), (36, 4)])
def test_groups(H, kv, bits):
    Batch([130, 7], H, kv, 64, 32, bits, seed=H).check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("page", [16, 48, 64, 112, 256])
def test_lengths_and_pages(page, bits):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 111, 113, 127, 128, 129, 255, 256, 257, 500, 1025]
    Batch(lens, 4, 2, 64, page, bits, seed=page).check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_long_sequence_in_many_parts(D, bits):
    Batch([20011], 4, 1, D, 64, bits, seed=D).check()


@pytest.mark.parametrize("bits", [8, 16])
def test_idle_places_and_a_wide_table(bits):
    """Lengths of zero and below give zeros; the table is far wider than any sequence."""
    b = Batch([0, 5, -3, 700, 0], 4, 2, 64, 16, bits, width=3000)
    got = b.check()
    assert not np.any(got[[0, 2, 4]])


@pytest.mark.parametrize("bits", [8, 16])
def test_many_sequences(bits):
    rng = np.random.default_rng(1)
    Batch([int(n) for n in rng.integers(0, 200, 300)], 8, 4, 64, 16, bits).check()


@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0, 1e-4])
@pytest.mark.parametrize("bits", [8, 16])
def test_scales(scale, bits):
    Batch([40, 333], 4, 2, 64, 16, bits, q_scale=1.0).check(scale)


@pytest.mark.parametrize("bits", [8, 16])
def test_large_scores(bits):
    Batch([1000, 200], 4, 1, 128, 16, bits, q_scale=100.0).check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_needles(page, bits):
    """Sequence s's query is the key at one place: its output is that value.  The token behind the length would
    have a larger score and is not seen."""
    rng = np.random.default_rng(page)
    places = [0, 1, 15, 16, 17, 31, 32, 47, 48, 63, 64, 100, 127, 128, 129, 255, 256, 300, 511, 512, 699]
    lens = [700] * len(places) + [p + 1 for p in places]
    places = places + places
    kv, D = 1, 64
    b = Batch(lens, 1, kv, D, page, bits, seed=page, spare=2 + len(lens))
    total = sum(lens)
    k = np.where(rng.random((kv, total, D)) < 0.5, -1.0, 1.0)
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]])
    import synth
    to = lambda a: synth.f32_to_bf16_bits(np.ascontiguousarray(a, np.float32))  # noqa: E731
    slots, extra_k, extra_slots = [], [], []
    free = sorted(set(range(b.cache.pages)) - {int(x) for i, n in enumerate(lens) for x in b.table[i, :-(-n // page)]})
    for i, n in enumerate(lens):
        slots += [int(b.table[i, j // page]) * page + j % page for j in range(n)]
        if n % page == 0 and n // page < b.width:
            b.table[i, n // page] = free.pop()
        if n // page < b.width:  # the token behind the last
            extra_slots.append(int(b.table[i, n // page]) * page + n % page)
            extra_k.append(k[:, starts[i] + places[i]] * 4)
    q = k[:, starts + np.array(places)].transpose(1, 0, 2) * 4
    b.k = to(k)
    b.cache.write(dev(b.k).transpose(0, 1), dev(b.v).transpose(0, 1), dev(np.array(slots, np.int32)))
    ek = dev(to(np.stack(extra_k)))
    b.cache.write(ek, torch.full_like(ek, 0x4700), dev(np.array(extra_slots, np.int32)))
    b.k64, b.q = k.astype(np.float64), to(q)
    b.dev_q, b.dev_table = dev(b.q), dev(b.table)
    got = b.check(4.0)
    want = b.v64[0, starts + np.array(places)]
    # every other key is at least 4 * 4 * 2 below in the exponent: the weights of up to 699 of them are below 1e-10.
    # The one weight is 1 times the value's scale (with 16 bits 1 itself): rounded to bf16 with 8 bits, 2^-8 of it,
    # and the output is rounded to bf16, 2^-8 of that
    err = np.abs(bf16_to_f64(got[:, 0]) - want)
    assert np.all(err <= np.abs(want) * ((1 + 2.0 ** -8) ** (2 if bits == 8 else 1) - 1) + 1e-6)


def test_pages_outside_the_cache_are_not_seen():
    """Their tokens drop out; a sequence of nothing else gives zeros."""
    b = Batch([200, 100, 64], 4, 2, 64, 16, 16, seed=2)
    keep = np.ones(sum(b.lens), bool)
    for seq, entry, page in ((0, 0, -1), (0, 3, b.cache.pages), (0, 12, 2 ** 31 - 1), (1, 6, -2 ** 31)):
        b.table[seq, entry] = page
        start = sum(b.lens[:seq]) + 16 * entry
        keep[start:min(start + 16, sum(b.lens[:seq + 1]))] = False
    b.table[2] = -1
    keep[300:] = False
    b.dev_table = dev(b.table)
    got = b.run()
    assert not np.any(got[2])
    for i, (a, e) in enumerate(((0, 200), (200, 300))):
        for h in range(2):
            k, v = b.k64[h, a:e][keep[a:e]], b.v64[h, a:e][keep[a:e]]
            q = bf16_to_f64(b.q[i, 2 * h:2 * h + 2])
            o, tol = attnref.attend(q, k, v, np.full(2, len(k) - 1), 0.125)
            attnref.assert_attn(got[i, 2 * h:2 * h + 2], o, tol, f"sequence {i}")


def test_lengths_past_the_table_are_cut_off():
    b = Batch([64, 32], 2, 1, 64, 16, 16, width=4)
    want = b.run().copy()
    b.dev_lens = dev(np.array([2 ** 31 - 1, 32], np.int32))
    assert np.array_equal(b.run(), want)


def test_a_page_shared_by_sequences():
    """A common prefix: two sequences name the same pages."""
    b = Batch([100, 100], 2, 1, 64, 16, 8, seed=3)
    b.table[1] = b.table[0]
    b.dev_table = dev(b.table)
    b.q[1] = b.q[0]
    b.dev_q = dev(b.q)
    got = b.run()
    assert np.array_equal(got[0], got[1])


def test_strides_of_queries_and_outputs():
    b = Batch([33, 250, 4], 6, 2, 64, 16, 8, seed=4)
    want = b.check()
    seqs, H, D = b.q.shape
    row = torch.full((seqs, H * D + 72), 77, dtype=torch.int16, device="cuda")
    row[:, 8:8 + H * D] = dev(b.q).view(seqs, H * D)
    out = torch.full((H, seqs + 2, D), 77, dtype=torch.int16, device="cuda")
    b.cache.attend(row[:, 8:8 + H * D].view(seqs, H, D), b.dev_table, b.dev_lens, o=out.transpose(0, 1)[:seqs])
    assert np.array_equal(host(out, np.uint16)[:, :seqs].transpose(1, 0, 2), want)
    assert bool((out[:, seqs:] == 77).all())


def test_repeats_itself():
    b = Batch([3000, 17, 900], 8, 2, 128, 16, 8, seed=5)
    first = b.run().copy()
    for _ in range(3):
        b.cache.workspace(3, 8, b.width).fill_(0xFF)  # (what it held does not matter)
        assert np.array_equal(b.run(), first)
