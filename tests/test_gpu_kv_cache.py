"""The paged cache on the GPU: what is written, what stays, what is read back."""
import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


def heads(x, layout):
    """Device tensor [M][kv][D] view of bits [kv][M][D], stored in the layout."""
    return dev(x).transpose(0, 1) if layout == "heads" else dev(np.ascontiguousarray(x.transpose(1, 0, 2)))


def filled(pages, page, kv, D, bits, seed):
    c = fq.KVCache(pages, page, kv, D, bits)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k, c.v, c.k_scale, c.v_scale):
        if t is not None:
            t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def bytes_of(c):
    return [None if t is None else host(t.view(torch.uint8)).copy() for t in (c.k, c.v, c.k_scale, c.v_scale)]


def check(M, kv, D, page, bits, layout, slots, pages, seed=0):
    rng = np.random.default_rng(seed)
    c = filled(pages, page, kv, D, bits, seed)
    before = bytes_of(c)
    x = [ref.bf16(rng, kv, M, D, scale=s) for s in (2.0, 0.3)]
    c.write(*(heads(t, layout) for t in x), dev(slots))
    after = bytes_of(c)
    ok = (slots >= 0) & (slots < pages * page)
    at = slots[ok].astype(np.int64)
    for i, t in enumerate(x):
        new = t.transpose(1, 0, 2)[ok]  # [M][kv][D]
        rows = before[i].reshape(pages, kv, page, -1).copy()
        if bits == 16:
            rows[at // page, :, at % page] = np.ascontiguousarray(new).view(np.uint8).reshape(len(at), kv, 2 * D)
            assert np.array_equal(after[i].reshape(rows.shape), rows)
        else:
            q, s = attnref.quant_heads(bf16_to_f64(new))
            rows[at // page, :, at % page] = q
            scales = before[2 + i].view(np.float32).reshape(pages, kv, page).copy()
            scales[at // page, :, at % page] = s
            # the quotient is a float32 value by definition: codes and scales are equal
            assert np.array_equal(after[i].reshape(rows.shape), rows)
            assert np.array_equal(after[2 + i].view(np.uint32).reshape(scales.shape), scales.view(np.uint32))
    # read back, with a few slots of no token among them
    ask = slots.copy()
    ask[:: 3] = -1
    if M > 4:
        ask[4] = pages * page
    got = c.read(dev(ask))
    good = (ask >= 0) & (ask < pages * page)
    for i, t in enumerate(x):
        bits_in = t.transpose(1, 0, 2)
        out = host(got[i].view(torch.int16), np.uint16)
        assert not np.any(out[~good])
        if bits == 16:
            assert np.array_equal(out[good], bits_in[good])
        else:
            q, s = attnref.quant_heads(bf16_to_f64(bits_in[good]))
            # one float32 product, one rounding to bf16
            want = torch.from_numpy((ref.TABLE[q].astype(np.float32) * s[..., None])).to(torch.bfloat16).view(torch.int16).numpy()
            assert np.array_equal(out[good].view(np.int16), want)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("layout", ["heads", "rows"])
@pytest.mark.parametrize("D,page", [(16, 16), (32, 48), (64, 16), (80, 64), (96, 32), (128, 64), (192, 16), (240, 112), (256, 256)])
def test_write_and_read(D, page, layout, bits):
    M, pages = 77, 9 if page < 64 else 4
    rng = np.random.default_rng(D)
    slots = rng.permutation(pages * page)[:M].astype(np.int32)
    slots[[5, 9]] = -1
    slots[7], slots[8] = pages * page, 2 ** 31 - 1
    slots[11] = -2 ** 31
    check(M, 3, D, page, bits, layout, slots, pages, seed=D)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("M,kv", [(1, 1), (1, 8), (23, 4), (1000, 2)])
def test_tokens_and_heads(M, kv, bits):
    pages, page = M // 16 + 2, 16
    check(M, kv, 128, page, bits, "heads", (np.arange(M) + 13).astype(np.int32), pages, seed=M)


def test_every_last_place_of_the_cache():
    pages, page, kv, D = 5, 16, 2, 64
    check(pages * page, kv, D, page, 8, "rows", np.arange(pages * page)[::-1].astype(np.int32).copy(), pages)


def test_codes_at_the_edges():
    """Zero heads, subnormal scales, the largest values."""
    x = np.zeros((1, 4, 64), np.float32)
    x[0, 1, :] = 3.38e38
    x[0, 2, :8] = [1e-38, -2e-39, 5e-39, 0, 1e-40, -1e-38, 3e-39, 1e-39]
    x[0, 3, 5] = -1.0
    import synth
    bits = synth.f32_to_bf16_bits(x)
    c = fq.KVCache(1, 16, 1, 64, 8)
    c.write(heads(bits, "heads"), heads(bits, "heads"), dev(np.arange(4, dtype=np.int32)))
    q, s = attnref.quant_heads(bf16_to_f64(bits))
    assert np.array_equal(host(c.k.view(torch.uint8))[0, 0, :4], q[0])
    assert np.array_equal(host(c.k_scale)[0, 0, :4], s[0])


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes: its last page."""
    pages, page, kv, D = 1 << 16, 64, 8, 256  # 8 GiB of codes each
    c = fq.KVCache(pages, page, kv, D, 8)
    rng = np.random.default_rng(3)
    slots = np.array([0, pages * page - 1, pages * page - page, pages // 2 * page + 3], np.int32)
    k, v = (ref.bf16(rng, kv, 4, D) for _ in range(2))
    c.write(heads(k, "heads"), heads(v, "heads"), dev(slots))
    for t, x in zip((c.k, c.v), (k, v)):
        q, _ = attnref.quant_heads(bf16_to_f64(x))
        for i, s in enumerate(slots):
            assert np.array_equal(host(t.view(torch.uint8)[int(s) // page, :, int(s) % page]), q[:, i])
    # attention over those four as the last tokens of a sequence whose pages lie there
    table = dev(np.array([[pages - 1]], np.int32))
    c.write(heads(k, "heads"), heads(v, "heads"), dev((np.arange(4) + (pages - 1) * page).astype(np.int32)))
    qq = ref.bf16(rng, 1, kv, D, scale=2.0)
    o = c.attend(dev(qq), table, dev(np.array([4], np.int32)))
    kq, vq = (ref.TABLE[a] * b[..., None] for a, b in (attnref.quant_heads(bf16_to_f64(x)) for x in (k, v)))
    got = host(o, np.uint16)
    for h in range(kv):
        want, tol = attnref.attend(bf16_to_f64(qq)[0, h:h + 1], kq[h], vq[h], [3], D ** -0.5)
        attnref.assert_attn(got[0, h:h + 1], want, tol, "far page")
    del c
    torch.cuda.empty_cache()
