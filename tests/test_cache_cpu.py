"""What KVCache refuses before it hands a pointer to the library.  The caches are built on the CPU; calls that pass every
check end at the binding, which takes GPU tensors only."""
import pytest
import torch

import w4a4_integer_gemm_amd as fq

P, S, KV, D, M, H = 6, 16, 2, 64, 5, 8


@pytest.fixture(scope="module", params=[8, 16])
def cache(request):
    return fq.KVCache(P, S, KV, D, request.param, device="cpu")


def heads(m=M, h=KV, d=D, dtype=torch.bfloat16):
    return torch.zeros(m, h, d, dtype=dtype)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_buffers():
    c = fq.KVCache(P, S, KV, D, 8, device="cpu")
    assert c.k.shape == c.v.shape == (P, KV, S, D) and c.k.dtype == torch.float8_e4m3fn
    assert c.k_scale.shape == c.v_scale.shape == (P, KV, S) and c.k_scale.dtype == torch.float32
    c = fq.KVCache(P, S, KV, D, 16, device="cpu")
    assert c.k.dtype == torch.bfloat16 and c.k_scale is None and c.v_scale is None


@pytest.mark.parametrize("args,match", [((P, S, KV, D, 4), "bits=4"), ((0, S, KV, D, 8), "0 pages"), ((P, S, 0, D, 8), "of 0 heads")])
def test_sizes_are_refused(args, match):
    with pytest.raises(ValueError, match=match):
        fq.KVCache(*args, device="cpu")


@pytest.mark.parametrize("k", [heads(), heads(dtype=torch.int16), heads(M, 3 * KV)[:, KV:2 * KV], heads(KV, M).transpose(0, 1),
                               heads(M, KV, 2 * D)[:, :, :D]])
def test_good_heads_reach_the_binding(cache, k):
    v = heads()
    for call in (lambda: cache.write(k, v, ints(M)), lambda: cache.write(v, k, ints(M)), lambda: cache.read(ints(M), k, v),
                 lambda: cache.read(ints(M)), lambda: cache.attend(heads(3, H), ints(3, 4), ints(3)),
                 lambda: cache.attend(heads(3, H), ints(3, 4), ints(3), o=heads(3, H)),
                 lambda: cache.attend(heads(3, H), ints(3, 4), ints(3), workspace=torch.zeros(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="GPU tensors"):
            call()


@pytest.mark.parametrize("t,match", [
    (heads(dtype=torch.float32), "dtype torch.float32"), (heads(dtype=torch.float16), "dtype torch.float16"),
    (heads(M + 1), r"is \(6, 2, 64\), not \(5, 2, 64\)"), (heads(M, KV + 1), r"not \(5, 2, 64\)"), (heads(M, KV, D - 16), "not"),
    (heads().view(M, KV * D), "not"), (torch.zeros(M, D, KV, dtype=torch.bfloat16).transpose(1, 2), "stride 2 along a head"),
    (heads().to("meta"), "is on meta, the cache on cpu"),
])
def test_heads_are_refused(cache, t, match):
    good = heads()
    for call in (lambda: cache.write(t, good, ints(M)), lambda: cache.write(good, t, ints(M)), lambda: cache.read(ints(M), k=t),
                 lambda: cache.read(ints(M), v=t)):
        with pytest.raises(ValueError, match=match):
            call()


@pytest.mark.parametrize("slots,match", [(torch.zeros(M, dtype=torch.int64), "torch.int64"), (ints(M, 1), "slots is"),
                                         (ints(2 * M)[::2], "strides"), (ints(M).to("meta"), "on meta")])
def test_slots_are_refused(cache, slots, match):
    with pytest.raises(ValueError, match=match):
        cache.write(heads(), heads(), slots)
    with pytest.raises(ValueError, match=match):
        cache.read(slots)


@pytest.mark.parametrize("kw,match", [
    (dict(q=heads(2, H)), "not"), (dict(q=heads(3, H, 32)), "not"), (dict(q=heads(3, H).float()), "dtype"),
    (dict(table=ints(12)), "page_table is"), (dict(table=ints(3, 8)[:, ::2]), "page_table is"),
    (dict(table=torch.zeros(3, 4, dtype=torch.int64)), "int64"), (dict(lens=ints(4)), "lens has 4 values"), (dict(lens=ints(3, 1)), "lens is"),
    (dict(o=heads(3, H + 1)), "o is"), (dict(o=heads(3, H).to("meta")), "o is on meta"),
    (dict(workspace=torch.zeros(8, dtype=torch.uint8, device="meta")), "workspace is on meta"),
])
def test_attend_refuses(cache, kw, match):
    args = dict(q=heads(3, H), table=ints(3, 4), lens=ints(3), o=None, workspace=None)
    args.update(kw)
    with pytest.raises(ValueError, match=match):
        cache.attend(args["q"], args["table"], args["lens"], o=args["o"], workspace=args["workspace"])


def test_strides_of_single_rows_and_heads_do_not_matter():
    """torch gives a dimension of one any stride."""
    c = fq.KVCache(P, S, 1, D, 16, device="cpu")
    t = torch.zeros(D, dtype=torch.bfloat16).as_strided((1, 1, D), (3, 1, 1))
    assert c._heads(t, "t", 1, 1) == (1, D, D)


def test_a_workspace_that_grew_keeps_the_one_before(cache):
    small = cache.workspace(1, H, 4)
    big = cache.workspace(64, H, 400)
    assert big.numel() > small.numel() and any(w is small for w in cache._ws_before)
    assert cache.workspace(2, H, 4) is big


def flat(n=4 * M * KV * D):
    return torch.zeros(n, dtype=torch.bfloat16)


@pytest.mark.parametrize("t,match", [
    (heads(1).expand(M, KV, D), "strides 0 from token"), (heads(M, 1).expand(M, KV, D), "and 0 from head"),
    (flat()[1:].as_strided((M, KV, D), (KV * D, D, 1), 1), "16 bytes"), (heads(M, KV, D + 16)[:, :, 4:D + 4], "16 bytes"),
    (heads(M, KV, D + 4)[:, :, :D], "multiples of 8"), (flat().as_strided((M, KV, D), (KV * D + 2, D, 1)), "multiples of 8"),
    (flat().as_strided((M, KV, D), (D // 2, M * D, 1)), "at least 64"), (flat().as_strided((M, KV, D), (KV * D, D - 8, 1)), "at least 64"),
])
def test_strides_and_starts_that_the_library_refuses_are_a_valueerror(cache, t, match):
    good = heads()
    q, table, lens = heads(M, KV), ints(M, 4), ints(M)
    for call in (lambda: cache.write(t, good, ints(M)), lambda: cache.write(good, t, ints(M)), lambda: cache.read(ints(M), k=t),
                 lambda: cache.read(ints(M), v=t), lambda: cache.attend(t, table, lens), lambda: cache.attend(q, table, lens, o=t)):
        with pytest.raises(ValueError, match=match):
            call()


@pytest.mark.parametrize("token,head", [(D, D), (2 * D, D + D // 2), (D + 8, 2 * D)])
def test_heads_that_overlap_are_inputs_only(cache, token, head):
    t = flat().as_strided((M, KV, D), (token, head, 1))
    apart = token >= head + D
    for call in (lambda: cache.read(ints(M), k=t), lambda: cache.read(ints(M), v=t),
                 lambda: cache.attend(heads(M, KV), ints(M, 4), ints(M), o=t)):
        with pytest.raises(ValueError, match="GPU tensors" if apart else "overlap"):
            call()
    with pytest.raises(ValueError, match="GPU tensors"):
        cache.write(t, heads(), ints(M))


def test_the_strides_taken_are_the_librarys():
    """Whatever passes the checks here passes the library's own, and the other way round."""
    c = fq.KVCache(P, S, 2, 16, 16, device="cpu")
    lib, dev = fq.lib(), 0x10000
    for token in (0, 8, 12, 16, 24, 32, 40, 48):
        for head in (0, 8, 16, 20, 24, 32, 48, 64):
            t = flat(1000).as_strided((3, 2, 16), (token, head, 1))
            for out in (False, True):
                try:
                    c._heads(t, "t", 3, 2, out)
                    ours = True
                except ValueError:
                    ours = False
                if out:
                    code = lib.fq_kv_read(dev, dev, None, None, 16, P, S, 0x10002, 3, 2, 16, dev, token, head, 2 * dev, 32, 16, None)
                else:
                    code = lib.fq_kv_write(dev, token, head, dev, 32, 16, 0x10002, 3, 2, 16, 16, P, S, dev, dev, None, None, None)
                # (the slots, looked at behind the strides, are misaligned: no call goes on to the device)
                assert ours == ("slots" in fq.last_error()), (token, head, out, code, fq.last_error())
