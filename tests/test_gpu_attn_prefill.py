"""Attention of packed prompts on the GPU against a plain 64-bit reference."""
import numpy as np
import pytest
import torch

import attnref
import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import bf16_to_f64, dev, host

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["auto", "rows", "64", "128", "small", "wide"], autouse=True)
def kernel(request, hook):
    """Every test on each of the kernels, and on the one that its sizes get."""
    hook(f"attn_prefill={request.param}")
    yield request.param


MARK = 0x1234


def strides(layout, heads, rows, D, pad):
    return (D, (rows + pad) * D) if layout == "heads" else (heads * D + 8 * pad, D)


def place(x, layout, pad):
    """Device buffer of bits [heads][rows][D] in a layout with `pad` rows (pieces of 8 values) of NaN between."""
    H, M, D = x.shape
    if layout == "heads":
        buf = np.full((H, M + pad, D), 0x7FC0, np.uint16)
        buf[:, :M] = x
    else:
        buf = np.full((M, H * D + 8 * pad), 0x7FC0, np.uint16)
        buf[:, :H * D] = x.transpose(1, 0, 2).reshape(M, H * D)
    return dev(buf)


def call(q, k, v, cu_q, cu_k, scale, causal, layout="rows", pad=1, out_layout="rows", stream=None, o=None):
    H, M, D = q.shape
    kv, Mk = k.shape[:2]
    o = dev(np.full((M + 1, H, D) if out_layout == "rows" else (H, M + 1, D), MARK, np.uint16)) if o is None else o
    ot, oh = (H * D, D) if out_layout == "rows" else (D, (M + 1) * D)
    up = lambda a: None if a is None else dev(np.asarray(a, np.int32))  # noqa: E731
    fq.fq_attn_prefill(place(q, layout, pad), *strides(layout, H, M, D, pad), place(k, layout, pad), *strides(layout, kv, Mk, D, pad),
                       place(v, layout, pad), *strides(layout, kv, Mk, D, pad), M, Mk, up(cu_q), up(cu_k), len(cu_q) - 1, H, kv, D,
                       scale, int(causal), o, ot, oh, stream)
    got = host(o, np.uint16)
    got = got.transpose(1, 0, 2) if out_layout == "rows" else got
    assert np.all(got[:, M] == MARK), "wrote past the last row"
    return got[:, :M]


def run(lens, more, H, kv, D, causal, layout="rows", seed=0, lead=0, tail=0, scale=None, q_scale=2.0, klens=None, **kw):
    """lead, tail: rows before the first and behind the last sequence, which hold NaN (and keep what o holds)."""
    rng = np.random.default_rng(seed)
    klens = [n + more for n in lens] if klens is None else klens
    cu_q = lead + np.concatenate([[0], np.cumsum(lens)])
    cu_k = lead + np.concatenate([[0], np.cumsum(klens)])
    M, Mk = int(cu_q[-1]) + tail, int(cu_k[-1]) + tail
    q, k, v = ref.bf16(rng, H, max(M, 1), D, scale=q_scale), ref.bf16(rng, kv, max(Mk, 1), D), ref.bf16(rng, kv, max(Mk, 1), D)
    for t, end in ((q, cu_q[-1]), (k, cu_k[-1]), (v, cu_k[-1])):
        t[:, :lead] = 0x7FC0
        t[:, end:] = 0xFF80  # -inf
    scale = D ** -0.5 if scale is None else scale
    same = np.array_equal(cu_q, cu_k) and M == Mk
    got = call(q, k, v, cu_q, None if same and seed % 2 == 0 else cu_k, scale, causal, layout, **kw)
    with np.errstate(invalid="ignore"):
        o, tol, inside = attnref.prefill(*(bf16_to_f64(t) for t in (q, k, v)), cu_q, cu_k, scale, causal)
    assert np.all(got[:, ~inside] == MARK), "wrote a row outside of every sequence"
    attnref.assert_attn(got[:, inside], o[:, inside], tol[:, inside], f"{lens} +{more} {H}/{kv}x{D} causal={causal}")
    return got


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 208, 256])
def test_head_sizes(D, causal):
    run([37, 150], 0, 4, 2, D, causal, seed=D)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 193, 255, 257, 300, 513])
def test_lengths(n, causal):
    for D in (64, 128, 256):
        run([n], 0, 2, 1, D, causal, seed=n)


@pytest.mark.parametrize("n", [300, 3])
@pytest.mark.parametrize("D", [144, 192, 208, 256])
def test_large_heads_with_many_groups_and_few(D, n):
    """Few rows: a group of columns has one workgroup, or two that share the values."""
    run([n], 40, 16, 2, D, 1)


@pytest.mark.parametrize("H,kv", [(1, 1), (3, 3), (8, 1), (28, 4), (7, 1), (40, 8), (36, 2)])
@pytest.mark.parametrize("layout", ["rows", "heads"])
def test_groups_and_layouts(H, kv, layout):
    for causal in (0, 1):
        run([70, 1, 130], 0, H, kv, 64, causal, layout, seed=H, out_layout="rows" if H % 2 else "heads")


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("lens", [[0], [0, 0, 5], [5, 0, 0, 7, 0], [1] * 70, [128] * 5, [127, 129, 128, 1, 255], [3, 200, 1, 0, 64, 65] * 12])
def test_packed_sequences(lens, causal):
    run(lens, 0, 2, 2, 64, causal, seed=len(lens), lead=5, tail=40)


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("more", [1, 63, 64, 100, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_prefix_behind_which_the_prompt_goes_on(more, causal, D):
    run([50, 1, 140], more, 4, 1, D, causal, seed=more, lead=3, tail=9)


@pytest.mark.parametrize("causal", [0, 1])
def test_fewer_keys_than_queries(causal):
    """Rows that see nothing are zero: keys missing at the front, or altogether."""
    got = run([10, 200, 64, 300], 0, 2, 1, 64, causal, klens=[0, 60, 65, 130], seed=1)
    assert not np.any(got[:, :10])
    if causal:
        assert not np.any(got[:, 10:10 + 140])


@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-3, 2.0, -1.0])
@pytest.mark.parametrize("causal", [0, 1])
def test_scales(scale, causal):
    run([90, 300], 0, 2, 1, 64, causal, scale=scale, seed=4)


def test_large_scores():
    """One key decides; the running maximum moves by hundreds, up and down."""
    run([400], 0, 2, 1, 128, 1, q_scale=60.0, seed=7)
    run([400], 0, 2, 1, 128, 0, q_scale=200.0, seed=8)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [0, 1])
def test_needles(D, causal):
    """Row i's score is large at the one key near[i] and nowhere else: its output is that key's value.  Causal: for
    some rows that key is the one behind the last that they see, and does not count."""
    import synth
    rng = np.random.default_rng(D)
    n, more = 333, 37
    m = n + more
    near = np.array([rng.integers(0, (i + more + 1) if causal else m) for i in range(n)])
    near[:: 5] = np.arange(n)[:: 5] + more if causal else m - 1  # the last that it sees
    near[1:: 7] = 0
    hidden = np.zeros(n, bool)
    if causal:
        hidden[2:n - 1:7] = True
        near[hidden] = np.arange(n)[hidden] + more + 1
    ks = np.where(rng.random((m, D)) < 0.5, -1.0, 1.0)  # (products of two of them are far below D)
    to = lambda a: synth.f32_to_bf16_bits(a.astype(np.float32))[None]  # noqa: E731
    q, k, v = to(ks[near] * 4), to(ks), to(rng.standard_normal((m, D)))
    got = call(q, k, v, [0, n], [0, m], 4.0, causal)
    o, tol, _ = attnref.prefill(*(bf16_to_f64(t) for t in (q, k, v)), [0, n], [0, m], 4.0, causal)
    attnref.assert_attn(got, o, tol, "needles")
    there = np.abs(o[0] - bf16_to_f64(v)[0, near]).max(1) < 1e-3
    assert np.array_equal(there, ~hidden)  # the construction


def test_long_sequence_rows():
    """A few thousand keys: rows at both ends and in the middle."""
    rng = np.random.default_rng(5)
    n, H, kv, D = 5000, 2, 1, 128
    q, k, v = ref.bf16(rng, H, n, D, scale=2.0), ref.bf16(rng, kv, n, D), ref.bf16(rng, kv, n, D)
    got = call(q, k, v, [0, n], None, D ** -0.5, 1)
    for i in (0, 1, 63, 64, 127, 128, 2500, 4096, 4990, 4999):
        for h in range(H):
            o, tol = attnref.attend(bf16_to_f64(q)[h, i:i + 1], bf16_to_f64(k)[0], bf16_to_f64(v)[0], [i], D ** -0.5)
            attnref.assert_attn(got[h, i:i + 1], o, tol, f"row {i}")


def test_offsets_cut_off_at_the_ends():
    """Offsets outside [0, M] and [0, M_k]: what lies outside is left out."""
    rng = np.random.default_rng(6)
    H, M, D = 2, 100, 64
    q, k, v = (ref.bf16(rng, H, M, D) for _ in range(3))
    want = call(q, k, v, [0, 40, 100], None, 0.125, 1)
    assert np.array_equal(call(q, k, v, [-7, 40, 1000], [-7, 40, 1000], 0.125, 1), want)


def test_offsets_beyond_32_bits():
    """Rows whose elements lie past 2^32 bytes from the first, in q, k, v and o."""
    rng = np.random.default_rng(9)
    D, M = 64, 300
    ld = 1 << 23  # 16 MiB a row: 300 rows are 5 GB
    ts = [torch.zeros(M * ld, dtype=torch.int16, device="cuda") for _ in range(4)]
    x = [ref.bf16(rng, 1, M, D) for _ in range(3)]
    for t, b in zip(ts, x):
        t.view(M, ld)[:, :D] = dev(b)[0]
    fq.fq_attn_prefill(ts[0], ld, D, ts[1], ld, D, ts[2], ld, D, M, M, dev(np.array([0, 10, M], np.int32)), None, 2, 1, 1, D, 0.125, 1,
                       ts[3], ld, D)
    o, tol, _ = attnref.prefill(*(bf16_to_f64(t) for t in x), [0, 10, M], [0, 10, M], 0.125, 1)
    attnref.assert_attn(host(ts[3].view(M, ld)[:, :D].contiguous(), np.uint16)[None], o, tol, "far rows")
    del ts
    torch.cuda.empty_cache()


def test_repeats_itself():
    rng = np.random.default_rng(10)
    q, k, v = ref.bf16(rng, 8, 700, 128), ref.bf16(rng, 2, 700, 128), ref.bf16(rng, 2, 700, 128)
    first = call(q, k, v, [0, 300, 700], None, 0.1, 1)
    for _ in range(3):
        assert np.array_equal(call(q, k, v, [0, 300, 700], None, 0.1, 1), first)
