"""The operators between the qkv site and the o site without a GPU: refusals, sizes, and where the paged cache's reads
go, for every lane of a decode call."""
import os
import shutil
import subprocess

import pytest

import w4a4_integer_gemm_amd as fq

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a4_integer_gemm_amd", "csrc")
DEV, BAD = 0x10000, 0x10004  # "device pointers", aligned and not; validation never reads them
ARG, SHAPE, UNSUPPORTED, ALIGN = 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


def norm(x=DEV, xt=512, xh=64, M=8, heads=8, q=4, k=2, D=64, gq=DEV, gk=DEV, eps=1e-6, rot=64, inter=0, freq=DEV, att=1.0, pos=DEV,
         pos0=0, y=2 * DEV, yt=512, yh=64):
    return fq.lib().fq_qk_norm_rope(x, xt, xh, M, heads, q, k, D, gq, gk, eps, rot, inter, freq, att, pos, pos0, y, yt, yh, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(x=None), ARG, "x_bf16 is NULL"), (dict(y=None), ARG, "y_bf16 is NULL"), (dict(freq=None), ARG, "freq is NULL"),
    (dict(M=0), SHAPE, "M=0"), (dict(M=2 ** 31 - 1), SHAPE, "M=2147483647"), (dict(M=2 ** 26), SHAPE, "too large for one launch"),
    (dict(D=24), SHAPE, "head_dim=24"), (dict(D=8), SHAPE, "head_dim=8"), (dict(D=272), SHAPE, "head_dim=272"),
    (dict(heads=0, q=0, k=0), SHAPE, "heads=0"), (dict(heads=70000), SHAPE, "heads=70000"),
    (dict(q=-1), SHAPE, "q_heads=-1"), (dict(k=-1), SHAPE, "k_heads=-1"), (dict(q=7, k=2), SHAPE, "at most heads=8"),
    (dict(q=2 ** 31 - 1, k=2 ** 31 - 1), SHAPE, "at most heads=8"),
    (dict(eps=-1.0), ARG, "eps=-1"), (dict(eps=NAN), ARG, "eps=nan"), (dict(rot=66), SHAPE, "rot_dim=66"),
    (dict(rot=7), SHAPE, "rot_dim=7"), (dict(rot=-2), SHAPE, "rot_dim=-2"), (dict(inter=2), ARG, "interleaved=2"),
    (dict(att=INF), ARG, "attn_scale=inf"), (dict(pos=None, pos0=2 ** 31 - 5), ARG, "passes the last position"),
    (dict(xt=56), SHAPE, "x_token=56 < head_dim=64"), (dict(xh=68), ALIGN, "x_head=68 is not a multiple of 8"),
    (dict(yt=64, yh=64), SHAPE, "make 8 heads of 8 tokens overlap"), (dict(x=BAD), ALIGN, "x_bf16"), (dict(y=BAD), ALIGN, "y_bf16"),
    (dict(y=DEV, yt=520), SHAPE, "in place"), (dict(gq=BAD), ALIGN, "q_gamma"), (dict(gk=BAD), ALIGN, "k_gamma"),
    (dict(freq=BAD), ALIGN, "freq"), (dict(pos=DEV + 2), ALIGN, "positions"),
])
def test_qk_norm_rope_refuses(kw, code, text):
    assert norm(**kw) == code and text in fq.last_error(), fq.last_error()


def write(k=DEV, kt=256, kh=64, v=DEV, vt=256, vh=64, slots=DEV, M=8, kv=4, D=64, bits=8, pages=10, page=16, kc=DEV, vc=DEV, ks=DEV,
          vs=DEV):
    return fq.lib().fq_kv_write(k, kt, kh, v, vt, vh, slots, M, kv, D, bits, pages, page, kc, vc, ks, vs, None)


def read(k=DEV, kt=256, kh=64, v=2 * DEV, vt=256, vh=64, slots=DEV, M=8, kv=4, D=64, bits=8, pages=10, page=16, kc=DEV, vc=DEV,
         ks=DEV, vs=DEV):
    return fq.lib().fq_kv_read(kc, vc, ks, vs, bits, pages, page, slots, M, kv, D, k, kt, kh, v, vt, vh, None)


CACHE = [
    (dict(kc=None), ARG, "k_cache is NULL"), (dict(vc=None), ARG, "v_cache is NULL"), (dict(bits=4), UNSUPPORTED, "kv_bits=4"),
    (dict(ks=None), ARG, "kv_bits=8 needs"), (dict(vs=None), ARG, "kv_bits=8 needs"), (dict(bits=16), ARG, "kv_bits=16 takes no"),
    (dict(D=72), SHAPE, "head_dim=72"), (dict(kv=0), SHAPE, "kv_heads=0"), (dict(kv=40000), SHAPE, "kv_heads=40000"),
    (dict(page=8), SHAPE, "page_size=8"), (dict(page=40), SHAPE, "page_size=40"), (dict(page=65536), SHAPE, "page_size=65536"),
    (dict(pages=0), SHAPE, "pages=0"), (dict(pages=1 << 27), SHAPE, "fewer than 2^31 tokens"), (dict(kc=BAD), ALIGN, "k_cache"),
    (dict(vc=BAD), ALIGN, "v_cache"), (dict(ks=BAD), ALIGN, "k_scale"), (dict(vs=BAD), ALIGN, "v_scale"),
]
ROWS = [
    (dict(M=0), SHAPE, "M=0"), (dict(M=2 ** 31 - 600), SHAPE, "too large for one launch"), (dict(slots=None), ARG, "slots is NULL"),
    (dict(slots=DEV + 2), ALIGN, "slots"), (dict(k=None), ARG, "k_bf16 is NULL"), (dict(v=None), ARG, "v_bf16 is NULL"),
    (dict(kt=56), SHAPE, "k_token=56"), (dict(vh=60), SHAPE, "v_head=60"), (dict(vt=260), ALIGN, "v_token=260"),
    (dict(k=BAD), ALIGN, "k_bf16"), (dict(v=BAD), ALIGN, "v_bf16"),
]


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("kw,code,text", CACHE + ROWS)
def test_cache_calls_refuse(call, kw, code, text):
    assert call(**kw) == code and text in fq.last_error(), fq.last_error()


@pytest.mark.parametrize("kw,code,text", [(dict(kt=64), SHAPE, "overlap"), (dict(vt=128), SHAPE, "overlap"),
                                          (dict(v=DEV), ARG, "k_bf16 and v_bf16 are the same")])
def test_cache_read_refuses_outputs(kw, code, text):
    assert read(**kw) == code and text in fq.last_error(), fq.last_error()


def prefill(q=DEV, qt=512, qh=64, k=DEV, kt=128, kh=64, v=DEV, vt=128, vh=64, M=100, Mk=100, cu=DEV, cuk=None, seqs=3, H=8, kv=2, D=64,
            scale=0.125, causal=1, o=2 * DEV, ot=512, oh=64):
    return fq.lib().fq_attn_prefill(q, qt, qh, k, kt, kh, v, vt, vh, M, Mk, cu, cuk, seqs, H, kv, D, scale, causal, o, ot, oh, None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(q=None), ARG, "q_bf16 is NULL"), (dict(k=None), ARG, "k_bf16 is NULL"), (dict(v=None), ARG, "v_bf16 is NULL"),
    (dict(o=None), ARG, "o_bf16 is NULL"), (dict(cu=None), ARG, "cu_q is NULL"), (dict(M=0), SHAPE, "M=0"), (dict(Mk=0), SHAPE, "M_k=0"),
    (dict(M=2 ** 31 - 1), SHAPE, "M=2147483647"), (dict(Mk=2 ** 31 - 1), SHAPE, "M_k=2147483647"), (dict(seqs=0), SHAPE, "seqs=0"),
    (dict(seqs=2 ** 21), SHAPE, "seqs=2097152"), (dict(M=2 ** 30), SHAPE, "too many for one launch"),
    (dict(H=0), SHAPE, "q_heads=0"), (dict(H=65536), SHAPE, "q_heads=65536"), (dict(kv=0), SHAPE, "kv_heads=0"),
    (dict(kv=3), SHAPE, "whole number of groups"), (dict(kv=16), SHAPE, "whole number of groups"), (dict(D=40), SHAPE, "head_dim=40"),
    (dict(D=512), SHAPE, "head_dim=512"), (dict(scale=INF), ARG, "scale=inf"), (dict(scale=NAN), ARG, "scale=nan"),
    (dict(causal=2), ARG, "causal=2"), (dict(qt=8), SHAPE, "q_token=8"), (dict(kh=72, D=64, kt=68), ALIGN, "k_token=68"),
    (dict(vt=1 << 25), SHAPE, "at most 2^24"), (dict(kt=(1 << 24) + 8), SHAPE, "at most 2^24"), (dict(ot=64), SHAPE, "overlap"),
    (dict(q=BAD), ALIGN, "q_bf16"), (dict(k=BAD), ALIGN, "k_bf16"), (dict(v=BAD), ALIGN, "v_bf16"), (dict(o=BAD), ALIGN, "o_bf16"),
    (dict(cu=DEV + 1), ALIGN, "cu_q"), (dict(cuk=DEV + 2), ALIGN, "cu_k"),
])
def test_prefill_refuses(kw, code, text):
    assert prefill(**kw) == code and text in fq.last_error(), fq.last_error()


def decode(q=DEV, qt=512, qh=64, seqs=3, H=8, kv=2, D=64, scale=0.125, kc=DEV, vc=DEV, ks=DEV, vs=DEV, bits=8, pages=10, page=16,
           table=DEV, width=4, lens=DEV, o=2 * DEV, ot=512, oh=64, ws=DEV, nbytes=1 << 30):
    return fq.lib().fq_attn_decode(q, qt, qh, seqs, H, kv, D, scale, kc, vc, ks, vs, bits, pages, page, table, width, lens, o, ot, oh,
                                   ws, nbytes, None)


@pytest.mark.parametrize("kw,code,text", CACHE + [
    (dict(q=None), ARG, "q_bf16 is NULL"), (dict(o=None), ARG, "o_bf16 is NULL"), (dict(table=None), ARG, "page_table is NULL"),
    (dict(lens=None), ARG, "lens is NULL"), (dict(ws=None), ARG, "workspace is NULL"), (dict(ws=DEV + 16), ALIGN, "256-byte"),
    (dict(nbytes=100), ARG, "workspace_bytes=100 <"), (dict(seqs=0), SHAPE, "seqs=0"), (dict(seqs=2 ** 24), SHAPE, "too many for one launch"),
    (dict(H=7), SHAPE, "whole number of groups"), (dict(width=0), SHAPE, "max_pages=0"), (dict(width=1 << 27), SHAPE, "at most 2^30"),
    (dict(scale=NAN), ARG, "scale=nan"), (dict(table=DEV + 2), ALIGN, "page_table"), (dict(lens=DEV + 2), ALIGN, "lens"),
    (dict(ot=64), SHAPE, "overlap"), (dict(qt=60), SHAPE, "q_token=60"), (dict(q=BAD), ALIGN, "q_bf16"), (dict(o=BAD), ALIGN, "o_bf16"),
])
def test_decode_refuses(kw, code, text):
    assert decode(**kw) == code and text in fq.last_error(), fq.last_error()


@pytest.mark.parametrize("call", [norm, write, read, prefill, decode])
def test_good_arguments_reach_the_device(call):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are none of this device's")
    assert call() == 5, fq.last_error()


def test_decode_workspace_never_shrinks():
    size = fq.fq_attn_decode_workspace_bytes
    for H, kv, D in ((1, 1, 16), (28, 4, 128), (8, 1, 256), (40, 2, 80), (64, 64, 64)):
        for seqs in (1, 2, 3, 7, 64, 127, 128, 129, 300, 5000):
            last = 0
            for n in (1, 16, 127, 128, 129, 1000, 4096, 100000, 1 << 20, 1 << 30):
                now = size(seqs, H, kv, D, n)
                assert now >= last and now % 256 == 0 and now >= seqs * (H * (D + 2) * 4 + 8)
                assert size(seqs + 1, H, kv, D, n) >= now
                last = now
    assert size(0, 8, 2, 64, 10) == 0 and size(1, 8, 3, 64, 10) == 0 and size(1, 8, 2, 20, 10) == 0 and size(1, 8, 2, 64, 0) == 0
    assert size(1, 8, 2, 64, (1 << 30) + 1) == 0


SRC = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "fq_paged.h"
using namespace fq;

int main() {
    long units = 0, wrong = 0;
    srand(1);
    // pages by multiplication
    for (int ps = 16; ps <= 32768; ps += 16) {
        const uint64_t magic = paged_magic(ps);
        const int most = kDecodeMaxLen;
        for (int k = 0; k < 400; ++k) {
            long t = k < 200 ? long(k) * ps / 16 / 16 * 16 : (long(rand()) << 10 ^ rand()) % most;
            if (k % 4 == 1) t = long(ps) * (k + rand() % (most / ps - k > 0 ? most / ps - k : 1));
            if (k % 4 == 2) t = long(ps) * (1 + rand() % (most / ps)) - 16;
            if (k % 4 == 3) t = most - 16 * (1 + k / 4);
            if (t < 0 || t >= most) continue;
            t = t / 16 * 16;
            wrong += paged_entry(int(t), most, magic) != t / ps;
            wrong += paged_entry(most - 1, most, magic) != (most - 1) / ps;
            wrong += paged_entry(int(t) + 64 < most ? int(t) + 64 : int(t), int(t) + 1, magic) != t / ps;
        }
    }
    // batches: every token of every sequence in one part, one wave, one tile; every row inside the cache
    const int lens[] = {-5, 0, 1, 15, 16, 17, 31, 33, 127, 128, 129, 500, 1023, 2000, 3001, 4097};
    const int sizes[] = {16, 48, 64, 112, 256};
    for (int ps : sizes)
        for (int seqs : {1, 2, 16, 64, 150})
            for (int heads : {1, 8, 40, 700}) {
                const int max_pages = 4097 / ps + 1, pages = 7, kv_heads = heads > 1 ? heads / 2 : 1;
                const int tiles = decode_head_tiles(heads, kv_heads), target = decode_target(kv_heads, tiles);
                std::vector<int> len(seqs);
                uint64_t sum = 0;
                for (int s = 0; s < seqs; ++s) {
                    const int want = lens[rand() % 16];
                    len[s] = paged_len(want, max_pages, ps);
                    if (len[s] != (want < 0 ? 0 : want > max_pages * ps ? max_pages * ps : want)) ++wrong;
                    sum += decode_units(len[s]);
                }
                const int per = decode_part_len(sum, target);
                if (per < kDecodeStep || per % kDecodeStep) ++wrong;
                int64_t parts = 0;
                const uint64_t magic = paged_magic(ps);
                for (int s = 0; s < seqs; ++s) {
                    const int count = decode_count(len[s], per);
                    parts += count;
                    std::vector<int> table(max_pages), seen(len[s], 0);
                    for (int& p : table) p = rand() % (pages + 4) - 2;  // some outside the cache
                    for (int part = 0; part < count; ++part) {
                        const int begin = part * per, end = begin + per < len[s] ? begin + per : len[s];
                        for (int wave = 0; wave < kDecodeWaves; ++wave)
                            for (int t = begin + kDecodeTile * wave; t < end; t += kDecodeTile * kDecodeWaves)
                                for (int i = 0; i < 2; ++i, ++units) {
                                    const int ti = t + kDecodeUnit * i, entry = paged_entry(ti, len[s], magic);
                                    if (entry < 0 || entry >= max_pages) { ++wrong; continue; }
                                    const PagedUnit u = paged_unit(table[entry], entry, ti, len[s], pages, ps);
                                    // 16 rows are read, whatever is valid
                                    const int64_t rows = int64_t(pages) * kv_heads * ps;
                                    for (int h = 0; h < kv_heads; ++h) {
                                        const int64_t row = paged_row(u.page, u.first, h, kv_heads, ps);
                                        if (row < 0 || row + kDecodeUnit > rows || u.first + kDecodeUnit > ps || u.first % 4) ++wrong;
                                    }
                                    for (int j = 0; j < kDecodeUnit; ++j) {
                                        const int tok = ti + j, p = tok < len[s] ? table[tok / ps] : -1;
                                        const bool there = tok < len[s] && p >= 0 && p < pages;
                                        if (there != (j < u.valid)) ++wrong;
                                        if (there && (u.page != p || u.first + j != tok % ps)) ++wrong;
                                        if (tok < len[s]) ++seen[tok];
                                    }
                                }
                    }
                    for (int n : seen) wrong += n != 1;
                }
                if (parts > decode_parts(seqs, heads, kv_heads, max_pages * ps)) ++wrong;
            }
    // no batch has more parts than its launch, and they fit the workspace
    for (int k = 0; k < 20000; ++k) {
        const int seqs = 1 + rand() % 200, kv = 1 + rand() % 40, q = kv * (1 + rand() % 40), top = 1 << (rand() % 31);
        const int target = decode_target(kv, decode_head_tiles(q, kv));
        std::vector<int> len(seqs);
        uint64_t sum = 0;
        for (int& n : len) sum += decode_units(n = rand() % 3 ? rand() % top : k % 2 ? top : 0);
        const int per = decode_part_len(sum, target);
        int64_t parts = 0;
        for (int n : len) parts += decode_count(n, per);
        const int64_t most = decode_parts(seqs, q, kv, top);
        if (parts > most || per < kDecodeStep) ++wrong;
        const DecodeWorkspace ws = decode_workspace(seqs, q, kv, 64, top);
        if (ws.stats < size_t(seqs) * 8 || ws.sums < ws.stats + size_t(most) * q * 8 || ws.bytes < ws.sums + size_t(most) * q * 256) ++wrong;
    }
    printf("%ld %ld\n", units, wrong);
    return 0;
}
"""


def test_paged_reads_stay_inside_the_cache_and_cover_every_token_once(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "paged.cpp", tmp_path / "paged"
    src.write_text(SRC)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    units, wrong = (int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert units > 10000 and wrong == 0


LONG = r"""
#include <cstdio>
#include <initializer_list>
#include "fq_paged.h"
using namespace fq;

int main() {
    const uint64_t wide = uint64_t(1) << 32;
    long wrong = 0;
    // parts are as long as they have to be, and no longer than a whole step more, on both sides of 2^32 units
    for (int32_t target : {1, 2, 3, 7, 37, 128, 512, 1023, 1024})
        for (uint64_t base : {uint64_t(target), wide / 2, wide - uint64_t(target), wide, 2 * wide, uint64_t(1) << 40})
            for (int64_t d = -1100; d <= 1100; ++d) {
                if (int64_t(base) + d < 1) continue;
                const uint64_t units = base + d;
                const unsigned __int128 tokens = (unsigned __int128)units * 64;
                unsigned __int128 least = (tokens + target - 1) / target, steps = (least + kDecodeStep - 1) / kDecodeStep;
                if (steps * kDecodeStep > (unsigned __int128)kDecodeMaxLen) steps = kDecodeMaxLen / kDecodeStep;
                const int64_t per = decode_part_len(units, target);
                // (units are rounded up once: at most one step more)
                if (per < int64_t(steps) * kDecodeStep || per > int64_t(steps + 1) * kDecodeStep || per > kDecodeMaxLen) ++wrong;
            }
    if (decode_part_len(0, 1024) != kDecodeStep) ++wrong;
    // batches of the longest sequences: no more parts than the launch and its workspace have
    for (int seqs : {1, 2, 255, 256, 257, 300, 4096})
        for (int kv : {1, 2, 3, 8, 32767})
            for (int tiles : {1, 2, 5})
                for (int less : {0, 1, 63, 64, 65, 64 * 1023, 64 * 1024, 1 << 29}) {
                    const int q = kv * (16 * (tiles - 1) + 1), target = decode_target(kv, decode_head_tiles(q, kv));
                    const int last = kDecodeMaxLen - less;
                    const uint64_t units = uint64_t(seqs - 1) * decode_units(kDecodeMaxLen) + decode_units(last);
                    const int per = decode_part_len(units, target);
                    const int64_t parts = int64_t(seqs - 1) * decode_count(kDecodeMaxLen, per) + decode_count(last, per);
                    if (parts > decode_parts(seqs, q, kv, kDecodeMaxLen)) ++wrong;
                }
    printf("%ld\n", wrong);
    return 0;
}
"""


def test_parts_of_the_longest_batches(tmp_path):
    """Sums of lengths around 2^32 units of 64 tokens: a part's length does not wrap, and no batch has more parts than
    its launch."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "long.cpp", tmp_path / "long"
    src.write_text(LONG)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    assert int(subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout) == 0


def test_hook_takes_the_prompt_kernels_and_nothing_else():
    L = fq.lib()
    try:
        for good in ("attn_prefill=rows", "attn_prefill=64", "attn_prefill=128", "attn_prefill=small", "attn_prefill=wide", "attn_prefill=auto", ""):
            assert L.fq_test_hook(good.encode()) == 0, good
        for bad in ("attn_prefill=32", "attn_prefill=", "attn_prefil=64"):
            assert L.fq_test_hook(bad.encode()) == 1, bad
    finally:
        L.fq_test_hook(b"")


@pytest.mark.parametrize("kernel,fits", [("rows", False), ("64", True), ("128", True), ("small", True), ("wide", False), ("auto", True)])
def test_a_forced_prompt_kernel_of_too_many_threads_is_refused(kernel, fits, hook):
    """The kernels have different rows and threads to a workgroup: each forced one's launch is checked, not the rule's."""
    import torch
    if fits and torch.cuda.is_available():
        pytest.skip("the pointers are none of this device's")
    hook(f"attn_prefill={kernel}")
    code = prefill(M=10 ** 8)
    assert code == (5 if fits else SHAPE) and (fits or "too many for one launch" in fq.last_error()), fq.last_error()


SEARCH = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "fq_paged.h"
using namespace fq;

int main() {
    long wrong = 0, most = 0;
    srand(2);
    for (int n : {1, 2, 63, 64, 65, 127, 128, 129, 1000, 4095, 4096, 4097, 5000, 100000, (1 << 18), (1 << 18) + 1, 1 << 20, (1 << 23) - 1}) {
        std::vector<long> at(n);
        long x = rand() % 3;
        for (long& a : at) a = x, x += 1 + (rand() % 4 ? 0 : rand() % 50);
        for (int k = 0; k < 300; ++k) {
            const long b = k < 3 ? k - 1 : k == 3 ? x + 5 : k == 4 ? at[n - 1] : rand() % (x + 1);
            long steps = 0;
            const int got = last_not_past(n, [&](int first, int step, int probes) {
                ++steps;
                if (probes < 1 || probes > 64) ++wrong;
                int c = 0;
                for (int p = 0; p < probes; ++p) {
                    const long i = first + long(p) * step;
                    if (i < 0 || i >= n) { ++wrong; continue; }
                    c += at[i] <= b;
                }
                return c;
            });
            // at[got] is not past b, the next one is
            if (got < -1 || got >= n || (got >= 0 && at[got] > b) || (got + 1 < n && at[got + 1] <= b)) ++wrong;
            if (n <= 64 ? steps != 1 : steps > (n <= 4096 ? 2 : n <= (1 << 18) ? 3 : 4)) ++wrong;
            most = steps > most ? steps : most;
        }
        // entries in no order: inside 0 .. n - 1 all the same, and it ends
        for (long& a : at) a = rand() % 1000 - 500;
        for (int k = 0; k < 50; ++k) {
            const int got = last_not_past(n, [&](int first, int step, int probes) {
                int c = 0;
                for (int p = 0; p < probes; ++p) {
                    const long i = first + long(p) * step;
                    if (i < 0 || i >= n) { ++wrong; continue; }
                    c += at[i] <= k * 20 - 500;
                }
                return c;
            });
            if (got < -1 || got >= n) ++wrong;
        }
    }
    printf("%ld %ld\n", most, wrong);
    return 0;
}
"""


def test_a_sequence_is_found_in_a_few_steps(tmp_path):
    """However many there are: looking at all of them in every workgroup would take the square of their number."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "search.cpp", tmp_path / "search"
    src.write_text(SEARCH)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    most, wrong = (int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert wrong == 0 and most == 4
