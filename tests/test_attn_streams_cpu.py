"""The stream that a caller names is the one that the library is given, for every call between the qkv site and the o site."""
import pytest
import torch

import w4a4_integer_gemm_amd as fq
from w4a4_integer_gemm_amd import _binding as B

HANDLE = 0x5150


class Stream:
    cuda_stream = HANDLE


class Buffer:
    """What the binding asks of a GPU tensor."""
    is_cuda = True

    def data_ptr(self):
        return 0x10000


class Library:
    """Takes every call, and keeps its arguments."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.real, name)

        def call(*args):
            assert len(args) == len(B.SIGNATURES[name][0])
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def library(monkeypatch):
    one = Library(fq.lib())
    monkeypatch.setattr(B, "lib", lambda: one)
    return one


T = Buffer()
CALLS = {
    "fq_qk_norm_rope": lambda **kw: B.fq_qk_norm_rope(T, 512, 64, 8, 8, 4, 2, 64, T, T, 1e-6, 64, 0, T, 1.0, T, 0, T, 512, 64, **kw),
    "fq_rope": lambda **kw: B.fq_rope(T, 512, 64, 8, 8, 6, 64, 64, 0, T, 1.0, T, 0, 0, T, 512, 64, **kw),
    "fq_kv_write": lambda **kw: B.fq_kv_write(T, 256, 64, T, 256, 64, T, 8, 4, 64, 8, 10, 16, T, T, T, T, **kw),
    "fq_kv_read": lambda **kw: B.fq_kv_read(T, T, T, T, 8, 10, 16, T, 8, 4, 64, T, 256, 64, T, 256, 64, **kw),
    "fq_attn_prefill": lambda **kw: B.fq_attn_prefill(T, 512, 64, T, 128, 64, T, 128, 64, 100, 100, T, None, 3, 8, 2, 64, 0.125, 1, T, 512, 64,
                                                      **kw),
    "fq_attn_decode": lambda **kw: B.fq_attn_decode(T, 512, 64, 3, 8, 2, 64, 0.125, T, T, T, T, 8, 10, 16, T, 4, T, T, 512, 64, T, 1 << 20, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_the_binding_hands_the_stream_on(name, library):
    CALLS[name](stream=Stream())
    (called, args), = library.calls
    assert called == name and args[-1] == HANDLE


@pytest.mark.parametrize("bits", [8, 16])
def test_the_cache_hands_the_stream_on(bits, library, monkeypatch):
    monkeypatch.setattr(B, "_dptr", lambda t: None if t is None else t.data_ptr())
    c = fq.KVCache(6, 16, 2, 64, bits, device="cpu")
    heads = lambda n, h: torch.zeros(n, h, 64, dtype=torch.bfloat16)  # noqa: E731
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c.write(heads(5, 2), heads(5, 2), ints(5), stream=Stream())
    c.read(ints(5), heads(5, 2), heads(5, 2), stream=Stream())
    c.attend(heads(3, 8), ints(3, 4), ints(3), o=heads(3, 8), workspace=torch.zeros(1 << 20, dtype=torch.uint8), stream=Stream())
    assert [n for n, _ in library.calls] == ["fq_kv_write", "fq_kv_read", "fq_attn_decode"]
    assert all(args[-1] == HANDLE for _, args in library.calls)
