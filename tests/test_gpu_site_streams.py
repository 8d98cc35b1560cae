"""Sites called with stream=: what they allocate belongs to that stream, so memory that the current stream has freed
but still writes is not handed out."""
import numpy as np
import pytest
import torch

import blockref as ref
import w4a4_integer_gemm_amd as fq
from fqtest import dev, host

pytestmark = pytest.mark.gpu

K, N, M = 512, 1024, 48


def sites():
    rng = np.random.default_rng(0)
    W = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    return rng, [lambda: fq.Fp8Site(W), lambda: fq.DeviceSite(W, 64, 8, 8)]


def pending_writes(nbytes):
    """A freed block of nbytes that work queued on the current stream fills with 7 some 20 ms from now."""
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(40_000_000)
    t.fill_(7)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("call", ["linear", "prologue", "heads"])
def test_allocations_of_a_call_on_a_stream(kind, call):
    rng, make = sites()
    x = dev(ref.bf16(rng, M, K))
    site = make[kind]()

    def run(s, stream=None):
        if call == "prologue":
            return s.prologue(x, stream=stream)
        if call == "heads":
            return (s.linear(x, head_dim=64, stream=stream) if kind == 0 else s.linear_heads(x, 64, stream=stream)),
        return s.linear(x, stream=stream),

    want = [host(t).copy() for t in run(site)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for size in {t.numel() * t.element_size() for t in run(site)} | {site.workspace(M).numel()}:
        fresh = make[kind]()  # (its workspace is allocated by the call)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        pending_writes(size)
        got = run(fresh, stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            a, b = (host(a)[:, :M], b[:, :M]) if a.dim() == 2 and a.dtype == torch.float32 else (host(a), b)
            assert np.array_equal(a, b), f"{call}: a block of {size} bytes was written by the other stream"
