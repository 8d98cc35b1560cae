"""Refusals of the FP8 calls whose arguments would give results that depend on timing."""
import pytest

import w4a4_integer_gemm_amd as fq

DEV, WS = 0x10000, 0x100000  # aligned "device pointers"; validation never reads them
M, N, K = 16, 128, 256


def gemm(m=M, ldr=N, hd=0, ldy=N):
    return fq.lib().fq_fp8_gemm(DEV, DEV, m, DEV, DEV, N, K, None, DEV, ldr, hd, DEV, ldy, None)


def linear(m=M, ldr=N, hd=0, ldy=N):
    return fq.lib().fq_fp8_linear(2 * DEV, m, K, K, None, 0.0, 2 * DEV, 2 * DEV, N, None, DEV, ldr, hd, DEV, ldy, WS, 1 << 20,
                                  None)


@pytest.mark.parametrize("call", [gemm, linear])
@pytest.mark.parametrize("kw", [dict(ldy=N + 8), dict(ldr=N + 8), dict(hd=64), dict(hd=8), dict(hd=N, ldr=N + 8)])
def test_output_over_a_residual_of_another_layout_is_refused(call, kw):
    """Workgroups would overwrite residual values that others have yet to read."""
    assert call(**kw) == 2, fq.last_error()
    assert "residual_bf16" in fq.last_error() and "layout" in fq.last_error()


@pytest.mark.parametrize("call", [gemm, linear])
@pytest.mark.parametrize("kw", [dict(), dict(ldy=N + 8, ldr=N + 8), dict(hd=N), dict(m=1, ldy=N + 8), dict(m=1, hd=64, ldr=N + 8)])
def test_output_over_a_residual_of_its_own_layout_passes_the_checks(call, kw):
    """(One token has one layout.)  What is reported without a device is the device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the pointers are none of this device's")
    assert call(**kw) == 5, fq.last_error()
