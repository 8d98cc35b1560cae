"""A FoldQuant linear site resident on the GPU (device buffers + calls into libfq).

Holds the packed weight codes, scales, folded gain, smoothing vector and the
workspace as torch tensors, and calls the C ABI on them.  Packing runs in
libfq's host packer; everything else runs in libfq's kernels.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import numpy as np

from . import _binding as B


def _to_dev(a: Optional[np.ndarray], device):
    import torch
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


def _allocating_on(stream):
    """Allocations for a call on `stream` (None: the current one) come from that stream's
    memory: a block that another stream's queued work still uses is not handed out."""
    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _bf16_types():
    """What holds bf16 values: the type itself, or its bits."""
    import torch
    return torch.bfloat16, torch.int16, torch.uint16


def _rows(site, t, name: str, rows: int, cols: int, exact: bool = False) -> int:
    """The row stride of t, bf16 rows of contiguous values on the site's device, at least
    rows x cols of them (exactly cols with `exact`): what the C ABI takes its pointer for."""
    shape, stride = t.shape, t.stride()
    if t.dtype not in site._bf16:
        raise ValueError(f"{name} has dtype {t.dtype}, not bfloat16 (or its bits as int16 or uint16)")
    if len(shape) != 2:
        raise ValueError(f"{name} has {len(shape)} dimensions, not 2")
    if shape[0] < rows or shape[1] < cols or (exact and shape[1] != cols):
        raise ValueError(f"{name} is {shape[0]} x {shape[1]}, not {rows} x {cols}")
    if stride[1] != 1:
        raise ValueError(f"{name} has stride {stride[1]} along its rows, not 1")
    if t.device != site.device:
        raise ValueError(f"{name} is on {t.device}, the site on {site.device}")
    return stride[0]


def _check_vectors(**vectors):
    for name, (v, n) in vectors.items():
        if v is not None and np.shape(v) != (n,):
            raise ValueError(f"{name} has shape {np.shape(v)}, not ({n},)")


def _check_heads(site, y, M: int, head_dim: int):
    """y is [N / head_dim][M][head_dim], contiguous bf16, on the site's device (or a flat buffer of them)."""
    if y.dtype not in site._bf16 or y.device != site.device:
        raise ValueError(f"y is {y.dtype} on {y.device}, not bfloat16 (or its bits) on {site.device}")
    shape = (site.N // head_dim, M, head_dim)
    if not (y.shape == shape or (y.dim() == 1 and y.numel() >= M * site.N)) or not y.is_contiguous():
        raise ValueError(f"y is {tuple(y.shape)} with strides {y.stride()}, not {shape}, contiguous")


class DeviceSite:
    """One linear site: x [M][K] bf16 -> y [M][N] bf16.

    gamma: RMSNorm gain (None for a quant-only site); ascale: smoothing vector;
    fold_into_gain: carry ascale inside the gain (gamma / a, fold before) rather
    than as an explicit divide in the prologue.

    Tensors hold bf16 or its bits (int16, uint16): x M x K, a residual and an output
    M x N, each or more (the first rows and columns are taken), the head layout's output
    [N / head_dim][M][head_dim], contiguous, all on the site's device; ValueError otherwise."""

    def __init__(self, W: np.ndarray, hblock: int, wbits: int, abits: int, gamma=None, ascale=None,
                 fold_after: int = 0, fold_into_gain: bool = True, bias=None, eps: float = 1e-6,
                 device="cuda", codes=None, wscale=None):
        import torch
        # (code bytes per row: K * bits / 8, with 6 bits for the E2M3 storage)
        self.N, self.K = W.shape if W is not None else (codes.shape[0], codes.shape[1] * 8 // wbits)
        self.hblock, self.wbits, self.abits = hblock, wbits, abits
        self.eps, self.fold_after = float(eps), int(fold_after)
        self._bf16 = _bf16_types()
        _check_vectors(gamma=(gamma, self.K), ascale=(ascale, self.K), bias=(bias, self.N))
        self.device = torch.device(device)
        if codes is None:
            codes, wscale = B.fq_pack_weights(W, ascale, fold_after, hblock, wbits)
        self.codes_host, self.wscale_host = codes, wscale
        self.codes = _to_dev(codes, self.device)
        self.device = self.codes.device
        self.wscale = _to_dev(wscale, self.device)
        if gamma is not None and fold_into_gain:
            if fold_after:
                raise ValueError("a gain fold is a fold before the rotation; pass fold_after=0")
            self.gamma_host = B.fq_fold_gain(gamma, ascale)
            self.ascale_host = None
        else:
            self.gamma_host = None if gamma is None else np.ascontiguousarray(gamma, np.float32)
            self.ascale_host = None if ascale is None else np.ascontiguousarray(ascale, np.float32)
        self.gamma = _to_dev(self.gamma_host, self.device)
        self.ascale = _to_dev(self.ascale_host, self.device)
        self.bias = _to_dev(None if bias is None else np.ascontiguousarray(bias, np.float32), self.device)
        self._ws, self._ws_size = None, 0
        self._ws_bytes = {}  # M -> fq_linear_workspace_bytes

    # -- buffers
    def workspace(self, M: int, stream=None):
        nbytes = self._ws_bytes.get(M)
        if nbytes is None:
            nbytes = self._ws_bytes[M] = B.fq_linear_workspace_bytes(M, self.K, self.abits)
        if self._ws is None or self._ws_size < nbytes:
            import torch
            with _allocating_on(stream):
                self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self._ws_size = nbytes
        return self._ws

    def empty_out(self, M: int, stream=None):
        import torch
        with _allocating_on(stream):
            return torch.empty((M, self.N), dtype=torch.int16, device=self.device)

    def empty_codes(self, M: int, stream=None):
        import torch
        with _allocating_on(stream):
            return (torch.empty(B.fq_act_bytes(M, self.K, self.abits), dtype=torch.uint8, device=self.device),
                    torch.empty(M, dtype=torch.float32, device=self.device))

    # -- checks
    def _check_codes(self, codes, scales, M: int):
        need = M * (self.K * self.abits // 8)
        if codes.numel() * codes.element_size() < need or not codes.is_contiguous():
            raise ValueError(f"codes are {need} contiguous bytes for M={M}, not {tuple(codes.shape)} of {codes.dtype}")
        if scales.element_size() != 4 or scales.numel() < M or not scales.is_contiguous():
            raise ValueError(f"scales are {M} float32 values, not {tuple(scales.shape)} of {scales.dtype}")
        if codes.device != self.device or scales.device != self.device:
            raise ValueError(f"codes are on {codes.device} and scales on {scales.device}, the site on {self.device}")

    # -- calls
    def prologue(self, x, codes=None, scales=None, stream=None):
        M = x.shape[0]
        ldx = _rows(self, x, "x", M, self.K)
        if codes is None:
            codes, scales = self.empty_codes(M, stream)
        else:
            self._check_codes(codes, scales, M)
        B.fq_prologue(x, M, self.K, ldx, self.gamma, self.eps, self.ascale, self.fold_after,
                      self.hblock, self.abits, codes, scales, stream)
        return codes, scales

    def gemm(self, codes, scales, M: int, residual=None, y=None, acc=None, stream=None):
        self._check_codes(codes, scales, M)
        ldr = 0 if residual is None else _rows(self, residual, "residual", M, self.N)
        y, ldy = (self.empty_out(M, stream), self.N) if y is None else (y, _rows(self, y, "y", M, self.N))
        if acc is not None and (acc.element_size() != 4 or acc.numel() < M * self.N or not acc.is_contiguous()):
            raise ValueError(f"acc is {M} x {self.N} int32, not {tuple(acc.shape)} of {acc.dtype}")
        B.fq_gemm(codes, scales, M, self.abits, self.codes, self.wscale, self.N, self.K, self.wbits, self.bias,
                  residual, ldr, y, ldy, acc, stream)
        return y

    def linear(self, x, residual=None, y=None, stream=None):
        M = x.shape[0]
        ldx = _rows(self, x, "x", M, self.K)
        ldr = 0 if residual is None else _rows(self, residual, "residual", M, self.N)
        y, ldy = (self.empty_out(M, stream), self.N) if y is None else (y, _rows(self, y, "y", M, self.N))
        ws = self.workspace(M, stream)
        B.fq_linear(x, M, self.K, ldx, self.gamma, self.eps, self.ascale, self.fold_after, self.hblock,
                    self.abits, self.codes, self.wscale, self.N, self.wbits, self.bias, residual,
                    ldr, y, ldy, ws, self._ws_size, stream)
        return y

    def linear_noalloc(self, x, residual=None, y=None, stream=None):
        """fq_linear_noalloc: as linear(), with the library's per-GPU scratch array as the workspace."""
        M = x.shape[0]
        ldx = _rows(self, x, "x", M, self.K)
        ldr = 0 if residual is None else _rows(self, residual, "residual", M, self.N)
        y, ldy = (self.empty_out(M, stream), self.N) if y is None else (y, _rows(self, y, "y", M, self.N))
        B.fq_linear_noalloc(x, M, self.K, ldx, self.gamma, self.eps, self.ascale, self.fold_after,
                            self.hblock, self.abits, self.codes, self.wscale, self.N, self.wbits, self.bias, residual,
                            ldr, y, ldy, stream)
        return y

    def linear_heads(self, x, head_dim: int, residual=None, y=None, stream=None):
        """fq_linear_heads: y is [N / head_dim][M][head_dim] (int16 tensor of bf16 bits)."""
        import torch
        M = x.shape[0]
        ldx = _rows(self, x, "x", M, self.K)
        ldr = 0 if residual is None else _rows(self, residual, "residual", M, self.N)
        if y is None:
            with _allocating_on(stream):
                y = torch.empty((self.N // head_dim, M, head_dim), dtype=torch.int16, device=self.device)
        else:
            _check_heads(self, y, M, head_dim)
        ws = self.workspace(M, stream)
        B.fq_linear_heads(x, M, self.K, ldx, self.gamma, self.eps, self.ascale, self.fold_after, self.hblock,
                          self.abits, self.codes, self.wscale, self.N, self.wbits, self.bias, residual,
                          ldr, head_dim, y, ws, self._ws_size, stream)
        return y

    def workspace_codes(self, M: int):
        """(codes, scales) views of the workspace after fq_linear."""
        import torch
        ws = self.workspace(M)
        nb = B.fq_act_bytes(M, self.K, self.abits)
        off = (nb + 255) // 256 * 256
        return ws[:nb], ws[off:off + 4 * M].view(torch.float32)

    @staticmethod
    def upload(a, device="cuda"):
        return _to_dev(a, device)


class Fp8Site:
    """One FP8 site with block scales: x [M][K] bf16 -> y [M][N] bf16.

    W float32 [N][K], or codes [N][K] and wscale [ceil(N / 128)][K / 128] as a
    checkpoint stores them (numpy arrays, or torch tensors already on the
    device); gamma: RMSNorm gain (None for a quant-only site).

    Tensors hold bf16 or its bits (int16, uint16); x is M x K, a residual or an output
    given for the row layout has M rows and N columns or more, one given for the head
    layout is [N / head_dim][M][head_dim], contiguous; codes, scales and the head layout's
    output may be flat buffers of that size.  All are on the site's device, which is the
    current one; ValueError otherwise.

    linear() uses the site's own workspace, which belongs to one call at a time: calls
    on two streams at once take two sites (of the same codes and wscale).  What a call
    with stream= allocates belongs to that stream.  A
    workspace that grew leaves the one before allocated, since a captured graph may
    still use it."""

    def __init__(self, W: Optional[np.ndarray] = None, gamma=None, bias=None, eps: float = 1e-6, device="cuda",
                 codes=None, wscale=None):
        import torch
        self.eps = float(eps)
        self._bf16 = _bf16_types()
        if codes is None:
            codes, wscale = B.fq_fp8_pack_weights(W)
        if wscale is None or len(codes.shape) != 2:
            raise ValueError("codes are a matrix and come with wscale")
        self.N, self.K = codes.shape
        self.codes = codes if isinstance(codes, torch.Tensor) else _to_dev(codes, torch.device(device))
        self.device = self.codes.device
        self.wscale = wscale if isinstance(wscale, torch.Tensor) else _to_dev(np.asarray(wscale, np.float32), self.device)
        if self.wscale.device != self.device:
            raise ValueError(f"wscale is on {self.wscale.device}, codes on {self.device}")
        if not (self.codes.is_contiguous() and self.wscale.is_contiguous()):
            raise ValueError("codes and wscale must be contiguous")
        if self.codes.element_size() != 1 or self.wscale.dtype != torch.float32:
            raise ValueError("codes are bytes and wscale is float32")
        if self.wscale.numel() != B.fq_fp8_wscale_count(self.N, self.K):
            raise ValueError(f"wscale has {self.wscale.numel()} values, not {B.fq_fp8_wscale_count(self.N, self.K)} "
                             f"for N={self.N} K={self.K}")
        _check_vectors(gamma=(gamma, self.K), bias=(bias, self.N))
        self.gamma = _to_dev(None if gamma is None else np.ascontiguousarray(gamma, np.float32), self.device)
        self.bias = _to_dev(None if bias is None else np.ascontiguousarray(bias, np.float32), self.device)
        self._ws, self._ws_size = None, 0
        self._ws_before = []
        self._ws_bytes = {}  # M -> fq_fp8_linear_workspace_bytes

    # -- buffers
    def workspace(self, M: int, stream=None):
        nbytes = self._ws_bytes.get(M)
        if nbytes is None:
            nbytes = self._ws_bytes[M] = B.fq_fp8_linear_workspace_bytes(M, self.K)
        if self._ws is None or self._ws_size < nbytes:
            import torch
            if self._ws is not None:
                self._ws_before.append(self._ws)
                nbytes = max(nbytes, 2 * self._ws_size)
            with _allocating_on(stream):
                self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self._ws_size = nbytes
        return self._ws

    def workspace_codes(self, M: int):
        """(codes [M][K], scales [K / 128][M]) views of the workspace after linear()."""
        import torch
        ws = self.workspace(M)
        nb = M * self.K
        off = (nb + 255) // 256 * 256
        sc = ws[off:off + 4 * B.fq_fp8_ascale_count(M, self.K)].view(torch.float32)
        return ws[:nb].view(M, self.K), sc.view(self.K // 128, -1)[:, :M]

    def empty_codes(self, M: int, stream=None):
        import torch
        with _allocating_on(stream):
            return (torch.empty((M, self.K), dtype=torch.uint8, device=self.device),
                    torch.empty((self.K // 128, -(-M // 4) * 4), dtype=torch.float32, device=self.device))

    # -- checks
    def _check_device(self):
        import torch
        if self.device.index is not None and torch.cuda.current_device() != self.device.index:
            raise ValueError(f"the site is on {self.device}, the current device is {torch.cuda.current_device()}")

    def _check_codes(self, codes, scales, M: int):
        import torch
        flat = codes.dim() == 1 and codes.numel() >= M * self.K
        if codes.element_size() != 1 or not (codes.shape == (M, self.K) or flat) or not codes.is_contiguous():
            raise ValueError(f"codes are {M} x {self.K} bytes, contiguous, not {tuple(codes.shape)} of {codes.dtype}")
        g, ld = self.K // 128, -(-M // 4) * 4
        flat = scales.dim() == 1 and scales.numel() >= g * ld and scales.stride() == (1,)
        rows = scales.dim() == 2 and scales.shape[0] == g and scales.shape[1] >= M and scales.stride() == (ld, 1)
        if scales.dtype != torch.float32 or not (rows or flat):
            raise ValueError(f"scales are float32 {g} x {M} in rows of {ld}, not {tuple(scales.shape)} of {scales.dtype} "
                             f"with strides {scales.stride()}")
        if codes.device != self.device or scales.device != self.device:
            raise ValueError(f"codes are on {codes.device} and scales on {scales.device}, the site on {self.device}")

    def _out(self, head_dim: int, y, M: int, stream):
        """(y, ldy) of a call: y as given, or a new one."""
        if y is None:
            import torch
            shape = (self.N // head_dim, M, head_dim) if head_dim else (M, self.N)
            with _allocating_on(stream):
                return torch.empty(shape, dtype=torch.int16, device=self.device), 0 if head_dim else self.N
        if not head_dim:
            return y, _rows(self, y, "y", M, self.N)
        _check_heads(self, y, M, head_dim)
        return y, 0

    # -- calls
    def prologue(self, x, codes=None, scales=None, stream=None):
        M = x.shape[0]
        ldx = _rows(self, x, "x", M, self.K, exact=True)
        self._check_device()
        if codes is None:
            codes, scales = self.empty_codes(M, stream)
        else:
            self._check_codes(codes, scales, M)
        B.fq_fp8_prologue(x, M, self.K, ldx, self.gamma, self.eps, codes, scales, stream)
        return codes, scales

    def gemm(self, codes, scales, M: int, residual=None, head_dim: int = 0, y=None, stream=None):
        """y [M][N], or [N / head_dim][M][head_dim], from codes that a prologue or fq_block_norm wrote."""
        self._check_codes(codes, scales, M)
        self._check_device()
        ldr = 0 if residual is None else _rows(self, residual, "residual", M, self.N)
        y, ldy = self._out(head_dim, y, M, stream)
        B.fq_fp8_gemm(codes, scales, M, self.codes, self.wscale, self.N, self.K, self.bias, residual, ldr, head_dim, y, ldy,
                      stream)
        return y

    def linear(self, x, residual=None, head_dim: int = 0, y=None, stream=None):
        M = x.shape[0]
        ldx = _rows(self, x, "x", M, self.K, exact=True)
        self._check_device()
        ldr = 0 if residual is None else _rows(self, residual, "residual", M, self.N)
        y, ldy = self._out(head_dim, y, M, stream)
        ws = self.workspace(M, stream)
        B.fq_fp8_linear(x, M, self.K, ldx, self.gamma, self.eps, self.codes, self.wscale, self.N, self.bias, residual, ldr,
                        head_dim, y, ldy, ws, self._ws_size, stream)
        return y
