"""A paged cache of keys and values on the GPU (device buffers + calls into libfq)."""
from __future__ import annotations

from typing import Optional

from . import _binding as B
from .site import _allocating_on, _bf16_types


class KVCache:
    """Keys and values of one layer in pages of page_size tokens: [pages][kv_heads][page_size][head_dim], bf16
    (bits 16) or e4m3 codes with a float32 scale for a token's head (bits 8).

    Which page holds which tokens of which sequence is the caller's: write() and read() take slots (int32 [M],
    page * page_size + place in the page), attend() a page table (int32 [seqs][max_pages]) and lengths (int32
    [seqs]), all on the device, so that one captured graph serves any batch.

    Heads are tensors [M][heads][head_dim] of bf16 or its bits (int16, uint16) with contiguous values that begin
    on 16 bytes, and strides from token to token and from head to head that are multiples of 8 and at least
    head_dim: a row-major projection's output as .view(M, heads, head_dim), the head layout's as
    .transpose(0, 1).  An output's heads do not overlap.  Everything is on the cache's device, which is the current
    one; ValueError otherwise.  Sizes and workspaces that the library refuses are an FqError.  That an output
    overlaps no input and no other output is the caller's to see to.

    attend() uses the cache's own workspace, which belongs to one call at a time: calls on two
    streams at once pass workspaces of their own.  What a call with stream= allocates belongs to that stream.  A
    workspace that grew leaves the one before allocated, since a captured graph may still use it."""

    def __init__(self, pages: int, page_size: int, kv_heads: int, head_dim: int, bits: int = 8, device="cuda"):
        import torch
        if bits not in (8, 16):
            raise ValueError(f"bits={bits}, not 8 or 16")
        if min(pages, page_size, kv_heads, head_dim) < 1:
            raise ValueError(f"{pages} pages of {page_size} tokens of {kv_heads} heads of {head_dim} values")
        self.pages, self.page_size, self.kv_heads, self.head_dim, self.bits = pages, page_size, kv_heads, head_dim, bits
        self._bf16 = _bf16_types()
        shape = (pages, kv_heads, page_size, head_dim)
        dtype = torch.float8_e4m3fn if bits == 8 else torch.bfloat16
        self.k, self.v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        self.k_scale, self.v_scale = ((torch.empty(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
                                      if bits == 8 else (None, None))
        self.device = self.k.device
        self._ws, self._ws_size = None, 0
        self._ws_before = []

    # -- checks
    def _check_device(self):
        import torch
        if self.device.index is not None and torch.cuda.current_device() != self.device.index:
            raise ValueError(f"the cache is on {self.device}, the current device is {torch.cuda.current_device()}")

    def _heads(self, t, name: str, rows: int, heads: Optional[int], out: bool = False):
        """(heads, token stride, head stride) of [rows][heads][head_dim]; out: they must not overlap."""
        shape, stride, D = t.shape, t.stride(), self.head_dim
        if t.dtype not in self._bf16:
            raise ValueError(f"{name} has dtype {t.dtype}, not bfloat16 (or its bits as int16 or uint16)")
        if len(shape) != 3 or shape[0] != rows or shape[2] != D or (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} is {tuple(shape)}, not ({rows}, {'heads' if heads is None else heads}, {D})")
        if stride[2] != 1:
            raise ValueError(f"{name} has stride {stride[2]} along a head's values, not 1")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        # (the stride of a dimension of one is never used, and torch allows it any value)
        n = shape[1]
        token, head = stride[0] if rows > 1 else n * D, stride[1] if n > 1 else D
        if token < D or head < D or token % 8 or head % 8:
            raise ValueError(f"{name} has strides {token} from token to token and {head} from head to head, not multiples "
                             f"of 8 that are at least {D}")
        if t.data_ptr() % 16:
            raise ValueError(f"{name} does not begin on 16 bytes")
        if out and token < (n - 1) * head + D and head < (rows - 1) * token + D:
            raise ValueError(f"{name} has strides {token} from token to token and {head} from head to head: heads overlap")
        return n, token, head

    def _ints(self, t, name: str, dims: int):
        import torch
        if t.dtype != torch.int32 or t.dim() != dims or not t.is_contiguous():
            raise ValueError(f"{name} is {tuple(t.shape)} of {t.dtype} with strides {t.stride()}, not {dims}-dimensional "
                             "contiguous int32")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")

    # -- buffers
    def workspace(self, seqs: int, q_heads: int, max_pages: int, stream=None):
        """The workspace of an attend() call of this size."""
        nbytes = B.fq_attn_decode_workspace_bytes(seqs, q_heads, self.kv_heads, self.head_dim, max_pages * self.page_size)
        if self._ws is None or self._ws_size < nbytes:
            import torch
            if self._ws is not None:
                self._ws_before.append(self._ws)
                nbytes = max(nbytes, 2 * self._ws_size)
            with _allocating_on(stream):
                self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            self._ws_size = nbytes
        return self._ws

    # -- calls
    def write(self, k, v, slots, stream=None):
        """Store token m's keys and values at slots[m]; a negative slot leaves it out."""
        self._ints(slots, "slots", 1)
        M = slots.shape[0]
        _, kt, kh = self._heads(k, "k", M, self.kv_heads)
        _, vt, vh = self._heads(v, "v", M, self.kv_heads)
        self._check_device()
        B.fq_kv_write(k, kt, kh, v, vt, vh, slots, M, self.kv_heads, self.head_dim, self.bits, self.pages, self.page_size,
                      self.k, self.v, self.k_scale, self.v_scale, stream)

    def read(self, slots, k=None, v=None, stream=None):
        """(k, v) bf16 [M][kv_heads][head_dim] of the tokens at slots; zeros for a negative slot."""
        self._ints(slots, "slots", 1)
        M = slots.shape[0]
        if k is None or v is None:
            import torch
            shape = (M, self.kv_heads, self.head_dim)
            with _allocating_on(stream):
                k = torch.empty(shape, dtype=torch.bfloat16, device=self.device) if k is None else k
                v = torch.empty(shape, dtype=torch.bfloat16, device=self.device) if v is None else v
        _, kt, kh = self._heads(k, "k", M, self.kv_heads, out=True)
        _, vt, vh = self._heads(v, "v", M, self.kv_heads, out=True)
        self._check_device()
        B.fq_kv_read(self.k, self.v, self.k_scale, self.v_scale, self.bits, self.pages, self.page_size, slots, M,
                     self.kv_heads, self.head_dim, k, kt, kh, v, vt, vh, stream)
        return k, v

    def attend(self, q, page_table, lens, scale: Optional[float] = None, o=None, workspace=None, stream=None):
        """o [seqs][q_heads][head_dim] of one token q of each sequence over its first lens[s] tokens (scale:
        head_dim^-1/2 unless given)."""
        self._ints(page_table, "page_table", 2)
        self._ints(lens, "lens", 1)
        seqs, max_pages = page_table.shape
        if lens.shape[0] != seqs:
            raise ValueError(f"lens has {lens.shape[0]} values, page_table {seqs} rows")
        H, qt, qh = self._heads(q, "q", seqs, None)
        if o is None:
            import torch
            with _allocating_on(stream):
                o = torch.empty((seqs, H, self.head_dim), dtype=q.dtype, device=self.device)
        _, ot, oh = self._heads(o, "o", seqs, H, out=True)
        self._check_device()
        if workspace is None:
            workspace = self.workspace(seqs, H, max_pages, stream)
        elif workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace is on {workspace.device}, the cache on {self.device}; it is contiguous")
        B.fq_attn_decode(q, qt, qh, seqs, H, self.kv_heads, self.head_dim,
                         self.head_dim ** -0.5 if scale is None else scale, self.k, self.v, self.k_scale, self.v_scale,
                         self.bits, self.pages, self.page_size, page_table, max_pages, lens, o, ot, oh, workspace,
                         workspace.numel() * workspace.element_size(), stream)
        return o
