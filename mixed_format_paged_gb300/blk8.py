"""``Blk8Cache``: the block-scaled 8-bit cache (mkv_blk8_*).  Holds codes, scales
and workspace as torch tensors and forwards to the C ABI; marshalling only."""
from __future__ import annotations

import torch

from . import binding as B
from .rope import current_stream, outputs

_I32 = torch.int32
_DTYPES = {torch.float32: B.MKV_F32, torch.bfloat16: B.MKV_BF16, torch.float16: B.MKV_F16}


class Blk8Cache:
    """K and V in E4M3 with one scale per (page, kv head), read through page
    tables and lengths on the device.  ``k``, ``v`` [layers, pages, Hkv, P, d]
    float8_e4m3fn and ``k_scale``, ``v_scale`` [layers, pages, Hkv] float32 are the
    cache itself: a program may fill, copy or move pages in them."""

    def __init__(self, num_layers: int, num_q_heads: int, num_kv_heads: int, head_dim: int, page_size: int,
                 num_pages: int, max_batch: int, device: str | torch.device = "cuda", host_only: bool = False, stream=None):
        B.lib()
        self.cfg = B.Blk8Config(num_layers, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, max_batch,
                                B.MKV_POOL_HOST_ONLY if host_only else 0)
        self.handle = None
        nbytes = B.mkv_blk8_workspace_bytes(self.cfg)
        self.host_only = host_only
        self.num_q_heads, self.num_kv_heads, self.head_dim = num_q_heads, num_kv_heads, head_dim
        self.page_size, self.num_pages, self.max_batch = page_size, num_pages, max_batch
        self.k = self.v = self.k_scale = self.v_scale = self.workspace = None
        if host_only:
            self.handle = B.mkv_blk8_create(self.cfg, None, None, None, None, None, 0, None)
            return
        shape = (num_layers, num_pages, num_kv_heads)
        self.k = torch.empty(*shape, page_size, head_dim, dtype=torch.float8_e4m3fn, device=device)
        self.v = torch.empty_like(self.k)
        self.k_scale = torch.zeros(shape, dtype=torch.float32, device=device)
        self.v_scale = torch.zeros(shape, dtype=torch.float32, device=device)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.k.device
        with torch.cuda.device(self.device):
            stream = torch.cuda.current_stream(self.device) if stream is None else stream
            self.handle = B.mkv_blk8_create(self.cfg, self.k, self.v, self.k_scale, self.v_scale, self.workspace, nbytes,
                                            stream)

    def close(self) -> None:
        if self.handle is not None:
            B.mkv_blk8_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _run(self, fn, *args, stream=None):
        """fn(handle, *args, stream) with the cache's device current."""
        if self.host_only:
            return fn(self.handle, *args, stream)
        if stream is None:
            stream = current_stream(self.device.index)
        if torch.cuda.current_device() == self.device.index:
            return fn(self.handle, *args, stream)
        with torch.cuda.device(self.device):
            return fn(self.handle, *args, stream)

    def _check(self, x: torch.Tensor, name: str, shape, dtypes, contiguous=True):
        if x.dtype not in dtypes:
            raise TypeError(f"{name} must be one of {sorted(str(d) for d in dtypes)}, got {x.dtype}")
        if x.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(x.shape)}")
        if contiguous and not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not self.host_only and x.device != self.device:
            raise ValueError(f"{name} must be on {self.device}")

    def _tables(self, lens, table):
        n = lens.shape[0]
        if not (lens.dtype is table.dtype is _I32 and lens.dim() == 1 and table.dim() == 2 and table.shape[0] == n
                and lens.is_contiguous() and table.is_contiguous()
                and (self.host_only or lens.device == table.device == self.device)):
            self._check(lens, "lens", (n,), (_I32,))
            if table.dim() != 2:
                raise ValueError("table must be [n, pages]")
            self._check(table, "table", (n, table.shape[1]), (_I32,))
        return n

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, cu_new: torch.Tensor, lens: torch.Tensor,
               table: torch.Tensor, stream=None):
        """Quantise k, v [tokens, Hkv, d] into the pages of their sequences:
        sequence i's last tokens are rows cu_new[i]:cu_new[i + 1] (int32 [n + 1],
        device); lens [n] counts them already; table [n, pages] int32."""
        n = self._tables(lens, table)
        T = k.shape[0]
        for name, x in (("k", k), ("v", v)):
            self._check(x, name, (T, self.num_kv_heads, self.head_dim), tuple(_DTYPES), contiguous=False)
            if x.dtype != k.dtype or x.stride(2) != 1:
                raise ValueError("k and v must share one dtype and have contiguous dims")
        self._check(cu_new, "cu_new", (n + 1,), (torch.int32,))
        # (strides of a dimension of size 1 say nothing)
        st = [x.stride(d) if x.shape[d] > 1 else 0 for x in (k, v) for d in (0, 1)]
        self._run(B.mkv_blk8_append, layer, n, T, k, v, _DTYPES[k.dtype], *st, cu_new, lens, table, table.shape[1],
                  stream=stream)

    def attention(self, layer: int, q: torch.Tensor, lens: torch.Tensor, table: torch.Tensor,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None, scale: float | None = None, stream=None):
        """Causal attention of each sequence's last nq tokens: q [n, nq, Hq, d] bf16
        or fp16 -> (out, of q's shape and dtype; lse [n, nq, Hq] fp32).  scale: of
        the scores, d ** -0.5 by default."""
        n = self._tables(lens, table)
        if q.dim() != 4:
            raise ValueError("q must be [n, nq, Hq, d]")
        nq = q.shape[1]
        shape = (n, nq, self.num_q_heads, self.head_dim)
        self._check(q, "q", shape, (torch.bfloat16, torch.float16))
        if out is None:
            out, = outputs(stream, q.device, lambda: torch.empty_like(q))
        else:
            self._check(out, "out", shape, (q.dtype,))
        if lse is None:
            lse, = outputs(stream, q.device, lambda: torch.empty(shape[:3], dtype=torch.float32, device=q.device))
        else:
            self._check(lse, "lse", shape[:3], (torch.float32,))
        scale = self.head_dim ** -0.5 if scale is None else scale
        self._run(B.mkv_blk8_attention, layer, n, nq, q, _DTYPES[q.dtype], scale, lens, table, table.shape[1], out, lse,
                  stream=stream)
        return out, lse

    def check_errors(self, stream=None):
        """Raise if a kernel met a page id or length out of range, or a wait ran out."""
        self._run(B.mkv_blk8_check_errors, stream=stream)
