"""``Rope``: rotary positions (mkv_rope).  Holds a frequency table (a plain host
value) and forwards to the C ABI; marshalling only."""
from __future__ import annotations

import torch

from . import binding as B

_DTYPES = {torch.float32: B.MKV_F32, torch.bfloat16: B.MKV_BF16, torch.float16: B.MKV_F16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def current_stream(index: int) -> int:
    """The current CUDA stream of device `index`, as the integer the C ABI takes
    (without the stream object that torch.cuda.current_stream builds)."""
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def outputs(stream, device: torch.device, *make):
    """New tensors make[i]() for a call on `stream` (None: the current one, which costs nothing more).  Where that is
    another one, their memory is `stream`'s, so that no earlier tensor's work on the current stream still uses it, and
    it is not given away, once they are freed, before the current stream is through with them."""
    if stream is not None and device.type == "cuda":
        raw = stream if isinstance(stream, int) else stream.cuda_stream
        current = torch.cuda.current_stream(device)
        if raw != current.cuda_stream:
            on = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
            with torch.cuda.stream(on):
                new = [f() for f in make]
            for x in new:
                x.record_stream(current)
            return new
    return [f() for f in make]


class Rope:
    """Rotary positions of the first `rot_dim` dims of a head; ``scaling`` is
    "none", "linear", "ntk", "yarn" or "wavelength" (see mkv_rope_scaling).
    ``inv_freq`` (rot_dim / 2 angles per position) with ``mscale`` replaces the
    frequencies of ``base`` and ``scaling``."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original_length: float = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 low_freq: float = 1.0, high_freq: float = 4.0, inv_freq=None, mscale: float = 1.0):
        if scaling not in B.MKV_ROPE_SCALINGS:
            raise ValueError(f"scaling {scaling!r}: one of {sorted(B.MKV_ROPE_SCALINGS)}")
        if inv_freq is not None:
            self.table = B.mkv_rope_from_frequencies(rot_dim, interleaved, mscale, inv_freq)
        else:
            self.table = B.mkv_rope_init(B.RopeConfig(rot_dim, int(interleaved), B.MKV_ROPE_SCALINGS[scaling], 0, base,
                                                      factor, original_length, beta_fast, beta_slow, low_freq, high_freq))
        self.rot_dim = rot_dim

    @property
    def inv_freq(self) -> list[float]:
        return list(self.table.inv_freq[:self.rot_dim // 2])

    @property
    def mscale(self) -> float:
        return self.table.mscale

    @staticmethod
    def _rows(name, x, out, tokens, d, like, stream):
        """(output, C arguments) of q or k; out None: a new contiguous tensor."""
        shape, st = x.shape, x.stride()
        if len(shape) != 3 or shape[0] != tokens or shape[2] != d or (d > 1 and st[2] != 1):
            raise ValueError(f"{name} must be [tokens, heads, d] with contiguous dims and q's tokens and d")
        if x is not like and not (x.dtype is like.dtype and x.device == like.device):
            raise TypeError("q, k and their outputs must share one dtype and device")
        heads = shape[1]
        if out is None:
            new = lambda: torch.empty_like(x, memory_format=torch.contiguous_format)  # noqa: E731
            out = new() if stream is None else outputs(stream, x.device, new)[0]
            return out, B.RopeRows(x.data_ptr(), out.data_ptr(), heads, 0, st[0], st[1], heads * d, d)
        so = out.stride()
        if out.shape != shape or (d > 1 and so[2] != 1):
            raise ValueError(f"the output of {name} must have its shape and contiguous dims")
        if not (out.dtype is like.dtype and out.device == like.device):
            raise TypeError("q, k and their outputs must share one dtype and device")
        return out, B.RopeRows(x.data_ptr(), out.data_ptr(), heads, 0, st[0], st[1], so[0], so[1])

    def __call__(self, q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor,
                 q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, inverse: bool = False,
                 stream=None):
        """Rotate q [T, Hq, d] and k [T, Hkv, d] (or None) at positions [T] (int32
        or int64, on the device).  Returns (q_out, k_out); pass q_out=q, k_out=k
        to work in place.  inverse: the transpose, i.e. the gradients of q and k
        from those of the outputs.  The call is not recorded by autograd, and
        refuses tensors that it would have to be recorded for."""
        dtype = _DTYPES.get(q.dtype)
        if dtype is None:
            raise TypeError("q must be float32, bfloat16 or float16")
        if torch.is_grad_enabled() and (q.requires_grad or k is not None and k.requires_grad or
                                        q_out is not None and q_out.requires_grad or k_out is not None and k_out.requires_grad):
            raise RuntimeError("Rope is not recorded by autograd: call it under torch.no_grad() (an autograd function's "
                               "forward is), with inverse=True for the gradients")
        T, d, device = q.shape[0], q.shape[-1], q.device
        pt = positions.dtype
        if (pt is not torch.int64 and pt is not torch.int32) or positions.shape != (T,) or not positions.is_contiguous():
            raise TypeError("positions must be a contiguous [T] int32 or int64 tensor")
        if positions.device != device or device.type != "cuda":
            raise TypeError("q and positions must be on one CUDA device")
        q_out, rows_q = self._rows("q", q, q_out, T, d, q, stream)
        rows_k = None
        if k is not None:
            k_out, rows_k = self._rows("k", k, k_out, T, d, q, stream)
        if stream is None:
            stream = current_stream(device.index)
        args = (self.table, T, d, positions, 8 if pt is torch.int64 else 4, rows_q, rows_k, dtype, inverse, stream)
        if device.index == torch.cuda.current_device():
            B.mkv_rope(*args)
        else:
            with torch.cuda.device(device):
                B.mkv_rope(*args)
        return q_out, k_out
