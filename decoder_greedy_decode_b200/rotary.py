"""Rotary positions (dec_rope_apply, and the rotation of dec_paged_append).

Marshalling only: the angle table is laid out once by dec_rope_phases (host),
the rotation runs in libdec.so's kernels.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import capi, tensors

SCALINGS = {"none": capi.DEC_ROPE_NONE, "linear": capi.DEC_ROPE_LINEAR,
            "ntk": capi.DEC_ROPE_NTK, "parts": capi.DEC_ROPE_PARTS}


class Rope:
    """A rotation of the first `rot_dim` elements of every head.

    interleaved  pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2)
    scaling      "none", "linear", "ntk" or "parts" (dec_rope_scaling), with
                 `factor`; "parts" needs `orig_ctx` and takes alpha, beta
    mscale       factor of the rotated elements; by default 1, and for "parts"
                 0.1 ln(factor) + 1 where factor is above 1
    """

    def __init__(self, rot_dim: int, theta: float = 1e6, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0, orig_ctx: float = 0.0,
                 alpha: float = 1.0, beta: float = 32.0, mscale: Optional[float] = None,
                 device="cuda"):
        if scaling not in SCALINGS:
            raise ValueError(f"scaling {scaling!r}: one of {sorted(SCALINGS)}")
        host = (ctypes.c_uint64 * max(1, rot_dim // 2))()
        capi.dec_rope_phases(rot_dim, theta, SCALINGS[scaling], factor, orig_ctx, alpha, beta, host)
        self.rot_dim, self.interleaved = rot_dim, bool(interleaved)
        if mscale is None:
            mscale = 0.1 * math.log(max(factor, 1.0)) + 1.0 if scaling == "parts" else 1.0
        self.mscale = float(mscale)
        bits = [p - (1 << 64) if p >= (1 << 63) else p for p in host]
        self.phases = torch.tensor(bits, dtype=torch.int64).to(device)
        self.c = capi.dec_rope(self.phases.data_ptr(), rot_dim, int(self.interleaved), self.mscale)
        self.device = self.phases.device
        self.pointer = ctypes.pointer(self.c)

    def apply(self, x: torch.Tensor, positions: torch.Tensor, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
        """Rotate x [tokens, heads, head_dim] (bf16 or fp32; heads contiguous,
        any token stride that is a multiple of 8) by int32 positions [tokens]
        into `out` (which may be x).  The row of a token at a negative position
        is copied as it is."""
        dev = self.device
        if tensors.elsewhere(dev, stream):
            with tensors.guard(dev, stream):
                return self.apply(x, positions, out)
        T, H, D = tensors.check_heads(x, "x", dev)
        if out is None:
            out = torch.empty((T, H, D), dtype=x.dtype, device=dev)
        elif out.dtype != x.dtype or tensors.check_heads(out, "out", dev) != (T, H, D):
            raise ValueError("out must have the shape and type of x")
        tensors.check_tensor(positions, "positions", torch.int32, (T,), dev)
        rc = capi.lib().dec_rope_apply(T, H, D, tensors.dtype_code(x, "x"), x.data_ptr(), x.stride(0),
                                       out.data_ptr(), out.stride(0), positions.data_ptr(),
                                       self.pointer, tensors.current_stream_of(dev))
        if rc:
            raise capi.DecError(rc, "dec_rope_apply")
        return out

