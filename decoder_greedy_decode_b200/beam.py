"""Beam search: the selection over beams and vocabulary, the contiguous cache
that follows the chosen beams, and the sequences that the choices spell
(dec_beam_select, dec_kv_reorder, dec_beam_backtrace).

Marshalling only: every operation runs in libdec.so's kernels.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import capi, tensors


_workspace = {}   # scratch bytes by (groups, beams, vocab, k, device)


class Selection(NamedTuple):
    scores: torch.Tensor    # fp32 [groups, k], best first
    parents: torch.Tensor   # int32 [groups, k], beam within the group
    tokens: torch.Tensor    # int32 [groups, k]
    done: Optional[torch.Tensor]   # uint8 [groups, k]; None without an end token


def _result(t, name: str, dtype, shape, like: torch.Tensor) -> torch.Tensor:
    """`t` if it is given and fits, else a new tensor on `like`'s device."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    tensors.check_tensor(t, name, dtype, shape, like.device)
    return t


def beam_select(logits: torch.Tensor, scores: torch.Tensor, k: Optional[int] = None,
                done: Optional[torch.Tensor] = None, eos: int = -1,
                out_scores: Optional[torch.Tensor] = None,
                out_parents: Optional[torch.Tensor] = None,
                out_tokens: Optional[torch.Tensor] = None,
                out_done: Optional[torch.Tensor] = None, stream=None) -> Selection:
    """The k best (beam, token) of every group by scores + log_softmax(logits).

    logits [groups, beams, vocab] (bf16 or fp32; rows contiguous, equally far
    apart), scores fp32 [groups, beams], done uint8 [groups, beams] (finished
    beams; needs eos).  k defaults to beams.  With k = beams out_scores may be
    scores and out_done done."""
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError("logits must be on a CUDA device")
    if tensors.elsewhere(dev, stream):
        with tensors.guard(dev, stream):
            return beam_select(logits, scores, k, done, eos, out_scores, out_parents, out_tokens,
                               out_done)
    if logits.dim() != 3 or logits.stride(2) != 1:
        raise ValueError("logits must be [groups, beams, vocab] with contiguous rows")
    G, W, V = logits.shape
    # the distance of neighbouring rows
    row = logits.stride(1) if W > 1 else logits.stride(0)
    if G > 1 and W > 1 and logits.stride(0) != W * row:
        raise ValueError("the rows of logits must be equally far apart")
    k = W if k is None else int(k)
    tensors.check_tensor(scores, "scores", torch.float32, (G, W), dev)
    if done is not None:
        tensors.check_tensor(done, "done", torch.uint8, (G, W), dev)
    nb = _workspace.get((G, W, V, k, dev.index))
    if nb is None:
        nb = _workspace[(G, W, V, k, dev.index)] = capi.lib().dec_beam_workspace_bytes(G, W, V, k)
    ws = torch.empty(nb or 256, dtype=torch.uint8, device=dev)
    shape = (G, max(k, 0))
    if out_scores is None and out_parents is None and out_tokens is None:
        # (one allocation for the three)
        bits, out_parents, out_tokens = scores.new_empty((3,) + shape, dtype=torch.int32).unbind()
        out_scores = bits.view(torch.float32)
    else:
        out_scores = _result(out_scores, "out_scores", torch.float32, shape, scores)
        out_parents = _result(out_parents, "out_parents", torch.int32, shape, scores)
        out_tokens = _result(out_tokens, "out_tokens", torch.int32, shape, scores)
    if out_done is not None or eos >= 0:
        out_done = _result(out_done, "out_done", torch.uint8, shape, scores)
    rc = capi.lib().dec_beam_select(
        G, W, V, k, tensors.dtype_code(logits, "logits"), logits.data_ptr(), row, scores.data_ptr(),
        None if done is None else done.data_ptr(), eos, out_scores.data_ptr(),
        out_parents.data_ptr(), out_tokens.data_ptr(),
        None if out_done is None else out_done.data_ptr(), ws.data_ptr(), nb,
        tensors.current_stream_of(dev))
    if rc:
        raise capi.DecError(rc, "dec_beam_select")
    return Selection(out_scores, out_parents, out_tokens, out_done)


def kv_reorder(values: torch.Tensor, parents: torch.Tensor, rows: torch.Tensor,
               scales: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """The first len(parents) sequences of a contiguous cache become copies of
    their parents, in place: values [n_layers, 2, batch, n_kv_heads, max_ctx,
    head_dim] (bf16, or uint8 E4M3 codes with scales), rows[b] rows of each;
    parents and rows int32."""
    if values.dim() != 6 or values.shape[1] != 2:
        raise ValueError("values must be [n_layers, 2, batch, n_kv_heads, max_ctx, head_dim]")
    L, _, B, H, ctx, D = values.shape
    dev = values.device
    if dev.type != "cuda":
        raise ValueError("values must be on a CUDA device")
    if tensors.elsewhere(dev, stream):
        with tensors.guard(dev, stream):
            return kv_reorder(values, parents, rows, scales, status)
    if values.dtype == torch.bfloat16 and scales is None:
        code = capi.DEC_KV_BF16
    elif values.dtype == torch.uint8 and scales is not None:
        code = capi.DEC_KV_FP8_E4M3
        tensors.check_tensor(scales, "scales", torch.float32, (L, 2, B, H, ctx), dev)
    else:
        raise ValueError("values must be bfloat16 without scales, or uint8 codes with scales")
    tensors.check_tensor(values, "values", values.dtype, None, dev)
    n = int(parents.numel())
    tensors.check_tensor(parents, "parents", torch.int32, (n,), dev)
    tensors.check_tensor(rows, "rows", torch.int32, (n,), dev)
    if status is not None:
        tensors.check_tensor(status, "status", torch.int32, (1,), dev)
    rc = capi.lib().dec_kv_reorder(
        L, H, D, code, B, ctx, values.data_ptr(), None if scales is None else scales.data_ptr(), n,
        parents.data_ptr(), rows.data_ptr(), None if status is None else status.data_ptr(),
        tensors.current_stream_of(dev))
    if rc:
        raise capi.DecError(rc, "dec_kv_reorder")


def backtrace(parents: torch.Tensor, tokens: torch.Tensor, stream=None) -> torch.Tensor:
    """The sequences [groups, beams, n_steps] that the choices of a search
    spell: parents, tokens int32 [n_steps, groups, beams]."""
    if parents.dim() != 3:
        raise ValueError("parents must be [n_steps, groups, beams]")
    n, G, W = parents.shape
    tensors.check_tensor(parents, "parents", torch.int32, None)
    tensors.check_tensor(tokens, "tokens", torch.int32, (n, G, W), parents.device)
    dev = parents.device
    if tensors.elsewhere(dev, stream):
        with tensors.guard(dev, stream):
            return backtrace(parents, tokens)
    out = torch.empty((G, W, n), dtype=torch.int32, device=dev)
    capi.dec_beam_backtrace(n, G, W, parents, tokens, out, tensors.current_stream_of(dev))
    return out
