"""ctypes binding of include/sdm_train.h: a route's balance, lookups, and the gradients
to a bank.

As in ``_binding``: argument marshalling only, contiguous tensors on one device,
work on torch's current stream of that device. A call's scratch memory is allocated with
the call, unless the caller gives a ``workspace`` of its own (a uint8 tensor).
"""

from __future__ import annotations

from typing import Optional, Union

import torch

from ._binding import _DTYPES, library
from ._memory import _INDEX, _VALUE, PackedBank, _at, _call, _check, _gather_sizes, _route_sizes, _score

SDM_GRAD_WRITE, SDM_GRAD_ADD = 0, 1

_F32 = (torch.float32,)


def _output(device: int, name: str, t: Optional[torch.Tensor], dtypes, shape, like: torch.Tensor) -> torch.Tensor:
    """`t` if it is given and of one of the dtypes and of the shape; else a new tensor of the first."""
    if t is None:
        return torch.empty(shape, dtype=dtypes[0], device=like.device)
    _check(device, name, t, dtypes, shape)
    return t


def _scratch(device: int, workspace: Optional[torch.Tensor], size: int, like: torch.Tensor) -> torch.Tensor:
    if workspace is None:
        return torch.empty((max(size, 16),), dtype=torch.uint8, device=like.device)
    _check(device, "workspace", workspace, (torch.uint8,), None)
    return workspace


def _chunks(device: int, tokens: int, chunk: Optional[int], valid: Optional[int], chunk_valid: Optional[torch.Tensor]):
    """chunk and valid with their defaults: one chunk of all tokens, all of them live."""
    if chunk is None:
        chunk = max(tokens, 1)
    if chunk_valid is not None:
        if chunk < 1 or tokens % chunk:
            raise ValueError(f"tokens ({tokens}) must be a multiple of chunk ({chunk})")
        _check(device, "chunk_valid", chunk_valid, (torch.int32,), (tokens // chunk,))
    return chunk, chunk if valid is None else valid


def sdm_route_balance(logits: torch.Tensor, idx: torch.Tensor, *, score: str = "softmax", chunk: Optional[int] = None,
                      valid: Optional[int] = None, chunk_valid: Optional[torch.Tensor] = None, per_chunk: bool = False,
                      scale: float = 1.0, stream_slots: int = 0, loss: Optional[torch.Tensor] = None,
                      counts: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                      coef: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """How evenly a route uses its keys (``sdm_route_balance`` of include/sdm_train.h).
    Returns (loss, counts, mean, coef): a scalar, int32 and float32 [sequences, keys] and
    float32 [sequences].

    logits [..., streams, keys] and idx [..., k] as ``sdm_route`` took and gave them. The
    tokens, numbered over the leading axes, are live as in a gather: below ``valid`` (or
    chunk_valid[t // chunk]) in their chunk (default: all of them, one chunk). With
    ``per_chunk`` each chunk is a sequence of its own, else all tokens are one. ``counts``
    and ``coef`` are what the backward call takes.
    """
    dev = logits.get_device()
    tokens, keys, streams = _route_sizes(logits)
    _check(dev, "logits", logits, _VALUE, None)
    if idx.dim() < 1:
        raise ValueError("idx must be [..., k]")
    k = idx.shape[-1]
    _check(dev, "idx", idx, _INDEX, logits.shape[:-1] + (k,))
    chunk, valid = _chunks(dev, tokens, chunk, valid, chunk_valid)
    sequences = (tokens // chunk if chunk >= 1 else 0) if per_chunk else 1
    loss = _output(dev, "loss", loss, _F32, (), logits)
    counts = _output(dev, "counts", counts, (torch.int32,), (sequences, keys), logits)
    mean = _output(dev, "mean", mean, _F32, (sequences, keys), logits)
    coef = _output(dev, "coef", coef, _F32, (sequences,), logits)
    lib = library()
    scratch = _scratch(dev, workspace, lib.sdm_route_balance_workspace(tokens, keys, chunk, int(per_chunk)), logits)
    _call(dev, lib.sdm_route_balance, logits.data_ptr(), _DTYPES[logits.dtype], tokens, keys, k, _score(score), chunk, valid,
          _at(chunk_valid), int(per_chunk), scale, max(streams, 1), stream_slots, idx.data_ptr(), _DTYPES[idx.dtype],
          counts.data_ptr(), mean.data_ptr(), coef.data_ptr(), loss.data_ptr(), scratch.data_ptr(), scratch.numel())
    return loss, counts, mean, coef


def sdm_route_balance_backward(logits: torch.Tensor, counts: torch.Tensor, coef: torch.Tensor, *,
                               dloss: Optional[torch.Tensor] = None, score: str = "softmax", chunk: Optional[int] = None,
                               valid: Optional[int] = None, chunk_valid: Optional[torch.Tensor] = None,
                               per_chunk: bool = False, dlogits: Optional[torch.Tensor] = None,
                               accumulate: bool = False) -> torch.Tensor:
    """Gradient of ``sdm_route_balance``'s loss with respect to its logits
    (``sdm_route_balance_backward`` of include/sdm_train.h): dlogits like logits, written
    whole, or with ``accumulate`` added to (to ``sdm_route_backward``'s, say).

    counts and coef as the balance gave them; dloss (default 1) a float32 scalar on the
    device; the other arguments as in the balance.
    """
    dev = logits.get_device()
    tokens, keys, _ = _route_sizes(logits)
    _check(dev, "logits", logits, _VALUE, None)
    chunk, valid = _chunks(dev, tokens, chunk, valid, chunk_valid)
    sequences = (tokens // chunk if chunk >= 1 else 0) if per_chunk else 1
    _check(dev, "counts", counts, (torch.int32,), (sequences, keys))
    _check(dev, "coef", coef, _F32, (sequences,))
    if dloss is not None:
        _check(dev, "dloss", dloss, _F32, None)
        if dloss.numel() != 1:
            raise ValueError(f"dloss must be one value, got {list(dloss.shape)}")
    if dlogits is None:
        if accumulate:
            raise ValueError("accumulate needs dlogits to add to")
        dlogits = torch.empty_like(logits)
    else:
        _check(dev, "dlogits", dlogits, (logits.dtype,), logits.shape)
    _call(dev, library().sdm_route_balance_backward, logits.data_ptr(), _DTYPES[logits.dtype], tokens, keys, _score(score),
          chunk, valid, _at(chunk_valid), int(per_chunk), counts.data_ptr(), coef.data_ptr(), _at(dloss), int(accumulate),
          dlogits.data_ptr())
    return dlogits


def _rng(device: int, rng: Optional[torch.Tensor]):
    if rng is not None:
        _check(device, "rng", rng, (torch.int64,), (2,))
    return _at(rng)


def sdm_lookup(bank: Union[PackedBank, torch.Tensor], idx: torch.Tensor, *, scale: float = 1.0, dropout: float = 0.0,
               rng: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scaled rows of a bank, with dropout (``sdm_lookup`` of include/sdm_train.h):
    [*idx.shape, head_dim] of out_dtype (default: that of a given ``out``, else the bank's,
    float32 of a packed bank).

    bank [num_slots, head_dim] float32 or bfloat16, or a PackedBank; idx int32 or int64 of
    any shape, a row outside the bank (-1, say) is 0. ``dropout`` (taken to the nearest
    2^-16) needs rng, int64 [2] on the device: a seed and an offset, from which the mask is
    computed here and again in ``sdm_lookup_grad``.
    """
    if out is not None and out_dtype not in (None, out.dtype):
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    if isinstance(bank, PackedBank):
        dev, hd, head, default = bank._device, bank.head_dim, bank._head, torch.float32
    else:
        dev = bank.get_device()
        if bank.dim() != 2:
            raise ValueError("bank must be [num_slots, head_dim]")
        _check(dev, "bank", bank, _VALUE, None)
        hd, default = bank.shape[1], bank.dtype
        head = (bank.data_ptr(), None, _DTYPES[bank.dtype], bank.shape[0], hd)
    _check(dev, "idx", idx, _INDEX, None)
    shape = idx.shape + (hd,)
    if out is None:
        out_dtype = default if out_dtype is None else out_dtype
        if out_dtype not in _VALUE:
            raise TypeError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
        out = torch.empty(shape, dtype=out_dtype, device=idx.device)
    else:
        _check(dev, "out", out, _VALUE, shape)
    _call(dev, library().sdm_lookup, *head, idx.numel(), idx.data_ptr(), _DTYPES[idx.dtype], scale, dropout, _rng(dev, rng),
          out.data_ptr(), _DTYPES[out.dtype])
    return out


def _dbank(device: int, dbank: Optional[torch.Tensor], bank_dtype: torch.dtype, num_slots: int, head_dim: int,
           accumulate: bool, like: torch.Tensor) -> torch.Tensor:
    if dbank is None:
        if accumulate:
            raise ValueError("accumulate needs dbank to add to")
        if bank_dtype not in _VALUE:
            raise TypeError(f"bank_dtype must be float32 or bfloat16, got {bank_dtype}")
        return torch.empty((num_slots, head_dim), dtype=bank_dtype, device=like.device)
    _check(device, "dbank", dbank, _VALUE, (num_slots, head_dim))
    return dbank


def sdm_lookup_grad(idx: torch.Tensor, dout: torch.Tensor, num_slots: int, *, scale: float = 1.0, dropout: float = 0.0,
                    rng: Optional[torch.Tensor] = None, bank_dtype: torch.dtype = torch.float32,
                    dbank: Optional[torch.Tensor] = None, accumulate: bool = False,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of a lookup with respect to its bank (``sdm_lookup_grad`` of
    include/sdm_train.h): dbank [num_slots, head_dim] of bank_dtype, written whole, or with
    ``accumulate`` given and added to (rows that idx does not name are not touched). A given
    dbank is float32 or bfloat16, whatever bank_dtype says.

    dout [*idx.shape, head_dim] float32 or bfloat16; idx, scale, dropout and rng as in the
    lookup.
    """
    dev = dout.get_device()
    if dout.dim() < 1:
        raise ValueError("dout must be [*idx.shape, head_dim]")
    hd = dout.shape[-1]
    _check(dev, "idx", idx, _INDEX, None)
    _check(dev, "dout", dout, _VALUE, idx.shape + (hd,))
    dbank = _dbank(dev, dbank, bank_dtype, num_slots, hd, accumulate, dout)
    lib = library()
    n = idx.numel()
    scratch = _scratch(dev, workspace, lib.sdm_bank_grad_workspace(n, num_slots, hd), dout)
    _call(dev, lib.sdm_lookup_grad, n, idx.data_ptr(), _DTYPES[idx.dtype], dout.data_ptr(), _DTYPES[dout.dtype], scale,
          dropout, _rng(dev, rng), dbank.data_ptr(), _DTYPES[dbank.dtype], num_slots, hd, int(accumulate),
          scratch.data_ptr(), scratch.numel())
    return dbank


def sdm_gather_bank_grad(idx0: torch.Tensor, w0: torch.Tensor, dout0: torch.Tensor, num_slots: int, *, chunk: int,
                         valid: Optional[int] = None, chunk_valid: Optional[torch.Tensor] = None,
                         idx1: Optional[torch.Tensor] = None, w1: Optional[torch.Tensor] = None,
                         dout1: Optional[torch.Tensor] = None, bank_dtype: torch.dtype = torch.float32,
                         dbank: Optional[torch.Tensor] = None, accumulate: bool = False,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of a gather's outputs with respect to its bank (``sdm_gather_bank_grad`` of
    include/sdm_train.h): dbank [num_slots, head_dim] of bank_dtype, written whole, or with
    ``accumulate`` given and added to (rows that no live token names are not touched). A given
    dbank is float32 or bfloat16, whatever bank_dtype says.

    idx0, w0 [tokens, width0], idx1, w1 and the padding as in the gather; dout0, dout1
    float32 [tokens, head_dim].
    """
    dev = dout0.get_device()
    if (idx1 is None) != (w1 is None) or (idx1 is None) != (dout1 is None):
        raise ValueError("give idx1, w1 and dout1 for a second operand, or none of them")
    tokens, width0, width1, valid = _gather_sizes(idx0, idx1, chunk, valid, chunk_valid, dev)
    _check(dev, "w0", w0, _VALUE, idx0.shape)
    if dout0.dim() != 2:
        raise ValueError("dout0 must be [tokens, head_dim]")
    hd = dout0.shape[1]
    _check(dev, "dout0", dout0, _F32, (tokens, hd))
    if idx1 is not None:
        _check(dev, "w1", w1, (w0.dtype,), idx1.shape)
        _check(dev, "dout1", dout1, _F32, (tokens, hd))
    dbank = _dbank(dev, dbank, bank_dtype, num_slots, hd, accumulate, dout0)
    lib = library()
    scratch = _scratch(dev, workspace, lib.sdm_bank_grad_workspace(tokens * (width0 + width1), num_slots, hd), dout0)
    _call(dev, lib.sdm_gather_bank_grad, tokens, chunk, valid, _at(chunk_valid), _DTYPES[idx0.dtype], _DTYPES[w0.dtype],
          idx0.data_ptr(), w0.data_ptr(), dout0.data_ptr(), width0, _at(idx1), _at(w1), _at(dout1), width1,
          dbank.data_ptr(), _DTYPES[dbank.dtype], num_slots, hd, int(accumulate), scratch.data_ptr(), scratch.numel())
    return dbank
