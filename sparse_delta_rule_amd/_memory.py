"""ctypes binding of include/sdm_memory.h: the slot router and packed banks.

As in ``_binding``: argument marshalling only, contiguous tensors on one device,
work on torch's current stream of that device.
"""

from __future__ import annotations

from typing import Optional, Union

import torch

from ._binding import _DTYPES, _raise, library

SDM_MX8, SDM_MX4 = 4, 5
SDM_MAX_KEYS = 65536

_SCORES = {"softmax": 0, "sigmoid": 1}
_KINDS = {"mx8": SDM_MX8, "mx4": SDM_MX4}
_INDEX = (torch.int32, torch.int64)
_VALUE = (torch.float32, torch.bfloat16)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _check(device: int, name: str, t: torch.Tensor, dtypes, shape):
    """A contiguous tensor of the device, of one of the dtypes and of the shape (None: any)."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has unsupported dtype {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if device < 0 or t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, the call on device {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_current_stream = torch._C._cuda_getCurrentRawStream  # the handle alone: a tenth of the stream object's cost


def _call(device: int, fn, *args):
    """The library's call on the device's current stream."""
    if torch.cuda.current_device() == device:
        rc = fn(*args, _current_stream(device))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _current_stream(device))
    if rc != 0:
        _raise(rc)


def _score(score: str) -> int:
    try:
        return _SCORES[score]
    except KeyError:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}") from None


def _route_sizes(logits: torch.Tensor):
    """tokens, keys and streams of logits [..., streams, keys]."""
    if logits.dim() < 1:
        raise ValueError("logits must be [..., keys]")
    keys = logits.shape[-1]
    return (logits.numel() // keys if keys else 0), keys, (logits.shape[-2] if logits.dim() > 1 else 1)


def sdm_route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None,
              groups: int = 1, kept_groups: Optional[int] = None, group_top: int = 1, normalise: bool = False,
              scale: float = 1.0, stream_slots: int = 0, idx_dtype: torch.dtype = torch.int64,
              w_dtype: torch.dtype = torch.float32, idx: Optional[torch.Tensor] = None,
              w: Optional[torch.Tensor] = None):
    """The k best keys of each token and their weights (``sdm_route`` of
    include/sdm_memory.h). Returns (idx, w), both [..., k].

    logits [..., keys] float32 or bfloat16; bias [keys] float32 is added to the scores
    for the choice alone; with ``groups`` the choice is from the ``kept_groups`` best
    groups (default: all). The last axis but one of logits counts streams: stream s's
    keys are slots s * stream_slots + key (stream_slots 0: the keys are the slots), so
    [streams, keys] and [steps, streams, keys] give what ``sdm_decode_step`` and
    ``sdm_decode_steps`` take. idx and w are allocated (idx_dtype, w_dtype) when not given.
    """
    dev = logits.get_device()
    tokens, keys, streams = _route_sizes(logits)
    _check(dev, "logits", logits, _VALUE, None)
    shape = logits.shape[:-1] + (k,)
    if idx is None:
        if idx_dtype not in _INDEX:
            raise TypeError(f"idx_dtype must be int32 or int64, got {idx_dtype}")
        idx = torch.empty(shape, dtype=idx_dtype, device=logits.device)
    else:
        _check(dev, "idx", idx, _INDEX, shape)
    if w is None:
        if w_dtype not in _VALUE:
            raise TypeError(f"w_dtype must be float32 or bfloat16, got {w_dtype}")
        w = torch.empty(shape, dtype=w_dtype, device=logits.device)
    else:
        _check(dev, "w", w, _VALUE, shape)
    if bias is not None:
        _check(dev, "bias", bias, (torch.float32,), (keys,))
    _call(dev, library().sdm_route, logits.data_ptr(), _DTYPES[logits.dtype], tokens, keys, k, _score(score),
          _at(bias), groups, groups if kept_groups is None else kept_groups, group_top, int(normalise), scale,
          max(streams, 1), stream_slots, idx.data_ptr(), _DTYPES[idx.dtype], w.data_ptr(), _DTYPES[w.dtype])
    return idx, w


def sdm_route_backward(logits: torch.Tensor, idx: torch.Tensor, dw: torch.Tensor, *, score: str = "softmax",
                       bias: Optional[torch.Tensor] = None, normalise: bool = False, scale: float = 1.0,
                       stream_slots: int = 0, dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``sdm_route``'s weights with respect to its logits
    (``sdm_route_backward`` of include/sdm_memory.h): dlogits like logits, written whole.

    idx as the route gave it, dw [..., k] float32 or bfloat16 the gradient of w; the other
    arguments as in the route.
    """
    dev = logits.get_device()
    tokens, keys, streams = _route_sizes(logits)
    _check(dev, "logits", logits, _VALUE, None)
    if idx.dim() < 1:
        raise ValueError("idx must be [..., k]")
    k = idx.shape[-1]
    shape = logits.shape[:-1] + (k,)
    _check(dev, "idx", idx, _INDEX, shape)
    _check(dev, "dw", dw, _VALUE, shape)
    if bias is not None:
        _check(dev, "bias", bias, (torch.float32,), (keys,))
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    else:
        _check(dev, "dlogits", dlogits, (logits.dtype,), logits.shape)
    _call(dev, library().sdm_route_backward, logits.data_ptr(), _DTYPES[logits.dtype], tokens, keys, k, _score(score),
          _at(bias), int(normalise), scale, max(streams, 1), stream_slots, idx.data_ptr(), _DTYPES[idx.dtype],
          dw.data_ptr(), _DTYPES[dw.dtype], dlogits.data_ptr())
    return dlogits


class PackedBank:
    """A bank in 8 ("mx8") or 4 ("mx4") bits: its code and scale arrays, laid out as
    include/sdm_memory.h says. Holds the two tensors, which must not be resized, and
    their addresses: its fields cannot be replaced, and a copy is a bank of the copied
    tensors."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, head_dim: int, kind: str = "mx8"):
        row, scale = self.row_bytes(head_dim, kind)
        if codes.dim() != 2:
            raise ValueError("codes must be [num_slots, row_bytes]")
        num_slots, device = codes.shape[0], codes.get_device()
        _check(device, "codes", codes, (torch.uint8,), (num_slots, row))
        _check(device, "scales", scales, (torch.uint8,), (num_slots, scale))
        self.__dict__.update(codes=codes, scales=scales, num_slots=num_slots, head_dim=head_dim, kind=kind,
                             dtype=_KINDS[kind], device=codes.device, _device=device,
                             _head=(codes.data_ptr(), scales.data_ptr(), _KINDS[kind], num_slots, head_dim))

    _FIELDS = frozenset(("codes", "scales", "num_slots", "head_dim", "kind", "dtype", "device", "_device", "_head"))

    def __setattr__(self, name, value):
        if name in self._FIELDS:
            raise AttributeError(f"{name} of a packed bank cannot be replaced: make another bank")
        super().__setattr__(name, value)

    def __reduce__(self):
        added = {name: value for name, value in self.__dict__.items() if name not in self._FIELDS}
        return type(self), (self.codes, self.scales, self.head_dim, self.kind), added

    @staticmethod
    def row_bytes(head_dim: int, kind: str = "mx8") -> tuple:
        """(bytes of a row of codes, bytes of a row of scales)."""
        if kind not in _KINDS:
            raise ValueError(f"kind must be one of {sorted(_KINDS)}, got {kind!r}")
        lib = library()
        got = lib.sdm_packed_row_bytes(_KINDS[kind], head_dim), lib.sdm_packed_scale_bytes(_KINDS[kind], head_dim)
        if got[0] == 0:
            raise ValueError(f"head_dim {head_dim} is out of range")
        return got

    @classmethod
    def empty(cls, num_slots: int, head_dim: int, kind: str = "mx8", device="cuda") -> "PackedBank":
        """A packed bank of zeros."""
        row, scale = cls.row_bytes(head_dim, kind)
        return cls(torch.zeros((num_slots, row), dtype=torch.uint8, device=device),
                   torch.zeros((num_slots, scale), dtype=torch.uint8, device=device), head_dim, kind)


def sdm_bank_pack(packed: PackedBank, rows: torch.Tensor, *, slots: Optional[torch.Tensor] = None,
                  row_idx: Optional[torch.Tensor] = None) -> PackedBank:
    """Quantise rows into slots of a packed bank (``sdm_bank_pack`` of
    include/sdm_memory.h), in place; returns the bank.

    rows [num_rows, head_dim] float32 or bfloat16. Row ``row_idx[i]`` (default i) goes to
    slot ``slots[i]`` (default i); both int32 or int64 of one shape. A negative slot
    stores nothing; a slot given twice must be given the same row, as with
    ``row_idx = slots`` to bring a packed copy of a bank up to date.
    """
    dev = packed._device
    if rows.dim() != 2:
        raise ValueError("rows must be [num_rows, head_dim]")
    _check(dev, "rows", rows, _VALUE, (rows.shape[0], packed.head_dim))
    n, index = rows.shape[0], torch.int64
    for name, t in (("row_idx", row_idx), ("slots", slots)):
        if t is not None:
            _check(dev, name, t, _INDEX, None)
            n, index = t.numel(), t.dtype
    if row_idx is not None and slots is not None and (row_idx.shape != slots.shape or row_idx.dtype != slots.dtype):
        raise ValueError("row_idx and slots must share shape and dtype")
    codes, scales, kind, num_slots, hd = packed._head
    _call(dev, library().sdm_bank_pack, codes, scales, kind, num_slots, hd, rows.data_ptr(), _DTYPES[rows.dtype],
          rows.shape[0], n, _at(row_idx), _at(slots), _DTYPES[index])
    return packed


def _gather_sizes(idx0, idx1, chunk, valid, chunk_valid, dev):
    """Checks of a gather's slots; returns (tokens, width0, width1, valid)."""
    if idx0.dim() != 2:
        raise ValueError("idx0 must be [tokens, width0]")
    _check(dev, "idx0", idx0, _INDEX, None)
    tokens, width1 = idx0.shape[0], 0
    if idx1 is not None:
        if idx1.dim() != 2 or idx1.shape[0] != tokens:
            raise ValueError("idx1 must be [tokens, width1]")
        _check(dev, "idx1", idx1, (idx0.dtype,), None)
        width1 = idx1.shape[1]
    if chunk_valid is not None:
        if chunk < 1 or tokens % chunk:
            raise ValueError(f"tokens ({tokens}) must be a multiple of chunk ({chunk})")
        _check(dev, "chunk_valid", chunk_valid, (torch.int32,), (tokens // chunk,))
    return tokens, idx0.shape[1], width1, chunk if valid is None else valid


def sdm_gather_packed(packed: PackedBank, idx0: torch.Tensor, w0: torch.Tensor, *, chunk: int,
                      valid: Optional[int] = None, chunk_valid: Optional[torch.Tensor] = None,
                      idx1: Optional[torch.Tensor] = None, w1: Optional[torch.Tensor] = None,
                      out0: Optional[torch.Tensor] = None, out1: Optional[torch.Tensor] = None):
    """``sdm_gather`` without a stash from a packed bank (``sdm_gather_packed`` of
    include/sdm_memory.h). Returns (out0, out1), float32 [tokens, head_dim]; out1 is None
    without a second operand."""
    dev = packed._device
    if (idx1 is None) != (w1 is None):
        raise ValueError("give both idx1 and w1 for a second operand, or neither")
    tokens, width0, width1, valid = _gather_sizes(idx0, idx1, chunk, valid, chunk_valid, dev)
    _check(dev, "w0", w0, _VALUE, idx0.shape)
    if w1 is not None:
        _check(dev, "w1", w1, (w0.dtype,), idx1.shape)
    shape = (tokens, packed.head_dim)
    if out0 is None:
        out0 = torch.empty(shape, dtype=torch.float32, device=packed.device)
    else:
        _check(dev, "out0", out0, (torch.float32,), shape)
    if idx1 is None:
        if out1 is not None:
            raise ValueError("out1 is given without a second operand")
    elif out1 is None:
        out1 = torch.empty(shape, dtype=torch.float32, device=packed.device)
    else:
        _check(dev, "out1", out1, (torch.float32,), shape)
    _call(dev, library().sdm_gather_packed, *packed._head, tokens, chunk, valid, _at(chunk_valid), _DTYPES[idx0.dtype],
          _DTYPES[w0.dtype], idx0.data_ptr(), w0.data_ptr(), width0, out0.data_ptr(), _at(idx1), _at(w1), width1,
          _at(out1))
    return out0, out1


def sdm_gather_weight_grad(bank: Union[PackedBank, torch.Tensor], idx0: torch.Tensor, dout0: torch.Tensor, *,
                           chunk: int, valid: Optional[int] = None, chunk_valid: Optional[torch.Tensor] = None,
                           idx1: Optional[torch.Tensor] = None, dout1: Optional[torch.Tensor] = None,
                           w_dtype: torch.dtype = torch.float32, dw0: Optional[torch.Tensor] = None,
                           dw1: Optional[torch.Tensor] = None):
    """Gradient of a gather's weights (``sdm_gather_weight_grad`` of
    include/sdm_memory.h). Returns (dw0, dw1), [tokens, width] of w_dtype; dw1 is None
    without a second operand.

    bank [num_slots, head_dim] float32 or bfloat16, or a PackedBank; idx0, idx1 and the
    padding as in the gather; dout0, dout1 float32 [tokens, head_dim].
    """
    if w_dtype not in _VALUE:
        raise TypeError(f"w_dtype must be float32 or bfloat16, got {w_dtype}")
    if isinstance(bank, PackedBank):
        dev = bank._device
        head = bank._head
        hd = bank.head_dim
    else:
        dev = bank.get_device()
        if bank.dim() != 2:
            raise ValueError("bank must be [num_slots, head_dim]")
        _check(dev, "bank", bank, _VALUE, None)
        hd = bank.shape[1]
        head = (bank.data_ptr(), None, _DTYPES[bank.dtype], bank.shape[0], hd)
    if (idx1 is None) != (dout1 is None):
        raise ValueError("give both idx1 and dout1 for a second operand, or neither")
    tokens, width0, width1, valid = _gather_sizes(idx0, idx1, chunk, valid, chunk_valid, dev)
    _check(dev, "dout0", dout0, (torch.float32,), (tokens, hd))
    if dw0 is None:
        dw0 = torch.empty(idx0.shape, dtype=w_dtype, device=bank.device)
    else:
        _check(dev, "dw0", dw0, _VALUE, idx0.shape)
    if idx1 is None:
        if dw1 is not None:
            raise ValueError("dw1 is given without a second operand")
    else:
        _check(dev, "dout1", dout1, (torch.float32,), (tokens, hd))
        if dw1 is None:
            dw1 = torch.empty(idx1.shape, dtype=dw0.dtype, device=bank.device)
        else:
            _check(dev, "dw1", dw1, (dw0.dtype,), idx1.shape)
    _call(dev, library().sdm_gather_weight_grad, *head, tokens, chunk, valid, _at(chunk_valid), _DTYPES[idx0.dtype],
          _DTYPES[dw0.dtype], idx0.data_ptr(), dout0.data_ptr(), width0, dw0.data_ptr(), _at(idx1), _at(dout1),
          width1, _at(dw1))
    return dw0, dw1
