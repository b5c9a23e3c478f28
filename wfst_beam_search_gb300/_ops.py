"""The second-pass operators on torch CUDA tensors.

One step of a small language model that reads the first-pass words: products
with 4-bit weights (``pack_quant``, ``matvec_quant``), the heads' norm and
rotation with the write into the paged cache (``norm_rotate``), attention of
one new token per lane over that cache (``attend_workspace``,
``attend_paged``) and the draw of the next token (``sample_tokens``).

As in the rest of the binding, the functions check and marshal arguments; the
work is done by the CUDA library (``include/wfst_gb300.h`` states layouts and
limits).  A call runs on ``stream``, by default torch's current stream of the
tensors' device; results are allocated on the stream the call runs on.  Inputs
that belong to another stream are the caller's to order, as anywhere in torch.
Wrong types, shapes or layouts raise ``TypeError`` or ``ValueError``, what the
library refuses raises ``WfstError``.  There are no backward passes: an input
that requires a gradient is refused while gradients are recorded.

A call for one token is over on the GPU before Python has asked its arguments
one by one what they are, so ``csrc/ops_binding.cpp`` asks them all and makes
the call; only when it finds something wrong do the functions here look for
what it is.
"""
from __future__ import annotations

import importlib.util
import os
import struct

import torch

from . import (WFST_ATTEND_ZEROED, WFST_BF16, WFST_F16, WFST_F32, _build, _check, load, wfst_attend_size,
               wfst_quant_pack, wfst_quant_size)

_HALF = {torch.float16: WFST_F16, torch.bfloat16: WFST_BF16}
_ANY = {torch.float32: WFST_F32, **_HALF}
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8

# the argument blocks of the C calls (``wfst_matvec_quant`` and so on, without tensors), field by field as the header
# declares them
_MATVEC = struct.Struct("4P2q7i4x").pack
_ROTATE = struct.Struct("11P14q11if").pack
_ATTEND = struct.Struct("8P12q11if").pack
_SAMPLE = struct.Struct("9Pq5i3f").pack


def _load_binding():
    load()
    if not os.path.exists(_build.BINDING):
        raise ImportError("ops_binding.so is not built (it needs torch and Python's headers); run __graft_entry__.build()")
    spec = importlib.util.spec_from_file_location("ops_binding", _build.BINDING)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_binding = _load_binding()


def _tensors(**named):
    for name, t in named.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")


def _on(stream, **first):
    """The context in which a call runs on ``stream``; ``first``: a tensor of its device."""
    _tensors(**first)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=next(iter(first.values())).device)
    return torch.cuda.stream(stream)


def _explain(dev, tensors):
    """Raise for the first of (name, tensor, dtype, shape) that is not a CUDA
    tensor of device ``dev``, that type and that shape."""
    for name, t, dtype, shape in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name} requires a gradient, and there is none to give: detach it, or use torch.no_grad()")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != dev or dev < 0:
            raise ValueError(f"{name} must be on the same CUDA device as the other tensors (there is no CPU path)")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _refused(rc, why):
    """Raise for what the binding returned instead of tensors: the library's
    error, or what ``why`` finds wrong with the arguments."""
    if rc < 0:
        _check(rc)
    why()
    raise ValueError("an argument does not fit its type")


def _last_axis(**tensors):
    for name, t in tensors.items():
        if t is not None and t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"{name} must have unit stride over its last axis")


def _contiguous(**tensors):
    for name, t in tensors.items():
        if isinstance(t, torch.Tensor) and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def _half_type(name, dtype):
    if dtype not in _HALF:
        raise TypeError(f"{name} must be float16 or bfloat16, got {dtype}")


# ------------------------------------------------------------------ 4-bit products

class QuantMatrix:
    """A matrix [n, k] in 4-bit codes, laid out for ``matvec_quant``."""

    __slots__ = ("packed", "n", "k", "group", "zeros", "dtype", "ptr", "device", "spec")

    def __init__(self, packed, n, k, group, zeros, dtype):
        self.packed, self.n, self.k, self.group, self.zeros, self.dtype = packed, n, k, group, zeros, dtype
        self.ptr, self.device = packed.data_ptr(), packed.get_device()
        self.spec = (self.ptr, _HALF[dtype], n, k, group, zeros, self.device)

    def __reduce__(self):    # a copy, or what is loaded from a file, has its own address
        return QuantMatrix, (self.packed, self.n, self.k, self.group, self.zeros, self.dtype)


def pack_quant(codes, scales, zeros=None, stream=None) -> QuantMatrix:
    """Lay out a matrix w[n, k] = scales[n, k // G] * (codes[n, k] - zeros[n, k // G]).

    codes: uint8 [n, k / 2], the even k in the lower half of a byte; scales
    and zeros: float16 or bfloat16 [n, k / G] with G 32, 64, 128 or 256
    (zeros None: 8 everywhere).  Done once per matrix."""
    if stream is not None:
        with _on(stream, codes=codes):
            return pack_quant(codes, scales, zeros)
    _tensors(codes=codes, scales=scales)
    dev = codes.get_device()
    _half_type("scales", scales.dtype)
    if codes.dim() != 2 or scales.dim() != 2:
        raise ValueError("codes must be [n, k / 2] and scales [n, k / group]")
    n, k, groups = codes.shape[0], 2 * codes.shape[1], scales.shape[1]
    _explain(dev, [("codes", codes, _U8, codes.shape), ("scales", scales, scales.dtype, (n, groups)),
                   ("zeros", zeros, scales.dtype, (n, groups))])
    if groups < 1 or k % groups:
        raise ValueError("the number of groups must divide k")
    codes, scales, zeros = codes.contiguous(), scales.contiguous(), None if zeros is None else zeros.contiguous()
    packed = torch.empty(wfst_quant_size(n, k, k // groups, zeros is not None), dtype=_U8, device=codes.device)
    wfst_quant_pack(codes.data_ptr(), scales.data_ptr(), 0 if zeros is None else zeros.data_ptr(), _HALF[scales.dtype],
                    n, k, k // groups, packed.data_ptr(), torch.cuda.current_stream(dev).cuda_stream)
    return QuantMatrix(packed, n, k, k // groups, int(zeros is not None), scales.dtype)


def matvec_quant(x, weights: QuantMatrix, bias=None, out=None, stream=None):
    """x [rows, k] times the packed matrix, transposed, plus ``bias`` [n]:
    [rows, n] of x's type, which is the scales' type.  Made for few rows (one
    new token per lane); any number is right."""
    if stream is not None:
        with _on(stream, x=x):
            return matvec_quant(x, weights, bias, out)
    y = _binding.matvec_quant(x, getattr(weights, "spec", None), bias, out)
    if y.__class__ is int:
        def why():
            _tensors(x=x)
            if not isinstance(weights, QuantMatrix):
                raise TypeError("weights must be a QuantMatrix (see pack_quant)")
            t, dev, n = weights.dtype, weights.device, weights.n
            rows = x.shape[0] if x.dim() else 0
            _explain(dev, [("x", x, t, (rows, weights.k)), ("bias", bias, t, (n,)), ("out", out, t, (rows, n))])
            _last_axis(x=x, out=out)
            _contiguous(bias=bias)
        _refused(y, why)
    return y


# ------------------------------------------------------------------ norm, rotation, cache

def norm_rotate(q, k, v, positions, table, q_gain, k_gain, k_pages, v_pages, slots, eps=1e-6, interleaved=False,
                out=None, stream=None):
    """The new tokens' heads: RMS norm of each head of q and k, rotation by
    position, k and v put into the cache.  Returns the new q.

    q [tokens, q_heads, d], k and v [tokens, kv_heads, d]; gains [d] or None;
    table float32 [contexts, rot], a position's rot/2 cosines and rot/2 sines;
    positions and slots int32 [tokens]; pages [pages, page_size, kv_heads, d]
    in any order of strides, updated in place (slot = page * page_size +
    place; negative: the token's k and v are not kept).  Pairs are (i, i +
    rot/2), or (2i, 2i + 1) if ``interleaved``.  ``out`` may be q itself."""
    if stream is not None:
        with _on(stream, q=q):
            return norm_rotate(q, k, v, positions, table, q_gain, k_gain, k_pages, v_pages, slots, eps, interleaved,
                               out)
    y = _binding.norm_rotate(q, k, v, positions, table, q_gain, k_gain, k_pages, v_pages, slots, eps, interleaved, out)
    if y.__class__ is int:
        def why():
            _tensors(q=q, k=k, v=v, positions=positions, table=table, k_pages=k_pages, v_pages=v_pages, slots=slots)
            _half_type("q", q.dtype)
            if q.dim() != 3 or k.dim() != 3 or k_pages.dim() != 4 or table.dim() != 2:
                raise ValueError("q, k and v must be [tokens, heads, d], pages [pages, page_size, heads, d], table "
                                 "[contexts, rot]")
            t, (tokens, _, d), hkv = q.dtype, q.shape, k.shape[1]
            cache = (*k_pages.shape[:2], hkv, d)
            _explain(q.get_device(), [
                ("q", q, t, q.shape), ("k", k, t, (tokens, hkv, d)), ("v", v, t, (tokens, hkv, d)),
                ("k_pages", k_pages, t, cache), ("v_pages", v_pages, t, cache), ("table", table, _F32, table.shape),
                ("positions", positions, _I32, (tokens,)), ("slots", slots, _I32, (tokens,)), ("q_gain", q_gain, t, (d,)),
                ("k_gain", k_gain, t, (d,)), ("out", out, t, q.shape)])
            _last_axis(q=q, k=k, v=v, k_pages=k_pages, v_pages=v_pages, out=out)
            _contiguous(table=table, positions=positions, slots=slots, q_gain=q_gain, k_gain=k_gain)
        _refused(y, why)
    return y


# ------------------------------------------------------------------ attention over the paged cache

def attend_workspace(device=None):
    """The workspace of ``attend_paged`` on a device.  Calls that share one
    must follow each other on a stream; make one for each stream that attends
    at the same time."""
    workspace = torch.empty(wfst_attend_size(), dtype=_U8, device="cuda" if device is None else device)
    workspace[:WFST_ATTEND_ZEROED].zero_()
    return workspace


def attend_paged(q, k_pages, v_pages, page_table, lengths, scale=None, window=0, sinks=0, workspace=None,
                 with_lse=False, out=None, stream=None):
    """Attention of one new token per lane over its paged cache.

    q [lanes, q_heads, d]; pages [pages, page_size, kv_heads, d] in any order
    of strides; page_table int32 [lanes, width]; lengths int32 [lanes], the
    new token among them.  ``scale`` is 1/sqrt(d) by default.  With ``window``
    a lane sees its last ``window`` tokens and the first ``sinks`` ones; table
    entries of tokens that are not seen are never read.  ``out`` may be q
    itself.  Returns o [lanes, q_heads, d], with ``with_lse`` also the float32 [lanes, q_heads] log of
    the sum of exponentials.  Without ``workspace`` (see
    ``attend_workspace``) the call makes one of its own, 34 MB."""
    if stream is not None:
        with _on(stream, q=q):
            return attend_paged(q, k_pages, v_pages, page_table, lengths, scale, window, sinks, workspace, with_lse,
                                out)
    y = _binding.attend_paged(q, k_pages, v_pages, page_table, lengths, scale, window, sinks, workspace, with_lse, out)
    if y.__class__ is int:
        def why():
            _tensors(q=q, k_pages=k_pages, v_pages=v_pages, page_table=page_table, lengths=lengths,
                     **({} if workspace is None else {"workspace": workspace}))
            _half_type("q", q.dtype)
            if q.dim() != 3 or k_pages.dim() != 4 or page_table.dim() != 2:
                raise ValueError("q must be [lanes, heads, d], pages [pages, page_size, heads, d], page_table "
                                 "[lanes, width]")
            t, (lanes, _, d) = q.dtype, q.shape
            cache, room = (*k_pages.shape[:3], d), 0 if workspace is None else workspace.numel()
            _explain(q.get_device(), [
                ("q", q, t, q.shape), ("k_pages", k_pages, t, cache), ("v_pages", v_pages, t, cache),
                ("page_table", page_table, _I32, (lanes, page_table.shape[1])), ("lengths", lengths, _I32, (lanes,)),
                ("workspace", workspace, _U8, (max(room, wfst_attend_size()),)),
                ("out", out, t, q.shape)])
            _last_axis(q=q, k_pages=k_pages, v_pages=v_pages, page_table=page_table, out=out)
            _contiguous(lengths=lengths, workspace=workspace)
        _refused(y, why)
    return y


# ------------------------------------------------------------------ the next token

def sample_tokens(logits, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """One token per lane from its logits [lanes, vocab] and a uniform number
    in [0, 1) (float32 [lanes]).  Returns (tokens int32, logprobs float32,
    kept int32), [lanes] each: the token, the log of its share of what was
    kept, and how many tokens were kept.

    Each setting is a number, or a tensor with one value per lane (float32;
    ``top_k`` int32).  top_k 0, top_p 1 and min_p 0 keep everything,
    temperature 0 takes the first largest logit."""
    if stream is not None:
        with _on(stream, logits=logits):
            return sample_tokens(logits, uniform, temperature, top_k, top_p, min_p)
    y = _binding.sample_tokens(logits, uniform, temperature, top_k, top_p, min_p)
    if y.__class__ is int:
        def why():
            _tensors(logits=logits, uniform=uniform)
            if logits.dtype not in _ANY:
                raise TypeError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
            if logits.dim() != 2:
                raise ValueError("logits must be [lanes, vocab]")
            lanes = logits.shape[:1]
            each = [(name, v, _I32 if name == "top_k" else _F32, lanes) for name, v in
                    (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p))
                    if isinstance(v, torch.Tensor)]
            _explain(logits.get_device(), [("logits", logits, logits.dtype, logits.shape),
                                           ("uniform", uniform, _F32, lanes), *each])
            _last_axis(logits=logits)
            _contiguous(uniform=uniform, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)
        _refused(y, why)
    return y
