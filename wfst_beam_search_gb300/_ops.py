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
library refuses raises ``WfstError``.
"""
from __future__ import annotations

import struct

import torch

from . import WFST_BF16, WFST_F16, WFST_F32, _check, load, wfst_attend_size, wfst_quant_pack, wfst_quant_size

_HALF = {torch.float16: WFST_F16, torch.bfloat16: WFST_BF16}
_ANY = {torch.float32: WFST_F32, **_HALF}
_raw_stream = torch._C._cuda_getCurrentRawStream

# the argument blocks of the C calls, field by field as the header declares them
_ROTATE = struct.Struct("11P14q10if4x").pack
_ATTEND = struct.Struct("8P12q10if4x").pack
_SAMPLE = struct.Struct("9Pq4i3f4x").pack

_lib = None


def _calls():
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


def _as_stream(stream, device):
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device=device)
    return stream


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _on(dev, name, t, dtype, *shape):
    """``t`` is a tensor of this type and shape on device number ``dev``."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same CUDA device as the other tensors")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    return t


def _cuda(name, t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return dev


# ------------------------------------------------------------------ 4-bit products

class QuantMatrix:
    """A matrix [n, k] in 4-bit codes, laid out for ``matvec_quant``."""

    __slots__ = ("packed", "n", "k", "group", "zeros", "dtype", "code", "ptr", "device")

    def __init__(self, packed, n, k, group, zeros, dtype):
        self.packed, self.n, self.k, self.group, self.zeros, self.dtype = packed, n, k, group, zeros, dtype
        self.code, self.ptr, self.device = _HALF[dtype], packed.data_ptr(), packed.get_device()


def pack_quant(codes, scales, zeros=None, stream=None) -> QuantMatrix:
    """Lay out a matrix w[n, k] = scales[n, k // G] * (codes[n, k] - zeros[n, k // G]).

    codes: uint8 [n, k / 2], the even k in the lower half of a byte; scales
    and zeros: float16 or bfloat16 [n, k / G] with G 32, 64, 128 or 256
    (zeros None: 8 everywhere).  Done once per matrix."""
    dev = _cuda("codes", codes)
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, codes.device)):
            return pack_quant(codes, scales, zeros)
    if codes.dtype is not torch.uint8:
        raise TypeError(f"codes must be uint8, got {codes.dtype}")
    if scales.dtype not in _HALF:
        raise TypeError(f"scales must be float16 or bfloat16, got {scales.dtype}")
    _need(codes.dim() == 2 and scales.dim() == 2 and scales.shape[0] == codes.shape[0],
          "codes must be [n, k / 2] and scales [n, k / group]")
    n, k, groups = codes.shape[0], 2 * codes.shape[1], scales.shape[1]
    _need(groups > 0 and k % groups == 0, "the number of groups must divide k")
    _on(dev, "scales", scales, scales.dtype, n, groups)
    if zeros is not None:
        zeros = _on(dev, "zeros", zeros, scales.dtype, n, groups).contiguous()
    codes, scales = codes.contiguous(), scales.contiguous()
    packed = torch.empty(wfst_quant_size(n, k, k // groups, zeros is not None), dtype=torch.uint8, device=codes.device)
    wfst_quant_pack(codes.data_ptr(), scales.data_ptr(), 0 if zeros is None else zeros.data_ptr(), n, k, k // groups,
                    packed.data_ptr(), _raw_stream(dev))
    return QuantMatrix(packed, n, k, k // groups, int(zeros is not None), scales.dtype)


def matvec_quant(x, weights: QuantMatrix, bias=None, out=None, stream=None):
    """x [rows, k] times the packed matrix, transposed, plus ``bias`` [n]:
    [rows, n] of x's type, which is the scales' type.  Made for few rows (one
    new token per lane); any number is right."""
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, x.device)):
            return matvec_quant(x, weights, bias, out)
    dev, n = weights.device, weights.n
    if x.dim() != 2 or x.stride(1) != 1 and x.shape[1] > 1:
        raise ValueError("x must be [rows, k] with unit stride over k")
    rows = x.shape[0]
    _on(dev, "x", x, weights.dtype, rows, weights.k)
    if bias is not None:
        _need(_on(dev, "bias", bias, weights.dtype, n).is_contiguous(), "bias must be contiguous")
    if out is None:
        out = torch.empty((rows, n), dtype=x.dtype, device=x.device)
    else:
        _need(_on(dev, "out", out, x.dtype, rows, n).stride(1) == 1 or n == 1, "out must have unit stride over n")
    rc = _calls().wfst_matvec_quant(weights.ptr, n, weights.k, weights.group, weights.zeros, weights.code, x.data_ptr(),
                                    x.stride(0) if rows > 1 else 0, rows, 0 if bias is None else bias.data_ptr(),
                                    out.data_ptr(), out.stride(0), _raw_stream(dev))
    if rc:
        _check(rc)
    return out


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
    dev = _cuda("q", q)
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, q.device)):
            return norm_rotate(q, k, v, positions, table, q_gain, k_gain, k_pages, v_pages, slots, eps, interleaved,
                               out)
    t = q.dtype
    if t not in _HALF:
        raise TypeError(f"q must be float16 or bfloat16, got {t}")
    if q.dim() != 3 or k.dim() != 3 or k_pages.dim() != 4 or table.dim() != 2:
        raise ValueError("q and k must be [tokens, heads, d], pages [pages, page_size, heads, d], table [contexts, rot]")
    tokens, hq, d = q.shape
    hkv = k.shape[1]
    pages, page = k_pages.shape[:2]
    contexts, rot = table.shape
    _on(dev, "k", k, t, tokens, hkv, d)
    _on(dev, "v", v, t, tokens, hkv, d)
    _on(dev, "k_pages", k_pages, t, pages, page, hkv, d)
    _on(dev, "v_pages", v_pages, t, pages, page, hkv, d)
    _on(dev, "table", table, torch.float32, contexts, rot)
    _on(dev, "positions", positions, torch.int32, tokens)
    _on(dev, "slots", slots, torch.int32, tokens)
    if out is None:
        out = torch.empty((tokens, hq, d), dtype=t, device=q.device)
    else:
        _on(dev, "out", out, t, tokens, hq, d)
    sq, sk, sv, so, kp, vp = q.stride(), k.stride(), v.stride(), out.stride(), k_pages.stride(), v_pages.stride()
    if not (sq[2] == sk[2] == sv[2] == so[2] == kp[3] == vp[3] == 1):
        raise ValueError("heads must have unit stride over d")
    if not (table.is_contiguous() and positions.is_contiguous() and slots.is_contiguous()):
        raise ValueError("table, positions and slots must be contiguous")
    gains = [0, 0]
    for i, w in enumerate((q_gain, k_gain)):
        if w is not None:
            _need(_on(dev, "gain", w, t, d).is_contiguous(), "gains must be contiguous")
            gains[i] = w.data_ptr()
    # a stride along an axis of one entry says nothing
    rc = _calls().wfst_norm_rotate(
        _ROTATE(q.data_ptr(), k.data_ptr(), v.data_ptr(), gains[0], gains[1], positions.data_ptr(), slots.data_ptr(),
                table.data_ptr(), out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                sq[0] if tokens > 1 else 0, sq[1] if hq > 1 else 0, sk[0] if tokens > 1 else 0, sk[1] if hkv > 1 else 0,
                sv[0] if tokens > 1 else 0, sv[1] if hkv > 1 else 0, so[0] if tokens > 1 else 0, so[1] if hq > 1 else 0,
                kp[0] if pages > 1 else 0, kp[1] if page > 1 else 0, kp[2] if hkv > 1 else 0,
                vp[0] if pages > 1 else 0, vp[1] if page > 1 else 0, vp[2] if hkv > 1 else 0,
                _HALF[t], tokens, hq, hkv, d, rot, bool(interleaved), contexts, pages, page, eps), _raw_stream(dev))
    if rc:
        _check(rc)
    return out


# ------------------------------------------------------------------ attention over the paged cache

def attend_workspace(device=None):
    """The workspace of ``attend_paged`` on a device.  Calls that share one
    must follow each other on a stream; make one for each stream that attends
    at the same time."""
    return torch.zeros(wfst_attend_size(), dtype=torch.uint8, device="cuda" if device is None else device)


def attend_paged(q, k_pages, v_pages, page_table, lengths, scale=None, window=0, sinks=0, workspace=None,
                 with_lse=False, out=None, stream=None):
    """Attention of one new token per lane over its paged cache.

    q [lanes, q_heads, d]; pages [pages, page_size, kv_heads, d] in any order
    of strides; page_table int32 [lanes, width]; lengths int32 [lanes], the
    new token among them.  ``scale`` is 1/sqrt(d) by default.  With ``window``
    a lane sees its last ``window`` tokens and the first ``sinks`` ones; table
    entries of tokens that are not seen are never read.  Returns o [lanes,
    q_heads, d], with ``with_lse`` also the float32 [lanes, q_heads] log of
    the sum of exponentials.  Without ``workspace`` (see
    ``attend_workspace``) the call makes one of its own."""
    dev = _cuda("q", q)
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, q.device)):
            return attend_paged(q, k_pages, v_pages, page_table, lengths, scale, window, sinks, workspace, with_lse,
                                out)
    t = q.dtype
    if t not in _HALF:
        raise TypeError(f"q must be float16 or bfloat16, got {t}")
    if q.dim() != 3 or k_pages.dim() != 4 or page_table.dim() != 2:
        raise ValueError("q must be [lanes, heads, d], pages [pages, page_size, heads, d], page_table [lanes, width]")
    lanes, hq, d = q.shape
    pages, page, hkv = k_pages.shape[:3]
    width = page_table.shape[1]
    _on(dev, "k_pages", k_pages, t, pages, page, hkv, d)
    _on(dev, "v_pages", v_pages, t, pages, page, hkv, d)
    _on(dev, "page_table", page_table, torch.int32, lanes, width)
    _on(dev, "lengths", lengths, torch.int32, lanes)
    if out is None:
        out = torch.empty((lanes, hq, d), dtype=t, device=q.device)
    else:
        _on(dev, "out", out, t, lanes, hq, d)
    lse = torch.empty((lanes, hq), dtype=torch.float32, device=q.device) if with_lse else None
    sq, so, st, kp, vp = q.stride(), out.stride(), page_table.stride(), k_pages.stride(), v_pages.stride()
    if not (sq[2] == so[2] == kp[3] == vp[3] == 1) or (st[1] != 1 and width > 1) or not lengths.is_contiguous():
        raise ValueError("heads must have unit stride over d, page_table over its width, lengths be contiguous")
    if workspace is None:
        workspace = attend_workspace(q.device)
    else:
        ws = workspace
        if ws.dtype is not torch.uint8 or ws.get_device() != dev or ws.numel() < _workspace_bytes():
            raise ValueError("workspace must come from attend_workspace of the same device")
    rc = _calls().wfst_attend_paged(
        _ATTEND(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), lengths.data_ptr(),
                out.data_ptr(), lse.data_ptr() if with_lse else 0, workspace.data_ptr(),
                sq[0] if lanes > 1 else 0, sq[1] if hq > 1 else 0, so[0], so[1], hq, st[0] if lanes > 1 else 0,
                kp[0] if pages > 1 else 0, kp[1] if page > 1 else 0, kp[2] if hkv > 1 else 0,
                vp[0] if pages > 1 else 0, vp[1] if page > 1 else 0, vp[2] if hkv > 1 else 0,
                _HALF[t], lanes, hq, hkv, d, width, pages, page, window, sinks,
                d ** -0.5 if scale is None else scale), _raw_stream(dev))
    if rc:
        _check(rc)
    return (out, lse) if with_lse else out


_ws_bytes = 0


def _workspace_bytes():
    global _ws_bytes
    if not _ws_bytes:
        _ws_bytes = wfst_attend_size()
    return _ws_bytes


# ------------------------------------------------------------------ the next token

def sample_tokens(logits, uniform, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """One token per lane from its logits [lanes, vocab] and a uniform number
    in [0, 1) (float32 [lanes]).  Returns (tokens int32, logprobs float32,
    kept int32), [lanes] each: the token, the log of its share of what was
    kept, and how many tokens were kept.

    Each setting is a number, or a tensor with one value per lane (float32;
    ``top_k`` int32).  top_k 0, top_p 1 and min_p 0 keep everything,
    temperature 0 takes the first largest logit."""
    dev = _cuda("logits", logits)
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, logits.device)):
            return sample_tokens(logits, uniform, temperature, top_k, top_p, min_p)
    code = _ANY.get(logits.dtype)
    if code is None:
        raise TypeError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [lanes, vocab] with unit stride over vocab")
    lanes, vocab = logits.shape
    _need(_on(dev, "uniform", uniform, torch.float32, lanes).is_contiguous(), "uniform must be contiguous")
    ptr = [0, 0, 0, 0]
    val = [temperature, top_p, min_p, top_k]
    for i, (name, v) in enumerate(zip(("temperature", "top_p", "min_p", "top_k"), val)):
        if isinstance(v, torch.Tensor):
            kind = torch.int32 if i == 3 else torch.float32
            _need(_on(dev, name, v, kind, lanes).is_contiguous(), f"{name} must be contiguous")
            ptr[i], val[i] = v.data_ptr(), 0
    res = torch.empty((3, lanes), dtype=torch.int32, device=logits.device)
    tokens, logprobs, kept = res.unbind()
    at = res.data_ptr()
    rc = _calls().wfst_sample_tokens(
        _SAMPLE(logits.data_ptr(), uniform.data_ptr(), ptr[0], ptr[1], ptr[2], ptr[3], at, at + 4 * lanes,
                at + 8 * lanes, logits.stride(0) if lanes > 1 else 0, code, lanes, vocab, val[3], val[0], val[1],
                val[2]), _raw_stream(dev))
    if rc:
        _check(rc)
    return tokens, logprobs.view(torch.float32), kept
