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

A call for one token is over on the GPU before Python has checked its
arguments one by one, so each function tests them all in one expression and
looks for the one that is wrong only when that fails.
"""
from __future__ import annotations

import struct

import torch

from . import (WFST_BF16, WFST_F16, WFST_F32, _check, load, wfst_attend_size, wfst_quant_pack,
               wfst_quant_size)

_HALF = {torch.float16: WFST_F16, torch.bfloat16: WFST_BF16}
_ANY = {torch.float32: WFST_F32, **_HALF}
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream
_empty = torch.empty

# the argument blocks of the C calls, field by field as the header declares them
def _block(fields):
    pack = struct.Struct(fields).pack

    def block(*values):
        try:
            return pack(*values)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"an argument does not fit its type: {e}") from None
    return block


_MATVEC = _block("4P2q7i4x")
_ROTATE = _block("11P14q11if")
_ATTEND = _block("8P12q11if")
_SAMPLE = _block("9Pq5i3f")

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


def _explain(dev, tensors):
    """Raise for the first of (name, tensor, dtype, shape) that is not a CUDA
    tensor of device ``dev``, that type and that shape."""
    for name, t, dtype, shape in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != dev or dev < 0:
            raise ValueError(f"{name} must be on the same CUDA device as the other tensors (there is no CPU path)")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _half_type(name, dtype):
    if dtype not in _HALF:
        raise TypeError(f"{name} must be float16 or bfloat16, got {dtype}")


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
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, codes.device)):
            return pack_quant(codes, scales, zeros)
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
    packed = _empty(wfst_quant_size(n, k, k // groups, zeros is not None), dtype=_U8, device=codes.device)
    wfst_quant_pack(codes.data_ptr(), scales.data_ptr(), 0 if zeros is None else zeros.data_ptr(), _HALF[scales.dtype],
                    n, k, k // groups, packed.data_ptr(), _raw_stream(dev))
    return QuantMatrix(packed, n, k, k // groups, int(zeros is not None), scales.dtype)


def matvec_quant(x, weights: QuantMatrix, bias=None, out=None, stream=None):
    """x [rows, k] times the packed matrix, transposed, plus ``bias`` [n]:
    [rows, n] of x's type, which is the scales' type.  Made for few rows (one
    new token per lane); any number is right."""
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, x.device)):
            return matvec_quant(x, weights, bias, out)
    t, dev, n, k = weights.dtype, weights.device, weights.n, weights.k
    shape, step = x.shape, x.stride()
    if not (x.dtype is t and x.get_device() == dev and len(shape) == 2 and shape[1] == k and step[1] == 1):
        _explain(dev, [("x", x, t, (shape[0] if len(shape) else 0, k))])
        raise ValueError("x must have unit stride over k")
    rows = shape[0]
    b = 0
    if bias is not None:
        if not (bias.dtype is t and bias.get_device() == dev and bias.shape == (n,) and bias.is_contiguous()):
            _explain(dev, [("bias", bias, t, (n,))])
            raise ValueError("bias must be contiguous")
        b = bias.data_ptr()
    if out is None:
        out = _empty((rows, n), dtype=t, device=x.device)
        line = n
    else:
        _explain(dev, [("out", out, t, (rows, n))])
        line = out.stride(0)
        if n > 1 and out.stride(1) != 1:
            raise ValueError("out must have unit stride over n")
    rc = (_lib or _calls()).wfst_matvec_quant(
        _MATVEC(weights.ptr, x.data_ptr(), b, out.data_ptr(), step[0], line, dev, weights.code, n, k, weights.group,
                weights.zeros, rows), _raw_stream(dev))
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
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, q.device)):
            return norm_rotate(q, k, v, positions, table, q_gain, k_gain, k_pages, v_pages, slots, eps, interleaved,
                               out)
    t, dev = q.dtype, q.get_device()
    try:
        tokens, hq, d = q.shape
        ks = k.shape
        _, hkv, _ = ks
        ps = k_pages.shape
        pages, page, _, _ = ps
        contexts, rot = table.shape
    except ValueError:
        raise ValueError("q, k and v must be [tokens, heads, d], pages [pages, page_size, heads, d], table "
                         "[contexts, rot]") from None
    code = _HALF.get(t)
    sq, sk, sv, kp, vp = q.stride(), k.stride(), v.stride(), k_pages.stride(), v_pages.stride()
    if not (code and dev >= 0 and k.dtype is t and v.dtype is t and k_pages.dtype is t and v_pages.dtype is t
            and table.dtype is _F32 and positions.dtype is _I32 and slots.dtype is _I32
            and k.get_device() == dev and v.get_device() == dev and k_pages.get_device() == dev
            and v_pages.get_device() == dev and table.get_device() == dev and positions.get_device() == dev
            and slots.get_device() == dev
            and ks == (tokens, hkv, d) and ks == v.shape and ps == (pages, page, hkv, d) and ps == v_pages.shape
            and positions.shape == (tokens,) and slots.shape == (tokens,)
            and sq[2] == sk[2] == sv[2] == kp[3] == vp[3] == 1
            and table.is_contiguous() and positions.is_contiguous() and slots.is_contiguous()):
        _half_type("q", t)
        _explain(dev, [("q", q, t, q.shape), ("k", k, t, (tokens, hkv, d)), ("v", v, t, (tokens, hkv, d)),
                       ("k_pages", k_pages, t, (pages, page, hkv, d)), ("v_pages", v_pages, t, (pages, page, hkv, d)),
                       ("table", table, _F32, (contexts, rot)), ("positions", positions, _I32, (tokens,)),
                       ("slots", slots, _I32, (tokens,))])
        raise ValueError("heads must have unit stride over d; table, positions and slots must be contiguous")
    g = h = 0
    if q_gain is not None:
        if not (q_gain.dtype is t and q_gain.get_device() == dev and q_gain.shape == (d,) and q_gain.is_contiguous()):
            _explain(dev, [("q_gain", q_gain, t, (d,))])
            raise ValueError("q_gain must be contiguous")
        g = q_gain.data_ptr()
    if k_gain is not None:
        if not (k_gain.dtype is t and k_gain.get_device() == dev and k_gain.shape == (d,) and k_gain.is_contiguous()):
            _explain(dev, [("k_gain", k_gain, t, (d,))])
            raise ValueError("k_gain must be contiguous")
        h = k_gain.data_ptr()
    if out is None:
        out = _empty((tokens, hq, d), dtype=t, device=q.device)
        so = (hq * d, d)
    else:
        _explain(dev, [("out", out, t, (tokens, hq, d))])
        so = out.stride()
        if so[2] != 1:
            raise ValueError("out must have unit stride over d")
    rc = (_lib or _calls()).wfst_norm_rotate(
        _ROTATE(q.data_ptr(), k.data_ptr(), v.data_ptr(), g, h, positions.data_ptr(), slots.data_ptr(),
                table.data_ptr(), out.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), sq[0], sq[1], sk[0], sk[1],
                sv[0], sv[1], so[0], so[1], kp[0], kp[1], kp[2], vp[0], vp[1], vp[2], dev, code, tokens, hq, hkv, d,
                rot, interleaved, contexts, pages, page, eps), _raw_stream(dev))
    if rc:
        _check(rc)
    return out


# ------------------------------------------------------------------ attention over the paged cache

_ws_bytes = 0


def _workspace_bytes():
    global _ws_bytes
    if not _ws_bytes:
        _ws_bytes = wfst_attend_size()
    return _ws_bytes


def attend_workspace(device=None):
    """The workspace of ``attend_paged`` on a device.  Calls that share one
    must follow each other on a stream; make one for each stream that attends
    at the same time."""
    return torch.zeros(_workspace_bytes(), dtype=_U8, device="cuda" if device is None else device)


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
    if stream is not None:
        with torch.cuda.stream(_as_stream(stream, q.device)):
            return attend_paged(q, k_pages, v_pages, page_table, lengths, scale, window, sinks, workspace, with_lse,
                                out)
    t, dev = q.dtype, q.get_device()
    try:
        lanes, hq, d = q.shape
        ps = k_pages.shape
        pages, page, hkv, _ = ps
        ts = page_table.shape
        _, width = ts
    except ValueError:
        raise ValueError("q must be [lanes, heads, d], pages [pages, page_size, heads, d], page_table "
                         "[lanes, width]") from None
    code = _HALF.get(t)
    sq, st, kp, vp = q.stride(), page_table.stride(), k_pages.stride(), v_pages.stride()
    if workspace is None:
        _half_type("q", t)
        _explain(dev, [("q", q, t, q.shape)])
        workspace = attend_workspace(q.device)
    if not (code and dev >= 0 and k_pages.dtype is t and v_pages.dtype is t and page_table.dtype is _I32
            and lengths.dtype is _I32 and k_pages.get_device() == dev and v_pages.get_device() == dev
            and page_table.get_device() == dev and lengths.get_device() == dev and workspace.get_device() == dev
            and ps == (pages, page, hkv, d) and ps == v_pages.shape and ts == (lanes, width)
            and lengths.shape == (lanes,) and sq[2] == kp[3] == vp[3] == 1 and (st[1] == 1 or width < 2)
            and lengths.is_contiguous() and workspace.dtype is _U8 and workspace.numel() >= _workspace_bytes()):
        _half_type("q", t)
        _explain(dev, [("q", q, t, q.shape), ("k_pages", k_pages, t, (pages, page, hkv, d)),
                       ("v_pages", v_pages, t, (pages, page, hkv, d)), ("page_table", page_table, _I32, (lanes, width)),
                       ("lengths", lengths, _I32, (lanes,)), ("workspace", workspace, _U8, (_workspace_bytes(),))])
        raise ValueError("heads must have unit stride over d, page_table over its width, lengths be contiguous")
    if out is None:
        out = _empty((lanes, hq, d), dtype=t, device=q.device)
        so = (hq * d, d)
    else:
        _explain(dev, [("out", out, t, (lanes, hq, d))])
        so = out.stride()
        if so[2] != 1:
            raise ValueError("out must have unit stride over d")
    lse, at = None, 0
    if with_lse:
        lse = _empty((lanes, hq), dtype=_F32, device=q.device)
        at = lse.data_ptr()
    rc = (_lib or _calls()).wfst_attend_paged(
        _ATTEND(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), lengths.data_ptr(),
                out.data_ptr(), at, workspace.data_ptr(), sq[0], sq[1], so[0], so[1], hq, st[0], kp[0], kp[1], kp[2],
                vp[0], vp[1], vp[2], dev, code, lanes, hq, hkv, d, width, pages, page, window, sinks,
                d ** -0.5 if scale is None else scale), _raw_stream(dev))
    if rc:
        _check(rc)
    return (out, lse) if with_lse else out


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
        with torch.cuda.stream(_as_stream(stream, logits.device)):
            return sample_tokens(logits, uniform, temperature, top_k, top_p, min_p)
    dev, code, shape, step = logits.get_device(), _ANY.get(logits.dtype), logits.shape, logits.stride()
    if not (code is not None and dev >= 0 and len(shape) == 2 and (step[1] == 1 or shape[1] < 2)
            and uniform.dtype is _F32 and uniform.get_device() == dev and uniform.shape == shape[:1]
            and uniform.is_contiguous()):
        if code is None:
            raise TypeError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
        _explain(dev, [("logits", logits, logits.dtype, shape), ("uniform", uniform, _F32, shape[:1])])
        raise ValueError("logits must be [lanes, vocab] with unit stride over vocab, uniform contiguous")
    lanes, vocab = shape
    ptr = [0, 0, 0, 0]
    val = [temperature, top_p, min_p, top_k]
    for i in range(4):
        v = val[i]
        if isinstance(v, torch.Tensor):
            _explain(dev, [(("temperature", "top_p", "min_p", "top_k")[i], v, _I32 if i == 3 else _F32, (lanes,))])
            if not v.is_contiguous():
                raise ValueError("settings must be contiguous")
            ptr[i], val[i] = v.data_ptr(), 0
    res = _empty((3, lanes), dtype=_I32, device=logits.device)
    at = res.data_ptr()
    rc = (_lib or _calls()).wfst_sample_tokens(
        _SAMPLE(logits.data_ptr(), uniform.data_ptr(), *ptr, at, at + 4 * lanes, at + 8 * lanes, step[0], dev, code,
                lanes, vocab, val[3], val[0], val[1], val[2]), _raw_stream(dev))
    if rc:
        _check(rc)
    tokens, logprobs, kept = res.unbind()
    return tokens, logprobs.view(_F32), kept
