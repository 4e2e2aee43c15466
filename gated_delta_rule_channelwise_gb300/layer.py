"""The operators around a layer's state: norm, 8-bit operands and their product, rotary positions.

Python side of ``include/cgdr_layer.h``, in the manner of :mod:`.serve`: each call checks types and shapes, packs
the argument block of its C entry point and runs it on the current CUDA stream (or ``stream``).  Every step runs
in the library's kernels and there is no CPU fallback.  The tensors of a call share one device, the current one.  Outputs that are
not given come from torch's caching allocator; no call needs a workspace.  An output may not overlap an input, other than
what is updated in place and the o of :func:`rms_norm`, which may be x.

* :func:`rms_norm`, :func:`rms_norm_fp8` -- root-mean-square norm with the residual's addition, the latter in 8 bits.
* :func:`fp8_quantize`, :func:`fp8_quantize_weight` -- rows and weights in 8 bits.
* :func:`fp8_matmul` -- the matrix product of such operands.
* :func:`rotary`, :func:`rotary_frequencies` -- rotary positions, and the frequencies of their usual scalings.

8 bits are ``torch.float8_e4m3fn`` with fp32 scales: a scale for each 128 values of a row (``[n, ceil(K/128)]``),
or for each 128 x 128 of a weight.  The scale is the largest magnitude times 1/448 (in fp32), 2^-126 at least, and a value is
``scale * e4m3``.  A NaN or an infinity makes its group's scale non-finite, and with it every value of the group.
"""
from __future__ import annotations

import math

import torch

from . import MATMUL_AUTO, CgdrError, _need_cuda, lib
from . import serve as _serve
from .serve import _CODES, _F32, _I32, Block, _address, _current, _fits, _i, _on, _on_device, _p, _refuse, _status_word, _strided

_E4M3, _F64 = torch.float8_e4m3fn, torch.float64

NORM = Block(*_i("n H C dtype"), ("eps", "f"), *_strided("x", "st", "sh"), *_strided("residual", "st", "sh"), *_p("weight"),
             *_strided("o", "st", "sh"), *_strided("y8", "st"), *_p("y_scale status"))
QUANTIZE = Block(*_i("n C dtype block_rows"), *_strided("x", "st"), *_strided("y8", "st"), *_p("y_scale status"))
MATMUL = Block(*_i("n N K o_dtype path wait_polls"), *_strided("x", "st"), *_p("x_scale"), *_strided("w", "st"), *_p("w_scale"),
               *_strided("o", "st"), *_p("status"))
ROTARY = Block(*_i("n Hq Hk D half dtype interleaved"), ("scale", "f"), *_strided("q", "st", "sh"), *_strided("k", "st", "sh"),
               *_p("positions freq status"))


def _groups(n):
    return -(-n // 128)


def _tokens(t, name):
    """(pointer, token stride, head stride) of [n, C] or [n, H, C]; of one token or head its stride says nothing, and 0 stands for it."""
    st, shape = t.stride(), t.shape
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s: innermost dimension must be contiguous" % name)
    return t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if len(st) == 3 and shape[1] > 1 else 0


_NONE = (0, 0, 0)


# --------------------------------------------------------------------------- norm


def _norm(x, weight, residual, eps, o, y, y_scale, status):
    device = x.get_device()
    if not (device >= 0 and device == _serve._here() and _on_device(weight, device) and _on_device(residual, device) and _on_device(o, device)
            and _on_device(y, device) and _on_device(y_scale, device)):
        _need_cuda(x, weight, residual, o, y, y_scale)
    dtype, shape = x.dtype, x.shape
    C = shape[-1]
    if not ((o is None or (o.dtype == dtype and o.shape == shape)) and (residual is None or (residual.dtype == dtype and residual.shape == shape))
            and _fits(weight, _F32, (C,))):
        _refuse([("weight", weight, _F32), ("residual", residual, dtype), ("o", o, dtype)],
                [("residual", residual, shape), ("o", o, shape), ("weight", weight, (C,))], [("weight", weight)])
    block = NORM.pack(shape[0], shape[1] if len(shape) == 3 else 1, C, _CODES.get(dtype, -1), eps, *_tokens(x, "x"),
                      *(_NONE if residual is None else _tokens(residual, "residual")), _address(weight),
                      *(_NONE if o is None else _tokens(o, "o")), *((0, 0) if y is None else _tokens(y, "y")[:2]), _address(y_scale),
                      0 if status is None else _status_word(status, device))
    st = lib().cgdr_norm(block, _current(device))
    if st:
        raise CgdrError(st, "cgdr_norm")


def _check_eps(eps):
    if not eps >= 0:
        raise ValueError("eps must not be below 0, got %s" % eps)    # the library would take its default


def rms_norm(x, weight, o=None, *, residual=None, eps=1e-6, status=None, stream=None):
    """Root-mean-square norm of the rows of ``x [n,C]`` or ``[n,H,C]`` (fp32 or bf16, C a multiple of 8, at most 32768):
    ``h = x + residual``, ``o = h / sqrt(mean(h^2) + eps) * weight``.  ``weight [C]`` is fp32 (None: ones).  ``residual``, like x, is
    optional and updated in place: it becomes h, rounded; o is formed from h in fp32.  x, residual and o may be strided in
    tokens and heads; rows are 16-byte aligned.  o may be x: the norm in place, of heads in a packed row for
    instance.  Returns o, like x."""
    if stream is not None:
        return _on(stream, rms_norm, x, weight, o, residual=residual, eps=eps, status=status)
    if x.dim() not in (2, 3):
        raise ValueError("x must be [n, C] or [n, H, C]")
    _check_eps(eps)
    if o is None:
        o = torch.empty(x.shape, dtype=x.dtype, device=x.device)    # dense, whatever x's strides are
    _norm(x, weight, residual, eps, o, None, None, status)
    return o


def _rows_of(n, C, dtype, device, step):
    """New rows, each beginning at a multiple of ``step`` values (16 bytes): dense, or with the least stride that gives that (one
    allocation either way; a view of padded rows would cost as much again)."""
    return torch.empty((n, C), dtype=dtype, device=device) if C % step == 0 else \
        torch.empty_strided((n, C), (C + -C % step, 1), dtype=dtype, device=device)


def _eight(shape, y, y_scale, device, rows=1):
    """The outputs in 8 bits of [n, C], the given ones or new."""
    n, C = shape
    scales = (_groups(n) if rows > 1 else n, _groups(C))
    if y is None:
        y = _rows_of(n, C, _E4M3, device, 16)
    elif y.dtype != _E4M3 or y.shape != shape:
        _refuse([("y", y, _E4M3)], [("y", y, shape)], [])
    if y_scale is None:
        y_scale = torch.empty(scales, dtype=_F32, device=device)
    elif not _fits(y_scale, _F32, scales):
        _refuse([("y_scale", y_scale, _F32)], [("y_scale", y_scale, scales)], [("y_scale", y_scale)])
    return y, y_scale


def rms_norm_fp8(x, weight, y=None, y_scale=None, *, residual=None, eps=1e-6, status=None, stream=None):
    """:func:`rms_norm` of ``x [n,C]`` with the output in 8 bits, as :func:`fp8_matmul` takes it.  Returns
    ``y [n,C]`` (``torch.float8_e4m3fn``) and ``y_scale [n, ceil(C/128)]`` (fp32)."""
    if stream is not None:
        return _on(stream, rms_norm_fp8, x, weight, y, y_scale, residual=residual, eps=eps, status=status)
    if x.dim() != 2:
        raise ValueError("x must be [n, C]")
    _check_eps(eps)
    y, y_scale = _eight(x.shape, y, y_scale, x.device)
    _norm(x, weight, residual, eps, None, y, y_scale, status)
    return y, y_scale


# --------------------------------------------------------------------------- 8 bits


def _quantize(x, rows, y, y_scale, status):
    if x.dim() != 2:
        raise ValueError("%s must be a matrix" % ("x" if rows == 1 else "w"))
    y, y_scale = _eight(x.shape, y, y_scale, x.device, rows)
    device = x.get_device()
    if not (device >= 0 and device == y.get_device() == y_scale.get_device() == _serve._here()):
        _need_cuda(x, y, y_scale)
    address, st, _ = _tokens(x, "x" if rows == 1 else "w")
    block = QUANTIZE.pack(x.shape[0], x.shape[1], _CODES.get(x.dtype, -1), rows, address, st, *_tokens(y, "y")[:2], y_scale.data_ptr(),
                          0 if status is None else _status_word(status, device))
    err = lib().cgdr_quantize(block, _current(device))
    if err:
        raise CgdrError(err, "cgdr_quantize")
    return y, y_scale


def fp8_quantize(x, y=None, y_scale=None, *, status=None, stream=None):
    """Rows ``x [n,K]`` (fp32 or bf16, K a multiple of 8, rows 16-byte aligned) in 8 bits: ``y [n,K]`` and
    ``y_scale [n, ceil(K/128)]``."""
    if stream is not None:
        return _on(stream, fp8_quantize, x, y, y_scale, status=status)
    return _quantize(x, 1, y, y_scale, status)


def fp8_quantize_weight(w, y=None, y_scale=None, *, status=None, stream=None):
    """A weight ``w [N,K]`` in 8 bits, with a scale for each block of 128 x 128: ``y [N,K]`` and
    ``y_scale [ceil(N/128), ceil(K/128)]``.  Done once, when a model is loaded."""
    if stream is not None:
        return _on(stream, fp8_quantize_weight, w, y, y_scale, status=status)
    return _quantize(w, 128, y, y_scale, status)


def fp8_matmul(x, x_scale, w, w_scale, o=None, *, dtype=torch.bfloat16, path=MATMUL_AUTO, status=None, wait_polls=0, stream=None):
    """``o = x w^T`` of 8-bit operands: ``x [n,K]`` with ``x_scale [n, ceil(K/128)]`` (as :func:`fp8_quantize` and
    :func:`rms_norm_fp8` leave them) and ``w [N,K]`` with ``w_scale [ceil(N/128), ceil(K/128)]``
    (:func:`fp8_quantize_weight`).  Any n, N and K; rows of x, w and o are 16-byte aligned (new outputs of all these calls
    have strides that give that).  Products are exact, sums fp32.  Returns o ``[n,N]``, the given one (fp32 or bf16) or a new one of
    ``dtype``.  ``path`` forces one of the two kernels for this call (``MATMUL_FEW``, ``MATMUL_TILES``).
    ``wait_polls``: polls of a bounded device wait (0: the default).  When one gives up o is undefined and ``status`` holds
    ``ERR_TIMEOUT``; without ``status`` nothing says so."""
    if stream is not None:
        return _on(stream, fp8_matmul, x, x_scale, w, w_scale, o, dtype=dtype, path=path, status=status, wait_polls=wait_polls)
    device = x.get_device()
    if not (device >= 0 and device == x_scale.get_device() == w.get_device() == w_scale.get_device() == _serve._here() and _on_device(o, device)):
        _need_cuda(x, x_scale, w, w_scale, o)
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x must be [n, K] and w [N, K]")
    n, K = x.shape
    N = w.shape[0]
    blocks = _groups(K)
    if o is None:
        o = _rows_of(n, N, dtype, x.device, 8 if dtype == torch.bfloat16 else 4)
    if not (x.dtype == _E4M3 and w.dtype == _E4M3 and w.shape[1] == K and o.shape == (n, N) and _fits(x_scale, _F32, (n, blocks))
            and _fits(w_scale, _F32, (_groups(N), blocks))):
        _refuse([("x", x, _E4M3), ("w", w, _E4M3), ("x_scale", x_scale, _F32), ("w_scale", w_scale, _F32)],
                [("w", w, (N, K)), ("o", o, (n, N)), ("x_scale", x_scale, (n, blocks)), ("w_scale", w_scale, (_groups(N), blocks))],
                [("x_scale", x_scale), ("w_scale", w_scale)])
    block = MATMUL.pack(n, N, K, _CODES.get(o.dtype, -1), path, wait_polls, *_tokens(x, "x")[:2], x_scale.data_ptr(), *_tokens(w, "w")[:2],
                        w_scale.data_ptr(), *_tokens(o, "o")[:2], 0 if status is None else _status_word(status, device))
    st = lib().cgdr_matmul(block, _current(device))
    if st:
        raise CgdrError(st, "cgdr_matmul")
    return o


# --------------------------------------------------------------------------- rotary positions


def rotary(q, k, positions, freq, *, interleaved=False, scale=1.0, status=None, stream=None):
    """Turn the first ``R = 2 * len(freq)`` channels of every head by the position of its token, in place: ``q [n,Hq,D]``
    and ``k [n,Hk,D]`` (fp32 or bf16, alike; k may be None), ``positions [n]`` int32 as :func:`~.serve.cache_plan`
    gives them (below 0: the token stays as it is), ``freq [R/2]`` fp64 radians a position (:func:`rotary_frequencies`).
    With ``a = position * freq[i]``, pair (u, v) becomes ``scale * (u cos a - v sin a, v cos a + u sin a)``; u and v are channels
    i and i + R/2, or 2 i and 2 i + 1 (``interleaved``).  Angles are formed in 64 bits.  q and k may be strided in
    tokens and heads (views of one packed row); heads are 16-byte aligned.  Returns q and k."""
    if stream is not None:
        return _on(stream, rotary, q, k, positions, freq, interleaved=interleaved, scale=scale, status=status)
    device = q.get_device()
    if not (device >= 0 and device == positions.get_device() == freq.get_device() == _serve._here() and _on_device(k, device)):
        _need_cuda(q, k, positions, freq)
    if q.dim() != 3 or freq.dim() != 1 or (k is not None and k.dim() != 3):
        raise ValueError("q must be [n, Hq, D], k [n, Hk, D] and freq [R / 2]")
    n, Hq, D = q.shape
    Hk = 0 if k is None else k.shape[1]
    if not (_fits(positions, _I32, (n,)) and freq.dtype == _F64 and freq.is_contiguous() and (k is None or (k.dtype == q.dtype and k.shape == (n, Hk, D)))):
        _refuse([("positions", positions, _I32), ("freq", freq, _F64), ("k", k, q.dtype)], [("positions", positions, (n,)), ("k", k, (n, Hk, D))],
                [("positions", positions), ("freq", freq)])
    block = ROTARY.pack(n, Hq, Hk, D, freq.shape[0], _CODES.get(q.dtype, -1), 1 if interleaved else 0, scale, *_tokens(q, "q"),
                        *(_tokens(k, "k") if Hk else _NONE), positions.data_ptr(), freq.data_ptr(),
                        0 if status is None else _status_word(status, device))
    st = lib().cgdr_rotary(block, _current(device))
    if st:
        raise CgdrError(st, "cgdr_rotary")
    return q, k


def rotary_frequencies(R, base=10000.0, *, scaling=None, factor=1.0, length=4096, fast=32.0, slow=1.0, device=None):
    """Frequencies for :func:`rotary` of R channels, ``base^(-2 i / R)``, scaled for contexts ``factor`` times as long as
    the ``length`` positions a model was trained on.  Returns ``(freq [R/2] fp64, scale)``.

    ``scaling``: None; ``"linear"`` divides every frequency by factor; ``"base"`` raises the base to ``base * factor^(R/(R-2))``,
    which keeps the fastest frequency and divides the slowest by factor; ``"turns"`` goes by how often a frequency turns
    within ``length``: ``fast`` times or more and it stays, ``slow`` or less and it is divided by factor, linear in the
    number of turns between; ``"ramp"`` goes by the pair's number between the (rounded) numbers that turn that often, and its
    scale is ``1 + 0.1 ln(factor)``."""
    if R <= 0 or R % 2:
        raise ValueError("R must be even and above 0, got %s" % R)
    if not (base > 0 and factor >= 1 and length > 0 and fast > slow > 0):
        raise ValueError("base, length and slow must be above 0, factor at least 1 and fast above slow")
    if scaling == "ramp" and base <= 1:
        raise ValueError("the ramp needs frequencies that fall: base must be above 1, got %s" % base)
    if scaling == "base" and R > 2:
        base = base * factor ** (R / (R - 2))
    i = torch.arange(0, R, 2, dtype=_F64)
    freq, scale = base ** (-i / R), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "turns":
        turns = length * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
    elif scaling == "ramp":
        def pair(turns):                              # whose frequency turns that often
            return R * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
        keep = 1 - ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
        scale = 1 + 0.1 * math.log(factor)
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, linear, base, turns or ramp, got %r" % (scaling,))
    return freq.to(device if device is not None else "cuda"), scale
