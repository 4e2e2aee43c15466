"""The operators around the delta rule: causal convolution, selective scan, 8-bit paged cache.

Python side of ``include/cgdr_serve.h``: each call checks types and shapes, packs the argument
block of its C entry point and runs it on the current CUDA stream (or ``stream``).  As for
:func:`~gated_delta_rule_channelwise_gb300.decode`, every step runs in the library's kernels and
there is no CPU fallback.  The tensors of a call share one device, the current one.  Outputs that
are not given, and workspaces, come from torch's caching allocator; with ``stream`` they are
allocated on that stream.  An output may not overlap an input, other than what is updated in place.

* :func:`conv_prefill`, :func:`conv_decode` -- short causal convolution with its state.
* :func:`scan_prefill`, :func:`scan_decode` -- selective state space scan.
* :func:`cache_plan` -- block tables and slots of a step, from the requests' lengths.
* :func:`cache_append` -- quantise new keys and values into the 8-bit cache.
* :func:`cache_attend` -- attention of the newest tokens over that cache.
"""
from __future__ import annotations

import struct

import torch

from . import ATTEND_AUTO, ATTEND_ROWS, ATTEND_TILES, BF16, F32, SIGNATURES, CgdrError, _need_cuda, lib  # noqa: F401

_F32, _I32 = torch.float32, torch.int32
_CODES = {torch.float32: F32, torch.bfloat16: BF16}
_NONE = (0, 0, 0)


class Block:
    """An argument block: (field, struct code) pairs in the order of the C struct.

    Packing with ``struct`` costs a tenth of filling a ``ctypes.Structure``, which matters for calls of
    a few microseconds.  ``@`` gives C's own alignment; the last code aligns the size to 8 bytes.
    """

    def __init__(self, *fields):
        self.fields = fields
        self._struct = struct.Struct("@" + "".join(code for _, code in fields) + "0q")
        self.pack, self.size = self._struct.pack, self._struct.size

    def offset(self, name):
        code = ""
        for field, c in self.fields:
            code += c
            if field == name:
                return struct.calcsize("@" + code) - struct.calcsize("@" + c)
        raise KeyError(name)


def _i(names):
    return [(n, "i") for n in names.split()]


def _p(names):
    return [(n, "P") for n in names.split()]


def _strided(name, *strides):
    return [(name, "P")] + [(name + "_" + s, "q") for s in strides]


CONV = Block(*_i("B T C W dtype silu n_tokens reserved"), *_strided("x", "sb", "st"), *_strided("o", "sb", "st"),
             *_p("weight bias state cu status"))
SCAN = Block(*_i("B T C N G dtype o_dtype softplus n_tokens reserved"), *_strided("x", "sb", "st"),
             *_strided("dt", "sb", "st"), *_strided("z", "sb", "st"), *_strided("Bm", "sb", "st"),
             *_strided("Cm", "sb", "st"), *_strided("o", "sb", "st"), *_p("A_log D dt_bias state cu status"))
PLAN = Block(*_i("B width page n_tokens F num_pages"), *_p("block_table"), ("table_sb", "q"),
             *_p("seq_lens new_lens free_pages free_count free_count_out kv_lens cu requests positions slots status"))
APPEND = Block(*_i("n Hkv D page dtype num_pages"), *_strided("k", "st", "sh"), *_strided("v", "st", "sh"),
               *_p("slots k_cache v_cache k_scale v_scale status"))
ATTEND = Block(*_i("B n Hq Hkv D page width dtype num_pages max_q max_kv path wait_polls"), ("scale", "f"), *_strided("q", "st", "sh"),
               *_strided("o", "st", "sh"), *_p("k_cache v_cache k_scale v_scale block_table"), ("table_sb", "q"),
               *_p("kv_lens cu status"))


def _on(stream, fn, *args, **kw):
    """fn with ``stream`` as the current one: what it allocates belongs to that stream, too."""
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


# The handle of a device's current stream, without the Stream object that torch.cuda.current_stream builds
# (2.9 us on a Grace host, as long as all the checks of a call).
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)

# The current device, without the initialisation check of torch.cuda.current_device: only asked beside a CUDA tensor.
_here = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _refuse(dtypes, shapes, dense):
    """Raises for what is wrong: (name, tensor, dtype), (name, tensor, shape) and (name, tensor) triples.

    The calls first test everything in one expression and come here only when it fails: naming the fault
    takes longer than the kernels of a small call."""
    for name, t, dtype in dtypes:
        if t is not None and t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    for name, t, shape in shapes:
        if t is not None and t.shape != tuple(shape):
            raise ValueError("%s must have shape %s, got %s" % (name, list(shape), list(t.shape)))
    for name, t in dense:
        if t is not None and not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    raise ValueError("the arguments do not agree")


def _fits(t, dtype, shape):
    """Whether a dense operand, which may be absent, has this type and shape."""
    return t is None or (t.dtype == dtype and t.shape == shape and t.is_contiguous())


def _address(t):
    return 0 if t is None else t.data_ptr()


def _status_word(status, device):
    if status.dtype != torch.int32 or status.numel() < 1 or not status.is_cuda:
        raise TypeError("status must be an int32 CUDA tensor")
    if status.get_device() != device:
        raise ValueError("status is on CUDA device %d, the other tensors on %d" % (status.get_device(), device))
    return status.data_ptr()


def _on_device(t, device):
    return t is None or t.get_device() == device


def _rows(t, name, step):
    """(pointer, batch stride, token stride) of [B, T, C] rows; with ``step`` of [B, C] or packed [n, C]: the
    stride of the first dimension then stands in for both."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError("%s: innermost dimension must be contiguous" % name)
    return (t.data_ptr(), st[0], st[0]) if step else (t.data_ptr(), st[0], st[1])


def _grouped(t, name, step, shape):
    """The same for [B, T, G, N], or [B, G, N] and packed [n, G, N], whose groups have to be dense."""
    st = t.stride()
    if (st[-1] != 1 and shape[-1] > 1) or (shape[-2] > 1 and st[-2] != shape[-1]):
        raise ValueError("%s: the last two dimensions must be contiguous" % name)
    return (t.data_ptr(), st[0], st[0]) if step else (t.data_ptr(), st[0], st[1])


def _heads(t, name):
    """(pointer, token stride, head stride) of [n, H, D]."""
    st = t.stride()
    if st[2] != 1 and t.shape[2] > 1:
        raise ValueError("%s: innermost dimension must be contiguous" % name)
    return t.data_ptr(), st[0], st[1]


def _sequences(x, state, cu):
    """Sequences of packed rows with offsets."""
    B = cu.numel() - 1
    if cu.dtype != torch.int32 or cu.dim() != 1 or B < 0 or not cu.is_contiguous():
        raise TypeError("cu_seqlens must be a dense int32 tensor of B + 1 offsets")
    if state.shape[0] != B:
        raise ValueError("state has %d sequences, cu_seqlens %d" % (state.shape[0], B))
    return B


# --------------------------------------------------------------------------- convolution


def _conv(x, weight, state, o, bias, silu, B, T, cu, status):
    """x is [B, T, C], or [B, C] / packed [n, C] (T is 1 / 0)."""
    device = x.get_device()
    if not (device >= 0 and device == weight.get_device() == state.get_device() == _here() and _on_device(bias, device)
            and _on_device(cu, device) and _on_device(o, device)):
        _need_cuda(x, weight, state, o, bias, cu)
    if o is None:
        o = torch.empty_like(x)
    dtype, shape = x.dtype, x.shape
    C, W, step = shape[-1], weight.shape[-1], len(shape) == 2
    if not (o.dtype == dtype and o.shape == shape and _fits(weight, _F32, (C, W)) and _fits(bias, _F32, (C,))
            and _fits(state, dtype, (B, W - 1, C))):
        _refuse([("weight", weight, _F32), ("bias", bias, _F32), ("state", state, dtype), ("o", o, dtype)],
                [("o", o, shape), ("weight", weight, (C, W)), ("bias", bias, (C,)), ("state", state, (B, W - 1, C))],
                [("weight", weight), ("bias", bias), ("state", state)])
    block = CONV.pack(B, T, C, W, _CODES.get(dtype, -1), 1 if silu else 0, 0 if cu is None else shape[0], 0, *_rows(x, "x", step),
                      *_rows(o, "o", step), weight.data_ptr(), _address(bias), state.data_ptr(), _address(cu),
                      0 if status is None else _status_word(status, device))
    st = lib().cgdr_conv(block, _current(device))
    if st:
        raise CgdrError(st, "cgdr_conv")
    return o


def conv_prefill(x, weight, state, o=None, *, bias=None, silu=True, cu_seqlens=None, status=None, stream=None):
    """Short causal convolution over prompts: ``x [B,T,C]``, or packed ``[n,C]`` with
    ``cu_seqlens [B+1]`` (int32, on the device).  ``weight [C,W]`` fp32 (W = 2, 3 or 4, the last
    column meets the current token), ``bias [C]`` fp32, SiLU unless ``silu=False``.  ``state [B,W-1,C]``
    in x's dtype holds the rows before x and is updated in place (zeros start a sequence).
    x and o may be strided in batch and tokens; rows are 16-byte aligned.  Returns o, like x."""
    if stream is not None:
        return _on(stream, conv_prefill, x, weight, state, o, bias=bias, silu=silu, cu_seqlens=cu_seqlens, status=status)
    if x.dim() != (3 if cu_seqlens is None else 2):
        raise ValueError("x must be [B, T, C], or packed [n, C] with cu_seqlens")
    B, T = x.shape[:2] if cu_seqlens is None else (_sequences(x, state, cu_seqlens), 0)
    return _conv(x, weight, state, o, bias, silu, B, T, cu_seqlens, status)


def conv_decode(x, weight, state, o=None, *, bias=None, silu=True, status=None, stream=None):
    """One token of :func:`conv_prefill` for every sequence: ``x [B,C]``."""
    if stream is not None:
        return _on(stream, conv_decode, x, weight, state, o, bias=bias, silu=silu, status=status)
    if x.dim() != 2:
        raise ValueError("x must be [B, C]")
    return _conv(x, weight, state, o, bias, silu, x.shape[0], 1, None, status)


# --------------------------------------------------------------------------- scan


def _scan(x, dt, A_log, Bm, Cm, state, o, D, z, dt_bias, softplus, B, T, cu, workspace, status):
    """x is [B, T, C], or [B, C] / packed [n, C] (T is 1 / 0)."""
    device = x.get_device()
    if not (device >= 0 and device == dt.get_device() == A_log.get_device() == Bm.get_device() == Cm.get_device()
            == state.get_device() == _here() and _on_device(o, device) and _on_device(D, device) and _on_device(z, device)
            and _on_device(dt_bias, device) and _on_device(cu, device) and _on_device(workspace, device)):
        _need_cuda(x, dt, A_log, Bm, Cm, state, o, D, z, dt_bias, cu, workspace)
    if o is None:
        o = torch.empty_like(x)
    dtype, shape = x.dtype, x.shape
    C, (G, N), step = shape[-1], Bm.shape[-2:], len(shape) == 2
    grouped = (*shape[:-1], G, N)
    if not (dt.dtype == dtype and dt.shape == shape and o.shape == shape and Bm.dtype == dtype and Bm.shape == grouped
            and Cm.dtype == dtype and Cm.shape == grouped and (z is None or (z.dtype == dtype and z.shape == shape))
            and _fits(A_log, _F32, (C, N)) and _fits(state, _F32, (B, C, N)) and _fits(D, _F32, (C,))
            and _fits(dt_bias, _F32, (C,))):
        _refuse([("A_log", A_log, _F32), ("state", state, _F32), ("D", D, _F32), ("dt_bias", dt_bias, _F32),
                 ("dt", dt, dtype), ("z", z, dtype), ("Bm", Bm, dtype), ("Cm", Cm, dtype)],
                [("dt", dt, shape), ("z", z, shape), ("o", o, shape), ("Bm", Bm, grouped), ("Cm", Cm, grouped),
                 ("A_log", A_log, (C, N)), ("state", state, (B, C, N)), ("D", D, (C,)), ("dt_bias", dt_bias, (C,))],
                [("A_log", A_log), ("state", state), ("D", D), ("dt_bias", dt_bias)])
    block = SCAN.pack(B, T, C, N, G, _CODES.get(dtype, -1), _CODES.get(o.dtype, -1), 1 if softplus else 0, 0 if cu is None else shape[0], 0,
                      *_rows(x, "x", step), *_rows(dt, "dt", step), *(_rows(z, "z", step) if z is not None else _NONE),
                      *_grouped(Bm, "Bm", step, grouped), *_grouped(Cm, "Cm", step, grouped), *_rows(o, "o", step), A_log.data_ptr(),
                      _address(D), _address(dt_bias), state.data_ptr(), _address(cu), 0 if status is None else _status_word(status, device))
    L = lib()
    need = 0 if T == 1 else L.cgdr_scan_workspace_size(block)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    st = L.cgdr_scan(block, workspace.data_ptr() if need else None, need, _current(device))
    if st:
        raise CgdrError(st, "cgdr_scan")
    return o


def scan_prefill(x, dt, A_log, Bm, Cm, state, o=None, *, D=None, z=None, dt_bias=None, softplus=True, cu_seqlens=None,
                 workspace=None, status=None, stream=None):
    """Selective state space scan over prompts: ``x, dt, z [B,T,C]``, ``Bm, Cm [B,T,G,N]`` (group g serves
    channels g C/G .. (g+1) C/G - 1), or the same packed ``[n,C]``, ``[n,G,N]`` with ``cu_seqlens [B+1]``.
    ``A_log [C,N]``, ``D [C]``, ``dt_bias [C]`` fp32; ``state [B,C,N]`` fp32, updated in place.

    With ``d = softplus(dt + dt_bias)``: ``h = exp(-exp(A_log) d) h + d x Bm``, ``o = Cm.h + D x``, times
    ``z / (1 + e^-z)`` if z is given.  N is 16, 32, 64 or 128 and C/G a multiple of 8.  Returns o: the given one
    (fp32 or bf16) or a new one like x.  ``workspace``: a buffer of :func:`scan_workspace_size` bytes or
    more keeps the call free of allocations."""
    if stream is not None:
        return _on(stream, scan_prefill, x, dt, A_log, Bm, Cm, state, o, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                   cu_seqlens=cu_seqlens, workspace=workspace, status=status)
    lead = 1 if cu_seqlens is not None else 2
    if x.dim() != lead + 1 or Bm.dim() != lead + 2:
        raise ValueError("x must be [B, T, C] and Bm [B, T, G, N], or packed [n, C] and [n, G, N] with cu_seqlens")
    B, T = x.shape[:2] if cu_seqlens is None else (_sequences(x, state, cu_seqlens), 0)
    return _scan(x, dt, A_log, Bm, Cm, state, o, D, z, dt_bias, softplus, B, T, cu_seqlens, workspace, status)


def scan_decode(x, dt, A_log, Bm, Cm, state, o=None, *, D=None, z=None, dt_bias=None, softplus=True, status=None,
                stream=None):
    """One token of :func:`scan_prefill` for every sequence: ``x, dt, z [B,C]``, ``Bm, Cm [B,G,N]``."""
    if stream is not None:
        return _on(stream, scan_decode, x, dt, A_log, Bm, Cm, state, o, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                   status=status)
    if x.dim() != 2 or Bm.dim() != 3:
        raise ValueError("x must be [B, C] and Bm [B, G, N]")
    return _scan(x, dt, A_log, Bm, Cm, state, o, D, z, dt_bias, softplus, x.shape[0], 1, None, None, status)


def scan_workspace_size(B, T, C, N, G=1, *, n_tokens=None, dtype=torch.bfloat16) -> int:
    """Bytes of workspace of a :func:`scan_prefill` of these sizes (``n_tokens``: packed, with T ignored)."""
    esz = 2 if dtype == torch.bfloat16 else 4
    fake = 1 << 20                                    # checked for alignment, never read
    rows = (fake, 0 if n_tokens is not None else C * T, C)
    groups = (fake, 0 if n_tokens is not None else G * N * T, G * N)
    block = SCAN.pack(B, T, C, N, G, _CODES[dtype], _CODES[dtype], 1, n_tokens or 0, 0, *rows, *rows, 0, 0, 0, *groups,
                      *groups, *rows, fake, 0, 0, fake, fake if n_tokens is not None else 0, 0)
    return lib().cgdr_scan_workspace_size(block)


# --------------------------------------------------------------------------- 8-bit cache


_MAX_KV = (1 << 30) - 1                               # cached tokens of a request at most
_PLAN_PARTS = frozenset(("slots", "kv_lens", "cu_seqlens", "free_count", "requests", "positions"))


class CachePlan:
    """What :func:`cache_plan` writes: see there.  One buffer holds it all; it is cut into tensors when one of
    them is first asked for, all at once (a view each costs as much as checking a call's arguments)."""

    def __init__(self, B, n_tokens, device="cuda"):
        self.B, self.n_tokens = B, n_tokens
        # slots [n] int64 first, then int32: kv_lens [B], cu_seqlens [B + 1], free_count [1], requests [n], positions [n]
        self._buffer = torch.empty(n_tokens + B + 1 + n_tokens, dtype=torch.int64, device=device)
        slots = self._buffer.data_ptr()
        kv = slots + 8 * n_tokens
        count = kv + 4 * (2 * B + 1)
        self._addresses = count, kv, kv + 4 * B, count + 4, count + 4 + 4 * n_tokens, slots

    def __getattr__(self, name):
        if name not in _PLAN_PARTS:
            raise AttributeError(name)
        B, n, parts = self.B, self.n_tokens, self.__dict__
        slots, parts["kv_lens"], parts["cu_seqlens"], parts["free_count"], parts["requests"], parts["positions"] = \
            self._buffer.view(_I32).unsafe_split_with_sizes((2 * n, B, B + 1, 1, n, n))
        parts["slots"] = slots.view(torch.int64)
        return parts[name]


def cache_plan(block_table, seq_lens, new_lens, free_pages, free_count, n_tokens, page, out=None, *, num_pages=None,
               status=None, stream=None):
    """Block tables and slots of a step, on the device.  Request b holds ``seq_lens[b]`` cached tokens in
    the first pages of its row of ``block_table [B,width]`` and gets ``new_lens[b]`` more; the pages it
    needs come off the top of the stack ``free_pages[:free_count]``, in request order, and are entered into
    block_table (in place).  All int32.  Returns a :class:`CachePlan` (``out``, or a new one; its ``kv_lens`` and
    ``free_count`` are the next step's ``seq_lens`` and ``free_count``, so steps that reuse buffers take turns with two):

    ``cu_seqlens`` prefix sums of new_lens; ``kv_lens = seq_lens + new_lens``; per packed new token its
    ``requests``, ``positions`` (place in the request) and ``slots`` (int64 ``page_number * page + place in
    the page``), -1 from the last new token to ``n_tokens``; ``free_count`` pages left.

    If the pages, the table's width or ``n_tokens`` do not suffice nothing is taken: every slot is -1, lengths
    and free count stay, and ``status`` receives ``ERR_CAPACITY`` (``ERR_INVALID_ARG`` for negative lengths
    and for free pages outside ``num_pages``, by default any number)."""
    if stream is not None:
        return _on(stream, cache_plan, block_table, seq_lens, new_lens, free_pages, free_count, n_tokens, page, out,
                   num_pages=num_pages, status=status)
    device = block_table.get_device()
    if not (device >= 0 and device == seq_lens.get_device() == new_lens.get_device() == free_pages.get_device()
            == free_count.get_device() == _here() and (out is None or out._buffer.get_device() == device)):
        _need_cuda(block_table, seq_lens, new_lens, free_pages, free_count, None if out is None else out._buffer)
    B, width = block_table.shape
    F = free_pages.numel()
    if out is None:
        out = CachePlan(B, n_tokens, block_table.device)
    elif out.B != B or out.n_tokens != n_tokens:
        raise ValueError("out is a plan of %d requests and %d tokens, not of %d and %d" % (out.B, out.n_tokens, B, n_tokens))
    if not (block_table.dtype == _I32 and _fits(seq_lens, _I32, (B,)) and _fits(new_lens, _I32, (B,))
            and _fits(free_pages, _I32, (F,)) and _fits(free_count, _I32, (1,))):
        named = [("seq_lens", seq_lens, B), ("new_lens", new_lens, B), ("free_pages", free_pages, F), ("free_count", free_count, 1)]
        _refuse([("block_table", block_table, _I32)] + [(name, t, _I32) for name, t, _ in named],
                [(name, t, (size,)) for name, t, size in named], [(name, t) for name, t, _ in named])
    sb, sw = block_table.stride()
    if sw != 1 and width > 1:
        raise ValueError("block_table: innermost dimension must be contiguous")
    block = PLAN.pack(B, width, page, n_tokens, F, 0x7FFFFFFF if num_pages is None else num_pages,
                      block_table.data_ptr(), sb, seq_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(),
                      free_count.data_ptr(), *out._addresses, 0 if status is None else _status_word(status, device))
    st = lib().cgdr_cache_plan(block, _current(device))
    if st:
        raise CgdrError(st, "cgdr_cache_plan")
    return out


def _check_cache(k_cache, v_cache, k_scale, v_scale):
    """(pages, Hkv, page, D) of a cache: int8 [pages, Hkv, page, D] with fp32 scales [pages, Hkv]."""
    device = k_cache.get_device()
    if not (device >= 0 and device == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == _here()):
        _need_cuda(k_cache, v_cache, k_scale, v_scale)
    shape = k_cache.shape
    if len(shape) != 4:
        raise ValueError("k_cache must be [pages, Hkv, page, D]")
    if not (_fits(k_cache, torch.int8, shape) and _fits(v_cache, torch.int8, shape) and _fits(k_scale, _F32, shape[:2])
            and _fits(v_scale, _F32, shape[:2])):
        _refuse([("k_cache", k_cache, torch.int8), ("v_cache", v_cache, torch.int8), ("k_scale", k_scale, _F32),
                 ("v_scale", v_scale, _F32)],
                [("v_cache", v_cache, shape), ("k_scale", k_scale, shape[:2]), ("v_scale", v_scale, shape[:2])],
                [("k_cache", k_cache), ("v_cache", v_cache), ("k_scale", k_scale), ("v_scale", v_scale)])
    return shape


def cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, *, status=None, stream=None):
    """Quantise ``k, v [n,Hkv,D]`` (fp32 or bf16) into the cache: ``k_cache, v_cache`` int8
    ``[pages,Hkv,page,D]``, ``k_scale, v_scale`` fp32 ``[pages,Hkv]``, all updated in place.  Token i goes to
    ``slots[i]`` (int64, as :func:`cache_plan` gives them: tokens of a page consecutive and ascending; below 0:
    nowhere).  A page's scale of a head is the largest magnitude in it times 1/127 (in fp32); where new values
    raise it, what the page holds is rounded to the larger scale.  A token at a page's offset 0 starts the page afresh.  A
    slot outside the cache is skipped and reported in ``status`` (``ERR_BOUNDS``)."""
    if stream is not None:
        return _on(stream, cache_append, k, v, slots, k_cache, v_cache, k_scale, v_scale, status=status)
    pages, Hkv, page, D = _check_cache(k_cache, v_cache, k_scale, v_scale)
    device = k.get_device()
    if not (device == v.get_device() == slots.get_device() == k_cache.get_device()):
        _need_cuda(k, v, slots, k_cache)
    n = k.shape[0]
    shape = (n, Hkv, D)
    if not (k.shape == shape and v.shape == shape and v.dtype == k.dtype and _fits(slots, torch.int64, (n,))):
        _refuse([("v", v, k.dtype), ("slots", slots, torch.int64)], [("k", k, shape), ("v", v, shape), ("slots", slots, (n,))],
                [("slots", slots)])
    block = APPEND.pack(n, Hkv, D, page, _CODES.get(k.dtype, -1), pages, *_heads(k, "k"), *_heads(v, "v"), slots.data_ptr(),
                        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                        0 if status is None else _status_word(status, device))
    st = lib().cgdr_cache_append(block, _current(device))
    if st:
        raise CgdrError(st, "cgdr_cache_append")


def cache_attend(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, o=None, *, max_q, max_kv=None,
                 scale=None, path=ATTEND_AUTO, workspace=None, status=None, wait_polls=0, stream=None):
    """Attention of the newest tokens over the cache (layout as in :func:`cache_append`).  ``q [n,Hq,D]`` (fp32 or
    bf16) packs the query tokens of all requests, ``cu_seqlens [B+1]`` says whose they are; they are the last of
    the ``kv_lens[b]`` cached tokens, each sees the tokens up to itself, and a row that sees nothing is zero.
    ``block_table [B,width]``, ``kv_lens``, ``cu_seqlens`` int32 as :func:`cache_plan` leaves them.  Query head h
    reads key-value head h / (Hq/Hkv); ``scale``, above 0, defaults to 1/sqrt(D).

    ``max_q`` and ``max_kv`` bound the requests' query and cached tokens on the host (default for max_kv: what
    the table holds); what exceeds them is cut off and reported in ``status`` (``ERR_CAPACITY``), and pages
    outside the cache are left out (``ERR_BOUNDS``).  Rows of q past ``cu_seqlens[B]`` are not computed.  Returns
    o ``[n,Hq,D]``, like q.  ``path`` forces one of the two kernels for this call (``ATTEND_ROWS``,
    ``ATTEND_TILES``; the latter covers bf16 with D = 128).  ``workspace``: a buffer of
    :func:`cache_attend_workspace_size` bytes (for dense q and o) or more keeps the call free of allocations.
    The choice goes by ``max_q`` and ``max_kv`` as if every request had them: a long prompt among many single
    tokens over long caches takes less time in a call of its own.
    ``wait_polls``: polls of a bounded device wait (0: the default; ``ERR_TIMEOUT`` in ``status`` when one gives up)."""
    if stream is not None:
        return _on(stream, cache_attend, q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, cu_seqlens, o,
                   max_q=max_q, max_kv=max_kv, scale=scale, path=path, workspace=workspace, status=status, wait_polls=wait_polls)
    if scale is not None and not scale > 0:
        raise ValueError("scale must be above 0, got %s" % scale)    # the library would take its default
    pages, Hkv, page, D = _check_cache(k_cache, v_cache, k_scale, v_scale)
    device = q.get_device()
    if not (device == block_table.get_device() == kv_lens.get_device() == cu_seqlens.get_device() == k_cache.get_device()
            and _on_device(o, device) and _on_device(workspace, device)):
        _need_cuda(q, o, block_table, kv_lens, cu_seqlens, workspace, k_cache)
    if o is None:
        o = torch.empty_like(q)
    n, Hq, Dq = q.shape
    if Dq != D:
        raise ValueError("q has head dimension %d, the cache %d" % (Dq, D))
    B, width = block_table.shape
    if not (o.dtype == q.dtype and o.shape == q.shape and block_table.dtype == _I32 and _fits(kv_lens, _I32, (B,))
            and _fits(cu_seqlens, _I32, (B + 1,))):
        _refuse([("o", o, q.dtype), ("block_table", block_table, _I32), ("kv_lens", kv_lens, _I32),
                 ("cu_seqlens", cu_seqlens, _I32)],
                [("o", o, q.shape), ("kv_lens", kv_lens, (B,)), ("cu_seqlens", cu_seqlens, (B + 1,))],
                [("kv_lens", kv_lens), ("cu_seqlens", cu_seqlens)])
    sb, sw = block_table.stride()
    if sw != 1 and width > 1:
        raise ValueError("block_table: innermost dimension must be contiguous")
    block = ATTEND.pack(B, n, Hq, Hkv, D, page, width, _CODES.get(q.dtype, -1), pages, max_q,
                        min(width * page, _MAX_KV) if max_kv is None else max_kv, path, wait_polls, 0.0 if scale is None else scale, *_heads(q, "q"), *_heads(o, "o"), k_cache.data_ptr(),
                        v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), sb,
                        kv_lens.data_ptr(), cu_seqlens.data_ptr(), 0 if status is None else _status_word(status, device))
    L = lib()
    need = L.cgdr_cache_attend_workspace_size(block)
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    st = L.cgdr_cache_attend(block, workspace.data_ptr() if need else None, need, _current(device))
    if st:
        raise CgdrError(st, "cgdr_cache_attend")
    return o


def cache_attend_workspace_size(B, n, Hq, Hkv, D, page, width, *, max_q, max_kv=None, dtype=torch.bfloat16,
                                path=ATTEND_AUTO) -> int:
    """Bytes of workspace of a :func:`cache_attend` of these sizes."""
    fake = 1 << 20                                    # checked for alignment, never read
    block = ATTEND.pack(B, n, Hq, Hkv, D, page, width, _CODES[dtype], 1, max_q,
                        min(width * page, _MAX_KV) if max_kv is None else max_kv, path, 0, 0.0, fake, Hq * D, D, fake, Hq * D, D, fake, fake, fake, fake, fake, width, fake, fake, 0)
    return lib().cgdr_cache_attend_workspace_size(block)
