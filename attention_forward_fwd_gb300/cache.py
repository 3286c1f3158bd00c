"""The quantised K/V cache and the rotary positions, for torch CUDA tensors.

A decoding step turns its q and k (``rotary``), writes k and v into the cache
(``kv4_write``) and attends over it (``kv4_attention``); ``kv4_read`` gives
plain K and V back, for the other attention calls.  As in the rest of the
package this module only marshals arguments (and records nothing for
autograd); the work runs in the library's kernels (``fa_kv4_*`` and
``fa_rotary`` in ``include/fa_gb300.h``, where the cache's format and the checks
on the device are described).

Every call takes ``page_table`` (int32 [B, max_pages]) and ``seq_lens`` (int32
[B], the tokens in the cache with the call's own), and concerns the LAST rows of
each sequence: S of them in batched tensors [B, S, heads, D], or
``cu_seqlens[b + 1] - cu_seqlens[b]`` in packed ones [total, heads, D].
"""
from __future__ import annotations

import ctypes
import functools
import struct

import attention_forward_fwd_gb300 as _fa

KV4_GROUP = 32   # values that share a scale

# A decoding step makes these calls for every layer and its kernels take
# microseconds.  So the common case goes through csrc/fa_binding.cpp, and the code
# here (other devices and streams, and what does not fit) looks at each property of a tensor
# once, in one expression, and finds out what was wrong only when that fails.
_pack_cache = struct.Struct("@5P8i").pack      # fa_kv4_cache_t
_pack3 = struct.Struct("@3q").pack             # strides
_pack2 = struct.Struct("@2q").pack
if struct.calcsize("@5P8i") != ctypes.sizeof(_fa.Kv4Cache):
    raise ImportError("fa_kv4_cache_t is not laid out as expected")

_torch = None


def _lib():
    """The library; torch too, which the package does not import by itself, and the
    native marshalling where it has been built."""
    global _torch, _native
    if _torch is None:
        import torch
        _torch = torch
        lib = _fa.library()
        _native = _load_native(lib)
    return _fa._LIB or _fa.library()


_native = None   # csrc/fa_binding.cpp


def _load_native(lib):
    import importlib.machinery
    import importlib.util

    from .build import BINDING_PATH, binding_built
    if not binding_built():
        return None
    loader = importlib.machinery.ExtensionFileLoader("fa_binding", BINDING_PATH)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("fa_binding", loader))
    loader.exec_module(module)
    module.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.fa_kv4_write, lib.fa_kv4_read, lib.fa_kv4_attention_workspace_size, lib.fa_kv4_attention, lib.fa_rotary)))
    return module


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _code(dtype):
    if dtype is _torch.bfloat16:
        return _fa.FA_BF16
    _need(dtype is _torch.float16, f"unsupported dtype {dtype}")
    return _fa.FA_F16


class _On:
    """The device and stream of a call that names a stream, or whose tensors are
    not on the current device.  Tensors that the call makes are made with
    that stream current, so that the allocator hands their memory out again in
    that stream's order; tensors that it is given are recorded on a stream that
    is not their own."""

    def __init__(self, device, stream):
        torch = _torch
        self.inner = None
        self.guard = torch.cuda.device(device)
        self.guard.__enter__()
        try:
            self.handle = _fa._stream_handle(stream)
            if self.handle != torch.cuda.current_stream(device).cuda_stream:
                self.target = (stream if isinstance(stream, torch.cuda.Stream)
                               else torch.cuda.default_stream(device) if self.handle == 0
                               else torch.cuda.ExternalStream(self.handle, device=device))
                inner = torch.cuda.stream(self.target)
                inner.__enter__()
                self.inner = inner
        except BaseException:
            self.guard.__exit__(None, None, None)
            raise

    def done(self, *tensors):
        if self.inner is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.target)
            self.inner.__exit__(None, None, None)
        self.guard.__exit__(None, None, None)


def _enter(device, stream):
    """(stream handle, _On or None): None when the call is for the current stream of the current device."""
    if stream is None and _torch.cuda.current_device() == device.index:
        return _current_stream(device.index), None
    on = _On(device, stream)
    return on.handle, on


def _current_stream(index):
    global _current_stream
    # the handle alone, where torch offers it: the Stream object costs 2 us a call
    raw = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    _current_stream = raw if raw is not None else (lambda i: _torch.cuda.current_stream(i).cuda_stream)
    return _current_stream(index)


def kv4_empty_cache(pages: int, H_kv: int, D: int, page_size: int = 64, device="cuda"):
    """(codes, scales) of an empty cache: uint8 [pages, 2, H_kv, page_size, D / 2]
    and bfloat16 [pages, 2, H_kv, page_size, D / 32] (4.5 bits a value)."""
    import torch
    _need(pages > 0 and H_kv > 0, "pages and H_kv must be positive")
    _need(D % KV4_GROUP == 0 and 0 < D <= 256, "D must be a multiple of 32 up to 256")
    _need(page_size > 0 and page_size % 16 == 0, "page_size must be a multiple of 16")
    codes = torch.full((pages, 2, H_kv, page_size, D // 2), 0x88, dtype=torch.uint8, device=device)
    scales = torch.zeros((pages, 2, H_kv, page_size, D // KV4_GROUP), dtype=torch.bfloat16, device=device)
    return codes, scales


def _cache(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, rows):
    """The call's fa_kv4_cache_t as bytes, then B, S, total, max_pages,
    page_size, H_kv and D; ``rows``: total of packed tensors, S of batched ones."""
    i32, dev = _torch.int32, codes.device
    csh, tsh = codes.shape, page_table.shape
    if len(csh) != 5 or len(tsh) != 2:
        _say_cache(codes, scales, page_table, seq_lens)
    pages, two, H_kv, P, half = csh
    B, max_pages = tsh
    if not (two == 2 and codes.is_cuda and codes.dtype is _torch.uint8 and codes.is_contiguous()
            and scales.dtype is _torch.bfloat16 and scales.shape == (pages, 2, H_kv, P, half // 16)
            and scales.is_contiguous() and page_table.dtype is i32 and page_table.is_contiguous()
            and seq_lens.dtype is i32 and seq_lens.shape == (B,) and seq_lens.is_contiguous()
            and scales.device == dev and page_table.device == dev and seq_lens.device == dev):
        _say_cache(codes, scales, page_table, seq_lens)
    if cu_seqlens is None:
        cu, S, total = 0, rows, 0
    else:
        _need(cu_seqlens.dtype is i32 and cu_seqlens.shape == (B + 1,) and cu_seqlens.is_contiguous()
              and cu_seqlens.device == dev,
              "cu_seqlens must be a contiguous int32 tensor [B + 1] on the cache's device")
        cu, total = cu_seqlens.data_ptr(), rows
        S = total if max_seqlen is None else int(max_seqlen)
    D = half * 2
    try:
        c = _pack_cache(codes.data_ptr(), scales.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), cu,
                        B, S, total, pages, max_pages, P, H_kv, D)
    except struct.error:
        raise ValueError("sizes must fit 32 bits") from None
    return c, B, S, total, max_pages, P, H_kv, D


def _say_cache(codes, scales, page_table, seq_lens):
    torch = _torch
    _need(codes.is_cuda and codes.dtype is torch.uint8 and codes.dim() == 5 and codes.is_contiguous()
          and codes.shape[1] == 2, "codes must be a contiguous uint8 CUDA tensor [pages, 2, H_kv, page_size, D / 2]")
    pages, _, H_kv, P, half = codes.shape
    _need(scales.dtype is torch.bfloat16 and scales.is_contiguous()
          and scales.shape == (pages, 2, H_kv, P, half // 16),
          "scales must be a contiguous bfloat16 tensor [pages, 2, H_kv, page_size, D / 32]")
    _need(page_table.dtype is torch.int32 and page_table.dim() == 2 and page_table.is_contiguous(),
          "page_table must be a contiguous int32 tensor [B, max_pages]")
    _need(seq_lens.dtype is torch.int32 and seq_lens.shape == (page_table.shape[0],) and seq_lens.is_contiguous(),
          "seq_lens must be a contiguous int32 tensor [B]")
    raise ValueError("codes, scales, page_table and seq_lens must be on one device")


def _rows(name, t, packed, B, heads, D, device):
    """Checks a tensor of the call's rows (heads: None for any); its strides (batch, row, head) as bytes."""
    sh, st = t.shape, t.stride()
    if packed:
        if len(sh) == 3 and sh[2] == D and (heads is None or sh[1] == heads) and st[2] == 1 and t.device == device:
            return _pack3(0, st[0], st[1])
    elif len(sh) == 4 and sh[3] == D and (heads is None or sh[2] == heads) and sh[0] == B and st[3] == 1 \
            and t.device == device:
        return _pack3(st[0], st[1], st[2])
    _need(t.device == device, f"{name} is on {t.device}, the cache on {device}")
    _need(len(sh) == (3 if packed else 4), f"{name} must be [B, S, heads, D], or [total, heads, D] with cu_seqlens")
    _need(st[-1] == 1, f"the last axis of {name} must be contiguous")
    raise ValueError(f"{name} has shape {tuple(sh)}: its batch, heads and D must match the cache")


def _check(rc, what):
    if rc != _fa.FA_OK:
        raise _fa.FaError(rc, what)


def kv4_write(k, v, codes, scales, page_table, seq_lens, cu_seqlens=None, max_seqlen=None, k_out=None,
              v_out=None, stream=None):
    """Quantises k and v into the cache at their sequences' last tokens.

    k, v: fp16 / bf16 [B, S, H_kv, D], or packed [total, H_kv, D] with
    ``cu_seqlens`` (int32 [B + 1]; ``max_seqlen``: the most rows of a sequence,
    checked on the device); only the last axis has to be contiguous (strides in
    multiples of 4 elements), so slices of a fused projection can be passed.
    ``k_out``, ``v_out`` (contiguous, like k and v; both or neither) receive
    what the cache now stands for.  Work is enqueued on ``stream`` (default:
    the current one) and not waited for.
    """
    lib = _lib()
    if stream is None and _native is not None:
        rc = _native.kv4_write(k, v, codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, k_out, v_out)
        if rc is not NotImplemented:
            return _check(rc, "fa_kv4_write") if rc is not None else None
    dev, packed, shape = codes.device, cu_seqlens is not None, k.shape
    dtype = _code(k.dtype)
    _need(v.dtype is k.dtype and v.shape == shape and len(shape) >= 3, "k and v must be alike")
    c, B, _, _, _, _, H_kv, D = _cache(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, shape[-3])
    ks = _rows("k", k, packed, B, H_kv, D, dev)
    vs = _rows("v", v, packed, B, H_kv, D, dev)
    ko = vo = None
    if k_out is not None or v_out is not None:
        _need(k_out is not None and v_out is not None, "k_out and v_out come together")
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            _need(t.shape == shape and t.dtype is k.dtype and t.is_contiguous() and t.device == dev,
                  f"{name} must be a contiguous tensor like k")
        ko, vo = k_out.data_ptr(), v_out.data_ptr()
    if 0 in shape:
        return
    handle, on = _enter(dev, stream)
    rc = lib.fa_kv4_write(c, k.data_ptr(), v.data_ptr(), ks, vs, ko, vo, dtype, handle)
    if on is not None:
        on.done(k, v, codes, scales, page_table, seq_lens, cu_seqlens, k_out, v_out)
    _check(rc, "fa_kv4_write")


def kv4_read(codes, scales, page_table, seq_lens, cu_seqlens=None, max_seqlen=None, total=None, dtype=None,
             k_out=None, v_out=None, stream=None):
    """k, v of the sequences' last tokens, as plain tensors.

    Packed [total, H_kv, D] with ``cu_seqlens`` and ``total`` (its last offset,
    which the host has to know), or batched [B, max_seqlen, H_kv, D].
    ``dtype``: torch.float16 (exact within its range) or torch.bfloat16
    (default).  Rows before a sequence's first token are zeros; packed rows
    outside every sequence are left as they were (of ``k_out``, ``v_out`` when
    given, else not defined).
    """
    lib = _lib()
    if stream is None and k_out is None and v_out is None and _native is not None and \
            (dtype is None or dtype is _torch.bfloat16 or dtype is _torch.float16):
        r = _native.kv4_read(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen,
                             max_seqlen if cu_seqlens is None else total, dtype is not _torch.float16)
        if type(r) is tuple:
            return r
        if r is not NotImplemented:
            _check(r, "fa_kv4_read")
    dev = codes.device
    if cu_seqlens is None:
        _need(max_seqlen is not None, "max_seqlen (the rows of a sequence) is needed without cu_seqlens")
        rows = int(max_seqlen)
    else:
        _need(total is not None, "total is needed with cu_seqlens")
        rows = int(total)
    c, B, _, _, _, _, H_kv, D = _cache(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, rows)
    shape = (B, rows, H_kv, D) if cu_seqlens is None else (rows, H_kv, D)
    if k_out is not None or v_out is not None:
        _need(k_out is not None and v_out is not None, "k_out and v_out come together")
        _need(dtype is None or dtype is k_out.dtype, "dtype and k_out's differ")
        dtype = k_out.dtype
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            _need(t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.device == dev,
                  f"{name} must be a contiguous tensor {shape} on the cache's device")
    elif dtype is None:
        dtype = _torch.bfloat16
    code = _code(dtype)
    _need(rows >= 0, "the number of rows must not be negative")
    handle, on = _enter(dev, stream)
    try:
        if k_out is None:
            k_out = _torch.empty(shape, dtype=dtype, device=dev)
            v_out = _torch.empty(shape, dtype=dtype, device=dev)
        rc = lib.fa_kv4_read(c, k_out.data_ptr(), v_out.data_ptr(), code, handle) if 0 not in shape else _fa.FA_OK
    finally:
        if on is not None:
            on.done(codes, scales, page_table, seq_lens, cu_seqlens, k_out, v_out)
    _check(rc, "fa_kv4_read")
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(device_index, B, S, total, max_pages, P, H_kv, D, H, dtype):
    """Workspace of a call's sizes on the current device (which device_index names)."""
    n = ctypes.c_size_t(0)
    # the sizes alone matter: 16 stands in for the pointers
    c = _pack_cache(16, 16, 16, 16, 16 if total else 0, B, S, total, 1, max_pages, P, H_kv, D)
    _check(int(_fa.library().fa_kv4_attention_workspace_size(c, H, dtype, ctypes.byref(n))),
           "fa_kv4_attention_workspace_size")
    return n.value


def kv4_attention(q, codes, scales, page_table, seq_lens, cu_seqlens=None, max_seqlen=None,
                  window_left: int = -1, scale: float | None = None, out=None, lse=None, with_lse: bool = True,
                  stream=None):
    """O, LSE of the queries q over the cache.

    q: fp16 / bf16 [B, S, H, D], or packed [total, H, D] with ``cu_seqlens``
    (and ``max_seqlen``, the most rows of a sequence); H a multiple of H_kv
    (query head h uses K/V head h // (H / H_kv)); only the last axis has to be
    contiguous (strides in multiples of 8 elements).  Row i of the n rows of
    sequence b is its token seq_lens[b] - n + i and sees the tokens up to
    itself, from ``window_left`` before itself on (-1: from the first).  The
    call's own k and v are written first (``kv4_write``).  Rows without a token
    are O = 0, LSE = -inf.  O is contiguous like q, LSE fp32 [B, H, S] or
    [H, total].  The workspace is made anew for each call.
    """
    lib = _lib()
    if stream is None and _native is not None:
        r = _native.kv4_attention(q, codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, window_left, scale,
                                  out, lse, bool(with_lse))
        if type(r) is tuple:
            return r
        if r is not NotImplemented:
            _check(r, "fa_kv4_attention")
    dev, packed, shape = codes.device, cu_seqlens is not None, q.shape
    dtype = _code(q.dtype)
    _need(len(shape) >= 3, "q must be [B, S, H, D], or [total, H, D] with cu_seqlens")
    rows, H = shape[-3], shape[-2]
    c, B, S, total, max_pages, P, H_kv, D = _cache(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, rows)
    qs = _rows("q", q, packed, B, None, D, dev)
    _need(H > 0 and H_kv > 0 and H % H_kv == 0, "the heads of q must be a multiple of the cache's H_kv")
    lse_shape = (H, rows) if packed else (B, H, rows)
    if out is not None:
        _need(out.shape == shape and out.dtype is q.dtype and out.is_contiguous() and out.device == dev,
              "out must be a contiguous tensor like q")
    if lse is not None:
        _need(lse.shape == lse_shape and lse.dtype is _torch.float32 and lse.is_contiguous() and lse.device == dev,
              f"lse must be a contiguous fp32 tensor {lse_shape}")
    window = max(-2, min(int(window_left), 0x7fffffff))   # a C int; positions are below that
    handle, on = _enter(dev, stream)
    try:
        if out is None:
            out = _torch.empty(shape, dtype=q.dtype, device=dev)
        if lse is None and with_lse:
            lse = _torch.empty(lse_shape, dtype=_torch.float32, device=dev)
        rc = _fa.FA_OK
        if 0 not in shape:
            n = _workspace_bytes(dev.index, B, S, total, max_pages, P, H_kv, D, H, dtype)
            # not kept: two captured graphs never share one
            ws = _torch.empty(n, dtype=_torch.uint8, device=dev) if n else None
            rc = lib.fa_kv4_attention(c, q.data_ptr(), qs, out.data_ptr(), lse.data_ptr() if lse is not None else None,
                                      H, window, D ** -0.5 if scale is None else float(scale), dtype,
                                      ws.data_ptr() if n else None, n, handle)
    finally:
        if on is not None:
            on.done(q, codes, scales, page_table, seq_lens, cu_seqlens, out, lse)
    _check(rc, "fa_kv4_attention")
    return out, lse


def rotary_frequencies(rotary_dim: int, sections, base: float = 10000.0, interleave_axes: bool = False,
                       per_axis: bool = False, device="cuda"):
    """(inv_freq float64, axes int32) for ``rotary``: rotary_dim / 2 frequencies
    base^(-2 f / rotary_dim), shared out to the axes.

    ``sections``: frequencies of each axis, in order (they sum to
    rotary_dim / 2).  ``interleave_axes`` deals them out in turn (axis 0, 1, 2,
    0, 1, 2, ... as long as an axis has some left) instead of section by
    section.  ``per_axis`` gives each axis a sequence of its own, base^(-i / n)
    for its n frequencies.
    """
    import torch
    sections = [int(s) for s in sections]
    half = rotary_dim // 2
    _need(rotary_dim > 0 and rotary_dim % 2 == 0 and sections and min(sections) >= 0 and sum(sections) == half,
          "sections must be non-negative and sum to rotary_dim / 2")
    _need(base > 0, "base must be positive")
    axes = []
    if interleave_axes:
        left = list(sections)
        while len(axes) < half:
            for a, n in enumerate(left):
                if n > 0:
                    axes.append(a)
                    left[a] -= 1
    else:
        axes = [a for a, n in enumerate(sections) for _ in range(n)]
    seen = [0] * len(sections)
    freq = []
    for f, a in enumerate(axes):
        freq.append(float(base) ** (-seen[a] / sections[a] if per_axis else -2.0 * f / rotary_dim))
        seen[a] += 1
    return (torch.tensor(freq, dtype=torch.float64, device=device),
            torch.tensor(axes, dtype=torch.int32, device=device))


def _tokens(name, t):
    """(stride between tokens, stride between heads) of t [..., heads, D], as bytes."""
    sh, st = t.shape, t.stride()
    if len(sh) == 3 and st[2] == 1:
        return _pack2(st[0], st[1])
    _need(st[-1] == 1 or sh[-1] == 1, f"the last axis of {name} must be contiguous")
    step, n = None, 1   # every token axis in one stride
    for size, s in zip(reversed(sh[:-2]), reversed(st[:-2])):
        if size == 1:
            continue
        if step is None:
            step = s
        _need(s == step * n, f"the token axes of {name} must be evenly spaced")
        n *= size
    return _pack2(step or 0, st[-2])


_NO_TENSOR = (None, None, None, None, 0)


def rotary(q, positions, inv_freq, axes, k=None, interleaved: bool = False, inverse: bool = False, q_out=None,
           k_out=None, stream=None):
    """q (and k) with rotary positions: returns q_out, or (q_out, k_out) with k.

    q [..., H, D], k [..., H_k, D]: fp16 / bf16 of the same tokens (only the
    last axis has to be contiguous); positions int32 [..., A], one for each
    axis; inv_freq float64 [F] and axes int32 [F] as ``rotary_frequencies``
    makes them (2 F <= D; elements from 2 F on are copied).  Pairs are
    (f, f + F), or (2 f, 2 f + 1) with ``interleaved``.  ``inverse`` turns back;
    it is also the gradient.  The outputs are new contiguous tensors unless
    given (``q_out=q``: in place).
    """
    lib = _lib()
    if stream is None and _native is not None:
        r = _native.rotary(q, positions, inv_freq, axes, k, interleaved, inverse, q_out, k_out)
        if type(r) is int:
            _check(r, "fa_rotary")
        elif r is not NotImplemented:
            return r
    torch = _torch
    dev, shape, F, psh = positions.device, q.shape, inv_freq.numel(), positions.shape
    dtype = _code(q.dtype)
    _need(len(shape) >= 2 and len(psh) >= 1, "q must be [..., H, D] and positions [..., A]")
    H, D, A, H2 = shape[-2], shape[-1], psh[-1], 0
    if not (q.is_cuda and q.device == dev and positions.dtype is torch.int32 and positions.is_contiguous()
            and psh[:-1] == shape[:-2] and A >= 1 and inv_freq.dtype is torch.float64 and inv_freq.shape == (F,)
            and inv_freq.is_contiguous() and axes.dtype is torch.int32 and axes.shape == (F,)
            and axes.is_contiguous() and inv_freq.device == dev and axes.device == dev and 0 < 2 * F <= D):
        _need(q.is_cuda and q.device == dev, "q and positions must be CUDA tensors of one device")
        _need(positions.dtype is torch.int32 and positions.is_contiguous() and psh[:-1] == shape[:-2] and A >= 1,
              "positions must be a contiguous int32 tensor [..., A] of q's tokens")
        _need(0 < 2 * F <= D, "2 F must be at most D")
        raise ValueError("inv_freq must be a contiguous float64 tensor [F] and axes an int32 one, on the "
                         "positions' device")
    if k is not None:
        ksh = k.shape
        _need(k.dtype is q.dtype and ksh[:-2] == shape[:-2] and ksh[-1] == D and k.device == dev,
              "k must have q's dtype, device, tokens and D")
        H2 = ksh[-2]
    for t, o in ((q, q_out), (k, k_out)):
        _need(o is None or (t is not None and o.shape == t.shape and o.dtype is t.dtype and o.device == dev),
              "an output must be like its input")
    handle, on = _enter(dev, stream)
    try:
        if q_out is None:
            q_out = torch.empty(shape, dtype=q.dtype, device=dev)
        first, second = _NO_TENSOR, _NO_TENSOR
        if H:
            first = (q.data_ptr(), _tokens("q", q), q_out.data_ptr(), _tokens("q_out", q_out), H)
        if k is not None:
            if k_out is None:
                k_out = torch.empty(ksh, dtype=q.dtype, device=dev)
            if H2:
                second = (k.data_ptr(), _tokens("k", k), k_out.data_ptr(), _tokens("k_out", k_out), H2)
        if not H:
            first, second = second, _NO_TENSOR
        rc, T = _fa.FA_OK, positions.numel() // A
        _need(max(T, A, H, H2) <= 0x7fffffff, "sizes must fit 32 bits")
        if T and H + H2:
            rc = lib.fa_rotary(*first, *second, positions.data_ptr(), inv_freq.data_ptr(), axes.data_ptr(), T, A, F,
                               D, 1 if interleaved else 0, 1 if inverse else 0, dtype, handle)
    finally:
        if on is not None:
            on.done(q, k, positions, inv_freq, axes, q_out, k_out)
    _check(rc, "fa_rotary")
    return q_out if k is None else (q_out, k_out)
