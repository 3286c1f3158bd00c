"""The quantised K/V cache and the rotary positions, for torch CUDA tensors.

A decoding step turns its q and k (``rotary``), writes k and v into the cache
(``kv4_write``) and attends over it (``kv4_attention``); ``kv4_read`` gives
plain K and V back, for the other attention calls.  As in the rest of the
package this module only marshals arguments; the work runs in the library's
kernels (``fa_kv4_*`` and ``fa_rotary`` in ``include/fa_gb300.h``, where the
cache's format and the checks on the device are described).

Every call takes ``page_table`` (int32 [B, max_pages]) and ``seq_lens`` (int32
[B], the tokens in the cache with the call's own), and concerns the LAST rows of
each sequence: S of them in batched tensors [B, S, heads, D], or
``cu_seqlens[b + 1] - cu_seqlens[b]`` in packed ones [total, heads, D].
"""
from __future__ import annotations

import ctypes
import functools

import attention_forward_fwd_gb300 as _fa

KV4_GROUP = 32   # values that share a scale

_Strides = ctypes.c_longlong * 3
_Pair = ctypes.c_longlong * 2


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _code(dtype):
    import torch
    if dtype is torch.bfloat16:
        return _fa.FA_BF16
    _need(dtype is torch.float16, f"unsupported dtype {dtype}")
    return _fa.FA_F16


class _On:
    """The device and stream of a call.  Tensors that the call makes are made
    with that stream current, so that the allocator hands their memory out
    again in that stream's order; tensors that it is given are recorded on a
    stream that is not their own."""

    def __init__(self, device, stream):
        import torch
        self.device = device
        self.guard = None if torch.cuda.current_device() == device.index else torch.cuda.device(device)
        self.given = stream is not None
        self.stream = stream

    def __enter__(self):
        import torch
        if self.guard is not None:
            self.guard.__enter__()
        self.inner = None
        if self.given:
            try:
                handle = _fa._stream_handle(self.stream)
                if handle != torch.cuda.current_stream(self.device).cuda_stream:
                    target = (self.stream if isinstance(self.stream, torch.cuda.Stream)
                              else torch.cuda.default_stream(self.device) if handle == 0
                              else torch.cuda.ExternalStream(handle, device=self.device))
                    self.inner = torch.cuda.stream(target)
                    self.inner.__enter__()
                    self.target = target
            except BaseException:
                if self.guard is not None:
                    self.guard.__exit__(None, None, None)
                raise
            self.handle = handle
        else:
            self.handle = torch.cuda.current_stream(self.device).cuda_stream
        return self

    def keep(self, *tensors):
        if self.inner is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.target)

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


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
    """The call's fa_kv4_cache_t; ``rows``: total of packed tensors, S of batched ones."""
    import torch
    _need(codes.is_cuda and codes.dtype is torch.uint8 and codes.dim() == 5 and codes.is_contiguous(),
          "codes must be a contiguous uint8 CUDA tensor [pages, 2, H_kv, page_size, D / 2]")
    pages, two, H_kv, P, half = codes.shape
    _need(two == 2, "codes must be [pages, 2, H_kv, page_size, D / 2]")
    _need(scales.dtype is torch.bfloat16 and scales.is_contiguous()
          and scales.shape == (pages, 2, H_kv, P, half // 16),
          "scales must be a contiguous bfloat16 tensor [pages, 2, H_kv, page_size, D / 32]")
    _need(page_table.dtype is torch.int32 and page_table.dim() == 2 and page_table.is_contiguous(),
          "page_table must be a contiguous int32 tensor [B, max_pages]")
    B = page_table.shape[0]
    _need(seq_lens.dtype is torch.int32 and seq_lens.shape == (B,) and seq_lens.is_contiguous(),
          "seq_lens must be a contiguous int32 tensor [B]")
    dev = codes.device
    _need(scales.device == dev and page_table.device == dev and seq_lens.device == dev,
          "codes, scales, page_table and seq_lens must be on one device")
    if cu_seqlens is None:
        cu, S, total = None, rows, 0
    else:
        _need(cu_seqlens.dtype is torch.int32 and cu_seqlens.shape == (B + 1,)
              and cu_seqlens.is_contiguous() and cu_seqlens.device == dev,
              "cu_seqlens must be a contiguous int32 tensor [B + 1] on the cache's device")
        cu, total = cu_seqlens.data_ptr(), rows
        S = total if max_seqlen is None else int(max_seqlen)
    return _fa.Kv4Cache(codes.data_ptr(), scales.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), cu,
                        B, S, total, pages, page_table.shape[1], P, H_kv, half * 2)


def _rows(name, t, cu_seqlens, B, heads, D, device):
    """Checks a tensor of the call's rows; its row count and element strides."""
    _need(t.device == device, f"{name} is on {t.device}, the cache on {device}")
    _need(t.dim() == (4 if cu_seqlens is None else 3),
          f"{name} must be [B, S, heads, D], or [total, heads, D] with cu_seqlens")
    _need(t.shape[-1] == D and (heads is None or t.shape[-2] == heads) and (cu_seqlens is not None or t.shape[0] == B),
          f"{name} has shape {tuple(t.shape)}: its batch, heads and D must match the cache")
    st = t.stride()
    _need(st[-1] == 1 or D == 1, f"the last axis of {name} must be contiguous")
    return t.shape[-3], _Strides(0 if cu_seqlens is not None else st[0], st[-3], st[-2])


def kv4_write(k, v, codes, scales, page_table, seq_lens, cu_seqlens=None, max_seqlen=None, k_out=None,
              v_out=None, stream=None):
    """Quantises k and v into the cache at their sequences' last tokens.

    k, v: fp16 / bf16 [B, S, H_kv, D] or packed [total, H_kv, D] with
    ``cu_seqlens`` (int32 [B + 1]; ``max_seqlen``: the most rows of a sequence, checked on the
    device); only the last axis has to be contiguous (strides in multiples of
    4 elements), so slices of a fused projection can be passed.  ``k_out``,
    ``v_out`` (contiguous, like k and v; both or neither) receive what the
    cache now stands for.  Work is enqueued on ``stream`` (default: the
    current one) and not waited for.
    """
    dev = codes.device
    dtype = _code(k.dtype)
    _need(v.dtype is k.dtype and v.shape == k.shape, "k and v must be alike")
    rows = k.shape[-3] if k.dim() >= 3 else 0
    c = _cache(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, rows)
    _, ks = _rows("k", k, cu_seqlens, c.B, c.H_kv, c.D, dev)
    _, vs = _rows("v", v, cu_seqlens, c.B, c.H_kv, c.D, dev)
    _need((k_out is None) == (v_out is None), "k_out and v_out come together")
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        _need(t is None or (t.shape == k.shape and t.dtype is k.dtype and t.is_contiguous() and t.device == dev),
              f"{name} must be a contiguous tensor like k")
    if k.numel() == 0:
        return
    with _On(dev, stream) as on:
        rc = _fa.library().fa_kv4_write(c, k.data_ptr(), v.data_ptr(), ks, vs,
                                        k_out.data_ptr() if k_out is not None else None,
                                        v_out.data_ptr() if v_out is not None else None, dtype, on.handle)
        on.keep(k, v, codes, scales, page_table, seq_lens, cu_seqlens, k_out, v_out)
    if rc != _fa.FA_OK:
        raise _fa.FaError(rc, "fa_kv4_write")


def kv4_read(codes, scales, page_table, seq_lens, cu_seqlens=None, max_seqlen=None, total=None, dtype=None,
             k_out=None, v_out=None, stream=None):
    """k, v of the sequences' last tokens, as plain tensors.

    Packed [total, H_kv, D] with ``cu_seqlens`` and ``total`` (its last offset, which the host has to know),
    or batched [B, max_seqlen, H_kv, D].  ``dtype``: torch.float16 (exact within its range) or torch.bfloat16
    (default).  Rows before a sequence's first token are zeros; packed rows
    outside every sequence are left as they were (of ``k_out``, ``v_out``, when given; else not defined).
    """
    import torch
    dev = codes.device
    _need((k_out is None) == (v_out is None), "k_out and v_out come together")
    if cu_seqlens is None:
        _need(max_seqlen is not None, "max_seqlen (the rows of a sequence) is needed without cu_seqlens")
        rows = int(max_seqlen)
    else:
        _need(total is not None, "total is needed with cu_seqlens")
        rows = int(total)
    c = _cache(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, rows)
    shape = (c.B, rows, c.H_kv, c.D) if cu_seqlens is None else (rows, c.H_kv, c.D)
    if k_out is not None:
        dtype = k_out.dtype
        for name, t in (("k_out", k_out), ("v_out", v_out)):
            _need(t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.device == dev,
                  f"{name} must be a contiguous tensor {shape} on the cache's device")
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _code(dtype)
    with _On(dev, stream) as on:
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=dev)
            v_out = torch.empty(shape, dtype=dtype, device=dev)
        rc = _fa.FA_OK
        if k_out.numel():
            rc = _fa.library().fa_kv4_read(c, k_out.data_ptr(), v_out.data_ptr(), code, on.handle)
        on.keep(codes, scales, page_table, seq_lens, cu_seqlens, k_out, v_out)
    if rc != _fa.FA_OK:
        raise _fa.FaError(rc, "fa_kv4_read")
    return k_out, v_out


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(device_index, B, S, total, max_pages, P, H_kv, D, H, dtype):
    """Workspace of a call's sizes on the current device (which device_index names)."""
    n = ctypes.c_size_t(0)
    one = ctypes.c_void_p(16)   # the sizes alone matter: stand-ins for the pointers
    c = _fa.Kv4Cache(one, one, one, one, one if total else None, B, S, total, 1, max_pages, P, H_kv, D)
    rc = int(_fa.library().fa_kv4_attention_workspace_size(c, H, dtype, ctypes.byref(n)))
    if rc != _fa.FA_OK:
        raise _fa.FaError(rc, "fa_kv4_attention_workspace_size")
    return n.value


def kv4_attention(q, codes, scales, page_table, seq_lens, cu_seqlens=None, max_seqlen=None,
                  window_left: int = -1, scale: float | None = None, out=None, lse=None, with_lse: bool = True,
                  stream=None):
    """O, LSE of the queries q over the cache.

    q: fp16 / bf16 [B, S, H, D] or packed [total, H, D] with ``cu_seqlens``
    (and ``max_seqlen``, the most rows of a sequence); H a multiple of H_kv
    (query head h uses K/V head h // (H / H_kv)); only the last axis has to be
    contiguous (strides in multiples of 8 elements).  Row i of the n rows of
    sequence b is its token seq_lens[b] - n + i and sees the tokens up to
    itself, from ``window_left`` before itself on (-1: from the first).  The
    call's own k and v are written first (``kv4_write``).  Rows without a
    token are O = 0, LSE = -inf.  O is contiguous like q, LSE fp32 [B, H, S] or [H, total].
    """
    import torch
    dev = codes.device
    dtype = _code(q.dtype)
    rows = q.shape[-3] if q.dim() >= 3 else 0
    c = _cache(codes, scales, page_table, seq_lens, cu_seqlens, max_seqlen, rows)
    _, qs = _rows("q", q, cu_seqlens, c.B, None, c.D, dev)
    H = q.shape[-2]
    _need(H > 0 and H % c.H_kv == 0, "the heads of q must be a multiple of the cache's H_kv")
    lse_shape = (c.B, H, rows) if cu_seqlens is None else (H, rows)
    _need(out is None or (out.shape == q.shape and out.dtype is q.dtype and out.is_contiguous() and out.device == dev),
          "out must be a contiguous tensor like q")
    _need(lse is None or (lse.shape == lse_shape and lse.dtype is torch.float32 and lse.is_contiguous()
                          and lse.device == dev), f"lse must be a contiguous fp32 tensor {lse_shape}")
    with _On(dev, stream) as on:
        made = out is None
        if made:
            out = torch.empty(q.shape, dtype=q.dtype, device=dev)
        if lse is None and with_lse:
            lse = torch.empty(lse_shape, dtype=torch.float32, device=dev)
        rc = _fa.FA_OK
        if q.numel():
            n = _workspace_bytes(dev.index, c.B, c.max_seqlen, c.total, c.max_pages, c.page_size, c.H_kv, c.D, H,
                                 dtype)
            # made anew for each call: two captured graphs never share one
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
            rc = _fa.library().fa_kv4_attention(
                c, q.data_ptr(), qs, out.data_ptr(), lse.data_ptr() if lse is not None else None, H,
                int(window_left), c.D ** -0.5 if scale is None else float(scale), dtype, ws.data_ptr(), n, on.handle)
        on.keep(q, codes, scales, page_table, seq_lens, cu_seqlens, out, lse)
    if rc != _fa.FA_OK:
        raise _fa.FaError(rc, "fa_kv4_attention")
    return out, lse


def rotary_frequencies(rotary_dim: int, sections, base: float = 10000.0, interleave_axes: bool = False,
                       per_axis: bool = False, device="cuda"):
    """(inv_freq float64, axes int32) for ``rotary``: rotary_dim / 2 frequencies
    base^(-2 f / rotary_dim) shared out to the axes.

    ``sections``: frequencies of each axis, in order (they sum to rotary_dim / 2).
    ``interleave_axes`` deals them out in turn (axis 0, 1, 2, 0, 1, 2, ... as
    long as an axis has some left) instead of section by section.
    ``per_axis`` gives each axis a sequence of its own, base^(-i / n) for its n frequencies.
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


def _turned(name, x, out, device):
    """Checks a tensor to be turned: (input strides, output strides)."""
    def strides(t, what):
        st, sh = t.stride(), t.shape
        _need(st[-1] == 1 or sh[-1] == 1, f"the last axis of {what} must be contiguous")
        # every token axis in one stride
        step, n = None, 1
        for size, s in zip(reversed(sh[:-2]), reversed(st[:-2])):
            if size == 1:
                continue
            if step is None:
                step = s
            _need(s == step * n, f"the token axes of {what} must be evenly spaced")
            n *= size
        return _Pair(step or 0, st[-2])
    _need(x.device == device, f"{name} is on {x.device}, the positions on {device}")
    _need(out.shape == x.shape and out.dtype is x.dtype and out.device == device, f"the output for {name} must be like it")
    return strides(x, name), strides(out, f"the output for {name}")


def rotary(q, positions, inv_freq, axes, k=None, interleaved: bool = False, inverse: bool = False, q_out=None,
           k_out=None, stream=None):
    """q (and k) with rotary positions: returns q_out, or (q_out, k_out) with k.

    q [..., H, D], k [..., H_k, D]: fp16 / bf16 of the same tokens (only the last axis has to be
    contiguous); positions int32 [..., A], one for each axis; inv_freq float64
    [F] and axes int32 [F] as ``rotary_frequencies`` makes them (2 F <= D; elements
    from 2 F on are copied).  Pairs are (f, f + F), or (2 f, 2 f + 1) with
    ``interleaved``.  ``inverse`` turns back; it is also the gradient.  The
    outputs are new contiguous tensors unless given (``q_out=q``: in place).
    """
    import torch
    dev = positions.device
    _need(q.is_cuda and dev.type == "cuda", "q and positions must be CUDA tensors")
    dtype = _code(q.dtype)
    _need(q.dim() >= 2 and positions.dtype is torch.int32 and positions.is_contiguous()
          and positions.dim() == q.dim() - 1 and positions.shape[:-1] == q.shape[:-2] and positions.shape[-1] >= 1,
          "positions must be a contiguous int32 tensor [..., A] of q's tokens")
    _need(inv_freq.dtype is torch.float64 and inv_freq.dim() == 1 and inv_freq.is_contiguous()
          and inv_freq.device == dev, "inv_freq must be a contiguous float64 tensor [F] on the positions' device")
    F, D, A = inv_freq.numel(), q.shape[-1], positions.shape[-1]
    _need(axes.dtype is torch.int32 and axes.shape == (F,) and axes.is_contiguous() and axes.device == dev,
          "axes must be a contiguous int32 tensor like inv_freq")
    _need(0 < 2 * F <= D, "2 F must be at most D")
    if k is not None:
        _need(k.dtype is q.dtype and k.shape[:-2] == q.shape[:-2] and k.shape[-1] == D,
              "k must have q's dtype, tokens and D")
    T = positions.numel() // A
    with _On(dev, stream) as on:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev) if q_out is None else q_out
        qx, qy = _turned("q", q, q_out, dev)
        kx = ky = None
        if k is not None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=dev) if k_out is None else k_out
            kx, ky = _turned("k", k, k_out, dev)
        rc = _fa.FA_OK
        H, H2 = q.shape[-2], (k.shape[-2] if k is not None else 0)
        if T and H + H2:
            if H == 0:   # only k has heads
                args = (k.data_ptr(), kx, k_out.data_ptr(), ky, H2, None, None, None, None, 0)
            else:
                args = (q.data_ptr(), qx, q_out.data_ptr(), qy, H,
                        k.data_ptr() if H2 else None, kx, k_out.data_ptr() if H2 else None, ky, H2)
            rc = _fa.library().fa_rotary(*args, positions.data_ptr(), inv_freq.data_ptr(), axes.data_ptr(), T, A, F,
                                         D, int(interleaved), int(inverse), dtype, on.handle)
        on.keep(q, k, positions, inv_freq, axes, q_out, k_out)
    if rc != _fa.FA_OK:
        raise _fa.FaError(rc, "fa_rotary")
    return q_out if k is None else (q_out, k_out)
