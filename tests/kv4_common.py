"""Helpers of the tests of the quantised cache (not collected by pytest)."""
import numpy as np

import fa_inputs
from oracle import kv4
from oracle.attention import decode

BITS = {"f16": 11, "bf16": 8}          # significant bits
EMIN = {"f16": -14, "bf16": -126}


def to16(x, dtype):
    """float64 -> 16-bit patterns."""
    if dtype == "bf16":
        return kv4.bf16_round(x)
    return np.asarray(x, np.float64).astype(np.float16).view(np.uint16)


def half_step(x, dtype):
    """Half the spacing of the type at |x|: its rounding's error."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** EMIN[dtype])))
    return 0.5 * np.exp2(e - (BITS[dtype] - 1))


class Setup:
    """A paged cache with sequences of the given lengths, on the host and (by
    ``cuda()``) on the GPU.  The pages are in random order, every byte that
    no token owns is set so that a read of it shows: codes at random, scales
    NaN."""

    def __init__(self, lens, H_kv, D, P, seed, spare=2, filled=True, loud=0.4):
        r = np.random.default_rng(seed)
        self.r, self.lens, self.H_kv, self.D, self.P = r, np.asarray(lens, np.int32), H_kv, D, P
        B = len(lens)
        self.B = B
        self.max_pages = max(1, -(-int(max(0, self.lens.max())) // P)) + 1
        own = [max(0, -(-int(n) // P)) for n in lens]
        self.pages = sum(own) + spare
        order = r.permutation(self.pages)
        self.table = np.full((B, self.max_pages), -7, np.int32)   # past the end: no page
        at = 0
        for b in range(B):
            self.table[b, :own[b]] = order[at:at + own[b]]
            at += own[b]
        self.codes = r.integers(0, 256, (self.pages, 2, H_kv, P, D // 2), dtype=np.uint8)
        self.scales = np.full((self.pages, 2, H_kv, P, D // 32), 0x7FC0, np.uint16)
        if filled:
            chan = np.exp(loud * r.standard_normal((2, H_kv, D)))
            for b in range(B):
                for which in (0, 1):
                    n = int(max(0, self.lens[b]))
                    x = r.standard_normal((n, H_kv, D)) * chan[which]
                    self.put(b, which, np.arange(n), x)

    def put(self, b, which, pos, x):
        n, s = kv4.quantise(x)
        pg, at = self.table[b, pos // self.P], pos % self.P
        self.codes[pg, which, :, at] = kv4.pack(n)
        self.scales[pg, which, :, at] = s

    def cuda(self):
        import torch
        return dict(codes=torch.from_numpy(self.codes.copy()).cuda(),
                    scales=torch.from_numpy(self.scales.copy()).view(torch.bfloat16).cuda(),
                    page_table=torch.from_numpy(self.table.copy()).cuda(),
                    seq_lens=torch.from_numpy(self.lens.copy()).cuda())

    def rows(self, b, which):
        return kv4.sequence_rows(self.codes, self.scales, self.table[b], int(max(0, self.lens[b])), which)


def attention_tolerance(q, k, o, a, lse, scale, dtype):
    """Bounds on |dO| and |dLSE| of one sequence, from the kernel's roundings.

    z: products of Q and the codes are exact; they are summed in fp32 by the
    tensor cores, 32 elements at a time from -8 sum q on, so that the terms
    are up to 16 scales where the values are up to 8: at most 2 (D / 16 + D / 32)
    roundings of 2^-23 (the tensor cores may truncate) of sum |q| 16 s <= 16 max|k| / 7 sum |q|
    (a group's scale is at least its largest value / 8, and its largest value at least 7 s),
    then the multiplication by scale log2 e and the exponential, 2^-22 of |z| + 2^-22.
    P s is rounded to fp16: 2^-11, and below 2^-21 of the largest by at most 2^-32 of it.
    O sums fp32; the result is rounded to its type.
    """
    D = q.shape[-1]
    H, Hkv = q.shape[1], k.shape[1]
    L = max(1, k.shape[0])
    kmax = np.abs(np.repeat(k, H // Hkv, 1)).max(axis=(0, 2)) if k.size else np.zeros(H)   # [H]
    qsum = np.abs(q).sum(-1)                                                               # [n, H]
    zabs = scale * qsum * kmax * 16 / 7
    dz = zabs * (3 * D / 16) * 2.0 ** -23 + zabs * 2.0 ** -22 + 2.0 ** -21                 # [n, H]
    steps = L / 16 * 2.0 ** -23   # the accumulator's own roundings, of sum p |v|
    tol_o = a * (2.0 ** -11 + 2 * dz[..., None] + steps + 2.0 ** -20) + a.max(initial=0) * L * 2.0 ** -31 \
        + half_step(np.abs(o) + a * 2.0 ** -10, dtype)
    tol_l = dz.T + np.where(np.isfinite(lse), np.abs(lse), 0) * 2.0 ** -22 + L * 2.0 ** -24
    return tol_o, tol_l
