"""The quantised cache and the rotary positions, on the host: the oracle
against the format's properties, and the refusals of the C-ABI and of the
Python calls (all before any launch)."""
import ctypes

import numpy as np
import pytest

import attention_forward_fwd_gb300 as fa
from oracle import kv4
from oracle.attention import decode

from kv4_common import to16


def test_bf16_rounding_matches_torch():
    import torch
    r = np.random.default_rng(0)
    x = np.concatenate([r.standard_normal(4000) * 10.0 ** r.integers(-38, 38, 4000), [0.0, 1.0, -1e-41, 2.0 ** -134,
                        1.5 * 2.0 ** -133, 1.00390625, 1.01171875]]).astype(np.float32)
    want = torch.from_numpy(x).bfloat16().view(torch.int16).numpy().view(np.uint16)
    got = kv4.bf16_round(x.astype(np.float64))
    zero = (got & 0x7FFF) == 0   # the sign of zero is not kept
    np.testing.assert_array_equal(np.where(zero, 0, got), np.where(zero, want & 0x7FFF, want))


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 256])
def test_packing_is_a_bijection(D):
    r = np.random.default_rng(D)
    n = r.integers(0, 16, (5, D)).astype(np.uint8)
    np.testing.assert_array_equal(kv4.unpack(kv4.pack(n)), n)
    one = np.zeros((D, D), np.uint8)
    np.fill_diagonal(one, 15)
    assert sorted(map(bytes, kv4.pack(one))) == sorted({bytes(x) for x in kv4.pack(one)})
    assert (kv4.pack(one) != 0).sum() == D


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_quantisation_error_and_exactness(dtype):
    r = np.random.default_rng(1)
    x = decode(to16(r.standard_normal((200, 64)) * 3, dtype), dtype)
    n, s = kv4.quantise(x)
    sv = np.repeat(decode(s, "bf16"), 32, -1)
    y = (n.astype(np.float64) - 8) * sv
    # half a step, or up to one (and the scale's rounding) where 8 s is cut to 7 s
    err = np.abs(y - x)
    cut = (n == 15) & (x / sv > 7.5)
    assert (err <= np.abs(sv) * 0.5 * (1 + 1e-12))[~cut].all()
    assert (err <= np.abs(sv) * (1 + 2.0 ** -5))[cut].all()
    # what the cache stands for is exact in fp16
    np.testing.assert_array_equal(y.astype(np.float16).astype(np.float64), y)
    # the extreme element of each group has the code 0
    g = x.reshape(200, 2, 32)
    first = np.abs(g).argmax(-1)
    assert (np.take_along_axis(n.reshape(200, 2, 32), first[..., None], -1) == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_ties_are_at_least_2_to_minus_13_apart(dtype):
    """The write kernel rounds x / s to multiples of 2^-14 before it rounds to
    integers: every quotient is a tie or at least 2^-13 away from one."""
    bits = {"f16": 11, "bf16": 8}[dtype]
    x = np.arange(2 ** (bits - 1), 2 ** bits, dtype=np.int64)
    s = np.arange(128, 256, dtype=np.int64)
    worst = 1.0
    for up in range(-8, 5):          # x / s 2^up for every pair of significands
        q = x[:, None] / s[None, :] * 2.0 ** (up - (bits - 8))
        q = q[(q > 0.4) & (q < 8.6)]
        d = np.abs(q - np.floor(q) - 0.5)
        d = d[d > 0]
        worst = min(worst, d.min(initial=1.0))
    assert worst >= 2.0 ** -13


def test_scale_of_special_groups():
    x = np.zeros((4, 32))
    x[1, 3] = np.inf
    x[2, 5] = np.nan
    x[3] = 2.0 ** -149
    n, s = kv4.quantise(x)
    assert (n == 8).all() and list(s[:, 0]) == [0, 0x7FC0, 0x7FC0, 0]
    x = np.zeros((1, 32))
    x[0, 4], x[0, 9] = 2.0, -2.0      # the first of equals gives the sign
    n, s = kv4.quantise(x)
    assert decode(s, "bf16")[0, 0] == -0.25 and n[0, 4] == 0 and n[0, 9] == 15


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.library()


def _cache(**change):
    d = dict(codes=4096, scales=8192, page_table=4096, seq_lens=4096, cu_seqlens=None, B=2, max_seqlen=3, total=0,
             pages=8, max_pages=4, page_size=32, H_kv=2, D=64)
    d.update(change)
    return ctypes.byref(fa.Kv4Cache(**d))


INV, UNS = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
BAD_CACHE = [
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(page_table=None), INV), (dict(seq_lens=None), INV),
    (dict(B=0), INV), (dict(max_seqlen=0), INV), (dict(H_kv=0), INV), (dict(pages=0), INV), (dict(max_pages=0), INV),
    (dict(page_size=0), INV), (dict(total=7), INV), (dict(cu_seqlens=4096, total=0), INV),
    (dict(D=16), UNS), (dict(D=80), UNS), (dict(D=288), UNS), (dict(D=0), UNS), (dict(page_size=24), UNS),
    (dict(page_size=8), UNS), (dict(codes=4096 + 8), UNS), (dict(scales=8192 + 2), UNS), (dict(page_table=4098), UNS),
    (dict(seq_lens=4097), UNS), (dict(cu_seqlens=4098, total=6), UNS), (dict(pages=1 << 26, page_size=32), UNS),
    (dict(max_pages=1 << 26, page_size=32), UNS), (dict(B=1 << 16, max_seqlen=1 << 16), UNS),
]
S3 = (ctypes.c_longlong * 3)(1024, 256, 64)
ODD3 = (ctypes.c_longlong * 3)(1024, 256, 62)


@pytest.mark.parametrize("change,status", BAD_CACHE)
def test_a_bad_cache_is_refused_by_every_call(lib, change, status):
    c = _cache(**change)
    n = ctypes.c_size_t(0)
    assert lib.fa_kv4_write(c, 4096, 4096, S3, S3, None, None, fa.FA_BF16, None) == status
    assert lib.fa_kv4_read(c, 4096, 4096, fa.FA_BF16, None) == status
    assert lib.fa_kv4_attention_workspace_size(c, 4, fa.FA_BF16, ctypes.byref(n)) == status
    assert lib.fa_kv4_attention(c, 4096, S3, 4096, None, 4, -1, 0.125, fa.FA_BF16, 4096, 1 << 30, None) == status
    assert lib.fa_kv4_write(None, 4096, 4096, S3, S3, None, None, fa.FA_BF16, None) == INV


def test_bad_arguments_are_refused(lib):
    c = _cache()
    w = lambda **k: lib.fa_kv4_write(c, *{**dict(K=4096, V=4096, ks=S3, vs=S3, ko=None, vo=None, dt=1), **k}.values(), None)
    for change, status in ((dict(K=None), INV), (dict(V=None), INV), (dict(ks=None), INV), (dict(vs=None), INV),
                           (dict(ko=4096), INV), (dict(vo=4096), INV), (dict(dt=2), INV), (dict(K=4100), UNS),
                           (dict(V=4098), UNS), (dict(ks=ODD3), UNS), (dict(vs=ODD3), UNS),
                           (dict(ko=4100, vo=4096), UNS)):
        assert w(**change) == status, change
    assert lib.fa_kv4_read(c, None, 4096, 1, None) == INV
    assert lib.fa_kv4_read(c, 4096, None, 1, None) == INV
    assert lib.fa_kv4_read(c, 4096, 4104, 1, None) == UNS
    assert lib.fa_kv4_read(c, 4096, 4096, -1, None) == INV
    base = dict(Q=4096, qs=S3, O=4096, L=None, H=4, w=-1, scale=0.125, dt=1, ws=4096, n=1 << 30)
    a = lambda **k: lib.fa_kv4_attention(c, *{**base, **k}.values(), None)
    odd = (ctypes.c_longlong * 3)(1024, 256, 68)
    for change, status in ((dict(Q=None), INV), (dict(O=None), INV), (dict(qs=None), INV), (dict(H=0), INV),
                           (dict(H=3), INV), (dict(w=-2), INV), (dict(scale=0.0), INV), (dict(scale=float("nan")), INV),
                           (dict(scale=float("inf")), INV), (dict(dt=5), INV), (dict(Q=4104), UNS), (dict(O=4104), UNS),
                           (dict(L=4098), UNS), (dict(qs=odd), UNS)):
        assert a(**change) == status, change


def test_rotary_refusals(lib):
    two = (ctypes.c_longlong * 2)(128, 64)
    base = dict(X=4096, xs=two, Y=4096, ys=two, H=2, X2=None, x2s=None, Y2=None, y2s=None, H2=0, pos=4096, f=4096,
                ax=4096, T=3, A=3, F=32, D=64, il=0, inv=0, dt=1)
    r = lambda **k: lib.fa_rotary(*{**base, **k}.values(), None)
    for change, status in ((dict(X=None), INV), (dict(Y=None), INV), (dict(xs=None), INV), (dict(ys=None), INV),
                           (dict(pos=None), INV), (dict(f=None), INV), (dict(ax=None), INV), (dict(T=0), INV),
                           (dict(H=0), INV), (dict(A=0), INV), (dict(F=0), INV), (dict(F=33), INV), (dict(H2=-1), INV),
                           (dict(H2=1), INV), (dict(dt=9), INV), (dict(D=512, F=200), UNS), (dict(X=4097), UNS),
                           (dict(pos=4098), UNS), (dict(f=4100), UNS), (dict(ax=4097), UNS), (dict(H=70000), UNS)):
        assert r(**change) == status, change


def test_python_calls_refuse_what_does_not_fit():
    import torch
    with pytest.raises(ValueError):
        fa.kv4_empty_cache(4, 2, 80, device="cpu")
    with pytest.raises(ValueError):
        fa.kv4_empty_cache(4, 2, 64, page_size=20, device="cpu")
    codes, scales = fa.kv4_empty_cache(4, 2, 64, page_size=16, device="cpu")
    assert codes.shape == (4, 2, 2, 16, 32) and scales.shape == (4, 2, 2, 16, 2)
    assert (codes == 0x88).all() and (scales == 0).all()
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: fa.kv4_write(q, q, codes, scales, table, lens),
                 lambda: fa.kv4_attention(q, codes, scales, table, lens),
                 lambda: fa.kv4_read(codes, scales, table, lens, max_seqlen=1)):
        with pytest.raises(ValueError):      # not on a GPU
            call()
    with pytest.raises(ValueError):
        fa.rotary(q, torch.zeros(1, 1, 3, dtype=torch.int32), *fa.rotary_frequencies(64, (32,), device="cpu"))
    with pytest.raises(ValueError):
        fa.rotary_frequencies(64, (16, 8), device="cpu")


def test_rotary_frequencies():
    f, a = fa.rotary_frequencies(16, (2, 3, 3), base=100.0, device="cpu")
    assert a.tolist() == [0, 0, 1, 1, 1, 2, 2, 2]
    np.testing.assert_allclose(f.numpy(), 100.0 ** (-np.arange(8) / 8), rtol=1e-15)
    f, a = fa.rotary_frequencies(16, (4, 2, 2), interleave_axes=True, per_axis=True, base=100.0, device="cpu")
    assert a.tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    np.testing.assert_allclose(f.numpy(), 100.0 ** -np.array([0, 0, 0, .25, .5, .5, .5, .75]), rtol=1e-15)


def test_status_codes_have_texts(lib):
    texts = {fa.fa_status_string(c) for c in (fa.FA_ERR_BAD_PAGES, fa.FA_ERR_BAD_AXIS, fa.FA_ERR_BAD_SEQLENS)}
    assert len(texts) == 3 and "unknown status" not in texts
