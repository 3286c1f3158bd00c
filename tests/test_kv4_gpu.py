"""The quantised cache on the GPU against the fp64 oracle: what is written
(codes and scales equal), what is read back (equal), attention over it (bounds
derived in kv4_common), and what the device refuses."""
import numpy as np
import pytest

import fa_inputs
from oracle import kv4
from oracle.attention import decode

from kv4_common import Setup, attention_tolerance, half_step, to16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import torch
    import attention_forward_fwd_gb300 as fa
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    fa.build()
    fa.fa_device_status(clear=True)
    return fa


@pytest.fixture(autouse=True)
def clean_status(fa):
    yield
    assert fa.fa_device_status(clear=True) == 0


def dev(bits, dtype):
    return fa_inputs.to_torch(np.ascontiguousarray(bits), dtype).cuda()


def host(t):
    import torch
    if t.dtype in (torch.float16, torch.bfloat16):
        return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


def cu_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def expected_write(s, b, x16, which, dtype, n):
    """Writes the n last tokens of sequence b from x16 [n, H_kv, D] into the setup's arrays."""
    pos = s.lens[b] - n + np.arange(n)
    s.put(b, which, pos[pos >= 0], decode(x16, dtype)[pos >= 0])


def read_values(s, b, which, n, dtype):
    """What a read of the n last tokens gives, as bits."""
    y = np.zeros((n, s.H_kv, s.D))
    have = s.rows(b, which)[-n:] if n else y
    y[n - len(have):] = have
    return to16(y, dtype)


# ------------------------------------------------------------------- write
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,H_kv,P", [(32, 1, 16), (64, 2, 16), (96, 3, 32), (128, 2, 64), (160, 1, 48),
                                      (192, 2, 16), (224, 1, 16), (256, 2, 32)])
@pytest.mark.parametrize("packed", [False, True])
def test_write_and_read_back(fa, dtype, D, H_kv, P, packed):
    import torch
    rows = [5, 0, 1, 37, 4] if packed else [6] * 4
    lens = [5, 3, 40, 64, 9] if packed else [6, 70, 9, 6]
    s = Setup(lens, H_kv, D, P, seed=D + P)
    c = s.cuda()
    total = sum(rows)
    k16, v16 = (to16(s.r.standard_normal((total + 3, H_kv, D)) * 4, dtype) for _ in (0, 1))
    cu = cu_of(rows)
    for b, n in enumerate(rows):
        for which, x in enumerate((k16, v16)):
            expected_write(s, b, x[cu[b]:cu[b] + n], which, dtype, n)
    k, v = dev(k16, dtype), dev(v16, dtype)
    if packed:
        kw = dict(cu_seqlens=torch.from_numpy(cu).cuda(), max_seqlen=max(rows))
    else:
        k, v = (t[:total].view(4, 6, H_kv, D) for t in (k, v))
        kw = {}
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    fa.kv4_write(k, v, **c, **kw, k_out=ko, v_out=vo)
    np.testing.assert_array_equal(c["codes"].cpu().numpy(), s.codes)
    np.testing.assert_array_equal(host(c["scales"]), s.scales)
    rkw = dict(cu_seqlens=kw["cu_seqlens"], max_seqlen=max(rows), total=total + 3) if packed else dict(max_seqlen=6)
    rk, rv = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    fa.kv4_read(**c, **rkw, k_out=rk, v_out=rv)
    for which, (o, r) in enumerate(((ko, rk), (vo, rv))):
        o, r = (decode(host(t), dtype).reshape(-1, H_kv, D) for t in (o, r))
        for b, n in enumerate(rows):
            want = decode(read_values(s, b, which, n, dtype), dtype)
            np.testing.assert_array_equal(o[cu[b]:cu[b] + n], want)
            np.testing.assert_array_equal(r[cu[b]:cu[b] + n], want)
        assert (o[total:] == 7).all() and (r[total:] == 7).all()    # rows behind the last sequence


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_write_of_special_values(fa, dtype):
    """Zeros, ties, equal extremes of both signs, subnormals, the largest
    values, infinities and NaN, next to ordinary rows."""
    D, n = 64, 40
    s = Setup([n], 1, D, 16, seed=3)
    x = s.r.standard_normal((n, 1, D))
    big, tiny = (3e38, 2.0 ** -133) if dtype == "bf16" else (65504.0, 2.0 ** -24)
    x[0] = 0
    x[1, 0, :32] = -0.0
    x[2, 0, 4], x[2, 0, 9], x[2, 0, 10:32] = 8.0, -8.0, 0.5      # ties: 0.5, 1.5, ... of a scale of 1
    x[3, 0] = (np.arange(64) % 17 - 8) * 0.5 + 0.25 * 0
    x[3, 0, 0] = -8.0
    x[4, 0] = np.where(np.arange(64) % 2, 4.0, -4.0)
    x[5] = tiny * s.r.integers(-3, 4, (1, D))
    x[6] = tiny * s.r.integers(-300, 300, (1, D))
    x[7] = big * s.r.uniform(-1, 1, (1, D))
    x[8, 0, 3] = np.inf
    x[9, 0, 40] = -np.inf
    x[10, 0, 31] = np.nan
    x[11, 0, 31], x[11, 0, 0] = np.nan, np.inf
    x[12, 0] = 8 * 2.0 ** -s.r.integers(0, 20, D).astype(float)
    x16 = to16(x, dtype)
    xd = decode(x16, dtype)
    import torch
    c = s.cuda()
    expected_write(s, 0, x16, 0, dtype, n)
    expected_write(s, 0, x16, 1, dtype, n)
    k = dev(x16[None], dtype)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    fa.kv4_write(k, k.clone(), **c, k_out=ko, v_out=vo)
    assert np.isnan(xd[10]).any()
    np.testing.assert_array_equal(host(c["scales"]), s.scales)
    np.testing.assert_array_equal(c["codes"].cpu().numpy(), s.codes)
    want = decode(read_values(s, 0, 0, n, dtype), dtype)
    np.testing.assert_array_equal(decode(host(ko), dtype)[0], want)
    # in place: the outputs over the inputs
    fa.kv4_write(k, k2 := k.clone(), **c, k_out=k, v_out=k2)
    np.testing.assert_array_equal(decode(host(k), dtype)[0], want)


def test_write_of_every_quotient(fa):
    """Every pair of fp16 significands that meets as element and extreme of a
    group, at quotients from 1/2 to 8: the codes are those of the exact quotient."""
    import torch
    r = np.random.default_rng(5)
    e = np.arange(1024, 2048)
    rows, x = 4096, np.empty((4096, 1, 64))
    x[:, 0, 0::32] = (r.choice(e, (rows, 2)) / 128.0) * r.choice([-1, 1], (rows, 2))
    rest = r.choice(e, (rows, 64)) * 2.0 ** (r.integers(-5, 0, (rows, 64)) - 7.0) * r.choice([-1, 1], (rows, 64))
    x[:, 0, np.arange(64) % 32 != 0] = rest[:, np.arange(64) % 32 != 0]
    # exact ties of the group's own scale
    ext = np.abs(x[:, 0, 0])
    s_ = decode(kv4.bf16_round(ext / 8), "bf16")
    for j in range(1, 9):
        t = (j - 0.5) * s_
        x[:, 0, j] = np.where(t.astype(np.float16).astype(np.float64) == t, t, x[:, 0, j])
    x16 = to16(x, "f16")
    s = Setup([rows], 1, 64, 64, seed=1, filled=False)
    c = s.cuda()
    expected_write(s, 0, x16, 0, "f16", rows)
    expected_write(s, 0, x16, 1, "f16", rows)
    k = dev(x16[None], "f16")
    fa.kv4_write(k, k, **c)
    np.testing.assert_array_equal(host(c["scales"]), s.scales)
    np.testing.assert_array_equal(c["codes"].cpu().numpy(), s.codes)


def test_write_takes_slices_of_a_projection(fa):
    import torch
    s = Setup([7, 20], 2, 64, 16, seed=9)
    qkv16 = to16(s.r.standard_normal((2, 3, 8, 64)), "bf16")
    c = s.cuda()
    for b in range(2):
        expected_write(s, b, qkv16[b, :, 4:6], 0, "bf16", 3)
        expected_write(s, b, qkv16[b, :, 6:8], 1, "bf16", 3)
    qkv = dev(qkv16, "bf16")
    fa.kv4_write(qkv[:, :, 4:6], qkv[:, :, 6:8], **c)
    np.testing.assert_array_equal(c["codes"].cpu().numpy(), s.codes)
    np.testing.assert_array_equal(host(c["scales"]), s.scales)
    # addresses that allow 8-byte accesses only
    flat = torch.zeros(qkv.numel() + 4, dtype=qkv.dtype, device="cuda")
    flat[4:] = qkv.flatten()
    odd = flat[4:].view(qkv.shape)
    w = {**c, "codes": torch.zeros_like(c["codes"]), "scales": torch.zeros_like(c["scales"])}
    fa.kv4_write(odd[:, :, 4:6], odd[:, :, 6:8], **w)
    z = {**c, "codes": torch.zeros_like(c["codes"]), "scales": torch.zeros_like(c["scales"])}
    fa.kv4_write(qkv[:, :, 4:6], qkv[:, :, 6:8], **z)
    assert torch.equal(w["codes"], z["codes"]) and torch.equal(w["scales"], z["scales"])
    # heads in front of rows: [B, H, S, D] seen as [B, S, H, D]
    t = qkv[:, :, 4:6].transpose(1, 2).contiguous().transpose(1, 2)
    fa.kv4_write(t, qkv[:, :, 6:8], **c)
    np.testing.assert_array_equal(c["codes"].cpu().numpy(), s.codes)


# --------------------------------------------------------------- attention
def run_attention(fa, s, dtype, H, rows, packed, window=-1, scale=None, q16=None, strided=False, check=True):
    import torch
    D = s.D
    cu = cu_of(rows)
    total = int(cu[-1])
    if q16 is None:
        q16 = to16(s.r.standard_normal((total, H, D)), dtype)
    q = dev(q16, dtype)
    if strided:
        wide = torch.zeros(total, H + 3, D + 8, dtype=q.dtype, device="cuda")
        wide[:, 1:H + 1, :D] = q
        q = wide[:, 1:H + 1, :D]
    if packed:
        kw = dict(cu_seqlens=torch.from_numpy(cu).cuda(), max_seqlen=max(rows))
    else:
        q = q.unflatten(0, (s.B, rows[0]))
        kw = {}
    o, lse = fa.kv4_attention(q, **s.cuda(), **kw, window_left=window, scale=scale)
    O, L = decode(host(o), dtype).reshape(total, H, D), lse.double().cpu().numpy()
    if not packed:
        L = L.transpose(1, 0, 2).reshape(H, total)
    sc = D ** -0.5 if scale is None else scale
    for b, n in enumerate(rows):
        at = slice(cu[b], cu[b] + n)
        qq = decode(q16[at], dtype)
        k, v = s.rows(b, 0), s.rows(b, 1)
        ro, rl, ra = kv4.attention(qq, k, v, sc, window)
        if check:
            to, tl = attention_tolerance(qq, k, ro, ra, rl, sc, dtype)
            assert np.isfinite(O[at]).all()
            worst = (np.abs(O[at] - ro) / to).max(initial=0)
            assert worst <= 1, f"sequence {b} (len {s.lens[b]}, n {n}): |dO| is {worst:.3g} of its bound"
            np.testing.assert_array_equal(np.isneginf(L[:, at]), np.isneginf(rl))
            fin = np.isfinite(rl)
            worst = (np.abs(L[:, at][fin] - rl[fin]) / tl[fin]).max(initial=0)
            assert worst <= 1, f"sequence {b}: |dLSE| is {worst:.3g} of its bound"
            assert (O[at][np.isneginf(rl).T] == 0).all()
    return O, L


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,H_kv,G,P", [(32, 1, 1, 16), (64, 2, 1, 16), (64, 1, 8, 32), (96, 1, 4, 48), (128, 2, 4, 64),
                                        (128, 1, 16, 16), (160, 1, 2, 16), (192, 1, 5, 32), (224, 1, 3, 16),
                                        (256, 2, 4, 32)])
def test_single_tokens(fa, dtype, D, H_kv, G, P):
    s = Setup(LENS, H_kv, D, P, seed=D + G)
    run_attention(fa, s, dtype, H_kv * G, [1] * len(LENS), packed=False)


@pytest.mark.parametrize("D,H_kv,G,P,n", [(64, 1, 4, 16, 3), (128, 2, 4, 32, 4), (128, 1, 1, 64, 16), (128, 1, 5, 48, 7),
                                          (256, 1, 4, 16, 2), (64, 1, 1, 16, 40), (96, 2, 2, 16, 33), (128, 2, 2, 64, 130),
                                          (256, 1, 2, 32, 70)])
@pytest.mark.parametrize("window", [-1, 0, 5, 40])
def test_several_tokens(fa, D, H_kv, G, P, n, window):
    lens = [0, 1, n, n + 1, 64, 150]
    s = Setup(lens, H_kv, D, P, seed=n)
    run_attention(fa, s, "bf16", H_kv * G, [n] * len(lens), packed=False, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,H_kv,G,P", [(32, 2, 2, 16), (64, 1, 4, 32), (96, 1, 1, 48), (128, 2, 5, 64), (160, 1, 2, 16),
                                        (192, 2, 1, 32), (224, 1, 3, 16), (256, 1, 4, 128)])
def test_parts_of_prompts(fa, dtype, D, H_kv, G, P):
    """More than 16 rows a K/V head, up to several row tiles; the whole
    sequence, its end, more rows than tokens, nothing cached, nothing at all."""
    lens, n = [0, 60, 129, 257, 600, 311], 129
    s = Setup(lens, H_kv, D, P, seed=D + P)
    run_attention(fa, s, dtype, H_kv * G, [n] * len(lens), packed=False)
    run_attention(fa, s, dtype, H_kv * G, [0, 60, 129, 257, 17, 1], packed=True, window=100, strided=True)


@pytest.mark.parametrize("D,G,n,L", [(128, 4, 20, 9000), (64, 8, 33, 5000), (256, 2, 40, 4000), (96, 1, 150, 6000)])
def test_prompts_whose_keys_are_shared_out(fa, D, G, n, L):
    s = Setup([L, L // 3, 5], 1, D, 64, seed=L)
    run_attention(fa, s, "bf16", G, [n] * 3, packed=False)
    run_attention(fa, s, "f16", G, [n] * 3, packed=False, window=L // 2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,H_kv,G,P", [(128, 2, 4, 32), (64, 1, 2, 16)])
def test_packed_sequences(fa, dtype, D, H_kv, G, P):
    rows = [1, 0, 4, 1, 90, 2, 0]
    lens = [65, 9, 4, 0, 100, 200, 0]
    s = Setup(lens, H_kv, D, P, seed=2)
    run_attention(fa, s, dtype, H_kv * G, rows, packed=True, strided=True)
    run_attention(fa, s, dtype, H_kv * G, rows, packed=True, window=20)


@pytest.mark.parametrize("B,L,H_kv,G,D,P", [(1, 9000, 1, 4, 128, 64), (1, 4097, 2, 8, 64, 16), (3, 2500, 1, 2, 256, 32),
                                            (40, 200, 2, 2, 64, 16), (150, 70, 1, 1, 32, 16),
                                            (300, 620, 1, 2, 32, 16)])
def test_ranges_that_cut_items(fa, B, L, H_kv, G, D, P):
    """Long contexts over many CTAs, many short ones in a CTA."""
    lens = [max(0, L - 37 * b % L) for b in range(B)]
    s = Setup(lens, H_kv, D, P, seed=B)
    run_attention(fa, s, "bf16", H_kv * G, [1] * B, packed=False)


@pytest.mark.parametrize("D,copies", [(64, 1), (64, 10), (160, 1), (160, 10)])
def test_peaky_scores_and_scales_of_every_size(fa, D, copies):
    """Scores that leave one key, values whose scales differ by 2^40 between
    tokens, tiny and huge queries; as a step and as a part of a prompt."""
    s = Setup([500], 1, D, 16, seed=4, loud=1.5)
    mag = np.exp2(s.r.integers(-20, 21, (500, 1, 1)).astype(float))
    s.put(0, 1, np.arange(500), s.r.standard_normal((500, 1, D)) * mag)
    q = s.r.standard_normal((4 * copies, 4, D)) * np.tile([1e-6, 1.0, 20.0, 200.0], copies)[:, None, None]
    run_attention(fa, s, "bf16", 4, [4 * copies], packed=False, q16=to16(q, "bf16"))
    # one value of scale for the whole call, far from one
    for mag in (2.0 ** -80, 2.0 ** 60):
        s.put(0, 1, np.arange(500), s.r.standard_normal((500, 1, D)) * mag)
        run_attention(fa, s, "bf16", 4, [4 * copies], packed=False, q16=to16(q, "bf16"))
    s.put(0, 1, np.arange(500), np.zeros((500, 1, D)))
    O, _ = run_attention(fa, s, "bf16", 4, [4 * copies], packed=False, q16=to16(q, "bf16"))
    assert (O == 0).all()


@pytest.mark.parametrize("D,heads", [(64, 2), (64, 4), (256, 4)])
def test_nan_reaches_its_rows_and_groups_only(fa, D, heads):
    """A NaN in a key makes the rows that see it NaN, one in a value its group
    of 32 elements; rows that do not see the token stay as they are."""
    n = 8
    for which in (0, 1):
        s = Setup([70], 1, D, 16, seed=6)
        q16 = to16(s.r.standard_normal((n, heads, D)), "f16")
        clean, _ = run_attention(fa, s, "f16", heads, [n], packed=False, q16=q16)
        bad = 66                                     # rows 0 .. 3 are tokens 62 .. 65
        s.scales[s.table[0, bad // 16], which, 0, bad % 16, 1] = 0x7FC0
        O, L = run_attention(fa, s, "f16", heads, [n], packed=False, q16=q16, check=False)
        np.testing.assert_array_equal(O[:4], clean[:4])
        if which == 0:
            assert np.isnan(O[4:]).all() and np.isnan(L[:, 4:]).all()
        else:
            assert np.isnan(O[4:, :, 32:64]).all()
            np.testing.assert_allclose(O[4:, :, :32], clean[4:, :, :32], rtol=2e-3, atol=1e-4)
            np.testing.assert_allclose(O[4:, :, 64:], clean[4:, :, 64:], rtol=2e-3, atol=1e-4)


@pytest.mark.parametrize("n", [2, 30])
def test_nan_in_a_query_stays_in_its_row(fa, n):
    s = Setup([50], 1, 64, 16, seed=7)
    q16 = to16(s.r.standard_normal((n, 4, 64)), "bf16")
    clean, cl = run_attention(fa, s, "bf16", 4, [n], packed=False, q16=q16)
    q16[1, 2, 5] = 0x7FC0
    q16[0, 3, 9] = 0x7F80
    O, L = run_attention(fa, s, "bf16", 4, [n], packed=False, q16=q16, check=False)
    hit = np.zeros((n, 4), bool)
    hit[1, 2] = hit[0, 3] = True
    assert np.isnan(O[hit]).all() and np.isnan(L.T[hit]).all()
    np.testing.assert_array_equal(O[~hit], clean[~hit])


# ------------------------------------------------------ what the device checks
def test_bad_pages_and_lengths_are_reported_and_left_out(fa):
    import torch
    s = Setup([40, 70, 33], 1, 64, 16, seed=8)
    c = s.cuda()
    q16 = to16(s.r.standard_normal((3, 1, 2, 64)), "bf16")
    q = dev(q16, "bf16")
    # a page number outside the cache in sequence 1: its 16 keys are left out
    for bad in (s.pages, -1, 2 ** 31 - 1, -2 ** 31):
        c["page_table"][1, 2] = bad
        o, lse = fa.kv4_attention(q, **c)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_PAGES
        k, v = (np.delete(s.rows(1, w), np.s_[32:48], 0) for w in (0, 1))
        ro, rl, ra = kv4.attention(decode(q16[1], "bf16"), k, v, 0.125)
        to, tl = attention_tolerance(decode(q16[1], "bf16"), k, ro, ra, rl, 0.125, "bf16")
        assert (np.abs(decode(host(o[1]), "bf16") - ro) <= to).all()
        assert (np.abs(lse[1].double().cpu().numpy() - rl) <= tl).all()
        # reading: the rows on the bad page stay as they were
        ko, vo = (torch.full((3, 40, 1, 64), 7.0, dtype=torch.float16, device="cuda") for _ in (0, 1))
        fa.kv4_read(**c, max_seqlen=40, k_out=ko, v_out=vo)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_PAGES
        K = ko[1].double().cpu().numpy()
        assert (K[2:18] == 7).all()                       # tokens 32 .. 47 of 30 .. 69
        np.testing.assert_array_equal(np.delete(K, np.s_[2:18], 0), np.delete(s.rows(1, 0)[30:], np.s_[2:18], 0))
        # writing: nothing of the cache changes for them
        x = torch.ones(3, 40, 1, 64, dtype=torch.float16, device="cuda")
        w = {**c, "codes": c["codes"].clone(), "scales": c["scales"].clone()}
        fa.kv4_write(x, x, **w)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_PAGES
        changed = {int(p) for p in (w["codes"] != c["codes"]).flatten(1).any(1).nonzero().flatten()}
        assert changed <= {int(p) for p in s.table.flatten() if p >= 0} - {int(s.table[1, 2])}
    # lengths outside: the sequence is skipped, the others are not
    c = s.cuda()
    for bad in (-1, s.max_pages * 16 + 1, 2 ** 31 - 1):
        c["seq_lens"][1] = bad
        out = torch.full((3, 1, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        o, lse = fa.kv4_attention(q, **c, out=out, lse=torch.full((3, 2, 1), 7.0, device="cuda"))
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_PAGES
        assert (o[1] == 7).all() and (lse[1] == 7).all()
        ro, rl, ra = kv4.attention(decode(q16[2], "bf16"), s.rows(2, 0), s.rows(2, 1), 0.125)
        assert (np.abs(decode(host(o[2]), "bf16") - ro) <= attention_tolerance(
            decode(q16[2], "bf16"), s.rows(2, 0), ro, ra, rl, 0.125, "bf16")[0]).all()
        x = torch.ones(3, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
        before, scales_before = c["codes"].clone(), c["scales"].clone()
        fa.kv4_write(x, x, **c)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_PAGES
        own = [int(p) for p in s.table[1] if p >= 0]
        assert torch.equal(before[own], c["codes"][own])
        c["codes"].copy_(before)
        c["scales"].copy_(scales_before)


def test_bad_offsets_are_reported_and_skipped(fa):
    import torch
    s = Setup([20, 20, 20], 1, 64, 16, seed=8)
    q = torch.zeros(12, 2, 64, dtype=torch.bfloat16, device="cuda")
    for cu in ([0, 4, 2, 12], [0, 4, 8, 13], [-1, 4, 8, 12], [0, 4, 2 ** 31 - 1, 12], [0, 4, 11, 12]):
        kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), max_seqlen=6)
        out = torch.full_like(q, 7.0)
        fa.kv4_attention(q, **s.cuda(), **kw, out=out)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_SEQLENS, cu
        x = torch.ones(12, 1, 64, dtype=torch.bfloat16, device="cuda")
        fa.kv4_write(x, x, **s.cuda(), **kw)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_SEQLENS, cu
        fa.kv4_read(**s.cuda(), **kw, total=12)
        assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_SEQLENS, cu


# ----------------------------------------------------------------- together
def test_rotate_write_attend_as_a_decoder_runs_them(fa):
    """A prompt of two sequences, then steps of one token: rotary positions,
    the write, attention over the cache; against the same in fp64 on the
    16-bit values that each call was given."""
    import torch
    r = np.random.default_rng(11)
    B, H, Hkv, D, P, dtype = 2, 4, 2, 64, 16, "bf16"
    n0 = [23, 40]
    s = Setup([0, 0], Hkv, D, P, seed=12, filled=False, spare=0)
    s.max_pages, s.pages = 4, 9
    s.table = np.arange(8, dtype=np.int32).reshape(2, 4) + 1
    s.codes = np.zeros((9, 2, Hkv, P, D // 2), np.uint8)
    s.scales = np.zeros((9, 2, Hkv, P, D // 32), np.uint16)
    freq, axes = fa.rotary_frequencies(D, (8, 12, 12))
    c = s.cuda()
    fnp, anp = freq.cpu().numpy(), axes.cpu().numpy()
    for step in range(4):
        rows = n0 if step == 0 else [1, 1]
        s.lens = s.lens + np.asarray(rows, np.int32)
        c["seq_lens"].copy_(torch.from_numpy(s.lens))
        cu, total = cu_of(rows), sum(rows)
        qkv16 = to16(r.standard_normal((total, H + 2 * Hkv, D)), dtype)
        pos = r.integers(0, 4000, (total, 3)).astype(np.int32)
        qkv = dev(qkv16, dtype)
        kw = dict(cu_seqlens=torch.from_numpy(cu).cuda(), max_seqlen=max(rows))
        q, k = fa.rotary(qkv[:, :H], torch.from_numpy(pos).cuda(), freq, axes, k=qkv[:, H:H + Hkv])
        fa.kv4_write(k, qkv[:, H + Hkv:], **c, **kw)
        o, lse = fa.kv4_attention(q, **c, **kw)
        x = decode(qkv16, dtype)
        want = kv4.rotary(x[:, :H + Hkv], pos, fnp, anp)
        got = np.concatenate([decode(host(q), dtype), decode(host(k), dtype)], 1)
        # each output is a rounding of a sum of two products in fp32
        assert (np.abs(got - want) <= half_step(want, dtype) * 1.02 + 2.0 ** -20 * np.abs(x).max()).all()
        for b, n in enumerate(rows):
            at = slice(cu[b], cu[b] + n)
            expected_write(s, b, host(k)[at], 0, dtype, n)
            expected_write(s, b, qkv16[at, H + Hkv:], 1, dtype, n)
            ro, rl, ra = kv4.attention(decode(host(q)[at], dtype), s.rows(b, 0), s.rows(b, 1), D ** -0.5)
            to, tl = attention_tolerance(decode(host(q)[at], dtype), s.rows(b, 0), ro, ra, rl, D ** -0.5, dtype)
            assert (np.abs(decode(host(o)[at], dtype) - ro) <= to).all()
            assert (np.abs(lse[:, at].double().cpu().numpy() - rl) <= tl).all()
        np.testing.assert_array_equal(c["codes"].cpu().numpy(), s.codes)


def test_read_back_feeds_the_plain_attention(fa):
    """K and V read back, through attention_forward_varlen, agree with
    attention over the cache."""
    import torch
    s = Setup([130, 60], 2, 128, 16, seed=13)
    c = s.cuda()
    cu = torch.tensor([0, 130, 190], dtype=torch.int32, device="cuda")
    k, v = fa.kv4_read(**c, cu_seqlens=cu, max_seqlen=130, total=190, dtype=torch.float16)
    q = dev(to16(s.r.standard_normal((190, 4, 128)), "f16"), "f16")
    o1, l1 = fa.attention_forward_varlen(q, k, v, cu, max_seqlen=130, causal=True)
    o2, l2 = fa.kv4_attention(q, **c, cu_seqlens=cu, max_seqlen=130)
    assert (o1.double() - o2.double()).abs().max().item() <= 2e-3
    assert (l1 - l2).abs().max().item() <= 1e-4


# ------------------------------------------------------- streams and graphs
def test_graphs_streams_and_repeats(fa):
    """The same bits on another stream, from two graphs replayed at once, and
    again and again."""
    import torch
    s = Setup([2000, 900, 0, 1], 2, 128, 64, seed=14)
    c = s.cuda()
    q = dev(to16(s.r.standard_normal((4, 1, 8, 128)), "bf16"), "bf16")
    q2 = dev(to16(s.r.standard_normal((4, 1, 8, 128)), "bf16"), "bf16")
    o, lse = fa.kv4_attention(q, **c)
    p, pl = fa.kv4_attention(q2, **c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, al = fa.kv4_attention(q, **c, stream=side)
    b, bl = fa.kv4_attention(q, **c, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for x, xl in ((a, al), (b, bl)):
        assert torch.equal(x, o) and torch.equal(xl, lse)
    graphs, outs = [], []
    for query in (q, q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(fa.kv4_attention(query, **c))
        graphs.append(g)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        for st, g in ((s1, graphs[0]), (s2, graphs[1])):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], o) and torch.equal(outs[0][1], lse)
    assert torch.equal(outs[1][0], p) and torch.equal(outs[1][1], pl)


def test_a_graph_follows_the_lengths(fa):
    """A captured step is replayed as the sequences grow: lengths, pages and
    rows are read on the device."""
    import torch
    s = Setup([30, 47], 1, 64, 16, seed=15)
    s.table[0, 2], s.table[1, 3] = s.pages - 1, s.pages - 2     # the spare pages
    c = s.cuda()
    k = torch.zeros(2, 1, 1, 64, dtype=torch.float16, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros(2, 1, 4, 64, dtype=torch.float16, device="cuda")
    fa.kv4_write(k, v, **{**c, "codes": c["codes"].clone(), "scales": c["scales"].clone()})   # the first launch
    fa.kv4_attention(q, **c)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.kv4_write(k, v, **c)
        o, lse = fa.kv4_attention(q, **c)
    for step in range(5):
        s.lens = s.lens + 1
        x = [to16(s.r.standard_normal(t.shape), "f16") for t in (k, v, q)]
        for t, bits in zip((k, v, q), x):
            t.copy_(dev(bits, "f16"))
        c["seq_lens"].copy_(torch.from_numpy(s.lens))
        g.replay()
        for b in range(2):
            expected_write(s, b, x[0][b], 0, "f16", 1)
            expected_write(s, b, x[1][b], 1, "f16", 1)
            ro, rl, ra = kv4.attention(decode(x[2][b], "f16"), s.rows(b, 0), s.rows(b, 1), 0.125)
            to, tl = attention_tolerance(decode(x[2][b], "f16"), s.rows(b, 0), ro, ra, rl, 0.125, "f16")
            assert (np.abs(decode(host(o[b]), "f16") - ro) <= to).all()
            assert (np.abs(lse[b].double().cpu().numpy() - rl) <= tl).all()


def test_offsets_past_32_bits(fa):
    """A cache of more than 4 GB of codes: the last pages are reached."""
    import torch
    D, Hkv, P, pages = 256, 8, 128, 18000          # 18000 x 2 x 8 x 128 x 128 B = 4.7 GB
    codes = torch.zeros(pages, 2, Hkv, P, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(pages, 2, Hkv, P, D // 32, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[pages - 1, pages - 2, 0]], dtype=torch.int32, device="cuda")
    s = Setup([200], Hkv, D, P, seed=16, filled=False)
    x16 = [to16(s.r.standard_normal((1, 200, Hkv, D)), "bf16") for _ in (0, 1)]
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    fa.kv4_write(dev(x16[0], "bf16"), dev(x16[1], "bf16"), codes, scales, table, lens)
    for which in (0, 1):
        expected_write(s, 0, x16[which][0], which, "bf16", 200)
    k, v = fa.kv4_read(codes, scales, table, lens, max_seqlen=200, dtype=torch.float16)
    np.testing.assert_array_equal(k[0].double().cpu().numpy(), s.rows(0, 0))
    np.testing.assert_array_equal(v[0].double().cpu().numpy(), s.rows(0, 1))
    q16 = to16(s.r.standard_normal((1, 1, Hkv, D)), "bf16")
    o, lse = fa.kv4_attention(dev(q16, "bf16"), codes, scales, table, lens)
    ro, rl, ra = kv4.attention(decode(q16[0], "bf16"), s.rows(0, 0), s.rows(0, 1), D ** -0.5)
    to, tl = attention_tolerance(decode(q16[0], "bf16"), s.rows(0, 0), ro, ra, rl, D ** -0.5, "bf16")
    assert (np.abs(decode(host(o[0]), "bf16") - ro) <= to).all()


def test_both_ways_of_marshalling_agree(fa, monkeypatch):
    """The native binding and the Python code make the same calls: results bit
    for bit, refusals alike."""
    import torch
    from attention_forward_fwd_gb300 import cache
    s = Setup([130, 7, 0], 2, 64, 16, seed=21)
    c = s.cuda()
    cu = torch.tensor([0, 100, 103, 103], dtype=torch.int32, device="cuda")
    qkv = dev(to16(s.r.standard_normal((103, 10, 64)), "bf16"), "bf16")
    freq, axes = fa.rotary_frequencies(64, (16, 16))
    pos = torch.arange(206, dtype=torch.int32, device="cuda").view(103, 2)

    def calls():
        w = {**c, "codes": c["codes"].clone(), "scales": c["scales"].clone()}
        kw = dict(cu_seqlens=cu, max_seqlen=100)
        q, k = fa.rotary(qkv[:, :6], pos, freq, axes, k=qkv[:, 6:8])
        (one,) = [fa.rotary(qkv[:, :6], pos, freq, axes, interleaved=True, inverse=True)]
        v = qkv[:, 8:]
        ko, vo = torch.empty_like(k), torch.empty(v.shape, dtype=v.dtype, device="cuda")
        assert fa.kv4_write(k, v, **w, **kw, k_out=ko, v_out=vo) is None
        out = [q, k, one, ko, vo, w["codes"], w["scales"], *fa.kv4_read(**w, **kw, total=103)]
        out += [*fa.kv4_read(**w, max_seqlen=5, dtype=torch.float16)]
        out += [*fa.kv4_attention(q, **w, **kw), *fa.kv4_attention(q, **w, **kw, window_left=9, scale=0.5)]
        o = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        p, none = fa.kv4_attention(q, **w, **kw, out=o, with_lse=False)
        assert p.data_ptr() == o.data_ptr() and none is None
        b = qkv[:3, :6].unsqueeze(1)
        out += [o, *fa.kv4_attention(b, **w), fa.rotary(b, pos[:3].unsqueeze(1), freq, axes)]
        for bad in (lambda: fa.kv4_attention(q[:, :5], **w, **kw), lambda: fa.kv4_attention(q.float(), **w, **kw),
                    lambda: fa.kv4_write(k, v[:50], **w, **kw), lambda: fa.kv4_attention(q, **w),
                    lambda: fa.rotary(q, pos.long(), freq, axes), lambda: fa.rotary(q, pos, freq, axes.long()),
                    lambda: fa.kv4_read(**{**w, "seq_lens": w["seq_lens"].long()}, max_seqlen=3),
                    lambda: fa.kv4_read(**w, cu_seqlens=cu), lambda: fa.kv4_attention(q, **w, **kw, out=o[:50]),
                    lambda: fa.kv4_attention(q.cpu(), **w, **kw)):
            with pytest.raises(ValueError):
                bad()
        for bad in (lambda: fa.kv4_attention(q, **w, **kw, window_left=-2), lambda: fa.kv4_attention(q, **w, **kw, scale=-1.0)):
            with pytest.raises(fa.FaError):
                bad()
        return out

    first = calls()
    monkeypatch.setattr(cache, "_native", None)
    for x, y in zip(first, calls(), strict=True):
        assert x.shape == y.shape and x.dtype == y.dtype and x.is_contiguous()
        assert torch.equal(x.view(torch.uint8) if x.dtype == torch.uint8 else torch.nan_to_num(x.float()),
                           y.view(torch.uint8) if y.dtype == torch.uint8 else torch.nan_to_num(y.float()))


def test_two_streams_at_once(fa):
    """Calls that overlap on two streams, cut and whole, steps and prompts,
    give what they give alone."""
    import torch
    s = Setup([5000, 300, 900], 2, 64, 16, seed=22)
    c = s.cuda()
    qs = [dev(to16(s.r.standard_normal((3, n, 4, 64)), "f16"), "f16") for n in (1, 1, 60, 40)]
    alone = [fa.kv4_attention(q, **c) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        got = []
        for q, st in zip(qs, streams):
            with torch.cuda.stream(st):
                got.append(fa.kv4_attention(q, **c))
        torch.cuda.synchronize()
        for (a, al), (b, bl) in zip(alone, got):
            assert torch.equal(a, b) and torch.equal(al, bl)


@pytest.mark.parametrize("L", [512, 513, 544, 545, 1024, 1056, 1057, 2048, 2080, 2081, 4096, 4128, 4129])
def test_contexts_around_the_cluster_sizes(fa, L):
    """Tables that end where a cluster of 1, 2, 4 or 8 CTAs does, and just behind;
    shorter sequences, of which some CTAs of the cluster get nothing."""
    s = Setup([L, 40, 0, L - 33], 1, 64, 16, seed=L)
    run_attention(fa, s, "bf16", 2, [1] * 4, packed=False)
    run_attention(fa, s, "f16", 3, [4, 0, 1, 4], packed=True, window=L // 3)


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("n", [4, 70])
def test_windows_of_any_int(fa, monkeypatch, native, n):
    """A window as far as an int goes, or farther, bounds nothing; rows before the
    first token stand at negative positions."""
    import torch
    from attention_forward_fwd_gb300 import cache
    if not native:
        monkeypatch.setattr(cache, "_native", None)
    s = Setup([150, 3, 0, 1], 2, 64, 16, seed=n)
    c = s.cuda()
    q = dev(to16(s.r.standard_normal((4, n, 4, 64)), "bf16"), "bf16")
    o, lse = fa.kv4_attention(q, **c)
    for window in (149, 2**31 - 1, 2**31, 2**32, 2**40):
        p, l2 = fa.kv4_attention(q, **c, window_left=window)
        assert torch.equal(o, p) and torch.equal(lse, l2)
    for window in (-2, -2**31, -2**32, -2**33 + 5):
        with pytest.raises(fa.FaError):
            fa.kv4_attention(q, **c, window_left=window)
