"""Rotary positions on the GPU against the fp64 oracle, their gradient against
the formula and against differences."""
import numpy as np
import pytest

import fa_inputs
from oracle import kv4
from oracle.attention import decode

from kv4_common import half_step, to16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import torch
    import attention_forward_fwd_gb300 as fa
    assert torch.cuda.is_available(), "the gpu tests need a CUDA device"
    fa.build()
    fa.fa_device_status(clear=True)
    return fa


def host(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def dev(bits, dtype):
    return fa_inputs.to_torch(np.ascontiguousarray(bits), dtype).cuda()


def check(got16, want, x, dtype):
    """One rounding of x cos + y sin: the angle is off by at most 2^-22 of a turn and sincospi, products and sum
    by a few 2^-24 (together below 2^-19 of |x| + |y|)."""
    top = np.abs(x).max()
    d = np.abs(decode(got16, dtype) - want)
    bound = half_step(np.abs(want) + 2.0 ** -18 * top, dtype) + 2.0 ** -18 * top
    assert (d <= bound).all(), f"worst {(d / bound).max()} of the bound"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hk,D,R,sections", [
    (1, 1, 1, 64, 64, (32,)), (5, 4, 2, 128, 128, (16, 24, 24)), (33, 3, 1, 96, 96, (48,)),
    (7, 2, 2, 128, 64, (10, 12, 10)), (2000, 4, 1, 64, 64, (16, 16)), (9, 2, 1, 80, 40, (20,)),
    (3, 1, 1, 2, 2, (1,)), (4, 2, 3, 72, 50, (5, 10, 10)), (6, 1, 2, 256, 256, (0, 64, 64)), (5, 1, 1, 37, 12, (6,)),
    (1500, 40, 8, 128, 128, (64,))])
@pytest.mark.parametrize("inverse", [False, True])
def test_turns(fa, dtype, interleaved, T, H, Hk, D, R, sections, inverse):
    import torch
    r = np.random.default_rng(T + D)
    freq, axes = fa.rotary_frequencies(R, sections)
    pos = r.integers(0, 1 << 20, (T, len(sections))).astype(np.int32)
    pos[0] = 0
    q16, k16 = (to16(r.standard_normal((T, h, D)), dtype) for h in (H, Hk))
    q, k = dev(q16, dtype), dev(k16, dtype)
    p = torch.from_numpy(pos).cuda()
    a, b = fa.rotary(q, p, freq, axes, k=k, interleaved=interleaved, inverse=inverse)
    for got, bits in ((a, q16), (b, k16)):
        x = decode(bits, dtype)
        check(host(got), kv4.rotary(x, pos, freq.cpu().numpy(), axes.cpu().numpy(), interleaved, inverse), x, dtype)
        np.testing.assert_array_equal(host(got)[..., R:], bits[..., R:])      # copied
    one = fa.rotary(q, p, freq, axes, interleaved=interleaved, inverse=inverse)
    assert torch.equal(one, a)
    fa.rotary(q, p, freq, axes, k=k, interleaved=interleaved, inverse=inverse, q_out=q, k_out=k)   # in place
    assert torch.equal(q, a) and torch.equal(k, b)
    assert fa.fa_device_status(clear=True) == 0


def test_strides_and_batches(fa):
    import torch
    r = np.random.default_rng(1)
    freq, axes = fa.rotary_frequencies(64, (16, 16))
    x16 = to16(r.standard_normal((2, 5, 9, 64)), "bf16")
    pos = r.integers(-1000, 1000, (2, 5, 2)).astype(np.int32)
    x, p = dev(x16, "bf16"), torch.from_numpy(pos).cuda()
    want = kv4.rotary(decode(x16, "bf16").reshape(10, 9, 64), pos.reshape(10, 2), freq.cpu().numpy(), axes.cpu().numpy())
    check(host(fa.rotary(x, p, freq, axes)).reshape(10, 9, 64), want, want, "bf16")
    # a slice of heads, in place: the others are left alone
    y = x.clone()
    fa.rotary(y[:, :, 2:6], p, freq, axes, k=y[:, :, 6:7], q_out=y[:, :, 2:6], k_out=y[:, :, 6:7])
    check(host(y[:, :, 2:7]).reshape(10, 5, 64), want[:, 2:7], want, "bf16")
    assert torch.equal(y[:, :, :2], x[:, :, :2]) and torch.equal(y[:, :, 7:], x[:, :, 7:])
    # an odd offset (2-byte accesses), a transposed head axis
    flat = torch.zeros(x.numel() + 3, dtype=x.dtype, device="cuda")
    flat[3:] = x.flatten()
    check(host(fa.rotary(flat[3:].view(x.shape), p, freq, axes)).reshape(10, 9, 64), want, want, "bf16")
    t = x[0].transpose(0, 1).contiguous().transpose(0, 1)
    check(host(fa.rotary(t, p[0], freq, axes)), want[:5], want, "bf16")
    with pytest.raises(ValueError):
        fa.rotary(x[:, ::2][:, :2], p[:, :2].contiguous(), freq, axes)     # tokens not evenly spaced


def test_far_positions(fa):
    """Up to the ends of int32 the angle stays within 2^-16 of a turn; up to 2^24 within 2^-22."""
    import torch
    freq, axes = fa.rotary_frequencies(64, (32,))
    pos = np.array([[0], [1], [(1 << 24) - 1], [-(1 << 24)], [2 ** 31 - 1], [-2 ** 31]], np.int32)
    x = np.zeros((6, 1, 64))
    x[..., :32] = 1.0
    got = decode(host(fa.rotary(dev(to16(x, "f16"), "f16"), torch.from_numpy(pos).cuda(), freq, axes)), "f16")
    want = kv4.rotary(x, pos, freq.cpu().numpy(), axes.cpu().numpy())
    err = np.abs(got - want).max((1, 2)) - 2.0 ** -12     # cos and sin are at most 1: half a step of fp16
    assert (err[:4] <= 2.0 ** -19).all() and (err[4:] <= 2 * np.pi * 2.0 ** -16).all()


def test_gradient(fa):
    """dX of sum(W y) is the inverse turn of W: against the formula's and
    against central differences of the fp64 definition."""
    import torch
    r = np.random.default_rng(2)
    freq, axes = fa.rotary_frequencies(32, (4, 6, 6))
    f, a = freq.cpu().numpy(), axes.cpu().numpy()
    pos = r.integers(0, 5000, (3, 3)).astype(np.int32)
    x, w16 = r.standard_normal((3, 2, 32)), to16(r.standard_normal((3, 2, 32)), "bf16")
    w = decode(w16, "bf16")
    for il in (False, True):
        got16 = host(fa.rotary(dev(w16, "bf16"), torch.from_numpy(pos).cuda(), freq, axes, interleaved=il, inverse=True))
        grad = np.empty_like(x)
        for i in np.ndindex(x.shape):
            up, down = x.copy(), x.copy()
            up[i] += 0.5
            down[i] -= 0.5                # the map is linear: any step is exact
            grad[i] = (w * (kv4.rotary(up, pos, f, a, il) - kv4.rotary(down, pos, f, a, il))).sum()
        check(got16, grad, w, "bf16")
        check(got16, kv4.rotary(w, pos, f, a, il, inverse=True), w, "bf16")


def test_bad_axis_is_reported(fa):
    import torch
    freq, axes = fa.rotary_frequencies(64, (32,))
    axes[3] = 5
    x = dev(to16(np.ones((2, 1, 64)), "bf16"), "bf16")
    y = fa.rotary(x, torch.full((2, 1), 7, dtype=torch.int32, device="cuda"), freq, axes)
    assert fa.fa_device_status(clear=True) == fa.FA_ERR_BAD_AXIS
    assert torch.equal(y[..., 3], x[..., 3]) and torch.equal(y[..., 35], x[..., 35])


def test_captured(fa):
    import torch
    freq, axes = fa.rotary_frequencies(128, (16, 24, 24))
    x = dev(to16(np.random.default_rng(3).standard_normal((4, 8, 128)), "bf16"), "bf16")
    pos = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    fa.rotary(x, pos, freq, axes)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = fa.rotary(x, pos, freq, axes)
    for p in (1, 77):
        pos.fill_(p)
        g.replay()
        assert torch.equal(y, fa.rotary(x, pos, freq, axes))


@pytest.mark.parametrize("T,H,Hk,D,F", [(200000, 1, 0, 16, 8), (90001, 2, 1, 64, 32), (30011, 1, 1, 256, 128),
                                        (25000, 1, 0, 40, 13), (5000, 3, 6, 96, 40)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens_of_few_heads(fa, T, H, Hk, D, F, interleaved):
    """However many tokens share a CTA, each is turned as in a call of its own few."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    q = torch.randn(T, H, D, generator=g, device="cuda").bfloat16()
    k = torch.randn(T, Hk, D, generator=g, device="cuda").bfloat16() if Hk else None
    pos = torch.randint(-1000, 1 << 20, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    freq, axes = fa.rotary_frequencies(2 * F, (F - F // 3, F // 3), interleave_axes=True)
    whole = fa.rotary(q, pos, freq, axes, k=k, interleaved=interleaved)
    whole = whole if Hk else (whole,)
    for lo, hi in ((0, 150), (T // 2 - 3, T // 2 + 140), (T - 131, T)):
        some = fa.rotary(q[lo:hi], pos[lo:hi], freq, axes, k=k[lo:hi] if Hk else None, interleaved=interleaved)
        for x, y in zip(whole, some if Hk else (some,)):
            assert torch.equal(x[lo:hi], y)
    assert fa.fa_device_status() == 0
