"""Cases of the quantised K/V cache operators and the rotary positions: what they compute, in plain torch, and the calls that reach the kernels.

The cache.  ``codes`` uint8 [pages, 2, H_kv, P, D / 2] and ``scales`` bf16 [pages, 2, H_kv, P, D / 32] hold K (index 0) and V (index 1) of P tokens a
page.  A row of D values (one token, one head) is cut in groups of 32 neighbours; a group has the scale s = -x_e / 8 rounded to bf16, x_e its element of
the largest magnitude (the first of equals), and each element the code n = clamp(rint(x / s), -8, 7) + 8, which stands for s * (n - 8).  A group of zeros
has s = 0 and codes 8, one with an infinity or a NaN has s = NaN and codes 8.  The code of element 32 g + 4 r + j of a row (j < 4, r < 8) is bits
4 j .. 4 j + 3 of the row's 16-bit word r * (D / 32) + g.

Sequence b has seq_lens[b] tokens in the pages page_table[b, :]; the n_b rows that a call brings for it are its last n_b tokens.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a step of 64 sequences being answered: one new token each goes into the cache (K and V are slices of a fused projection)
        dict(name="write step b64", op="write", B=64, n=1, L=2048, Hkv=8, D=128, P=64, dtype="bf16", ragged=True, values=False, fused=True),
        # prompts of up to 8191 tokens, packed; the values the cache stands for come back for the attention of the same pass
        dict(name="write prompts", op="write", B=6, n=8191, L=8191, Hkv=8, D=128, P=64, dtype="bf16", ragged=True, values=True, fused=True),
        # one long document in fp16 with narrow heads and small pages
        dict(name="write document f16", op="write", B=1, n=65536, L=65536, Hkv=4, D=64, P=16, dtype="f16", ragged=False, values=False, fused=False),
        # one sequence read back, for a kernel that wants plain K and V
        dict(name="read one", op="read", B=1, L=1999, Hkv=8, D=128, P=64, dtype="bf16", ragged=False),
        # a batch read back packed
        dict(name="read batch", op="read", B=16, L=8192, Hkv=8, D=128, P=32, dtype="f16", ragged=True),
        # the smallest answer: one short chat, one token
        dict(name="attend one", op="attend", B=1, n=1, L=320, H=16, Hkv=16, D=64, P=16, dtype="f16", ragged=False, window=-1),
        # a step of 64 sequences being answered, some slots of the batch empty
        dict(name="attend step b64", op="attend", B=64, n=1, L=4096, H=32, Hkv=8, D=128, P=64, dtype="bf16", ragged=True, window=-1),
        # one token over a long context
        dict(name="attend long", op="attend", B=2, n=1, L=131072, H=32, Hkv=8, D=128, P=64, dtype="bf16", ragged=False, window=-1),
        # four drafted tokens checked at once, wide heads, a sliding window
        dict(name="attend draft", op="attend", B=16, n=4, L=8192, H=16, Hkv=4, D=256, P=32, dtype="bf16", ragged=True, window=4096),
        # the next 2000 tokens of a prompt, over what is in the cache
        dict(name="attend prompt", op="attend", B=1, n=2000, L=16384, H=32, Hkv=8, D=128, P=64, dtype="bf16", ragged=False, window=-1),
        # rotary positions of a step: a token each, queries and keys
        dict(name="rotate step b64", op="rotate", T=64, H=32, Hkv=8, D=128, dtype="bf16", axes=3, interleaved=False, inverse=False, far=1 << 20),
        # of a video's patches: three axes; and back, as for the gradient
        dict(name="rotate video", op="rotate", T=32760, H=16, Hkv=16, D=128, dtype="bf16", axes=3, interleaved=False, inverse=True, far=1 << 14),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "rotate"])
    dtype, D = rng.choice(["bf16", "f16"]), rng.choice([32, 64, 64, 96, 128, 128, 128, 192, 256])
    if op == "rotate":
        Hkv = rng.choice([1, 2, 4, 8, 16])
        H = Hkv * rng.choice([1, 2, 4])
        T = _log(rng, 1, 32760 * 32 * 128 // ((H + Hkv) * D))
        return dict(op=op, T=T, H=H, Hkv=Hkv, D=D, dtype=dtype, axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, far=_log(rng, 16, 1 << 20))
    Hkv, P = rng.choice([1, 2, 4, 8, 16]), rng.choice([16, 32, 48, 64, 128])
    ragged = rng.random() < 0.6
    if op != "attend":
        rows = _log(rng, 1, 16 * 8192 * 8 * 128 // (Hkv * D))
        B = min(rows, _log(rng, 1, 64))
        L = rows // B
        if op == "read":
            return dict(op=op, B=B, L=L, Hkv=Hkv, D=D, P=P, dtype=dtype, ragged=ragged)
        n = L if rng.random() < 0.6 else _log(rng, 1, L)
        return dict(op=op, B=B, n=n, L=L, Hkv=Hkv, D=D, P=P, dtype=dtype, ragged=ragged, values=rng.random() < 0.5, fused=rng.random() < 0.5)
    G = rng.choice([1, 2, 4, 5, 8, 16])
    if rng.random() < 0.65:  # a step, or a few drafted tokens
        n = rng.choice([1, 1, 1, 2, 3, 4, 7])
        keys = _log(rng, 1, 64 * 4096 * 8 * 128 // (Hkv * D))
        B = min(keys, _log(rng, 1, 128))
        L = min(131072, keys // B)
    else:  # part of a prompt
        Hkv = min(Hkv, 8)
        most = 2000 * 16384 * 32 * 128 // (Hkv * G * D)  # query rows x keys, at most the listed prompt's work
        n = _log(rng, 8, 2000)
        L = max(n, _log(rng, n, max(n, min(16384, most // n))))
        B = 1 if n * L > most // 2 else rng.choice([1, 2])
    window = -1 if rng.random() < 0.7 else _log(rng, 1, L)
    return dict(op=op, B=B, n=n, L=L, H=Hkv * G, Hkv=Hkv, D=D, P=P, dtype=dtype, ragged=ragged, window=window)


def _lengths(case):
    """(tokens in the cache, rows of the call) of each sequence: fixed by the case, so that its work is."""
    B, L = case["B"], case["L"]
    r = np.random.RandomState(B * 131 + L)
    lens = np.full(B, L, np.int64)
    if case["ragged"] and B > 1:
        lens = r.randint(max(1, L // 8), L + 1, B)
        lens[0] = L
        if case["op"] == "attend" and B > 2:
            lens[B // 2] = 0  # a slot of the batch without a sequence
    if case["op"] == "read":
        rows = lens.copy()
    elif case["op"] == "write" and case["n"] > 1:
        rows = np.minimum(lens, case["n"])
    else:
        rows = np.full(B, case["n"], np.int64)
    return lens, rows


def _packed(case):
    """Writes and reads of more than one token a sequence come packed; steps and queries as a batch [B, n, ...]."""
    return case["op"] == "read" or (case["op"] == "write" and case["n"] > 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "rotate":
        T, H, A = case["T"], case["H"], case["axes"]
        half = D // 2
        cuts = [half * (a + 1) // A for a in range(A)]
        axes = torch.tensor([sum(f >= c for c in cuts) for f in range(half)], dtype=torch.int32, device="cuda")
        inv_freq = torch.tensor([10000.0 ** (-2.0 * f / D) for f in range(half)], dtype=torch.float64, device="cuda")
        qk = randn(T, H + Hkv, D).to(dt)
        pos = torch.randint(0, case["far"], (T, A), generator=g, device="cuda", dtype=torch.int32)
        return dict(case=case, q=qk[:, :H], k=qk[:, H:], pos=pos, inv_freq=inv_freq, axes=axes)
    B, P = case["B"], case["P"]
    lens, rows = _lengths(case)
    per = -(-max(1, case["L"]) // P)
    pages = B * per + 3
    table = torch.randperm(pages, generator=g, device="cuda")[: B * per].to(torch.int32).reshape(B, per)
    st = dict(case=case, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if _packed(case):
        cu = np.concatenate([[0], np.cumsum(rows)])
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        st["total"], st["most"] = int(cu[-1]), int(rows.max())
    if case["op"] == "write":
        st["codes"] = torch.zeros(pages, 2, Hkv, P, D // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros(pages, 2, Hkv, P, D // 32, dtype=torch.bfloat16, device="cuda")
        T = st["total"] if _packed(case) else B * case["n"]
        x = randn(T, 4 * Hkv if case["fused"] else 2 * Hkv, D)
        x *= torch.exp(0.5 * randn(D))  # some channels are louder than others
        x = x.to(dt)
        k, v = x[:, -2 * Hkv : -Hkv], x[:, -Hkv:]
        if not case["fused"]:
            k, v = k.contiguous(), v.contiguous()
        st["k"], st["v"] = (k, v) if _packed(case) else (k.unflatten(0, (B, case["n"])), v.unflatten(0, (B, case["n"])))
        st["k_out"] = torch.zeros(st["k"].shape, dtype=dt, device="cuda") if case["values"] else None
        st["v_out"] = torch.zeros(st["v"].shape, dtype=dt, device="cuda") if case["values"] else None
    else:
        # K and V as the cache meets them, one value of scale for each channel; what lies past the sequences' ends is whatever was there before
        loud = torch.exp(0.4 * randn(2, 1, 1, D))
        st["codes"] = torch.empty(pages, 2, Hkv, P, D // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(pages, 2, Hkv, P, D // 32, dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 26) // (2 * Hkv * P * D))
        for i in range(0, pages, step):
            x = randn(min(step, pages - i), 2, Hkv, P, D)
            st["codes"][i : i + step], st["scales"][i : i + step] = _quantise((x * loud).to(dt))
        if case["op"] == "attend":
            st["q"] = (0.7 * randn(B, case["n"], case["H"], D)).to(dt)
    return st


# ---------------------------------------------------------------- the plain forms


def _quantise(x):
    """(codes, scales) of rows [..., D]."""
    D = x.shape[-1]
    N = D // 32
    x = x.float().unflatten(-1, (N, 32))
    e = x.gather(-1, x.abs().argmax(-1, keepdim=True))
    ok = x.isfinite().all(-1, keepdim=True)
    s = (e / -8).bfloat16()
    some = ok & (s != 0)
    s = torch.where(some, s, torch.where(ok, 0.0, math.nan).to(s.dtype))
    n = torch.where(some, (x / s.float()).round().clamp(-8, 7) + 8, 8.0).to(torch.uint8)
    n = n.unflatten(-1, (8, 4)).transpose(-3, -2).flatten(-3).unflatten(-1, (D // 2, 2))
    return n[..., 0] | (n[..., 1] << 4), s.squeeze(-1)


def _values(codes, scales):
    """What codes [..., D / 2] and scales [..., D / 32] stand for, in 32 bits."""
    N = scales.shape[-1]
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).unflatten(-1, (8, N, 4)).transpose(-3, -2).flatten(-2)
    return ((n.float() - 8) * scales.float().unsqueeze(-1)).flatten(-2)


def _places(st):
    """Packed rows' (page, place in the page), from the page table."""
    case = st["case"]
    lens = st["lens"].long()
    if "cu" in st:
        cu = st["cu"].long()
        row = torch.arange(st["total"], device="cuda")
        b = torch.searchsorted(cu, row, right=True) - 1
        pos = lens[b] - (cu[b + 1] - row)
    else:
        b = torch.arange(case["B"], device="cuda").repeat_interleave(case["n"])
        pos = lens[b] - case["n"] + torch.arange(case["n"], device="cuda").repeat(case["B"])
    return st["table"][b, pos // case["P"]].long(), pos % case["P"]


def _write(st):
    page, at = _places(st)
    k, v = (x.flatten(0, -3) for x in (st["k"], st["v"]))
    codes, scales = _quantise(torch.stack((k, v), 1))
    st["codes"][page, :, :, at], st["scales"][page, :, :, at] = codes, scales
    out = [st["codes"], st["scales"]]
    if st["k_out"] is not None:
        x = _values(codes, scales).to(k.dtype)
        st["k_out"].copy_(x[:, 0].view(st["k_out"].shape))
        st["v_out"].copy_(x[:, 1].view(st["v_out"].shape))
        out += [st["k_out"], st["v_out"]]
    return out


def _read(st):
    page, at = _places(st)
    x = _values(st["codes"][page, :, :, at], st["scales"][page, :, :, at]).to(DT[st["case"]["dtype"]])
    return [x[:, 0].contiguous(), x[:, 1].contiguous()]


def _attend(st):
    case, q = st["case"], st["q"]
    B, n, H, D = q.shape
    Hkv, dev = case["Hkv"], q.device
    table = st["table"].long()
    # [B, pages, H_kv, P, ...] -> [B, H_kv, L, D]
    k, v = (_values(st["codes"][table, i], st["scales"][table, i]).transpose(1, 2).flatten(2, 3) for i in (0, 1))
    L = k.shape[2]
    s = torch.matmul(q.float().unflatten(2, (Hkv, H // Hkv)).permute(0, 2, 3, 1, 4).flatten(2, 3), k.transpose(2, 3)) * D**-0.5
    s = s.unflatten(2, (H // Hkv, n))
    pos = st["lens"].long()[:, None] - n + torch.arange(n, device=dev)
    j = torch.arange(L, device=dev)
    seen = j <= pos[..., None]
    if case["window"] >= 0:
        seen &= j >= pos[..., None] - case["window"]
    s.masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (H // Hkv, n)) / torch.where(l == 0, 1.0, l)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(q.dtype)
    return [o, (m + l.log()).squeeze(-1).flatten(1, 2)]


def _rotate(st):
    case = st["case"]
    a = st["pos"][:, st["axes"].long()].double() * st["inv_freq"]
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    s = -s if case["inverse"] else s

    def turn(x):
        x = x.float()
        x = x.unflatten(-1, (-1, 2)) if case["interleaved"] else x.unflatten(-1, (2, -1)).transpose(-1, -2)
        y = torch.stack((x[..., 0] * c - x[..., 1] * s, x[..., 1] * c + x[..., 0] * s), -1)
        return (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2).to(DT[case["dtype"]])

    return [turn(st["q"]), turn(st["k"])]


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"write": _write, "read": _read, "attend": _attend, "rotate": _rotate}[op](st)
    import attention_forward_fwd_gb300 as fa

    if op == "write":
        fa.kv4_write(st["k"], st["v"], st["codes"], st["scales"], st["table"], st["lens"], cu_seqlens=st.get("cu"), max_seqlen=st.get("most"), k_out=st["k_out"], v_out=st["v_out"])
        return [x for x in (st["codes"], st["scales"], st["k_out"], st["v_out"]) if x is not None]
    if op == "read":
        return list(fa.kv4_read(st["codes"], st["scales"], st["table"], st["lens"], cu_seqlens=st["cu"], max_seqlen=st["most"], total=st["total"], dtype=DT[st["case"]["dtype"]]))
    if op == "attend":
        return list(fa.kv4_attention(st["q"], st["codes"], st["scales"], st["table"], st["lens"], window_left=st["case"]["window"]))
    return list(fa.rotary(st["q"], st["pos"], st["inv_freq"], st["axes"], k=st["k"], interleaved=st["case"]["interleaved"], inverse=st["case"]["inverse"]))


def work(case):
    D, Hkv = case["D"], case["Hkv"]
    if case["op"] == "rotate":
        x = case["T"] * (case["H"] + Hkv) * D
        return {"bytes": 4 * x + 4 * case["T"] * case["axes"], "flops": 3 * x}
    lens, rows = _lengths(case)
    row4 = Hkv * (D // 2 + D // 16)  # K or V of a token, quantised
    T = int(rows.sum())
    if case["op"] == "write":
        return {"bytes": 2 * T * (row4 + Hkv * D * (4 if case["values"] else 2)), "flops": 2 * T * Hkv * D * 3}
    if case["op"] == "read":
        return {"bytes": 2 * T * (row4 + Hkv * D * 2), "flops": 2 * T * Hkv * D}
    n, H, w = case["n"], case["H"], case["window"]
    pairs = tokens = 0
    for m in lens.tolist():
        pos = np.maximum(np.arange(m - n, m), -1)
        first = np.maximum(pos - w, 0) if w >= 0 else np.zeros_like(pos)
        pairs += int((pos + 1 - first).sum())
        tokens += int(pos[-1] + 1 - first[0])
    return {"bytes": 2 * tokens * row4 + case["B"] * n * H * (4 * D + 4), "flops": 4 * pairs * H * D}


# ---------------------------------------------------------------- the definition, in 64 bits


def _row_values(codes, scales):
    """What rows of codes [..., D / 2] (uint8) and scales stand for, in 64 bits, element by element of the definition."""
    D, N = codes.shape[-1] * 2, scales.shape[-1]
    d = torch.arange(D, device=codes.device)
    word, bit = (d % 32) // 4 * N + d // 32, 4 * (d % 4)
    n = (codes[..., 2 * word + bit // 8].long() >> (bit % 8)) & 15
    return (n - 8).double() * scales.double()[..., d // 32]


def exact(case, seed):
    st = prepare(case, seed)
    dev = "cuda"
    if case["op"] == "rotate":
        D, half = case["D"], case["D"] // 2
        f = torch.arange(half, device=dev)
        at = torch.stack((2 * f, 2 * f + 1) if case["interleaved"] else (f, f + half))
        sign = -1.0 if case["inverse"] else 1.0
        out = []
        for x in (st["q"], st["k"]):
            y = torch.empty(x.shape, dtype=torch.float64, device=dev)
            for i in range(0, x.shape[0], 4096):
                z = torch.complex(x[i : i + 4096][..., at[0]].double(), x[i : i + 4096][..., at[1]].double())
                angle = sign * st["inv_freq"] * st["pos"][i : i + 4096].double()[:, st["axes"].long()]
                z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
                y[i : i + 4096, :, at[0]], y[i : i + 4096, :, at[1]] = z.real, z.imag
            out.append(y)
        return out
    lens, rows = _lengths(case)
    P, table = case["P"], st["table"].long()
    if case["op"] == "read":
        k, v = [], []
        for b, m in enumerate(lens.tolist()):
            j = torch.arange(m, device=dev)
            page = table[b, j // P]
            k.append(_row_values(st["codes"][page, 0, :, j % P], st["scales"][page, 0, :, j % P]))
            v.append(_row_values(st["codes"][page, 1, :, j % P], st["scales"][page, 1, :, j % P]))
        return [torch.cat(k), torch.cat(v)]
    if case["op"] == "write":
        if case["values"] is False:
            return [None, _exact_scales(case, st, lens, rows)]
        return [None, _exact_scales(case, st, lens, rows)] + [_exact_values(x) for x in (st["k"], st["v"])]
    B, n, H, D, Hkv, w = case["B"], case["n"], case["H"], case["D"], case["Hkv"], case["window"]
    o, lse = torch.zeros(B, n, H, D, dtype=torch.float64, device=dev), torch.full((B, H, n), -math.inf, dtype=torch.float64, device=dev)
    for b, m in enumerate(lens.tolist()):
        j = torch.arange(m, device=dev)
        page = table[b, j // P]
        for h in range(Hkv):
            if not m:
                continue
            k, v = (_row_values(st["codes"][page, i, h, j % P], st["scales"][page, i, h, j % P]) for i in (0, 1))
            for i in range(0, n, 256):
                at = torch.arange(i, min(n, i + 256), device=dev)
                pos = m - n + at
                hid = (j[None] > pos[:, None]) | ((j[None] < pos[:, None] - w) if w >= 0 else False)
                for hq in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                    z = (st["q"][b, at, hq].double() @ k.T / math.sqrt(D)).masked_fill(hid, -math.inf)
                    lse[b, hq, at] = torch.logsumexp(z, -1)
                    o[b, at, hq] = torch.nan_to_num(torch.softmax(z, -1)) @ v
    return [o, lse]


def _exact_group(x):
    """(scale, x) of the groups of rows [..., D], in 64 bits; the scale as bf16 holds it."""
    x = x.double().unflatten(-1, (-1, 32))
    first = (x.abs() == x.abs().amax(-1, keepdim=True)).double().argmax(-1, keepdim=True)
    return (-x.gather(-1, first) / 8).bfloat16().double(), x


def _exact_values(x):
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    flat, to = x.flatten(0, -3), out.flatten(0, -3)
    for i in range(0, flat.shape[0], 4096):
        s, y = _exact_group(flat[i : i + 4096])
        to[i : i + 4096] = ((y / torch.where(s == 0, 1.0, s)).round().clamp(-8, 7) * s).flatten(-2)
    return out


def _exact_scales(case, st, lens, rows):
    scales = st["scales"].double()
    for i, x in enumerate((st["k"], st["v"])):
        flat, at = x.flatten(0, -3), 0
        for b, (m, r) in enumerate(zip(lens.tolist(), rows.tolist())):
            j = torch.arange(m - r, m, device=x.device)
            s = _exact_group(flat[at : at + r])[0].squeeze(-1)
            scales[st["table"][b, j // case["P"]].long(), i, :, j % case["P"]] = s + 0.0
            at += r
    return scales
