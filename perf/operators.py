"""Measured cases of the windowed attention, its single-token forms and the 4-bit KV cache.

Every case is one pass through one operator: forward over a prompt ("prefill"), forward and backward ("train"), one
query per sequence over a bf16 cache ("decode") or a 4-bit cache ("decode4"), and rows quantised into a 4-bit cache
and read back ("write").  ``run`` computes them in plain torch, or with the package where ``own`` is true.

Key j is visible to query i, at position p = i + Nk - Nq, iff j <= p and (j > p - window or j < sinks); a decode
query sits at p = length - 1.  Query head h reads key/value head h // (H // Hkv).

4-bit cache: the d channels of a row form groups of 32.  A group has step = bf16(max|x| / 7) and codes
clamp(round_half_even(x / step), -7, 7) + 8, and stands for step * (code - 8).  Group g's channels are cut into units
(8 channels for K, 4 for V); unit u of group g is stored at unit position u * (d / 32) + g of the row, a unit's first
channel in its lowest nibble.
"""
import math

import torch

own = False

GROUP = 32
K_UNIT, V_UNIT = 8, 4


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a few short prompts of odd lengths behind a cached prefix: latency
        dict(name="prefill_short", kind="prefill", B=3, H=8, Hkv=2, Nq=77, Nk=333, d=64, window=100, sinks=3),
        # one chunk of a long prompt against the prefix that is already cached
        dict(name="prefill_chunk", kind="prefill", B=1, H=32, Hkv=8, Nq=512, Nk=8192, d=128, window=1024, sinks=4),
        # a long document in one go
        dict(name="prefill_long", kind="prefill", B=1, H=16, Hkv=16, Nq=65536, Nk=65536, d=128, window=4096, sinks=4),
        # a training step of a small model
        dict(name="train_small", kind="train", B=2, H=8, Hkv=8, Nq=1024, Nk=1024, d=64, window=256, sinks=0),
        # a training step with shared key/value heads
        dict(name="train_shared", kind="train", B=4, H=16, Hkv=4, Nq=4096, Nk=4096, d=128, window=1024, sinks=4),
        # a long training sequence of odd length and window
        dict(name="train_odd", kind="train", B=1, H=16, Hkv=16, Nq=16301, Nk=16301, d=64, window=777, sinks=5),
        # one user's next token: latency
        dict(name="decode_one", kind="decode", B=1, H=32, Hkv=32, Lmax=8192, lmin=8000, d=128, window=1024, sinks=4),
        # the next token of a full batch, ragged lengths
        dict(name="decode_batch", kind="decode", B=32, H=32, Hkv=8, Lmax=8192, lmin=1024, d=128, window=4096, sinks=4),
        # each sequence's newest token enters the cache
        dict(name="write_token", kind="write", B=32, Hkv=8, T=1, Lmax=8192, d=128),
        # prompts of ragged lengths enter the cache
        dict(name="write_prompt", kind="write", B=4, Hkv=8, T=4096, Lmax=8192, d=128),
        # one long conversation's next token, the whole cache visible
        dict(name="decode4_one", kind="decode4", B=1, H=16, Hkv=4, Lmax=65536, lmin=65000, d=128, window=65536, sinks=0),
        # the next token of a full batch, the whole cache visible
        dict(name="decode4_batch", kind="decode4", B=32, H=32, Hkv=8, Lmax=8192, lmin=1024, d=128, window=8192,
             sinks=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prefill", "train", "decode", "decode4", "write"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 16])
    G = rng.choice([1, 1, 2, 4, 5, 8, 12])
    H = Hkv * G
    if kind in ("prefill", "train"):
        top = 65536 if kind == "prefill" else 16384
        # a training sequence of one token, or a window of one, has gradients that are zero by cancellation
        least = 64 if kind == "train" else 1
        N = _log(rng, least, top)
        Nq = N if kind == "train" or rng.random() < 0.5 else _log(rng, 1, N)
        window = _log(rng, 1 + least // 8, 4096)
        # within the largest listed case's work: pairs x channels
        B = _log(rng, 1, 16)
        most = 16 * 65536 * 4096 * 128 if kind == "prefill" else 4 * 16 * 4096 * 1024 * 128
        while B > 1 and B * H * Nq * min(window + 128, N) * d > most:
            B //= 2
        while B * H * Nq * min(window + 128, N) * d > most and window > 16:
            window //= 2
        return dict(kind=kind, B=B, H=H, Hkv=Hkv, Nq=Nq, Nk=N, d=d, window=window,
                    sinks=rng.choice([0, 1, 4, 5, 64, 130]))
    Lmax = _log(rng, 1, 65536 if kind == "decode4" else 8192)
    B = _log(rng, 1, 32)
    while B > 1 and B * Hkv * Lmax * d > 32 * 8 * 8192 * 128:
        B //= 2
    if kind == "write":
        return dict(kind=kind, B=B, Hkv=Hkv, T=rng.choice([1, _log(rng, 1, min(Lmax, 4096))]), Lmax=Lmax, d=d)
    window = rng.choice([Lmax, _log(rng, 1, Lmax)])
    return dict(kind=kind, B=B, H=H, Hkv=Hkv, Lmax=Lmax, lmin=_log(rng, 1, Lmax), d=d, window=window,
                sinks=rng.choice([0, 1, 4, 7, 64]))


# ------------------------------------------------------------------------------------------------ work
def _visible(p, window, sinks):
    """How many keys a query at position p sees."""
    if p < 0:
        return 0
    lo = max(0, p - window + 1)
    return p + 1 - lo + min(sinks, lo)


def _pairs(c):
    off = c["Nk"] - c["Nq"]
    return sum(_visible(i + off, c["window"], c["sinks"]) for i in range(c["Nq"]))


def work(case):
    c = case
    d = c["d"]
    if c["kind"] in ("prefill", "train"):
        pairs = _pairs(c) * c["B"] * c["H"]
        rows, kv = c["B"] * c["H"] * c["Nq"], c["B"] * c["Hkv"] * c["Nk"]
        fwd_bytes = rows * (2 * d * 2 + 4) + kv * 2 * d * 2
        if c["kind"] == "prefill":
            return {"bytes": fwd_bytes, "flops": 4 * d * pairs}
        # q, dO, o, lse, dq once each; k, v, dk, dv once each (the forward's o and lse stay in the output)
        return {"bytes": rows * (4 * d * 2 + 4) + kv * 4 * d * 2, "flops": 14 * d * pairs}
    if c["kind"] == "write":
        # the numbers of new rows are uniform in [max(1, T / 2), T]
        rows = c["B"] * c["Hkv"] * (max(1, c["T"] // 2) + c["T"])
        packed = d // 2 + 2 * (d // GROUP)
        return {"bytes": rows * (2 * d * 2 + packed), "flops": 4 * d * rows}
    # lengths are uniform in [lmin, Lmax]
    mean = sum(_visible(L - 1, c["window"], c["sinks"]) for L in range(c["lmin"], c["Lmax"] + 1)) \
        / (c["Lmax"] - c["lmin"] + 1)
    row = 2 * d if c["kind"] == "decode" else d // 2 + 2 * (d // GROUP)
    keys = mean * c["B"]
    return {"bytes": int(keys * c["Hkv"] * 2 * row + c["B"] * c["H"] * (2 * d * 2 + 4)),
            "flops": int(4 * d * keys * c["H"])}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _outliers(k):
    """Keys have a few large channels, the same for every token."""
    k[..., 3::48] *= 4
    return k


def _inputs(c, seed):
    g = _gen(seed)
    d = c["d"]
    if c["kind"] in ("prefill", "train"):
        t = {"q": _randn(g, c["B"], c["H"], c["Nq"], d), "k": _randn(g, c["B"], c["Hkv"], c["Nk"], d),
             "v": _randn(g, c["B"], c["Hkv"], c["Nk"], d)}
        if c["kind"] == "train":
            t["do"] = _randn(g, c["B"], c["H"], c["Nq"], d)
        return t
    B, Hkv = c["B"], c["Hkv"]
    if c["kind"] == "write":
        T, Lmax = c["T"], c["Lmax"]
        lens = torch.randint(max(1, T // 2), T + 1, (B,), generator=g, device="cuda", dtype=torch.int64)
        starts = (torch.rand(B, generator=g, device="cuda", dtype=torch.float64) * (Lmax - lens + 1)).long()
        return {"k": _outliers(_randn(g, B, Hkv, T, d)), "v": _randn(g, B, Hkv, T, d), "starts": starts.int(),
                "lens": lens.int()}
    lens = torch.randint(c["lmin"], c["Lmax"] + 1, (B,), generator=g, device="cuda", dtype=torch.int64).int()
    return {"q": _randn(g, B, c["H"], 1, d), "k": _outliers(_randn(g, B, Hkv, c["Lmax"], d)),
            "v": _randn(g, B, Hkv, c["Lmax"], d), "lens": lens}


def _order(d, unit):
    """channel -> nibble position in the stored row."""
    ch = torch.arange(d, device="cuda")
    grp, inner = ch // GROUP, ch % GROUP
    return (inner // unit * (d // GROUP) + grp) * unit + inner % unit


def _pack(x, unit):
    """bf16 rows [..., d] -> (codes [..., d / 2] uint8, steps [..., d / 32] bf16)."""
    d = x.shape[-1]
    f = x.float().unflatten(-1, (d // GROUP, GROUP))
    steps = (f.abs().amax(-1) / 7).to(torch.bfloat16)
    s = steps.float().unsqueeze(-1)
    n = torch.where(s > 0, torch.round(f / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(f))
    c = (n.clamp(-7, 7) + 8).to(torch.uint8).flatten(-2)
    stored = torch.empty_like(c)
    stored[..., _order(d, unit)] = c
    return (stored[..., 0::2] | (stored[..., 1::2] << 4)).contiguous(), steps.contiguous()


def _unpack(codes, steps, unit):
    """(codes, steps) -> float32 rows [..., d]."""
    d = 2 * codes.shape[-1]
    stored = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    c = stored[..., _order(d, unit)].float() - 8
    return (c.unflatten(-1, (d // GROUP, GROUP)) * steps.float().unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    c, t = case, _inputs(case, seed)
    d = c["d"]
    st = {"case": c, "scale": 1 / math.sqrt(d), "t": t}
    if c["kind"] == "write":
        rows = (c["B"], c["Hkv"], c["Lmax"])
        st["cache"] = tuple(torch.zeros(*rows, n, dtype=ty, device="cuda") for n, ty in
                            ((d // 2, torch.uint8), (d // GROUP, torch.bfloat16)) * 2)
        st["out"] = (torch.zeros_like(t["k"]), torch.zeros_like(t["v"]))
    elif c["kind"] == "decode4":
        kc, ks = _pack(t.pop("k"), K_UNIT)
        vc, vs = _pack(t.pop("v"), V_UNIT)
        st["cache"] = (kc, ks, vc, vs)
    if c["kind"] in ("decode", "decode4"):
        st["longest"] = int(t["lens"].max())
    if own:
        import io_aware_exact_32_b200 as fa
        st["fa"] = fa
        if c["kind"] in ("decode", "decode4"):
            B, H = c["B"], c["H"]
            n = fa.fa_decode_window_workspace_size(B, H, c["Hkv"], c["Lmax"], d, c["window"], c["sinks"])
            st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
            st["o"] = torch.empty(B, H, 1, d, dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty(B, H, dtype=torch.float32, device="cuda")
        elif c["kind"] == "train":
            n = fa.fa_bwd_window_workspace_size(c["B"], c["H"], c["Hkv"], c["Nq"], c["Nk"], d, c["window"], c["sinks"])
            st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        if c["kind"] in ("write", "decode4"):
            st["kv4"] = fa.KV4Cache(*st["cache"])
    return st


# ------------------------------------------------------------------------------------------------ the package's operators
def _run_own(st):
    fa, c, t = st["fa"], st["case"], st["t"]
    w = (c.get("window"), c.get("sinks"))
    if c["kind"] == "prefill":
        return fa.attention_forward_window(t["q"], t["k"], t["v"], *w, scale=st["scale"])
    if c["kind"] == "train":
        o, lse = fa.attention_forward_window(t["q"], t["k"], t["v"], *w, scale=st["scale"])
        return (o, lse) + tuple(fa.attention_backward_window(t["q"], t["k"], t["v"], o, lse, t["do"], *w,
                                                             scale=st["scale"], workspace=st["ws"]))
    if c["kind"] == "write":
        fa.fa_kv4_write(t["k"], t["v"], st["kv4"], t["starts"], t["lens"])
        fa.fa_kv4_read(st["kv4"], st["out"][0], st["out"][1], t["starts"], t["lens"])
        return st["out"]
    if c["kind"] == "decode":
        fa.fa_decode_window(t["q"], t["k"], t["v"], t["lens"], *w, st["o"], st["lse"], st["ws"], scale=st["scale"])
    else:
        fa.fa_decode_kv4(t["q"], st["kv4"], t["lens"], *w, st["o"], st["lse"], st["ws"], scale=st["scale"])
    return st["o"], st["lse"]


# ------------------------------------------------------------------------------------------------ plain form
def _chunks(c, rows=1024):
    """Query chunks with the keys they can see: (i0, i1, number of sink keys apart, first and last window key)."""
    off = c["Nk"] - c["Nq"]
    for i0 in range(0, c["Nq"], rows):
        i1 = min(i0 + rows, c["Nq"])
        lo = min(max(0, i0 + off - c["window"] + 1), c["Nk"])
        hi = max(lo, i1 + off)
        yield i0, i1, min(c["sinks"], lo), lo, hi


def _mask(c, i0, i1, ns, lo, hi):
    off = c["Nk"] - c["Nq"]
    pos = (torch.arange(i0, i1, device="cuda") + off).unsqueeze(1)
    keys = torch.cat((torch.arange(ns, device="cuda"), torch.arange(lo, hi, device="cuda"))).unsqueeze(0)
    return (keys <= pos) & ((keys > pos - c["window"]) | (keys < c["sinks"]))


def _softmax(s, mask):
    s = torch.where(mask, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(s - base)
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l > 0, l, torch.ones_like(l))
    return p, (base + torch.log(l)).squeeze(-1)


def _attend_plain(st, train):
    c, t, scale = st["case"], st["t"], st["scale"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    q = t["q"].float().view(B, Hkv, H // Hkv, c["Nq"], d)
    k, v = t["k"].float(), t["v"].float()
    o, lse = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
    if train:
        do = t["do"].float().view_as(q)
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    rows = max(64, min(1024, (1 << 29) // max(1, B * H * min(c["Nk"], c["window"] + c["sinks"] + 1024))))
    for i0, i1, ns, lo, hi in _chunks(c, rows):
        if ns + hi - lo == 0:
            o[..., i0:i1, :] = 0
            lse[..., i0:i1] = -math.inf
            continue
        kc = torch.cat((k[:, :, :ns], k[:, :, lo:hi]), 2).unsqueeze(2)
        vc = torch.cat((v[:, :, :ns], v[:, :, lo:hi]), 2).unsqueeze(2)
        qc = q[..., i0:i1, :]
        p, l = _softmax(qc @ kc.transpose(-1, -2) * scale, _mask(c, i0, i1, ns, lo, hi))
        oc = p @ vc
        o[..., i0:i1, :], lse[..., i0:i1] = oc, l
        if train:
            doc = do[..., i0:i1, :]
            dp = doc @ vc.transpose(-1, -2)
            ds = p * (dp - (doc * oc).sum(-1, keepdim=True))
            dq[..., i0:i1, :] = ds @ kc * scale
            gk = (ds.transpose(-1, -2) @ qc).sum(2) * scale
            gv = (p.transpose(-1, -2) @ doc).sum(2)
            for grad, part in ((dk, gk), (dv, gv)):
                grad[:, :, :ns] += part[:, :, :ns]
                grad[:, :, lo:hi] += part[:, :, ns:]
    out = (o.to(torch.bfloat16).view(B, H, c["Nq"], d), lse.view(B, H, c["Nq"]))
    if train:
        out += (dq.to(torch.bfloat16).view(B, H, c["Nq"], d), dk.to(torch.bfloat16), dv.to(torch.bfloat16))
    return out


def _decode_plain(st):
    c, t = st["case"], st["t"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    n = st["longest"]
    if c["kind"] == "decode":
        k, v = t["k"][:, :, :n].float(), t["v"][:, :, :n].float()
    else:
        kc, ks, vc, vs = (x[:, :, :n] for x in st["cache"])
        k, v = _unpack(kc, ks, K_UNIT), _unpack(vc, vs, V_UNIT)
    keys = torch.arange(n, device="cuda").unsqueeze(0)
    pos = (t["lens"].long() - 1).unsqueeze(1)
    mask = (keys <= pos) & ((keys > pos - c["window"]) | (keys < c["sinks"]))
    q = t["q"].float().view(B, Hkv, H // Hkv, d)
    p, lse = _softmax(q @ k.transpose(-1, -2) * st["scale"], mask[:, None, None])
    return (p @ v).to(torch.bfloat16).view(B, H, 1, d), lse.view(B, H)


def _write_plain(st):
    c, t = st["case"], st["t"]
    kc, ks, vc, vs = st["cache"]
    step = torch.arange(c["T"], device="cuda").unsqueeze(0)
    b, r = ((step < t["lens"].unsqueeze(1)).nonzero(as_tuple=True))
    at = t["starts"].long()[b] + r
    for x, codes, steps, unit, out in ((t["k"], kc, ks, K_UNIT, st["out"][0]), (t["v"], vc, vs, V_UNIT, st["out"][1])):
        cc, ss = _pack(x, unit)
        codes[b, :, at], steps[b, :, at] = cc[b, :, r], ss[b, :, r]
        out[b, :, r] = _unpack(codes[b, :, at], steps[b, :, at], unit).to(torch.bfloat16)
    return st["out"]


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind in ("prefill", "train"):
        return _attend_plain(state, kind == "train")
    if kind == "write":
        return _write_plain(state)
    return _decode_plain(state)


# ------------------------------------------------------------------------------------------------ definition in 64 bits
def _values64(x):
    """What a 4-bit row of bf16 x stands for, in float64."""
    g = x.double().reshape(*x.shape[:-1], -1, GROUP)
    step = (g.abs().max(dim=-1, keepdim=True).values / 7).to(torch.bfloat16).double()
    n = torch.where(step == 0, 0.0, torch.round(g / step))
    return (torch.minimum(torch.maximum(n, torch.full_like(n, -7.0)), torch.full_like(n, 7.0)) * step).reshape(x.shape)


def exact(case, seed):
    c = case
    d, scale = c["d"], 1 / math.sqrt(c["d"])
    t = _inputs(c, seed)
    if c["kind"] == "write":
        live = torch.arange(c["T"], device="cuda").view(1, 1, -1, 1) < t["lens"].view(-1, 1, 1, 1)
        return tuple(torch.where(live, _values64(t[n]), 0.0) for n in ("k", "v"))
    G = c["H"] // c["Hkv"]
    if c["kind"] in ("decode", "decode4"):
        q = t["q"].double()
        o = torch.zeros_like(q)
        lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device="cuda")
        for b, L in enumerate(t["lens"].tolist()):
            idx = torch.tensor([j for j in range(L) if j >= L - c["window"] or j < c["sinks"]], device="cuda")
            k, v = t["k"][b][:, idx], t["v"][b][:, idx]
            k, v = (k.double(), v.double()) if c["kind"] == "decode" else (_values64(k), _values64(v))
            for h in range(c["H"]):
                x = scale * (k[h // G] @ q[b, h, 0])
                lse[b, h] = torch.logsumexp(x, 0)
                o[b, h, 0] = torch.exp(x - lse[b, h]) @ v[h // G]
        return o, lse
    if 56 * d * _pairs(c) * c["B"] * c["H"] > 2e14:
        return None
    off = c["Nk"] - c["Nq"]
    o = torch.zeros(c["B"], c["H"], c["Nq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["H"], c["Nq"]), -math.inf, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(o)
    dk = torch.zeros(c["B"], c["Hkv"], c["Nk"], d, dtype=torch.float64, device="cuda")
    dv = torch.zeros_like(dk)
    span = 2048
    for b in range(c["B"]):
        for h in range(c["H"]):
            K, V = t["k"][b, h // G].double(), t["v"][b, h // G].double()
            for r0 in range(max(0, -off), c["Nq"], span):
                r1 = min(r0 + span, c["Nq"])
                p = torch.arange(r0 + off, r1 + off, device="cuda")
                first = max(0, r0 + off - c["window"] + 1)
                idx = torch.arange(r1 + off, device="cuda")
                idx = idx[(idx >= first) | (idx < c["sinks"])]
                hide = (idx[None] > p[:, None]) | ((p[:, None] - idx[None] >= c["window"]) & (idx[None] >= c["sinks"]))
                Q = t["q"][b, h, r0:r1].double()
                x = (scale * (Q @ K[idx].T)).masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, 1)
                w = torch.exp(x - z[:, None])
                out = w @ V[idx]
                o[b, h, r0:r1], lse[b, h, r0:r1] = out, z
                if c["kind"] == "train":
                    g = t["do"][b, h, r0:r1].double()
                    ds = w * (g @ V[idx].T - (g * out).sum(1, keepdim=True)) * scale
                    dq[b, h, r0:r1] = ds @ K[idx]
                    dk[b, h // G].index_add_(0, idx, ds.T @ Q)
                    dv[b, h // G].index_add_(0, idx, w.T @ g)
    return (o, lse, dq, dk, dv) if c["kind"] == "train" else (o, lse)
