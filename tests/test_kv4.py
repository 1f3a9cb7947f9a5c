"""The 4-bit KV cache (write, read, single-token attention over it) and the windowed single-token attention over a bf16
cache: definitions and refusals (CPU), kernels against the definitions (GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gpu_common as gc
import io_aware_exact_32_b200 as fa
from oracle import attention as A
from oracle import kv4 as Q
from oracle import windowed as OW

NULL = ctypes.c_void_p(0)
A16 = ctypes.c_void_p(0x10000)      # fake, aligned, never dereferenced
MIS = ctypes.c_void_p(0x10008)


# ------------------------------------------------------------------------------------------------ the definitions
def test_quantise_by_hand():
    x = np.zeros(32)
    x[:6] = [7.0, -7.0, 0.5, 1.5, 2.5, -3.4]   # step 1: ties go to even
    c, s = Q.quantise(x)
    assert Q.bf16_value(s).tolist() == [1.0]
    assert (c[:6].astype(int) - 8).tolist() == [7, -7, 0, 2, 2, -3] and np.all(c[6:] == 8)
    assert Q.values(c, s)[:6].tolist() == [7, -7, 0, 2, 2, -3]
    c, s = Q.quantise(np.zeros(64))
    assert np.all(c == 8) and np.all(Q.values(c, s) == 0)
    x[3] = np.nan
    c, s = Q.quantise(x)
    assert np.all(np.isnan(Q.values(c, s)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
def test_pack_round_trip_and_order(d, which):
    rng = np.random.default_rng(d)
    c = rng.integers(0, 16, (3, d)).astype(np.uint8)
    p = Q.pack(c, which)
    assert p.shape == (3, d // 2) and np.array_equal(Q.unpack(p, which), c)
    # the second unit of group 0 follows the first units of all groups
    u = Q.UNIT[which]
    at = (d // 32) * u
    assert (p[0, at // 2] & 15) == c[0, u] and (p[0, 0] & 15) == c[0, 0]


def test_quantisation_error_is_half_a_step():
    x = torch.randn(50, 128, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).double().numpy()
    c, s = Q.quantise(x)
    err = np.abs(Q.values(c, s) - x).reshape(50, 4, 32)
    # half a step, and at the clamp 7 |amax / 7 - step| <= 7 * 2^-8 step besides
    assert np.all(err <= Q.bf16_value(s)[..., None] * 0.5 * (1 + 1e-9))


def test_decode_definition_is_plain_decode_for_a_window_over_everything():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((2, 3, 8)), rng.standard_normal((2, 3, 9, 8)), rng.standard_normal((2, 3, 9, 8))
    L = np.array([9, 4])
    r = OW.decode(q, k, v, L, 9, 0, 0.4)
    o, lse = A.decode_forward(q, k, v, L, 0.4)
    assert np.allclose(r["o"], o, atol=1e-13) and np.allclose(r["lse"], lse, atol=1e-13)


# ------------------------------------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def L():
    return fa.lib()


def dec(L, q4, q=A16, seq=A16, ws=A16, ws_bytes=1 << 30, steps=A16, k=A16, Lmax=4096, window=100, sinks=4, B=2, H=4,
        Hkv=2, d=128, scale=0.088):
    if q4:
        return L.fa_decode_kv4(q, k, steps, A16, A16, seq, Lmax, window, sinks, A16, A16, B, H, Hkv, d, scale, ws,
                               ws_bytes, NULL)
    return L.fa_decode_window(q, k, A16, seq, Lmax, window, sinks, A16, A16, B, H, Hkv, d, scale, ws, ws_bytes, NULL)


@pytest.mark.parametrize("q4", [False, True])
def test_decode_refusals(L, q4):
    assert dec(L, q4, d=96) == 2
    assert dec(L, q4, Hkv=3) == 1
    assert dec(L, q4, Hkv=0) == 1
    assert dec(L, q4, window=0) == 1
    assert dec(L, q4, sinks=-1) == 1
    assert dec(L, q4, Lmax=0) == 1
    assert dec(L, q4, Lmax=(1 << 24) + 1) == 2
    assert dec(L, q4, scale=float("nan")) == 1
    assert dec(L, q4, q=NULL) == 1
    assert dec(L, q4, k=NULL) == 1
    assert dec(L, q4, k=MIS) == 3
    assert dec(L, q4, seq=NULL) == 1
    assert dec(L, q4, seq=ctypes.c_void_p(0x10002)) == 3
    assert dec(L, q4, ws=NULL) == 4
    assert dec(L, q4, ws_bytes=8) == 4
    assert dec(L, q4, ws=ctypes.c_void_p(0x10010)) == 3
    assert dec(L, q4, B=0) == 0
    if q4:
        assert dec(L, q4, steps=NULL) == 1
        assert dec(L, q4, steps=MIS) == 3


def test_decode_workspace(L):
    f = L.fa_decode_window_workspace_size
    up = lambda rows: (rows * 130 * 4 + 255) // 256 * 256                    # noqa: E731  d = 128: fp32 O, m, l a row
    assert f(1, 4, 2, 4096, 128, 64, 0) == up(2 * 2 * 8)                     # 4 bits: a step a head, two slots of 8 rows
    assert f(1, 40, 1, 4096, 128, 250, 10) == up(2 * 15 * 8)                 # three steps of 128 for each of five blocks of heads
    assert f(64, 64, 64, 1 << 20, 128, 1 << 24, 4) == up(64 * 64 * 256)      # bf16: no more than 256 parts
    assert f(2, 4, 3, 4096, 128, 100, 4) == 0
    assert f(2, 4, 2, 0, 128, 100, 4) == 0
    assert f(0, 4, 2, 4096, 128, 100, 4) == 0
    assert f(64, 64, 64, 1 << 24, 128, 1 << 24, 4) > 0
    assert f(1 << 15, 64, 64, 1 << 24, 128, 1 << 24, 4) == 0                 # 2^38 steps are not counted


@pytest.mark.parametrize("name", ["fa_kv4_write", "fa_kv4_read"])
def test_rows_refusals(L, name):
    def call(null=None, mis=None, starts=A16, lens=NULL, B=1, Hkv=2, T=3, Lmax=64, d=128):
        args = [A16] * 6
        if null is not None:
            args[null] = NULL
        if mis is not None:
            args[mis] = MIS
        return getattr(L, name)(*args, starts, lens, B, Hkv, T, Lmax, d, NULL)

    for i in range(6):
        assert call(null=i) == 1
        assert call(mis=i) == 3
    assert call(d=32) == 2
    assert call(T=-1) == 1
    assert call(Lmax=0) == 1
    assert call(Lmax=(1 << 24) + 1) == 2
    assert call(B=-1) == 1
    assert call(starts=ctypes.c_void_p(0x10002)) == 3
    assert call(lens=ctypes.c_void_p(0x10001)) == 3
    assert call(T=0, null=0) == 0
    assert call(B=0) == 0


def test_binding_refusals():
    bf = torch.bfloat16
    cache = fa.kv4_cache(2, 2, 16, 64, "cpu")
    q = torch.zeros(2, 4, 1, 64, dtype=bf)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_kv4(q, cache, n)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fa_kv4_write(torch.zeros(2, 2, 3, 64, dtype=bf), torch.zeros(2, 2, 3, 64, dtype=bf), cache)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_window(q, torch.zeros(2, 2, 16, 64, dtype=bf), torch.zeros(2, 2, 16, 64, dtype=bf), n, 4)
    with pytest.raises(ValueError, match="head dim"):
        fa.kv4_cache(1, 1, 4, 96, "cpu")
    with pytest.raises(ValueError, match="KV4Cache"):
        fa._kv4_dims(cache[:3], torch.device("cpu"))


# ------------------------------------------------------------------------------------------------ write and read
def _bf(*shape, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * spread).to(torch.bfloat16)


def _awkward(d):
    """Rows of a [*, d] bf16 tensor: ties, zeros, lone outliers, the smallest and largest magnitudes, equal entries."""
    rows = [torch.arange(d) % 15 * 0.5 - 3.5, torch.zeros(d), torch.full((d,), -2.0), torch.full((d,), 1e-3)]
    r = torch.full((d,), 0.01)
    r[::32] = 300.0
    rows.append(r)
    rows.append(torch.linspace(-1, 1, d) * 2.0 ** -126)
    rows.append(torch.linspace(-1, 1, d) * 2.0 ** -130)      # steps below the normal range
    rows.append(torch.linspace(-1, 1, d) * 3.3e38)
    rows.append((torch.arange(d) % 2 * 2 - 1) * (torch.arange(d) % 8 + 0.5) * 7 / 7.5)
    r = torch.linspace(-1, 1, d)
    r[40 % d] = float("nan")
    rows.append(r)
    r = torch.linspace(-1, 1, d)
    r[5] = float("-inf")
    rows.append(r)
    return torch.stack(rows).to(torch.bfloat16)


def _np(t):
    return t.double().cpu().numpy()


def _bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_written_bytes_and_read_back_are_the_definitions(d):
    x = torch.cat([_awkward(d), _bf(40, d, seed=d), _bf(20, d, seed=d + 1, spread=1e-4)])
    T = x.shape[0]
    k, v = x.view(1, 1, T, d), x.flip(0).contiguous().view(1, 1, T, d)
    cache = fa.kv4_cache(1, 1, T, d, gc.DEV)
    fa.fa_kv4_write(k.to(gc.DEV), v.to(gc.DEV), cache)
    kr, vr = fa.kv4_read(cache, T)
    for which, src, codes, steps, back in (("k", k, cache.k_codes, cache.k_steps, kr), ("v", v, cache.v_codes, cache.v_steps, vr)):
        c, s = Q.quantise(_np(src))
        assert np.array_equal(codes.cpu().numpy(), Q.pack(c, which)), which
        nan = s == 0x7FFF
        assert np.array_equal(_bits(steps)[~nan], s[~nan]) and np.all(np.isnan(_np(steps)[nan])), which
        want = Q.values(c, s)
        got = _np(back)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fin = ~np.isnan(want)
        assert np.array_equal(Q.bf16_bits(got[fin]) & 0x7FFF, Q.bf16_bits(want[fin]) & 0x7FFF)   # zeros of either sign
        assert np.all(got[fin] * want[fin] >= 0)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_writes_touch_their_rows_only(d):
    """Sequences at their own positions with their own row counts; rows past a sequence's, and positions outside the
    cache, are neither written nor read."""
    B, Hkv, T, Lmax = 5, 3, 9, 21
    starts = torch.tensor([0, 12, 17, -3, 20], dtype=torch.int32)
    lens = torch.tensor([9, 4, 9, 9, 0], dtype=torch.int32)
    k, v = _bf(B, Hkv, T, d, seed=1), _bf(B, Hkv, T, d, seed=2)
    cache = fa.kv4_cache(B, Hkv, Lmax, d, gc.DEV)
    for t in cache:
        t.view(torch.uint8).fill_(0x5A)
    fa.fa_kv4_write(k.to(gc.DEV), v.to(gc.DEV), cache, starts.to(gc.DEV), lens.to(gc.DEV))
    want = {n: np.full(t.shape, 0x5A, np.uint8) if t.dtype == torch.uint8 else np.full(t.shape, 0x5A5A, np.uint16)
            for n, t in cache._asdict().items()}
    kb, vb = torch.full((B, Hkv, T, d), 3.0, dtype=torch.bfloat16), torch.full((B, Hkv, T, d), -3.0, dtype=torch.bfloat16)
    wk, wv = _np(kb), _np(vb)
    for which, src, back in (("k", k, wk), ("v", v, wv)):
        c, s = Q.quantise(_np(src))
        for b in range(B):
            for t in range(int(lens[b])):
                pos = int(starts[b]) + t
                if 0 <= pos < Lmax:
                    want[which + "_codes"][b, :, pos] = Q.pack(c[b, :, t], which)
                    want[which + "_steps"][b, :, pos] = s[b, :, t]
                    back[b, :, t] = Q.bf16_value(Q.bf16_bits(Q.values(c[b, :, t], s[b, :, t])))
    for n, t in cache._asdict().items():
        got = t.cpu().numpy() if t.dtype == torch.uint8 else _bits(t)
        assert np.array_equal(got, want[n]), n
    kb, vb = kb.to(gc.DEV), vb.to(gc.DEV)
    fa.fa_kv4_read(cache, kb, vb, starts.to(gc.DEV), lens.to(gc.DEV))
    assert np.array_equal(_np(kb), wk) and np.array_equal(_np(vb), wv)


@pytest.mark.gpu
def test_row_at_a_time_equals_all_at_once():
    B, Hkv, T, d = 3, 2, 7, 128
    k, v = _bf(B, Hkv, T, d, seed=5).to(gc.DEV), _bf(B, Hkv, T, d, seed=6).to(gc.DEV)
    a, b = fa.kv4_cache(B, Hkv, 16, d, gc.DEV), fa.kv4_cache(B, Hkv, 16, d, gc.DEV)
    starts = torch.tensor([0, 9, 4], dtype=torch.int32, device=gc.DEV)
    fa.fa_kv4_write(k, v, a, starts)
    for t in range(T):
        fa.fa_kv4_write(k[:, :, t:t + 1].contiguous(), v[:, :, t:t + 1].contiguous(), b, starts + t)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------------------------------------ single-token attention
def _within(got, ref, bound, what):
    got = _np(got)
    inf = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), inf), f"{what}: -inf pattern"
    err = np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, ref))
    assert np.all(np.isfinite(err)), f"{what}: non-finite"
    worst = np.max(err / (bound + 1e-30), initial=0.0)
    assert worst <= 1, f"{what}: {worst:.2f} x the bound"


def _case(B, H, Hkv, Lmax, d, lens, seed, vscale=None):
    q = _bf(B, H, 1, d, seed=seed)
    k, v = _bf(B, Hkv, Lmax, d, seed=seed + 1), _bf(B, Hkv, Lmax, d, seed=seed + 2)
    k[..., 3::48] *= 4
    if vscale is not None:
        v = (v.float() * vscale).to(torch.bfloat16)
    return q, k, v, torch.tensor(lens, dtype=torch.int32)


def _visible_rows(lens, Lmax, window, sinks):
    m = np.zeros((len(lens), Lmax), bool)
    for b, n in enumerate(lens):
        if n:
            m[b, :n] = OW.visible(1, n, window, sinks)[0]
    return torch.from_numpy(m)


def _run_decode(q4, case, window, sinks):
    """Kernel and definition; invisible cache rows are poisoned."""
    q, k, v, lens = case
    scale = 1 / math.sqrt(q.shape[-1])
    L = lens.tolist()
    hidden = ~_visible_rows(L, k.shape[2], window, sinks)
    qd, nd = q.to(gc.DEV), lens.to(gc.DEV)
    if q4:
        (kc, ks), (vc, vs) = Q.quantise(_np(k)), Q.quantise(_np(v))
        r = Q.decode(_np(q)[:, :, 0], kc, ks, vc, vs, L, window, sinks, scale)
        cache = fa.kv4_cache(k.shape[0], k.shape[1], k.shape[2], k.shape[3], gc.DEV)
        fa.fa_kv4_write(k.to(gc.DEV), v.to(gc.DEV), cache)
        for b in range(len(L)):
            at = hidden[b].to(gc.DEV)
            cache.k_steps[b, :, at] = float("nan")
            cache.v_steps[b, :, at] = float("nan")
        o, lse = fa.decode_kv4(qd, cache, nd, window, sinks, scale=scale)
    else:
        r = OW.decode(_np(q)[:, :, 0], _np(k), _np(v), L, window, sinks, scale)
        # the weights enter as two bf16 terms (2^-17): only the output's own rounding and fp32 remain
        r["o_bound"] = r["o_bound"] * 0 + 2.0 ** -8 * np.abs(r["o"]) + (r["o_bound"] - 2 * 2.0 ** -8 * np.abs(r["o"])) / 4
        kp, vp = k.clone(), v.clone()
        for b in range(len(L)):
            kp[b, :, hidden[b]] = float("nan")
            vp[b, :, hidden[b]] = float("nan")
        o, lse = fa.decode_window(qd, kp.to(gc.DEV), vp.to(gc.DEV), nd, window, sinks, scale=scale)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == 0
    _within(o[:, :, 0], r["o"], r["o_bound"], "O")
    _within(lse, r["lse"], r["lse_bound"], "LSE")
    return o, lse


DECODE = [  # B, H, Hkv, Lmax, d, lens, window, sinks
    (1, 1, 1, 1, 64, [1], 1, 0),
    (2, 2, 1, 1, 128, [1, 0], 4, 2),
    (3, 4, 4, 37, 128, [37, 16, 17], 64, 0),
    (3, 4, 2, 300, 64, [300, 0, 120], 100, 4),
    (2, 5, 1, 700, 128, [700, 65], 33, 3),
    (2, 8, 1, 500, 64, [499, 500], 500, 0),
    (2, 12, 1, 260, 128, [260, 255], 128, 5),       # two passes of 8 and 4 heads
    (1, 40, 2, 333, 64, [333], 200, 1),             # groups of twenty
    (4, 6, 3, 1500, 128, [1500, 1, 15, 800], 1, 0),  # each sees itself alone
    (2, 4, 2, 1000, 64, [1000, 700], 256, 300),     # many sinks
    (2, 4, 2, 1000, 128, [1000, 40], 1 << 24, 1 << 20),
    (2, 4, 2, 200, 128, [10000, -5], 50, 4),        # lengths outside the cache are clamped
]


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("B,H,Hkv,Lmax,d,lens,window,sinks", DECODE)
def test_decode(B, H, Hkv, Lmax, d, lens, window, sinks, q4):
    clamped = [min(max(n, 0), Lmax) for n in lens]
    case = _case(B, H, Hkv, Lmax, d, clamped, seed=Lmax + H)
    if clamped != lens:
        ref = _run_decode(q4, case, window, sinks)
        q, k, v, _ = case
        n = torch.tensor(lens, dtype=torch.int32, device=gc.DEV)
        cache = fa.kv4_cache(B, Hkv, Lmax, d, gc.DEV)
        fa.fa_kv4_write(k.to(gc.DEV), v.to(gc.DEV), cache)
        o, lse = fa.decode_kv4(q.to(gc.DEV), cache, n, window, sinks) if q4 else \
            fa.decode_window(q.to(gc.DEV), k.to(gc.DEV), v.to(gc.DEV), n, window, sinks)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
        return
    _run_decode(q4, case, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_ragged_batch_with_empty_sequences(q4):
    """Sequences of one chunk, several, and none."""
    lens = [700, 0, 0, 65, 64, 1, 1300, 0, 129, 5] * 5 + [0]
    _run_decode(q4, _case(len(lens), 16, 16, 1300, 64, lens, seed=11), 1200, 6)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_many_sequences(q4):
    """Short ragged sequences."""
    lens = [(37 * i) % 150 for i in range(101)]
    _run_decode(q4, _case(101, 2, 1, 150, 64, lens, seed=17), 100, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_one_long_sequence(q4):
    """One unit in many chunks."""
    _run_decode(q4, _case(1, 3, 1, 20000, 128, [19999], seed=18), 1 << 20, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_same_bits_every_time(q4):
    case = _case(7, 8, 2, 900, 128, [900, 3, 450, 899, 0, 77, 64], seed=19)
    a, b = _run_decode(q4, case, 800, 4), _run_decode(q4, case, 800, 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** -18, 2.0 ** 12, 2.0 ** 60])
def test_values_of_any_size(scale):
    """The weights times the steps stay in fp16's range whatever V's size."""
    _run_decode(True, _case(2, 4, 2, 300, 128, [300, 190], seed=12, vscale=scale), 280, 4)


@pytest.mark.gpu
def test_values_whose_size_changes_along_the_cache():
    """V grows by 2^24 along the sequence, and shrinks again: the running bound moves, the early sums fade."""
    Lmax = 1024
    ramp = 2.0 ** (torch.arange(Lmax).float() / Lmax * 24).floor()
    for r in (ramp, ramp.flip(0)):
        _run_decode(True, _case(1, 4, 2, Lmax, 128, [Lmax], seed=13, vscale=r.view(1, 1, Lmax, 1)), Lmax, 0)


@pytest.mark.gpu
def test_queries_of_any_size():
    q, k, v, n = _case(1, 4, 2, 200, 64, [200], seed=14)
    for f in (2.0 ** -30, 2.0 ** 5):
        _run_decode(True, ((q.float() * f).to(torch.bfloat16), k, v, n), 200, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_a_visible_nan_is_not_lost(q4):
    """A NaN in a visible row of V makes the output of its heads NaN there, and leaves the other sequence alone."""
    q, k, v, n = _case(2, 4, 2, 500, 128, [500, 300], seed=15)
    ref = _run_decode(q4, (q, k, v, n), 500, 0)[0]
    v = v.clone()
    v[0, 1, 77, 5] = float("nan")
    kd, vd = k.to(gc.DEV), v.to(gc.DEV)
    if q4:
        cache = fa.kv4_cache(2, 2, 500, 128, gc.DEV)
        fa.fa_kv4_write(kd, vd, cache)
        o, _ = fa.decode_kv4(q.to(gc.DEV), cache, n.to(gc.DEV))
    else:
        o, _ = fa.decode_window(q.to(gc.DEV), kd, vd, n.to(gc.DEV), 500)
    assert torch.all(torch.isnan(o[0, 2:, 0, 5])) and torch.equal(o[1], ref[1]) and torch.equal(o[0, :2], ref[0, :2])


@pytest.mark.gpu
def test_window_decode_equals_split_decode_over_everything():
    q, k, v, n = _case(3, 4, 4, 900, 128, [900, 17, 512], seed=16)
    a = fa.decode_window(q.to(gc.DEV), k.to(gc.DEV), v.to(gc.DEV), n.to(gc.DEV), 900)
    b = fa.decode_splitkv(q.to(gc.DEV), k.to(gc.DEV), v.to(gc.DEV), n.to(gc.DEV))
    # both round an fp32 result once: a bf16 step where they fall on either side of a tie
    assert torch.all((a[0].float() - b[0].float()).abs() <= 2.0 ** -7 * b[0].float().abs() + 2.0 ** -12)
    assert torch.all((a[1] - b[1]).abs() < 1e-4)


@pytest.mark.gpu
def test_generation_together():
    """A prompt through the windowed forward, its keys and values into the 4-bit cache, then tokens one by one: each
    written, then attended to, on a side stream and from a captured graph; every output against the definition."""
    B, H, Hkv, P, d, W, S, steps = 2, 6, 3, 150, 64, 64, 4, 5
    Lmax = P + steps
    q, k, v = _bf(B, H, Lmax, d, seed=21), _bf(B, Hkv, Lmax, d, seed=22), _bf(B, Hkv, Lmax, d, seed=23)
    prompts = torch.tensor([P, 97], dtype=torch.int32)
    qd, kd, vd = gc.to_dev(q, k, v)
    cache = fa.kv4_cache(B, Hkv, Lmax, d, gc.DEV)
    o, _ = fa.attention_forward_window(*(t[:, :, :P].contiguous() for t in (qd, kd, vd)), W, S)
    r = OW.attention(_np(q[:, :, :P]), _np(k[:, :, :P]), _np(v[:, :, :P]), W, S, 1 / math.sqrt(d))
    _within(o, r["o"], r["o_bound"], "prompt")
    fa.fa_kv4_write(kd[:, :, :P].contiguous(), vd[:, :, :P].contiguous(), cache, None, prompts.to(gc.DEV))
    # static buffers of one decoding step
    nq = torch.empty(B, H, 1, d, dtype=torch.bfloat16, device=gc.DEV)
    nk, nv = (torch.empty(B, Hkv, 1, d, dtype=torch.bfloat16, device=gc.DEV) for _ in range(2))
    at, n = prompts.to(gc.DEV), prompts.to(gc.DEV) + 1
    out, lse = torch.empty_like(nq), torch.empty(B, H, device=gc.DEV)
    ws = torch.empty(max(256, fa.fa_decode_window_workspace_size(B, H, Hkv, Lmax, d, W, S)), dtype=torch.uint8, device=gc.DEV)

    def step():
        fa.fa_kv4_write(nk, nv, cache, at)
        fa.fa_decode_kv4(nq, cache, n, W, S, out, lse, ws)
        at.add_(1)
        n.add_(1)

    side = torch.cuda.Stream()
    graph = None
    for i in range(steps):
        for b in range(B):
            p = int(prompts[b]) + i
            nq[b, :, 0], nk[b, :, 0], nv[b, :, 0] = qd[b, :, p], kd[b, :, p], vd[b, :, p]
        if i == 0:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        lens = (prompts + i + 1).tolist()
        (kc, ks), (vc, vs) = Q.quantise(_np(k)), Q.quantise(_np(v))
        pq = np.stack([_np(q)[b, :, lens[b] - 1] for b in range(B)])
        r = Q.decode(pq, kc, ks, vc, vs, lens, W, S, 1 / math.sqrt(d))
        _within(out[:, :, 0], r["o"], r["o_bound"], f"token {i}")
    assert fa.fa_get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_two_streams_at_once(q4):
    """Overlapping calls with workspaces of their own."""
    cases = [_case(4, 8, 2, 3000, 128, [3000, 1, 2999, 700], seed=30 + i) for i in range(2)]
    want = [_run_decode(q4, c, 2500, 4) for c in cases]
    args, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for q, k, v, n in cases:
        kv = (k.to(gc.DEV), v.to(gc.DEV))
        if q4:
            cache = fa.kv4_cache(4, 2, 3000, 128, gc.DEV)
            fa.fa_kv4_write(*kv, cache)
            kv = (cache,)
        args.append((q.to(gc.DEV), *kv, n.to(gc.DEV), 2500, 4))
    torch.cuda.synchronize()
    f = fa.decode_kv4 if q4 else fa.decode_window
    for _ in range(5):
        outs = []
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                outs.append(f(*a))
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True])
def test_lse_is_optional(q4):
    q, k, v, n = _case(2, 4, 2, 400, 64, [400, 0], seed=33)
    ref = _run_decode(q4, (q, k, v, n), 300, 2)
    o = torch.full((2, 4, 1, 64), 9.0, dtype=torch.bfloat16, device=gc.DEV)
    ws = torch.empty(fa.fa_decode_window_workspace_size(2, 4, 2, 400, 64, 300, 2), dtype=torch.uint8, device=gc.DEV)
    kd, vd = k.to(gc.DEV), v.to(gc.DEV)
    if q4:
        cache = fa.kv4_cache(2, 2, 400, 64, gc.DEV)
        fa.fa_kv4_write(kd, vd, cache)
        fa.fa_decode_kv4(q.to(gc.DEV), cache, n.to(gc.DEV), 300, 2, o, None, ws)
    else:
        fa.fa_decode_window(q.to(gc.DEV), kd, vd, n.to(gc.DEV), 300, 2, o, None, ws)
    assert torch.equal(o, ref[0])


@pytest.mark.gpu
def test_caches_beyond_32_bit_offsets():
    """A cache of more than 2^32 bytes (bf16) and 2^31 codes (4 bits): rows at its end are written and attended to."""
    Hkv, Lmax, d, W, S = 3, 1 << 23, 128, 90, 3
    lens = [Lmax - 1]
    q = _bf(1, 6, 1, d, seed=40)
    rows = torch.cat([torch.arange(S), torch.arange(Lmax - 1 - W, Lmax - 1)])
    k, v = _bf(1, Hkv, rows.numel(), d, seed=41), _bf(1, Hkv, rows.numel(), d, seed=42)
    scale = 1 / math.sqrt(d)
    n = torch.tensor(lens, dtype=torch.int32, device=gc.DEV)
    kc = torch.empty(1, Hkv, Lmax, d, dtype=torch.bfloat16, device=gc.DEV)
    vc = torch.empty_like(kc)
    at = rows.to(gc.DEV)
    kc[:, :, at], vc[:, :, at] = k.to(gc.DEV), v.to(gc.DEV)
    assert kc.numel() * 2 > 1 << 32
    o, lse = fa.decode_window(q.to(gc.DEV), kc, vc, n, W, S, scale=scale)
    r = OW.decode(_np(q)[:, :, 0], _np(k), _np(v), [rows.numel()], rows.numel(), 0, scale)
    _within(o[:, :, 0], r["o"], r["o_bound"], "O")
    del kc, vc
    cache = fa.KV4Cache(*(torch.empty(1, Hkv, Lmax, m, dtype=t, device=gc.DEV)
                          for m, t in ((d // 2, torch.uint8), (d // 32, torch.bfloat16)) * 2))
    for first, count in ((0, S), (Lmax - 1 - W, W)):
        part = slice(0, S) if first == 0 else slice(S, S + W)
        start = torch.tensor([first], dtype=torch.int32, device=gc.DEV)
        fa.fa_kv4_write(k[:, :, part].contiguous().to(gc.DEV), v[:, :, part].contiguous().to(gc.DEV), cache, start)
    o, lse = fa.decode_kv4(q.to(gc.DEV), cache, n, W, S, scale=scale)
    (kq, ks), (vq, vs) = Q.quantise(_np(k)), Q.quantise(_np(v))
    r = Q.decode(_np(q)[:, :, 0], kq, ks, vq, vs, [rows.numel()], rows.numel(), 0, scale)
    _within(o[:, :, 0], r["o"], r["o_bound"], "O, 4 bits")
    _within(lse, r["lse"], r["lse_bound"], "LSE, 4 bits")
    kr, _ = fa.kv4_read(cache, W, torch.tensor([Lmax - 1 - W], dtype=torch.int32, device=gc.DEV))
    want = Q.values(kq, ks)[:, :, S:]
    assert np.array_equal(Q.bf16_bits(_np(kr)) & 0x7FFF, Q.bf16_bits(want) & 0x7FFF)
