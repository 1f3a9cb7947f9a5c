"""Sliding-window attention with sinks and shared key/value heads: the float64 definition (CPU), the refusals (CPU), and
the kernels against the definition (GPU), elementwise within the rounding bounds of oracle/windowed.py."""
import ctypes
import math

import numpy as np
import pytest
import torch

import gpu_common as gc
import io_aware_exact_32_b200 as fa
from oracle import attention as A
from oracle import windowed as OW
from tolerances import check_grad

NULL = ctypes.c_void_p(0)
A16 = ctypes.c_void_p(0x10000)      # fake, aligned, never dereferenced
MIS = ctypes.c_void_p(0x10008)


# ------------------------------------------------------------------------------------------------ the definition
def test_definition_is_causal_attention_for_a_window_over_everything():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal((1, 2, n, 8)) for n in (5, 9, 9))
    r = OW.attention(q, k, v, 9, 0, 0.3)
    o, lse = A.attention_forward(q, k, v, 0.3, True)
    assert np.allclose(r["o"], o, atol=1e-13) and np.allclose(r["lse"], lse, atol=1e-13)
    r2 = OW.attention(q, k, v, 3, 9, 0.3)   # every key a sink
    assert np.array_equal(r2["o"], r["o"])


def test_visible_by_hand():
    m = OW.visible(4, 6, 2, 1).astype(int)   # positions 2 .. 5
    assert m.tolist() == [[1, 1, 1, 0, 0, 0], [1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    m = OW.visible(4, 2, 1, 0).astype(int)   # positions -2 .. 1: two rows see nothing
    assert m.tolist() == [[0, 0], [0, 0], [1, 0], [0, 1]]


def test_definition_gradients_match_differences():
    """dQ, dK, dV of sum(O * dO) against central differences, with shared heads and rows that see nothing."""
    rng = np.random.default_rng(1)
    q, do = (rng.standard_normal((1, 4, 7, 4)) for _ in range(2))
    k, v = (rng.standard_normal((1, 2, 6, 4)) for _ in range(2))
    r = OW.attention(q, k, v, 2, 1, 0.5, do)
    h = 1e-6
    for x, g in ((q, r["dq"]), (k, r["dk"]), (v, r["dv"])):
        for idx in rng.choice(x.size, 12, replace=False):
            at = np.unravel_index(idx, x.shape)
            old = x[at]
            f = []
            for s in (h, -h):
                x[at] = old + s
                f.append((OW.attention(q, k, v, 2, 1, 0.5)["o"] * do).sum())
            x[at] = old
            assert abs((f[0] - f[1]) / (2 * h) - g[at]) < 1e-7


# ------------------------------------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def L():
    return fa.lib()


def fwd(L, q=A16, k=A16, o=A16, B=1, H=4, Hkv=2, Nq=128, Nk=128, d=64, window=16, sinks=4, scale=0.125):
    return L.fa_fwd_window(q, k, A16, o, A16, B, H, Hkv, Nq, Nk, d, window, sinks, scale, NULL)


def test_forward_refusals(L):
    assert fwd(L, d=96) == 2
    assert fwd(L, window=0) == 1
    assert fwd(L, window=-3) == 1
    assert fwd(L, sinks=-1) == 1
    assert fwd(L, Hkv=3) == 1
    assert fwd(L, Hkv=0) == 1
    assert fwd(L, Hkv=-2) == 1
    assert fwd(L, Hkv=8) == 1
    assert fwd(L, Nq=(1 << 24) + 1) == 2
    assert fwd(L, scale=float("inf")) == 1
    assert fwd(L, q=NULL) == 1
    assert fwd(L, o=MIS) == 3
    assert fwd(L, k=MIS) == 3
    assert fwd(L, B=0) == 0
    assert fwd(L, Nq=0, q=NULL, o=NULL) == 0
    assert fwd(L, H=0, Hkv=0) == 0


def bwd(L, ws=A16, ws_bytes=1 << 30, null=None, mis=None, H=4, Hkv=2, window=16, sinks=4, d=64):
    args = [A16] * 9
    if null is not None:
        args[null] = NULL
    if mis is not None:
        args[mis] = MIS
    return L.fa_bwd_window(*args, ws, ws_bytes, 1, H, Hkv, 300, 300, d, window, sinks, 0.125, NULL)


def test_backward_refusals(L):
    assert bwd(L, d=80) == 2
    assert bwd(L, Hkv=3) == 1
    assert bwd(L, window=0) == 1
    assert bwd(L, sinks=-1) == 1
    for i in range(9):
        assert bwd(L, null=i) == 1
        assert bwd(L, mis=i) == 3
    assert bwd(L, ws=NULL) == 4
    need = L.fa_bwd_window_workspace_size(1, 4, 2, 300, 300, 64, 16, 4)
    assert bwd(L, ws_bytes=need - 1) == 4
    assert bwd(L, ws=ctypes.c_void_p(0x10010)) == 3


def test_workspace_sizes(L):
    f = L.fa_bwd_window_workspace_size
    base = L.fa_bwd_workspace_size(2, 8, 4096, 64)
    assert f(2, 8, 8, 4096, 4096, 64, 256, 0) == base                # nothing is cut
    assert f(2, 8, 8, 4096, 4096, 64, 4096, 4) == base               # the window covers everything
    cut = f(2, 8, 8, 4096, 4096, 64, 256, 4) - base
    assert cut > 0 and cut % (2 * 8 * 2 * 128 * 64 * 4) == 0         # whole fp32 dV and dK tiles
    assert f(2, 8, 3, 4096, 4096, 64, 256, 4) == 0                   # 3 does not divide 8
    assert f(2, 8, 8, 4096, 4096, 96, 256, 4) == 0
    assert f(2, 8, 8, 0, 4096, 64, 256, 4) == 0


def test_binding_refusals():
    q = torch.zeros(1, 4, 16, 64, dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.attention_forward_window(q, k, k, 4)
    with pytest.raises(ValueError, match="window"):
        fa.attention_forward_window(q, k, k, 0)
    with pytest.raises(ValueError, match="sinks"):
        fa.attention_forward_window(q, k, k, 4, -1)
    with pytest.raises(ValueError, match="share"):
        fa.attention_forward_window(q, torch.zeros(1, 3, 16, 64, dtype=torch.bfloat16), k, 4)
    with pytest.raises(ValueError, match="shape"):
        fa.attention_forward_window(q, torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16), k, 4)


# ------------------------------------------------------------------------------------------------ kernels
def _inputs(B, H, Hkv, Nq, Nk, d, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    return mk(B, H, Nq, d), mk(B, Hkv, Nk, d), mk(B, Hkv, Nk, d), mk(B, H, Nq, d)


def _within(got, ref, bound, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    inf = np.isneginf(ref)
    assert np.array_equal(np.isneginf(got), inf), f"{what}: -inf pattern"
    err = np.abs(np.where(inf, 0.0, got) - np.where(inf, 0.0, ref))
    assert np.all(np.isfinite(err)), f"{what}: non-finite"
    bad = err > bound + 1e-30
    assert not bad.any(), f"{what}: {int(bad.sum())} beyond the bound, worst {np.max(err / (bound + 1e-30)):.2f} x at " \
                          f"{np.unravel_index(np.argmax(err / (bound + 1e-30)), err.shape)}"


def _check(x, window, sinks, backward=True):
    q, k, v, do = x
    scale = 1 / math.sqrt(q.shape[-1])
    r = OW.attention(*(t.double().numpy() for t in (q, k, v)), window, sinks, scale,
                     do.double().numpy() if backward else None)
    qd, kd, vd, dod = gc.to_dev(q, k, v, do)
    o, lse = fa.attention_forward_window(qd, kd, vd, window, sinks, scale=scale)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == 0
    _within(o, r["o"], r["o_bound"], "O")
    _within(lse, r["lse"], r["lse_bound"], "LSE")
    if backward:
        grads = fa.attention_backward_window(qd, kd, vd, o, lse, dod, window, sinks, scale=scale)
        torch.cuda.synchronize()
        assert fa.fa_get_device_error() == 0
        for n, t in zip(("dq", "dk", "dv"), grads):
            _within(t, r[n], r[n + "_bound"], n)
            # A window of one key has P = 1 and dS = 0: dq and dk are rounding alone.
            if window > 1 and min(q.shape[2], k.shape[2]) > 1:
                check_grad(gc.f64(t), r[n], n)


SHAPES = [  # B, H, Hkv, Nq, Nk, d, window, sinks
    (1, 1, 1, 1, 1, 64, 1, 0),
    (2, 2, 1, 1, 1, 128, 5, 3),
    (1, 2, 2, 128, 128, 64, 32, 0),
    (1, 2, 2, 129, 129, 128, 1, 0),        # each row sees itself alone
    (1, 2, 1, 300, 300, 64, 100, 4),
    (2, 4, 2, 257, 513, 128, 128, 1),      # a chunk behind a prefix
    (1, 3, 3, 77, 333, 64, 129, 7),
    (1, 6, 2, 700, 700, 128, 127, 130),    # sinks across two tiles
    (1, 2, 2, 640, 640, 64, 640, 0),       # plain causal
    (1, 2, 2, 640, 640, 128, 1 << 20, 1 << 20),
    (1, 2, 1, 400, 250, 64, 60, 2),        # 150 rows see nothing
    (1, 2, 1, 500, 100, 128, 128, 0),      # whole tiles of rows see nothing
    (1, 1, 1, 1300, 1300, 128, 200, 260),
    (1, 8, 1, 200, 200, 64, 33, 5),        # one key/value head for all
    (2, 6, 3, 333, 333, 128, 70, 8),
    (1, 2, 2, 200, 500, 128, 64, 2),       # a chunk that lies beyond the sinks' windows altogether
    (1, 2, 1, 500, 300, 64, 90, 8),        # rows that see nothing, then sinks in and out of their windows
    (1, 2, 1, 300, 300, 128, 299, 1),      # one row beyond the sink's window
    (1, 2, 1, 256, 256, 64, 5, 8),         # sinks that leave the window one by one
    (1, 4, 2, 700, 700, 64, 40, 32),       # the widest narrow sink tile
    (1, 4, 2, 700, 700, 128, 40, 33),      # the first wide one
    (1, 10, 2, 130, 390, 64, 300, 64),     # groups of five
    (3, 1, 1, 1, 700, 128, 256, 4),        # one query
]


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,window,sinks", SHAPES)
def test_forward_and_backward(B, H, Hkv, Nq, Nk, d, window, sinks):
    _check(_inputs(B, H, Hkv, Nq, Nk, d, seed=Nq + Nk + window + sinks), window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,N,d,window,sinks", [(8, 20, 5, 515, 64, 130, 4), (2, 80, 80, 300, 128, 64, 1),
                                                      (1, 150, 75, 390, 128, 190, 133)])
def test_two_tile_items(B, H, Hkv, N, d, window, sinks):
    """Enough work for the persistent two-tile forward; several items per CTA."""
    _check(_inputs(B, H, Hkv, N, N, d, seed=B + H), window, sinks)


@pytest.mark.gpu
def test_long_sequence_with_cut_sinks():
    """A sink tile's walk over all query blocks is cut into shares; 4096 rows, small window."""
    x = _inputs(1, 2, 1, 4096, 4096, 64, seed=9)
    assert fa.fa_bwd_window_workspace_size(1, 2, 1, 4096, 4096, 64, 100, 3) > fa.fa_bwd_workspace_size(1, 2, 4096, 64)
    _check(x, 100, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,Nq,Nk,d,window,sinks", [
    (1, 16, 1, 700, 700, 64, 300, 0),
    (1, 16, 1, 700, 700, 128, 300, 4),      # sinks cut apart
    (1, 12, 1, 650, 650, 64, 650, 5),       # sinks among the others
    (2, 16, 2, 257, 900, 128, 513, 130),    # keys that no query sees; two sink tiles
    (1, 16, 1, 900, 430, 64, 200, 3),       # queries that see nothing
    (1, 24, 2, 129, 129, 128, 40, 1),
])
def test_few_key_tiles_with_long_walks(B, H, Hkv, Nq, Nk, d, window, sinks):
    """Every key tile's walk is cut into shares: partials for whole key tiles in the workspace, dK and dV the same bits
    run to run."""
    need = fa.fa_bwd_window_workspace_size(B, H, Hkv, Nq, Nk, d, window, sinks)
    tiles = (need - fa.fa_bwd_workspace_size(B, H, Nq, d)) // (2 * 128 * d * 4)
    assert tiles >= 2 * B * Hkv * ((Nk + 127) // 128)
    x = _inputs(B, H, Hkv, Nq, Nk, d, seed=Nq + H)
    _check(x, window, sinks)
    q, k, v, do = gc.to_dev(*x)
    o, lse = fa.attention_forward_window(q, k, v, window, sinks)
    ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=gc.DEV)  # its contents do not matter: NaN
    a = fa.attention_backward_window(q, k, v, o, lse, do, window, sinks, workspace=ws[:need])
    b = fa.attention_backward_window(q, k, v, o, lse, do, window, sinks)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert torch.all(ws[need:] == 0xFF)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_equals_the_plain_kernels(d):
    """A window over everything and one key/value head per query head: the same bits as fa_fwd."""
    q, k, v, _ = gc.to_dev(*_inputs(2, 3, 3, 700, 700, d, seed=3))
    o, lse = fa.attention_forward_window(q, k, v, 700)
    o2, lse2 = fa.attention_forward(q, k, v, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.gpu
def test_reproducible_gradients_of_shared_heads():
    """dK and dV are the same bits run to run, cut sinks included."""
    q, k, v, do = gc.to_dev(*_inputs(1, 8, 2, 2000, 2000, 64, seed=4))
    o, lse = fa.attention_forward_window(q, k, v, 64, 5)
    a = fa.attention_backward_window(q, k, v, o, lse, do, 64, 5)
    b = fa.attention_backward_window(q, k, v, o, lse, do, 64, 5)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


@pytest.mark.gpu
def test_empty_sizes():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=gc.DEV)  # noqa: E731
    o, lse = fa.attention_forward_window(z(1, 2, 5, 64), z(1, 1, 0, 64), z(1, 1, 0, 64), 3, 1)   # no key
    assert torch.all(o == 0) and torch.all(lse == -math.inf)
    dq, dk, dv = fa.attention_backward_window(z(1, 2, 5, 64), z(1, 1, 0, 64), z(1, 1, 0, 64), o, lse, z(1, 2, 5, 64), 3)
    assert torch.all(dq == 0) and dk.numel() == 0
    q = z(1, 2, 0, 64)                                                                            # no query
    k = torch.ones(1, 1, 9, 64, dtype=torch.bfloat16, device=gc.DEV)
    o, lse = fa.attention_forward_window(q, k, k, 3, 1)
    dk = torch.full_like(k, 7.0)
    dv = torch.full_like(k, 7.0)
    fa.fa_bwd_window(q, k, k, o, q, lse, q, dk, dv, torch.empty(256, dtype=torch.uint8, device=gc.DEV), 3, 1)
    assert torch.all(dk == 0) and torch.all(dv == 0)


@pytest.mark.gpu
def test_other_stream_and_graph_replay():
    """Forward and backward on a side stream, then captured into a graph and replayed on new inputs."""
    x = gc.to_dev(*_inputs(1, 4, 2, 513, 513, 64, seed=5))
    y = gc.to_dev(*_inputs(1, 4, 2, 513, 513, 64, seed=6))
    W, S = 90, 2
    ws = torch.empty(fa.fa_bwd_window_workspace_size(1, 4, 2, 513, 513, 64, W, S), dtype=torch.uint8, device=gc.DEV)
    o, lse = torch.empty_like(x[0]), torch.empty(1, 4, 513, device=gc.DEV)
    g = [torch.empty_like(t) for t in x[:3]]

    def step(a):
        fa.fa_fwd_window(a[0], a[1], a[2], o, lse, W, S)
        fa.fa_bwd_window(a[0], a[1], a[2], o, a[3], lse, *g, ws, W, S)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(y)
    s.synchronize()
    want = [t.clone() for t in (o, lse, g[1], g[2])]
    buf = [t.clone() for t in x]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(buf)
    for d_, s_ in zip(buf, y):
        d_.copy_(s_)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((o, lse, g[1], g[2]), want):
        assert torch.equal(a, b)


def _same_gradients(a, b):
    """dk and dv the same bits; dq's reduce-adds may meet in another order: its fp32 sums then differ by a few 2^-24 of
    their terms, and a bf16 result by one step of 2^-7 of itself at most where that crosses a rounding boundary."""
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    x, y = a[0].float(), b[0].float()
    assert torch.all((x - y).abs() <= 2.0 ** -7 * torch.maximum(x.abs(), y.abs()) + 1e-4 * x.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,N,d,window,sinks", [(4, 2, 900, 64, 200, 3), (16, 1, 700, 128, 300, 4), (8, 8, 300, 128, 50, 0)])
def test_calls_one_after_another_share_a_workspace(H, Hkv, N, d, window, sinks):
    """A call's kernels start before the ones ahead of them have ended; the next call's must not disturb them."""
    xs = [gc.to_dev(*_inputs(1, H, Hkv, N, N, d, seed=s)) for s in (21, 22)]
    fw = [fa.attention_forward_window(*x[:3], window, sinks) for x in xs]
    ws = torch.empty(fa.fa_bwd_window_workspace_size(1, H, Hkv, N, N, d, window, sinks), dtype=torch.uint8, device=gc.DEV)
    want = []
    for x, (o, lse) in zip(xs, fw):
        want.append(fa.attention_backward_window(*x[:3], o, lse, x[3], window, sinks))
        torch.cuda.synchronize()
    got = [fa.attention_backward_window(*xs[i % 2][:3], *fw[i % 2], xs[i % 2][3], window, sinks, workspace=ws)
           for i in range(40)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        _same_gradients(want[i % 2], g)


@pytest.mark.gpu
def test_two_streams_at_once():
    """Forward and backward on two streams that overlap, each with its own workspace."""
    xs = [gc.to_dev(*_inputs(1, 8, 2, 1100, 1100, d, seed=d)) for d in (64, 128)]
    want = []
    for x in xs:
        o, lse = fa.attention_forward_window(*x[:3], 250, 4)
        want.append((o, lse, fa.attention_backward_window(*x[:3], o, lse, x[3], 250, 4)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(15):
        for x, s, out in zip(xs, streams, got):
            with torch.cuda.stream(s):
                o, lse = fa.attention_forward_window(*x[:3], 250, 4)
                out.append((o, lse, fa.attention_backward_window(*x[:3], o, lse, x[3], 250, 4)))
    torch.cuda.synchronize()
    for w, out in zip(want, got):
        for o, lse, g in out:
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
            _same_gradients(w[2], g)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_at_any_16_byte_offset(d):
    """o, dk and dv that are 16- but not 32-byte aligned take other stores: the same bits."""
    q, k, v, do = gc.to_dev(*_inputs(1, 4, 2, 300, 300, d, seed=7))
    W, S = 90, 3
    o, lse = fa.attention_forward_window(q, k, v, W, S)
    g = fa.attention_backward_window(q, k, v, o, lse, do, W, S)

    def shifted(t):
        buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device=t.device)
        x = buf[8:8 + t.numel()].view(t.shape)
        assert x.data_ptr() % 32 == 16
        return x

    o2, g2 = shifted(o), [shifted(t) for t in (q, k, v)]
    fa.fa_fwd_window(q, k, v, o2, lse, W, S)
    ws = torch.empty(fa.fa_bwd_window_workspace_size(1, 4, 2, 300, 300, d, W, S), dtype=torch.uint8, device=gc.DEV)
    fa.fa_bwd_window(q, k, v, o2, do, lse, *g2, ws, W, S)
    assert torch.equal(o, o2) and torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])


@pytest.mark.gpu
def test_window_larger_than_any_sequence():
    q, k, v, _ = gc.to_dev(*_inputs(1, 2, 1, 150, 200, 64, seed=8))
    a = fa.attention_forward_window(q, k, v, 1 << 40, 1 << 40)
    b = fa.attention_forward_window(q, k, v, 200)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,d,sinks", [(16, 16, 128, 4), (16, 4, 128, 40), (16, 16, 64, 0), (16, 2, 64, 4)])
def test_waits_give_up_and_the_device_stays_usable(H, Hkv, d, sinks):
    """With the limit of the kernels' waits lowered, a healthy forward or backward gives up, reports it, and the next
    call on the device gives the results of before."""
    x = gc.to_dev(*_inputs(1, H, Hkv, 4096, 4096, d, seed=10))
    o, lse = fa.attention_forward_window(*x[:3], 500, sinks)
    g = fa.attention_backward_window(*x[:3], o, lse, x[3], 500, sinks)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == 0
    for call in (lambda: fa.attention_forward_window(*x[:3], 500, sinks),
                 lambda: fa.attention_backward_window(*x[:3], o, lse, x[3], 500, sinks)):
        fa.fa_debug_set_wait_limit(300)
        try:
            call()
            torch.cuda.synchronize()
            status = fa.fa_get_device_error()
        finally:
            fa.fa_debug_set_wait_limit(0)
        assert status == 6, status
    o2, lse2 = fa.attention_forward_window(*x[:3], 500, sinks)
    g2 = fa.attention_backward_window(*x[:3], o2, lse2, x[3], 500, sinks)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == 0
    for a, b in zip((o, lse) + g[1:], (o2, lse2) + g2[1:]):
        assert torch.equal(a, b)
