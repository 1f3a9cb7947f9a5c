"""The allocating wrappers on a stream that is not the current one (`stream=`): what a call allocates for itself is given
back in that stream's order, and what it fills is filled there."""
import math

import pytest
import torch

import gpu_common as gc
import io_aware_exact_32_b200 as fa

pytestmark = pytest.mark.gpu


def _bf(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(gc.DEV)


def _cache(k, v):
    cache = fa.kv4_cache(*k.shape, gc.DEV)
    fa.fa_kv4_write(k, v, cache)
    return cache


def _calls():
    """name -> (call with stream=, the function of the module that allocates for it)."""
    q, k, v, do = (_bf(1, 4, 300, 64, seed=i) for i in range(4))
    ks, vs = k[:, :2].contiguous(), v[:, :2].contiguous()
    x1 = _bf(2, 4, 1, 128, seed=5)
    kc, vc = _bf(2, 2, 700, 128, seed=6), _bf(2, 2, 700, 128, seed=7)
    kf, vf = _bf(2, 4, 700, 128, seed=8), _bf(2, 4, 700, 128, seed=9)
    n = torch.tensor([700, 300], dtype=torch.int32, device=gc.DEV)
    cache = _cache(kc, vc)
    o, lse = fa.attention_forward(q, k, v, causal=True)
    ow, lw = fa.attention_forward_window(q, ks, vs, 90, 3)
    q8 = [_bf(1, 2, 256, 128, seed=10 + i) for i in range(3)]
    return {
        "attention_backward": (lambda stream: fa.attention_backward(q, k, v, o, lse, do, True, stream=stream, deterministic=True), "_workspace"),
        "attention_backward_window": (lambda stream: fa.attention_backward_window(q, ks, vs, ow, lw, do, 90, 3, stream=stream)[1:], "_workspace"),
        "decode_splitkv": (lambda stream: fa.decode_splitkv(x1, kf, vf, n, stream=stream), "_workspace"),
        "decode_window": (lambda stream: fa.decode_window(x1, kc, vc, n, 600, 4, stream=stream), "_workspace"),
        "decode_kv4": (lambda stream: fa.decode_kv4(x1, cache, n, 600, 4, stream=stream), "_workspace"),
        "attention_forward_fp8": (lambda stream: fa.attention_forward_fp8(*q8, stream=stream), "quantize_fp8"),
    }


NAMES = ["attention_backward", "attention_backward_window", "decode_splitkv", "decode_window", "decode_kv4",
         "attention_forward_fp8"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_is_not_handed_out_while_it_runs(name, raw, monkeypatch):
    """The call waits on a busy side stream; what the current stream allocates meanwhile is other memory."""
    call, allocator = _calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    taken = []
    original = getattr(fa, allocator)

    def recording(*args, **kw):
        out = original(*args, **kw)
        for t in out if isinstance(out, tuple) else (out,):
            taken.append((t.data_ptr(), t.numel() * t.element_size()))
        return out

    monkeypatch.setattr(fa, allocator, recording)
    side = torch.cuda.Stream()
    handle = side.cuda_stream if raw else side
    call(handle)   # the stream's pool gets its memory here: cudaMalloc would wait for the sleep below
    torch.cuda.synchronize()
    taken.clear()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = call(handle)
    assert taken
    mine = []
    for _ in range(3):
        for _, size in taken:
            mine.append(torch.empty(size, dtype=torch.uint8, device=gc.DEV))
            mine[-1].fill_(0xFF)
    for t in mine:
        for start, size in taken:
            assert t.data_ptr() + t.numel() <= start or start + size <= t.data_ptr()
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("raw", [False, True])
def test_rows_read_back_on_an_idle_stream_while_the_current_one_is_busy(raw):
    """The zeros past the cache's end are written ahead of the rows, on the call's own stream."""
    k, v = _bf(2, 2, 50, 64, seed=20), _bf(2, 2, 50, 64, seed=21)
    cache = _cache(k, v)
    starts = torch.tensor([45, 3], dtype=torch.int32, device=gc.DEV)
    want = fa.kv4_read(cache, 20, starts)
    assert torch.all(want[0][0, :, 5:] == 0) and torch.all(torch.any(want[0][1] != 0, dim=-1))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = fa.kv4_read(cache, 20, starts, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_the_default_streams_raw_handle():
    q, k, v, do = (_bf(1, 2, 200, 64, seed=30 + i) for i in range(4))
    o, lse = fa.attention_forward_window(q, k, v, 50, 2, scale=1 / math.sqrt(64))
    a = fa.attention_backward_window(q, k, v, o, lse, do, 50, 2, stream=0)
    torch.cuda.synchronize()
    b = fa.attention_backward_window(q, k, v, o, lse, do, 50, 2)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
