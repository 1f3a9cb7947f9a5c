"""Single-token attention over a 4-bit cache whose values differ in size: from group to group of a row, from row to row,
and up to the ends of bf16.  Each 32-channel group is judged by its own values, and the LSE, which does not depend on
them, by the scores alone."""
import math

import numpy as np
import pytest
import torch

import gpu_common as gc
import io_aware_exact_32_b200 as fa
from oracle import kv4 as Q

GROUP = Q.GROUP


def _bf(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _np(t):
    return t.double().cpu().numpy()


def _case(B, H, Hkv, L, d, seed):
    return _bf(B, H, 1, d, seed=seed), _bf(B, Hkv, L, d, seed=seed + 1), _bf(B, Hkv, L, d, seed=seed + 2)


def _definition(q, k, v, lens, window, sinks):
    (kc, ks), (vc, vs) = Q.quantise(_np(k)), Q.quantise(_np(v))
    return Q.decode(_np(q)[:, :, 0], kc, ks, vc, vs, lens, window, sinks, 1 / math.sqrt(q.shape[-1]))


def _kernel(q, k, v, lens, window, sinks):
    cache = fa.kv4_cache(*k.shape, gc.DEV)
    fa.fa_kv4_write(k.to(gc.DEV), v.to(gc.DEV), cache)
    o, lse = fa.decode_kv4(q.to(gc.DEV), cache, torch.tensor(lens, dtype=torch.int32, device=gc.DEV), window, sinks)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == 0
    return _np(o)[:, :, 0], _np(lse)


def _compare(o, lse, r):
    """Elementwise within the definition's bounds; the smallest bf16 results (below 2^-126) may be flushed."""
    assert np.all(np.abs(lse - r["lse"]) <= r["lse_bound"]), \
        f"LSE: {np.max(np.abs(lse - r['lse']) / r['lse_bound']):.2f} x the bound"
    err, bound = np.abs(o - r["o"]), r["o_bound"] + 2.0 ** -126
    assert np.all(np.isfinite(err)), "O: non-finite"
    assert np.all(err <= bound), f"O: {np.max(err / bound):.2f} x the bound at {np.unravel_index(np.argmax(err / bound), err.shape)}"


def _check(q, k, v, lens=None, window=None, sinks=0):
    L = k.shape[2]
    lens = [L] * k.shape[0] if lens is None else lens
    window = L if window is None else window
    _compare(*_kernel(q, k, v, lens, window, sinks), _definition(q, k, v, lens, window, sinks))


def _scaled_group(v, g, power):
    """Group g of every row times 2^power."""
    v = v.clone()
    v[..., GROUP * g:GROUP * (g + 1)] = (v[..., GROUP * g:GROUP * (g + 1)].double() * 2.0 ** power).to(torch.bfloat16)
    return v


# ------------------------------------------------------------------------------------------------ the bounds themselves
def test_a_groups_bound_does_not_depend_on_its_neighbours():
    """Scaling one group of V scales that group's output and bound, and nothing else."""
    q, k, v = _case(1, 2, 1, 50, 64, seed=1)
    a, b = _definition(q, k, v, [50], 50, 0), _definition(q, k, _scaled_group(v, 1, -24), [50], 50, 0)
    for n in ("o", "o_bound"):
        assert np.array_equal(a[n][..., :GROUP], b[n][..., :GROUP]), n
        assert np.allclose(a[n][..., GROUP:] * 2.0 ** -24, b[n][..., GROUP:], rtol=1e-12, atol=0), n
    assert np.array_equal(a["lse"], b["lse"]) and np.array_equal(a["lse_bound"], b["lse_bound"])


def test_the_bounds_see_a_lost_group():
    """A group lost to its neighbours' size (an output of zeros, or off by a sixth) is beyond its bound."""
    q, k, v = _case(1, 2, 1, 1000, 128, seed=2)
    r = _definition(q, k, _scaled_group(v, 2, -24), [1000], 1000, 0)
    for factor in (0.0, 5 / 6):
        o = r["o"].copy()
        o[..., 2 * GROUP:3 * GROUP] *= factor
        with pytest.raises(AssertionError, match="O: "):
            _compare(o, r["lse"], r)
    _compare(r["o"], r["lse"], r)


# ------------------------------------------------------------------------------------------------ the kernel
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("power", [-20, -28, -60, 20, 28, 100])
def test_one_group_of_another_size(d, power):
    q, k, v = _case(2, 4, 2, 1000, d, seed=3)
    _check(q, k, _scaled_group(v, d // 64, power), lens=[1000, 333])


@pytest.mark.gpu
def test_every_group_of_another_size():
    q, k, v = _case(1, 10, 1, 700, 128, seed=4)
    for g, power in enumerate((-90, 60, -3, 110)):
        v = _scaled_group(v, g, power)
    _check(q, k, v, window=600, sinks=5)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_query_and_key_groups_of_another_size(d):
    """A group of q 2^-16 of the others against keys 2^16 larger there: its part of the scores counts as much."""
    q, k, v = _case(1, 4, 2, 300, d, seed=15)
    _check(_scaled_group(q, 1, -16), _scaled_group(k, 1, 16), v)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [20, 28, 60])
@pytest.mark.parametrize("at", [0, 3, 64, 500, 999])
def test_a_row_of_large_values_and_no_weight(at, power):
    """One key whose score is far below the others' has values 2^power larger: where it comes first, in the middle and
    last.  Its contribution (about 2^(power - 40) of the others') is small, or all that counts; theirs stays what it is."""
    q, k, v = _case(1, 4, 2, 1000, 128, seed=5)
    q[:, 1::2] *= 0.25
    for h in range(2):
        # key `at` lies against the sum of its two heads' queries: scores of about -28 (nats) for the first
        s = q[0, 2 * h, 0].float()
        k[0, h, at] = (-s * (28 * math.sqrt(128) / (s * s).sum())).to(torch.bfloat16)
    v[:, :, at] = (v[:, :, at].double() * 2.0 ** power).to(torch.bfloat16)
    _check(q, k, v)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [20, 28])
def test_heads_that_look_at_different_rows(power):
    """Rows of large values that one head of a key/value head attends to and another does not."""
    q, k, v = _case(1, 2, 1, 900, 128, seed=6)
    q[0, 1] = -q[0, 0]
    rows = torch.arange(7, 900, 90)
    s = q[0, 0, 0].float()
    k[0, 0, rows] = (s * (20 * math.sqrt(128) / (s * s).sum())).to(torch.bfloat16)   # scores +20 and -20
    v[0, 0, rows] = (v[0, 0, rows].double() * 2.0 ** power).to(torch.bfloat16)
    _check(q, k, v)


@pytest.mark.gpu
@pytest.mark.parametrize("order", [1, -1])
def test_scores_that_rise_while_values_shrink(order):
    """The early keys' weights fade by 2^200 as the scores rise, their values are 2^60 larger; and the other way round."""
    L = 1024
    q, k, v = _case(1, 4, 1, L, 64, seed=7)
    q[0, :] = q[0, :1]
    s = q[0, 0, 0].float()
    ramp = torch.linspace(-70, 70, L)[:, None]
    k[0, 0] = (s * ramp * (math.sqrt(64) / (s * s).sum())).to(torch.bfloat16)
    v = (v.double() * (2.0 ** torch.linspace(60, 0, L, dtype=torch.float64).floor())[:, None]).to(torch.bfloat16)
    if order < 0:
        k, v = k.flip(2), v.flip(2)
    _check(q, k.contiguous(), v.contiguous())


@pytest.mark.gpu
@pytest.mark.parametrize("L", [5, 700, 20000])
@pytest.mark.parametrize("d", [64, 128])
def test_values_at_the_top_of_bf16(d, L):
    """V up to 3e38: no sum of weighted values leaves fp32's range, and the LSE is that of small values."""
    q, k, _ = _case(1, 3, 1, L, d, seed=8)
    v = (torch.rand(1, 1, L, d, generator=torch.Generator().manual_seed(9)) * 2 - 1).double()
    big = (v * 3e38).to(torch.bfloat16)
    _check(q, k, big)
    a, b = _kernel(q, k, big, [L], L, 0), _kernel(q, k, v.to(torch.bfloat16), [L], L, 0)
    assert np.array_equal(a[1], b[1])


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
def test_all_values_at_the_top_of_bf16(sign):
    """Equal values, whose mean is as large as they are."""
    q, k, v = _case(2, 4, 2, 3000, 128, seed=10)
    v = torch.full_like(v, sign * 3e38)
    _check(q, k, v, lens=[3000, 130])


@pytest.mark.gpu
def test_one_key_far_above_the_others_with_values_at_the_top():
    """The other keys' weights are 2^-14 of the first one's: their sum still counts in O and LSE."""
    q, k, v = _case(1, 2, 1, 20000, 128, seed=11)
    q[0, 1] = q[0, 0]
    s = q[0, 0, 0].float()
    k[0, 0, 17] = (s * (14 * math.log(2) + 2) * (math.sqrt(128) / (s * s).sum())).to(torch.bfloat16)
    _check(q, k, _scaled_group(_scaled_group(v, 0, 122), 3, 122))


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-80, -100, -112])
def test_values_near_the_bottom_of_bf16(power):
    q, k, v = _case(1, 4, 2, 600, 64, seed=12)
    for g in range(2):
        v = _scaled_group(v, g, power)
    _check(q, k, v)


@pytest.mark.gpu
def test_rows_of_zeros_before_and_after_values():
    """Groups of zeros (step 0) set no size; the rows after them do."""
    q, k, v = _case(1, 2, 1, 400, 128, seed=13)
    v[:, :, :130] = 0
    v[:, :, 200:210] = 0
    v[..., 32:64] = 0
    _check(q, k, v)


@pytest.mark.gpu
def test_a_visible_nan_keeps_to_its_group():
    """A NaN in one group of a visible row: the other groups' channels and the LSE are as without it."""
    q, k, v = _case(1, 4, 2, 500, 128, seed=14)
    ref = _kernel(q, k, v, [500], 500, 0)
    v[0, 1, 77, 37] = float("nan")
    o, lse = _kernel(q, k, v, [500], 500, 0)
    assert np.all(np.isnan(o[0, 2:, 32:64])) and np.array_equal(lse, ref[1])
    o[0, 2:, 32:64] = ref[0][0, 2:, 32:64]
    assert np.array_equal(o, ref[0])
