"""The bound of kv8_weights_ref on the CPU: what the roundings it allows leave
stays inside, and mistakes planted in the plain form do not."""
import math

import pytest
import torch

import kv8_weights_ref as wr
import prefix_cache_ref as ref

F64, BF = torch.float64, torch.bfloat16


def case(gap, sink_value=0.02, P=900, block=64):
    g = torch.Generator().manual_seed(int(gap * 16) + block)
    return wr.sink_inputs(g, P, 8, gap, sink_value, 3, block)


def ordinary(P=900, block=64):
    g = torch.Generator().manual_seed(P)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    codes = [(40 * r(1, 1, P, 256)).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-7, -4, (1, 1, -(-P // block)), generator=g).float()) for _ in range(2)]
    return r(1, 2, 40, 256).to(BF), (*codes, *scales, block), r(1, 1, 40, 256).to(BF), r(1, 1, 40, 256).to(BF)


def held(a, carry, other=None):
    """wr.off of a form that carries its weights so (on `other` inputs than the bound's)."""
    vis = torch.ones(1, a[1][0].shape[2], dtype=torch.bool)
    o, _, far, _ = wr.attention(*a, vis)
    return wr.off(wr.with_weights(*(other or a), vis, carry), o, far)


def test_roundings_match_the_types():
    x = torch.cat([torch.randn(4000, dtype=F64) * 2.0 ** e for e in (-30, -20, -16, -14, -9, -6, 0, 6, 7)])
    for t, bits, low in ((torch.float8_e4m3fn, 3, -6), (torch.float8_e5m2, 2, -14), (torch.float16, 10, -14)):
        y = x.clamp(-400, 400).float().double()
        assert torch.equal(wr.to_type(y, bits, low), y.float().to(t).to(F64))
    assert torch.equal(wr.bf16(x), x.float().to(BF).to(F64))


@pytest.mark.parametrize("gap", [0, 8, 10, 11, 12, 14, 18])
def test_stepped_weights_stay_inside(gap):
    for sink in (0.0, 0.02, 1.0):
        for block in (16, 64):
            assert held(case(gap, sink, block=block), wr.stepped_weights)[0] <= 1


@pytest.mark.parametrize("gap", [0, 8, 10, 12, 14])
def test_stepped_weights_are_no_worse_than_bf16_ones(gap):
    for sink in (0.0, 0.02, 1.0):
        a = case(gap, sink)
        assert held(a, wr.stepped_weights)[1] <= 1.1 * held(a, wr.bf16_weights)[1]


def test_size_of_the_error():
    worst, rms = held(ordinary(), wr.stepped_weights)
    assert worst <= 1 and rms <= wr.RMS
    spread = math.sqrt(1 / 3) * math.sqrt(3 / (8 * math.log(2)))   # of a half step's error, relative
    assert abs(2.0 ** -8 * spread - 1.66e-3) < 1e-5 and abs(2.0 ** -7 * spread ** 2 - 1.41e-3) < 1e-5
    assert abs(math.hypot(2.0 ** -8, 2.0 ** -7 * spread) * spread - 2.18e-3) < 1e-5


@pytest.mark.parametrize("gap", [10, 11, 12, 14])
def test_one_window_for_all_weights_is_found(gap):
    """An absolute smallest step of 2^-14 of the row's largest weight."""
    def window(suffix, prefix, scale):
        return suffix, torch.round(prefix * 2.0 ** 14) / 2.0 ** 14 * scale
    assert held(case(gap), window)[0] > 1


def test_planted_mistakes_are_found():
    a = ordinary()
    q, (k8, v8, s_k, s_v, block), ks, vs = a
    exactly = lambda s, p, scale: (s, p * scale)  # noqa: E731
    assert held(a, exactly)[0] <= 1
    assert held(a, lambda s, p, scale: (s, wr.to_type(p, 3, -40) * scale))[1] > wr.RMS  # the first term alone
    assert held(a, lambda s, p, scale: (s, wr.to_type(p, 5, -40) * scale))[1] > wr.RMS  # six bits of a weight
    assert held(a, lambda s, p, scale: (s, 0 * p))[0] > 1  # no prefix
    assert held(a, lambda s, p, scale: (s, p * scale.roll(block)))[0] > 1
    assert held(a, exactly, (q, (k8, v8, s_k.roll(1, 2), s_v, block), ks, vs))[0] > 1
    # values scaled by 2^-12, and the unit of the weights not
    small = (q, (k8, v8, s_k, s_v * 2.0 ** -12, block), ks, (vs.float() * 2.0 ** -12).to(BF))
    assert held(small, wr.stepped_weights)[0] <= 1
    assert held(small, lambda s, p, scale: (s, torch.round(p * 16) / 16 * scale))[0] > 1


def test_rows_of_zeros_with_a_scale_of_their_own():
    """A 16-row block without a value, whose scale is 1, does not set the unit of the
    block it shares a step with: as if its weights were zero; they were not, the others would be lost."""
    q, (k8, v8, s_k, s_v, _), ks, vs = ordinary(block=16)
    v8 = v8.clone()
    v8.view(torch.uint8)[:, :, 32:48] = 0
    s_v = s_v * 2.0 ** -40
    s_v[:, :, 2] = 1.0
    a = (q, (k8, v8, s_k, s_v, 16), ks, (vs.float() * 2.0 ** -40).to(BF))
    dead = torch.ones(900, dtype=F64)
    dead[32:48] = 0
    assert held(a, lambda s, p, scale: wr.stepped_weights(s, p * dead, scale))[0] <= 1
    lone = (q[:, :, :4], (k8[:, :, 32:64], v8[:, :, 32:64], s_k[:, :, 2:4], s_v[:, :, 2:4], 16), ks[:, :, :4], a[3][:, :, :4])
    vis = torch.ones(1, 32, dtype=torch.bool)
    o = wr.attention(*lone, vis)[0]
    assert wr.off(wr.with_weights(*lone, vis, wr.stepped_weights), o, torch.zeros_like(o))[1] > 0.1
