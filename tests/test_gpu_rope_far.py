"""wide_rope at near and far positions against the formula in 64-bit mantissas
(numpy's longdouble), element by element.

Bound: cos and sin are off by 4 * 2^-24 (the angle within half a turn rounded to
fp32, 2^-25 half turns or 1.6 * 2^-24 radians; the functions, 2^-24; the
amplitude's rounding and the product with it, 2^-24 in all) and by the angle's own
error in double: relative to it, 2 powers and their product 3, the division by the
factor 1, by 2 pi (itself rounded) 2, the product with the position 1, so under
8 * 2^-53; the ramp's g, from a ratio of at most 4 / 3 times its own 4 roundings,
and its products make it under 16.  The rotation multiplies and adds in fp32
(2^-24 of each product, together under 4 * 2^-24 (|a| + |b|)) and rounds once:
    |err| <= A (|a| + |b|) (8 * 2^-24 + k * 2^-53 |angle|) + 2^-24 |out|."""
import numpy as np
import pytest

from tests._util import from_dev

pytestmark = pytest.mark.gpu
POSITIONS = [0, 1, -1, 5, 4095, -4096, 100003, 1 << 20, -(1 << 24) + 1, 1 << 26, -(1 << 26), 1 << 29, 2 ** 31 - 1,
             -2 ** 31]


def _frequencies(rot, theta, factor, low, high, original):
    L = np.longdouble
    f = L(theta) ** (-(L(2) * np.arange(rot // 2).astype(L)) / L(rot))
    if factor == 1.0:
        return f
    if original == 0:
        return f / L(factor)
    r = L(original) * f / (2 * np.arccos(L(-1)))
    g = np.clip((r - L(low)) / (L(high) - L(low)), L(0), L(1))
    return f * (g + (1 - g) / L(factor))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [128, 64, 20])
@pytest.mark.parametrize("theta,factor,low,high,original,amp,k", [
    (5e5, 1.0, 0.0, 0.0, 0, 1.0, 8), (1e4, 4.0, 0.0, 0.0, 0, 1.0, 8), (5e5, 0.25, 0.0, 0.0, 0, 1.0, 8),
    (5e5, 8.0, 1.0, 4.0, 8192, 1.2079, 16)])
def test_rope_at_any_position(layout, rot, theta, factor, low, high, original, amp, k):
    import torch
    import token_level_dynamic_b200 as w
    assert np.finfo(np.longdouble).nmant >= 63
    x = torch.randn((len(POSITIONS), 3, 128), generator=torch.Generator().manual_seed(rot))
    pos = np.array(POSITIONS, dtype=np.int64)
    cfg = w.wide_rope_config(rot, theta, w.WIDE_ROPE_HALF if layout == "half" else w.WIDE_ROPE_INTERLEAVED,
                             factor=factor, low_freq=low, high_freq=high, original_len=original, amplitude=amp)
    got = from_dev(w.wide_rope(x.cuda(), torch.from_numpy(pos.astype(np.int32)).cuda(), cfg))
    xl = x.numpy().astype(np.longdouble)
    ang = pos.astype(np.longdouble)[:, None] * _frequencies(rot, theta, factor, low, high, original)
    c, s = (f(ang)[:, None] * np.longdouble(amp) for f in (np.cos, np.sin))
    h = rot // 2
    ia, ib = (np.arange(h), np.arange(h) + h) if layout == "half" else (2 * np.arange(h), 2 * np.arange(h) + 1)
    a, b = xl[..., ia], xl[..., ib]
    slack = amp * (np.abs(a) + np.abs(b)) * (8 * 2.0 ** -24 + k * 2.0 ** -53 * np.abs(ang)[:, None])
    for at, ref in ((ia, a * c - b * s), (ib, b * c + a * s)):
        err = np.abs(got[..., at] - ref)
        assert np.all(err <= slack + 2.0 ** -24 * (np.abs(ref) + slack)), float(np.max(err / slack))
    assert np.array_equal(got[..., rot:], from_dev(x)[..., rot:])
