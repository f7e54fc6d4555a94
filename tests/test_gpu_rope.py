"""wide_rope on the GPU against the fp64 oracle.

Bound, element by element: the rotation is one product and one fused
multiply-add in fp32 on cos and sin that are within 4 units of 2^-24 (one turn
reduced exactly, cospi / sinpi of a rounded fp32 argument: 2^-24 * pi of angle
and about 2 units of the functions), times the amplitude rounded to fp32, so
    |err| <= 8 * 2^-24 * A (|a| + |b|) + half a step of the element type."""
import numpy as np
import pytest

from oracle import serving
from tests._util import from_dev

pytestmark = pytest.mark.gpu


def _case(T, n, hd, dtype, seed, far=100000):
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((T, n, hd)).astype(np.float32)).to(dtype)
    return x, rng.integers(-far, far, T).astype(np.int32)


def _check(got, x, pos, rot, layout, scaling, amplitude, dtype):
    import torch
    xf = from_dev(x)
    ref = serving.rope(xf, pos, rot, layout, amplitude, **scaling)
    mag = np.abs(xf)
    h = rot // 2
    ia, ib = (np.arange(h), np.arange(h) + h) if layout == "half" else (2 * np.arange(h), 2 * np.arange(h) + 1)
    bound = np.zeros_like(ref)
    bound[..., ia] = bound[..., ib] = 8 * 2.0 ** -24 * amplitude * (mag[..., ia] + mag[..., ib])
    bound += torch.finfo(dtype).eps / 2 * (np.abs(ref) + bound)
    bound[..., rot:] = 0.0                                    # copied
    err = np.abs(from_dev(got) - ref)
    assert np.all(err <= bound), float(np.max(err - bound))


SCALINGS = [({}, 1.0), (dict(factor=4.0), 1.0),
            (dict(factor=8.0, low=1.0, high=4.0, original=8192), 1.2079)]


def _cfg(w, rot, layout, scaling, amplitude):
    return w.wide_rope_config(rot, 5e5, w.WIDE_ROPE_HALF if layout == "half" else w.WIDE_ROPE_INTERLEAVED,
                              factor=scaling.get("factor", 1.0), low_freq=scaling.get("low", 0.0),
                              high_freq=scaling.get("high", 0.0), original_len=scaling.get("original", 0),
                              amplitude=amplitude)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,n,hd,rot", [
    (1, 1, 128, 128), (8, 40, 128, 128), (33, 5, 128, 64), (7, 3, 96, 36), (5, 2, 80, 18),
    (3, 7, 64, 2), (2, 1, 256, 256), (1, 3, 2, 2), (700, 4, 128, 128), (2, 33, 1024, 250)])
def test_rope_matches_the_definition(layout, dt, T, n, hd, rot):
    import torch
    import token_level_dynamic_b200 as w
    dtype = getattr(torch, dt)
    scaling, amp = SCALINGS[(T + rot) % 3]
    x, pos = _case(T, n, hd, dtype, T * 1000 + rot)
    xd = x.cuda()
    got = w.wide_rope(xd, torch.from_numpy(pos).cuda(), _cfg(w, rot, layout, scaling, amp))
    torch.cuda.synchronize()
    _check(got, x, pos, rot, layout, scaling, amp, dtype)
    assert torch.equal(xd.cpu(), x)


def test_rope_far_positions():
    import torch
    import token_level_dynamic_b200 as w
    x, _ = _case(6, 2, 128, torch.float32, 3)
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 24], dtype=np.int32)
    got = w.wide_rope(x.cuda(), torch.from_numpy(pos).cuda(), w.wide_rope_config(128))
    ref = serving.rope(from_dev(x), pos, 128)
    # the double product is 2^-53 of up to 2^31 radians off on either side: 2^-21 of angle in all
    tol = 8 * 2.0 ** -24 + np.where(np.abs(pos.astype(np.int64)) > 1 << 26, 2.0 ** -20, 0.0)
    assert np.all(np.abs(from_dev(got) - ref) <= tol[:, None, None] * 10)


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides_in_place_and_unaligned(layout, dt):
    """A fused QKV row's heads, heads-major output, one element past a 16-byte
    boundary, a broadcast input, and in place: same values as the plain call,
    and nothing around the rows is touched."""
    import torch
    import token_level_dynamic_b200 as w
    dtype = getattr(torch, dt)
    x, pos = _case(9, 6, 64, dtype, 5)
    p, cfg = torch.from_numpy(pos).cuda(), _cfg(w, 48, layout, *SCALINGS[2])
    ref = w.wide_rope(x.cuda(), p, cfg)
    fused = torch.full((9, 10 * 64 + 3), 7.0, dtype=dtype, device="cuda")
    for off in (0, 1, 64):
        fused.fill_(7.0)
        view = fused.as_strided((9, 6, 64), (fused.stride(0), 64, 1), off)
        view.copy_(x)
        heads_major = torch.empty((6, 9, 64), dtype=dtype, device="cuda").transpose(0, 1)
        assert torch.equal(w.wide_rope(view, p, cfg, out=heads_major), ref)
        assert w.wide_rope(view, p, cfg, out=view) is view
        assert torch.equal(view, ref)
        assert torch.all(fused[:, :off] == 7) and torch.all(fused[:, off + 6 * 64:] == 7)
    one = x[:, :1].cuda().expand(9, 6, 64)
    assert torch.equal(w.wide_rope(one, p, cfg), w.wide_rope(one.contiguous(), p, cfg))


def test_rope_gradient_is_the_rotation_back():
    """The gradient by differences of sum(c * rope(x)) equals rope(c, -position)
    (fp32; central differences of a linear map are exact up to rounding)."""
    import torch
    import token_level_dynamic_b200 as w
    x, pos = _case(2, 1, 32, torch.float32, 8)
    p, cfg = torch.from_numpy(pos).cuda(), _cfg(w, 20, "interleaved", *SCALINGS[2])
    c = torch.randn(2, 1, 32, generator=torch.Generator().manual_seed(1)).cuda()
    g = w.wide_rope(c, -p, cfg).cpu().double()
    for t in range(2):
        for d in range(32):
            e = torch.zeros(2, 1, 32, device="cuda")
            e[t, 0, d] = 1.0
            hi, lo = (w.wide_rope(x.cuda() + s * e, p, cfg).double() for s in (1.0, -1.0))
            diff = float(((hi - lo) * c.double()).sum()) / 2
            assert abs(diff - float(g[t, 0, d])) <= 64 * 2.0 ** -24 * 20


def test_rope_no_tokens_other_stream_and_graph():
    import torch
    import token_level_dynamic_b200 as w
    cfg = w.wide_rope_config(128)
    e = w.wide_rope(torch.empty((0, 3, 128), dtype=torch.bfloat16, device="cuda"),
                    torch.empty(0, dtype=torch.int32, device="cuda"), cfg)
    assert e.shape == (0, 3, 128)
    x, pos = _case(40, 8, 128, torch.bfloat16, 9)
    xd, p = x.cuda(), torch.from_numpy(pos).cuda()
    ref, out = w.wide_rope(xd, p, cfg), torch.empty_like(xd)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    w.wide_rope(xd, p, cfg, out=out, stream=st)
    st.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.wide_rope(xd, p, cfg, out=out)
    p.add_(5)
    xd.mul_(0.5)
    graph.replay()
    assert torch.equal(out, w.wide_rope(xd, p, cfg))
