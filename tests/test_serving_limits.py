"""Refusals at the ends of the parameters' ranges: what would reach a kernel as an
infinity or a zero is answered on the host (CPU only; pointers are never
dereferenced, and the calls that pass have nothing to enqueue)."""
import ctypes

import pytest

from tests.test_serving_args import P, _cache, _rope_cfg, native  # noqa: F401


@pytest.mark.parametrize("bad", [dict(amplitude=1e39), dict(amplitude=1e-60), dict(amplitude=float("inf")),
                                 dict(factor=1e-305), dict(theta=1e-308), dict(theta=1e-305, factor=0.5)])
def test_rope_parameters_that_are_not_finite_in_the_kernel(native, bad):  # noqa: F811
    L, cfg = native.lib(), _rope_cfg(native, **bad)
    d = native.WideRopeDims(0, 40, 128, 0, 0, 0, 0, 0)
    assert L.wide_rope(None, None, None, ctypes.byref(d), ctypes.byref(cfg), None) == native.WIDE_EINVAL
    c, rows = _cache(native), native.WideKVRows(0, 0, 0, 0, 0)
    assert L.wide_kv_append(P, P, ctypes.byref(c), None, None, None, ctypes.byref(rows), ctypes.byref(cfg),
                            None) == native.WIDE_EINVAL


@pytest.mark.parametrize("good", [dict(amplitude=3e38), dict(amplitude=1e-40), dict(factor=1e-250),
                                  dict(theta=1e308), dict(theta=1e-5), dict(factor=1e300)])
def test_rope_parameters_at_the_ends_of_their_range(native, good):  # noqa: F811
    L, cfg = native.lib(), _rope_cfg(native, **good)
    d = native.WideRopeDims(0, 40, 128, 0, 0, 0, 0, 0)
    assert L.wide_rope(None, None, None, ctypes.byref(d), ctypes.byref(cfg), None) == native.WIDE_OK


@pytest.mark.parametrize("scale,ok", [(1e-45, True), (2.0 ** 127, True), (2.36e38, False), (3.4e38, False)])
def test_attention_scales_that_the_kernels_can_hold(native, scale, ok):  # noqa: F811
    """The kernels multiply by scale * log2(e): an infinity makes NaN of scores of zero."""
    L, d, c = native.lib(), native.WideAttnTreeDims(8, 4096, 32, scale), _cache(native)
    assert (L.wide_attn_tree_workspace_bytes(ctypes.byref(c), ctypes.byref(d)) > 0) == ok
    c = _cache(native, n_seq=0, k=None, v=None, ks=None, vs=None)
    assert L.wide_attn_tree(None, ctypes.byref(c), None, None, None, None, None, ctypes.byref(d), None, 0,
                            None) == (native.WIDE_OK if ok else native.WIDE_EINVAL)


def test_sizes_past_the_documented_limits(native):  # noqa: F811
    """(the ones that test_serving_args.py does not have)"""
    L, cfg = native.lib(), _rope_cfg(native, rot_dim=2)
    for heads, hd, tokens in ((65536, 2, 1), (1, 2, (1 << 28) + 1), (1025, 1024, 1)):
        d = native.WideRopeDims(tokens, heads, hd, 0, 1 << 30, hd, 1 << 30, hd)
        assert L.wide_rope(P, P, P, ctypes.byref(d), ctypes.byref(cfg), None) == native.WIDE_EUNSUPPORTED
    for kw, seq_len in ((dict(n_seq=(1 << 24) + 1), 1), (dict(n_kv=1025), 1), (dict(cap=(1 << 30) + 1), 1),
                        (dict(n_seq=1), (1 << 24) + 1), (dict(n_seq=1 << 20), 257)):
        c, rows = _cache(native, **kw), native.WideKVRows(seq_len, 1 << 20, 128, 1 << 20, 128)
        assert L.wide_kv_append(P, P, ctypes.byref(c), None, None, None, ctypes.byref(rows), None,
                                None) == native.WIDE_EUNSUPPORTED
        assert L.wide_kv_read(P, P, ctypes.byref(c), None, None, ctypes.byref(rows),
                              None) == native.WIDE_EUNSUPPORTED
    # n_seq * n_kv * cap; the work's places
    for c, draft, n_q in ((dict(n_seq=1, n_kv=2, cap=1 << 30), 1, 2), (dict(n_seq=1024, n_kv=1, cap=1 << 20), 1024, 1)):
        c, d = _cache(native, **c), native.WideAttnTreeDims(draft, n_q * 128, n_q, 0.1)
        assert L.wide_attn_tree_workspace_bytes(ctypes.byref(c), ctypes.byref(d)) == 0
        assert L.wide_attn_tree(P, ctypes.byref(c), P, None, None, None, P, ctypes.byref(d), P, 1 << 40,
                                None) == native.WIDE_EUNSUPPORTED
