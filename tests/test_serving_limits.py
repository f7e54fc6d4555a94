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
