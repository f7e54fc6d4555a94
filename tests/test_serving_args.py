"""Refusals of the rotation, cache and tree-attention entry points: answered
on the host, before anything is enqueued (CPU only; pointers are never
dereferenced)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def native():
    from token_level_dynamic_b200 import _native
    return _native


P = ctypes.c_void_p(1 << 20)
MIS2, MIS1 = ctypes.c_void_p((1 << 20) + 2), ctypes.c_void_p((1 << 20) + 1)


def _rope_cfg(n, **kw):
    c = dict(rot_dim=128, layout=0, theta=5e5, factor=1.0, low_freq=0.0, high_freq=0.0,
             original_len=0, amplitude=1.0)
    c.update(kw)
    return n.WideRopeConfig(*c.values())


def test_rope_refusals(native):
    L, D = native.lib(), native.WideRopeDims
    ok, cfg = D(8, 40, 128, 0, 5120, 128, 5120, 128), _rope_cfg(native)
    call = lambda d=ok, c=cfg, x=P, p=P, o=P: L.wide_rope(  # noqa: E731
        x, p, o, ctypes.byref(d), ctypes.byref(c), None)
    for bad in (dict(rot_dim=0), dict(rot_dim=127), dict(rot_dim=130), dict(rot_dim=258),
                dict(layout=2), dict(theta=0.0), dict(theta=float("nan")), dict(factor=0.0),
                dict(factor=float("inf")), dict(amplitude=0.0), dict(original_len=-1),
                dict(factor=2.0, original_len=4096, low_freq=4.0, high_freq=4.0),
                dict(factor=2.0, original_len=4096, low_freq=-1.0, high_freq=4.0)):
        assert call(c=_rope_cfg(native, **bad)) == native.WIDE_EINVAL, bad
    for bad in (D(-1, 40, 128, 0, 5120, 128, 5120, 128), D(8, 0, 128, 0, 5120, 128, 5120, 128),
                D(8, 40, 64, 0, 5120, 128, 5120, 128),           # rot_dim > head_dim
                D(8, 40, 128, 7, 5120, 128, 5120, 128),
                D(8, 40, 128, 0, -5120, 128, 5120, 128),
                D(8, 40, 128, 0, 5120, 128, 0, 128),             # output tokens overlap
                D(8, 40, 128, 0, 5120, 128, 5120, 64)):          # output heads overlap
        assert call(d=bad) == native.WIDE_EINVAL
    assert call(x=None) == call(p=None) == call(o=None) == native.WIDE_EINVAL
    # in place needs the same strides
    assert call(d=D(8, 40, 128, 0, 10240, 128, 5120, 128)) == native.WIDE_EINVAL
    assert call(x=MIS1) == call(p=MIS2) == native.WIDE_EUNSUPPORTED
    for uns in (D(8, 2, 2048, 0, 5120, 2048, 5120, 2048), D(8, 2, 131, 0, 5120, 131, 5120, 131),
                D(8, 70000, 128, 0, 1 << 30, 128, 1 << 30, 128)):
        assert call(d=uns) == native.WIDE_EUNSUPPORTED
    assert L.wide_rope(None, None, None, ctypes.byref(D(0, 40, 128, 0, 0, 0, 0, 0)),
                       ctypes.byref(cfg), None) == native.WIDE_OK
    assert L.wide_rope(P, P, P, None, ctypes.byref(cfg), None) == native.WIDE_EINVAL
    assert L.wide_rope(P, P, P, ctypes.byref(ok), None, None) == native.WIDE_EINVAL


def _cache(n, kind=1, k=1 << 20, v=1 << 20, ks=1 << 20, vs=1 << 20, n_seq=2, cap=64, n_kv=8, hd=128):
    return n.WideKVCache(k, v, ks, vs, n_seq, cap, n_kv, hd, kind)


def test_kv_refusals(native):
    L, R = native.lib(), native.WideKVRows
    rows = R(4, 1024, 128, 1024, 128)

    def both(c=None, r=rows, k=P, v=P, start=P, count=P):
        c = _cache(native) if c is None else c
        a = L.wide_kv_append(k, v, ctypes.byref(c), start, count, None, ctypes.byref(r), None, None)
        b = L.wide_kv_read(k, v, ctypes.byref(c), start, count, ctypes.byref(r), None)
        assert a == b, (a, b)
        return a

    for bad in (_cache(native, kind=3), _cache(native, kind=-1), _cache(native, k=None),
                _cache(native, ks=None), _cache(native, n_seq=-1), _cache(native, cap=0),
                _cache(native, n_kv=0), _cache(native, hd=0)):
        assert both(bad) == native.WIDE_EINVAL
    for uns in (_cache(native, hd=64), _cache(native, k=(1 << 20) + 8), _cache(native, ks=(1 << 20) + 2),
                _cache(native, n_kv=2000), _cache(native, cap=1 << 31)):
        assert both(uns) == native.WIDE_EUNSUPPORTED
    assert both(k=None) == native.WIDE_EINVAL
    assert both(r=R(-1, 1024, 128, 1024, 128)) == native.WIDE_EINVAL
    assert both(r=R(4, -8, 128, 1024, 128)) == native.WIDE_EINVAL
    assert both(r=R(4, 1028, 128, 1024, 128)) == native.WIDE_EUNSUPPORTED      # not 16-byte pieces
    assert both(k=ctypes.c_void_p((1 << 20) + 8)) == native.WIDE_EUNSUPPORTED
    assert both(start=MIS2) == both(count=MIS2) == native.WIDE_EUNSUPPORTED
    assert both(r=R(0, 0, 0, 0, 0)) == native.WIDE_OK                          # no tokens
    assert both(_cache(native, n_seq=0, k=None, v=None, ks=None, vs=None)) == native.WIDE_OK
    # rows that would overlap are refused as a destination
    c = _cache(native)
    assert L.wide_kv_read(P, P, ctypes.byref(c), None, None, ctypes.byref(R(4, 64, 128, 1024, 128)),
                          None) == native.WIDE_EINVAL
    # rotation: at most the head, and in the half layout whole 16-element steps
    for kw, want in ((dict(rot_dim=256), native.WIDE_EINVAL), (dict(rot_dim=24), native.WIDE_EUNSUPPORTED),
                     (dict(theta=-1.0), native.WIDE_EINVAL)):
        cfg = _rope_cfg(native, **kw)
        assert L.wide_kv_append(P, P, ctypes.byref(c), None, None, None, ctypes.byref(rows),
                                ctypes.byref(cfg), None) == want
    assert L.wide_kv_append(P, P, None, None, None, None, ctypes.byref(rows), None,
                            None) == native.WIDE_EINVAL
    assert L.wide_kv_append(P, P, ctypes.byref(c), None, None, None, None, None,
                            None) == native.WIDE_EINVAL


def test_attn_tree_refusals(native):
    L, D = native.lib(), native.WideAttnTreeDims
    ok, c = D(8, 4096, 32, 0.088), _cache(native)
    ws = L.wide_attn_tree_workspace_bytes(ctypes.byref(c), ctypes.byref(ok))
    assert ws > 0

    def call(d=ok, c=c, q=P, cl=P, dl=None, tm=None, hm=None, o=P, w=P, n=ws):
        return L.wide_attn_tree(q, ctypes.byref(c), cl, dl, tm, hm, o, ctypes.byref(d), w, n, None)

    for bad in (D(0, 4096, 32, 0.088), D(8, 4096, 0, 0.088), D(8, 4096, 30, 0.088),
                D(8, 4096, 32, 0.0), D(8, 4096, 32, -1.0), D(8, 4096, 32, float("nan")),
                D(8, 4096, 32, float("inf")), D(8, -8, 32, 0.088)):
        assert call(d=bad) == native.WIDE_EINVAL
        assert L.wide_attn_tree_workspace_bytes(ctypes.byref(c), ctypes.byref(bad)) == 0
    assert call(d=D(8, 2048, 32, 0.088)) == native.WIDE_EINVAL                # tokens of q overlap
    for uns in (D(1025, 4096, 32, 0.088), D(8, 4100, 32, 0.088), D(8, 1 << 20, 8 * 33, 0.088)):
        assert call(d=uns) == native.WIDE_EUNSUPPORTED
    assert call(c=_cache(native, n_seq=600)) == native.WIDE_EUNSUPPORTED       # more than 4096 units
    assert call(c=_cache(native, hd=64)) == native.WIDE_EUNSUPPORTED
    for kw in (dict(q=None), dict(cl=None), dict(o=None), dict(w=None)):
        assert call(**kw) == native.WIDE_EINVAL
    for kw in (dict(q=ctypes.c_void_p((1 << 20) + 8)), dict(o=ctypes.c_void_p((1 << 20) + 8)),
               dict(cl=MIS2), dict(dl=MIS2), dict(tm=MIS2), dict(hm=MIS2),
               dict(w=ctypes.c_void_p((1 << 20) + 16))):
        assert call(**kw) == native.WIDE_EUNSUPPORTED
    assert call(n=ws - 1) == native.WIDE_EWORKSPACE
    assert call(c=_cache(native, n_seq=0, k=None, v=None, ks=None, vs=None)) == native.WIDE_OK


def test_status_string_names_the_range_bit(native):
    assert b"range" in native.lib().wide_status_string(native.WIDE_DEV_BAD_RANGE)


def test_bindings_check_dtypes_and_shapes():
    """What the C ABI cannot see stops in the binding; well-formed CPU tensors
    get as far as the device check."""
    import torch
    import token_level_dynamic_b200 as w
    bf = torch.bfloat16
    cfg = w.wide_rope_config(128)
    x, pos = torch.zeros(4, 2, 128, dtype=bf), torch.zeros(4, dtype=torch.int32)
    for args in ((x.half(), pos, cfg), ):
        with pytest.raises((TypeError, ValueError)):
            w.wide_rope(*args)
    with pytest.raises(ValueError):
        w.wide_rope(x[0], pos, cfg)
    with pytest.raises(ValueError):
        w.wide_rope(x, pos, cfg, out=x.float())
    with pytest.raises(ValueError):
        w.wide_rope(x.transpose(1, 2), pos, cfg)                   # elements not contiguous
    with pytest.raises(ValueError, match="CUDA tensor"):
        w.wide_rope(x, pos, cfg)

    cache = w.wide_kv_cache(2, 2, 8, torch.int8, device="cpu")
    assert cache["k_scale"].shape == (2, 2, 8, 4)
    with pytest.raises(TypeError):
        w.wide_kv_cache(2, 2, 8, torch.float16, device="cpu")
    k = torch.zeros(4, 2, 128, dtype=bf)
    with pytest.raises(ValueError):
        w.wide_kv_append(k[:3], k[:3], cache)                      # 3 rows, 2 sequences
    with pytest.raises(ValueError):
        w.wide_kv_append(k.float(), k, cache)
    with pytest.raises(ValueError):
        w.wide_kv_append(k[:, :1], k, cache)
    with pytest.raises(ValueError, match="CUDA tensor"):
        w.wide_kv_append(k, k, cache)
    with pytest.raises(ValueError):
        w.wide_kv_read(cache, None, 2, k=k.float())
    with pytest.raises(ValueError, match="CUDA tensor"):
        w.wide_kv_read(cache, None, 2)

    q, cl = torch.zeros(4, 4, 128, dtype=bf), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        w.wide_attn_tree(q.float(), cache, cl)
    with pytest.raises(ValueError):
        w.wide_attn_tree(q[:3], cache, cl)
    with pytest.raises(ValueError):
        w.wide_attn_tree(q, cache, cl, tree_mask=torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        w.wide_attn_tree(q, cache, cl, head_mask=torch.zeros(4, 1, dtype=torch.int64))
    with pytest.raises(ValueError):
        w.wide_attn_tree(q, {"k": cache["k"], "v": cache["v"]}, cl)  # 8 bits without scales
    with pytest.raises(TypeError):
        w.wide_attn_tree(q, {"k": cache["k"], "v": cache["v"].float()}, cl)
    with pytest.raises(ValueError):
        w.wide_attn_tree(q, cache, cl, out=q.float())
    with pytest.raises(ValueError, match="CUDA tensor"):
        w.wide_attn_tree(q, cache, cl)
