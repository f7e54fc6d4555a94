"""wide_kv_append / wide_kv_read on the GPU against the fp64 oracle.

Without a rotation both are exact: codes, scale bytes and the values read back
equal the definition's bit for bit.  With one, K is rotated in fp32 (error
<= 8 * 2^-24 A (|a| + |b|), see test_gpu_rope) before its one rounding, so a
value is at most half a code step of its block plus that from the exact
rotation: e4m3 half a step is 2^-4 of the value or 2^-10 of the scale, int8
2^-1 of the scale, bf16 2^-8 of the value."""
import numpy as np
import pytest

from oracle import serving
from tests._util import from_dev

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "i8"]


def _dtype(kind):
    import torch
    return {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[kind]


def _rows(T, n_kv, seed, special=True):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((2, T, n_kv, 128)) * np.exp(rng.uniform(-12, 12, (2, T, n_kv, 1)))
    x[:, :, :, 5] *= 30.0
    if special:
        x[0, 0, 0, 0:32] = 0.0
        x[1, 0, 0, 96:128] = 0.0
        x[0, -1, -1, 40] = np.inf
        x[1, -1, -1, 127] = np.nan
        x[0, 0, -1, 64:96] = 3e38 * rng.uniform(-1, 1, 32)
        x[1, -1, 0, 32:64] = 1e-39 * rng.uniform(-1, 1, 32)
        x[1, -1, 0, 0:32] = 2.0 ** -120 * rng.uniform(-1, 1, 32)
    t = torch.from_numpy(x).to(torch.bfloat16).cuda()
    return t[0], t[1]


def _bits(t):
    import torch
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()


def _fill(cache, value):
    import torch
    for t in cache.values():
        t.view(torch.uint8).fill_(value)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_seq,seq_len,n_kv,cap", [(1, 1, 1, 1), (16, 1, 8, 70), (3, 17, 3, 40), (2, 130, 8, 200),
                                                    (5, 7, 33, 9)])
def test_append_then_read_is_exact(kind, n_seq, seq_len, n_kv, cap):
    import torch
    import token_level_dynamic_b200 as w
    rng = np.random.default_rng(n_seq * seq_len)
    k, v = _rows(n_seq * seq_len, n_kv, 4)
    count = rng.integers(0, seq_len + 1, n_seq).astype(np.int32)
    count[0] = seq_len
    start = rng.integers(0, cap - seq_len + 1, n_seq).astype(np.int32)
    cache = w.wide_kv_cache(n_seq, n_kv, cap, _dtype(kind))
    _fill(cache, 0x2a)
    st, ct = torch.from_numpy(start).cuda(), torch.from_numpy(count).cuda()
    w.wide_clear_device_status()
    w.wide_kv_append(k, v, cache, st, count=ct)
    ko, vo = (torch.full_like(k, 7.0) for _ in range(2))
    w.wide_kv_read(cache, st, seq_len, count=ct, k=ko, v=vo)
    torch.cuda.synchronize()
    assert w.wide_get_device_status() == 0
    for name, src, back in (("k", k, ko), ("v", v, vo)):
        codes = np.full((n_seq, n_kv, cap, 128), 0x2a2a if kind == "bf16" else 0x2a,
                        dtype=np.int16 if kind == "bf16" else np.uint8)
        scale = np.full((n_seq, n_kv, cap, 4), 0x2a, dtype=np.uint8)
        want = np.full(src.shape, 7.0)
        for s in range(n_seq):
            m = int(count[s])
            rows = src[s * seq_len:s * seq_len + m]
            if kind == "bf16":
                codes[s, :, start[s]:start[s] + m] = _bits(rows).transpose(1, 0, 2)
                want[s * seq_len:s * seq_len + m] = from_dev(rows)
            else:
                c, b = serving.kv_encode(from_dev(rows), kind)
                codes[s, :, start[s]:start[s] + m] = c.view(np.uint8).transpose(1, 0, 2)
                scale[s, :, start[s]:start[s] + m] = b.transpose(1, 0, 2)
                want[s * seq_len:s * seq_len + m] = serving.kv_decode(c, b, kind)
        assert np.array_equal(_bits(cache[name]), codes), name
        if kind != "bf16":
            assert np.array_equal(cache[name + "_scale"].cpu().numpy(), scale), name
        assert np.array_equal(from_dev(back), want, equal_nan=True), name


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout,rot", [("half", 128), ("half", 48), ("half", 16), ("interleaved", 128),
                                        ("interleaved", 34), ("interleaved", 2)])
@pytest.mark.parametrize("given", [False, True])
def test_append_rotates_keys(kind, layout, rot, given):
    import torch
    import token_level_dynamic_b200 as w
    n_seq, seq_len, n_kv = 3, 6, 5
    rng = np.random.default_rng(rot)
    k, v = _rows(n_seq * seq_len, n_kv, 6, special=False)
    start = np.array([3, 1000, 60000], dtype=np.int32)
    pos = (start[:, None] + np.arange(seq_len)).reshape(-1).astype(np.int32)
    if given:
        pos = rng.integers(0, 1 << 20, n_seq * seq_len).astype(np.int32)
    amp = 1.25
    cfg = w.wide_rope_config(rot, 1e4, w.WIDE_ROPE_HALF if layout == "half" else w.WIDE_ROPE_INTERLEAVED,
                             factor=8.0, low_freq=1.0, high_freq=4.0, original_len=8192, amplitude=amp)
    cache = w.wide_kv_cache(n_seq, n_kv, 60100, _dtype(kind))
    st = torch.from_numpy(start).cuda()
    w.wide_kv_append(k, v, cache, st, rope=cfg, positions=torch.from_numpy(pos).cuda() if given else None)
    ko, vo = w.wide_kv_read(cache, st, seq_len)
    kf = from_dev(k)
    ref = serving.rope(kf, pos, rot, layout, amp, theta=1e4, factor=8.0, low=1.0, high=4.0, original=8192)
    mag = np.abs(kf)
    h = rot // 2
    ia, ib = (np.arange(h), np.arange(h) + h) if layout == "half" else (2 * np.arange(h), 2 * np.arange(h) + 1)
    slack = np.zeros_like(ref)
    slack[..., ia] = slack[..., ib] = 8 * 2.0 ** -24 * amp * (mag[..., ia] + mag[..., ib])
    if kind == "bf16":
        bound = slack + 2.0 ** -8 * (np.abs(ref) + slack)
        assert np.array_equal(from_dev(vo), from_dev(v))
    else:
        top = np.max((np.abs(ref) + slack).reshape(*ref.shape[:-1], 4, 32), -1)
        scale = np.repeat(2.0 ** np.ceil(np.log2(top / serving.KV_MAX[kind])), 32, -1)
        half = scale / 2 if kind == "i8" else np.maximum(2.0 ** -4 * (np.abs(ref) + slack), scale * 2.0 ** -10)
        bound = half + slack
        c, b = serving.kv_encode(from_dev(v), kind)
        assert np.array_equal(from_dev(vo), serving.kv_decode(c, b, kind))
    err = np.abs(from_dev(ko) - ref)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("kind", KINDS)
def test_strided_rows_and_defaults(kind):
    """K and V as views of a fused projection's output; start and count left
    out; the same rows read back into a strided destination."""
    import torch
    import token_level_dynamic_b200 as w
    qkv = torch.randn(2 * 5, 4 * 128 + 2 * 2 * 128 + 8, device="cuda").to(torch.bfloat16)
    k, v = (qkv.as_strided((10, 2, 128), (qkv.stride(0), 128, 1), 512 + 256 * i) for i in range(2))
    a, b = w.wide_kv_cache(2, 2, 5, _dtype(kind)), w.wide_kv_cache(2, 2, 5, _dtype(kind))
    w.wide_kv_append(k, v, a)
    w.wide_kv_append(k.contiguous(), v.contiguous(), b, torch.zeros(2, dtype=torch.int32, device="cuda"),
                     count=torch.full((2,), 5, dtype=torch.int32, device="cuda"))
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), n
    back = torch.full_like(qkv, 9.0)
    kb, vb = (back.as_strided((10, 2, 128), (back.stride(0), 128, 1), 512 + 256 * i) for i in range(2))
    w.wide_kv_read(a, None, 5, k=kb, v=vb)
    kr, vr = w.wide_kv_read(b, None, 5)
    assert torch.equal(kb, kr) and torch.equal(vb, vr)
    assert torch.all(back[:, :512] == 9) and torch.all(back[:, 1024:] == 9)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_out_of_range_are_flagged_and_skipped(kind):
    import torch
    import token_level_dynamic_b200 as w
    k, v = _rows(4 * 3, 2, 11, special=False)
    cache = w.wide_kv_cache(4, 2, 8, _dtype(kind))
    _fill(cache, 0x2a)
    good = {n: t.clone() for n, t in cache.items()}
    start = torch.tensor([2, 6, -1, 0], dtype=torch.int32, device="cuda")
    count = torch.tensor([3, 3, 1, 4], dtype=torch.int32, device="cuda")     # 1: one row past the end, 3: too many
    w.wide_kv_append(k, v, good, torch.tensor([2, 6, 0, 0], dtype=torch.int32, device="cuda"),
                     count=torch.tensor([3, 2, 0, 0], dtype=torch.int32, device="cuda"))
    w.wide_clear_device_status()
    w.wide_kv_append(k, v, cache, start, count=count)
    assert w.wide_get_device_status() == w.WIDE_DEV_BAD_RANGE
    for n in cache:
        assert torch.equal(cache[n].view(torch.uint8), good[n].view(torch.uint8)), n
    w.wide_clear_device_status()
    ko, vo = (torch.full_like(k, float("nan")) for _ in range(2))
    w.wide_kv_read(cache, start, 3, count=count, k=ko, v=vo)
    assert w.wide_get_device_status() == w.WIDE_DEV_BAD_RANGE
    w.wide_clear_device_status()
    there = torch.zeros(12, dtype=torch.bool, device="cuda")
    there[[0, 1, 2, 3, 4]] = True
    assert torch.isnan(ko[~there]).all() and torch.isnan(vo[~there]).all()
    assert torch.isfinite(ko[there]).all() and torch.isfinite(vo[there]).all()


def test_long_cache_offsets_pass_32_bits():
    """Rows past 2^31 elements of the cache (3 GB of codes)."""
    import torch
    import token_level_dynamic_b200 as w
    n_kv, cap = 16, 3 << 19
    cache = {"k": torch.empty((1, n_kv, cap, 128), dtype=torch.int8, device="cuda"),
             "v": torch.empty((1, n_kv, cap, 128), dtype=torch.int8, device="cuda"),
             "k_scale": torch.empty((1, n_kv, cap, 4), dtype=torch.uint8, device="cuda"),
             "v_scale": torch.empty((1, n_kv, cap, 4), dtype=torch.uint8, device="cuda")}
    k, v = _rows(5, n_kv, 12, special=False)
    start = torch.tensor([cap - 5], dtype=torch.int32, device="cuda")
    w.wide_kv_append(k, v, cache, start)
    ko, vo = w.wide_kv_read(cache, start, 5)
    for src, got in ((k, ko), (v, vo)):
        assert np.array_equal(from_dev(got), serving.kv_decode(*serving.kv_encode(from_dev(src), "i8"), "i8"))


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_append_read_stream_and_graph(kind):
    import torch
    import token_level_dynamic_b200 as w
    k, v = _rows(8, 4, 13, special=False)
    start = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    cfg = w.wide_rope_config(128)
    cache, ref = (w.wide_kv_cache(2, 4, 20, _dtype(kind)) for _ in range(2))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    w.wide_kv_append(k, v, cache, start, rope=cfg, stream=st)
    st.synchronize()
    w.wide_kv_append(k, v, ref, start, rope=cfg)
    assert all(torch.equal(cache[n].view(torch.uint8), ref[n].view(torch.uint8)) for n in cache)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.wide_kv_append(k, v, cache, start, rope=cfg)
        w.wide_kv_read(cache, start, 4, k=ko, v=vo)
    k.neg_()
    start.add_(4)
    graph.replay()
    w.wide_kv_append(k, v, ref, start, rope=cfg)
    kr, vr = w.wide_kv_read(ref, start, 4)
    assert torch.equal(ko, kr) and torch.equal(vo, vr)
