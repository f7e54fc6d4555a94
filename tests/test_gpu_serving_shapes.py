"""wide_rope, wide_kv_append / wide_kv_read and wide_attn_tree at sizes that
take other paths of their kernels: pieces of 16 bytes that fill a block, several
tokens a block with odd heads, chunks of one sequence that begin before the
cache, cache rows past 2^31 bytes.  Oracles and bounds as in test_gpu_rope.py
and test_gpu_kv_cache.py."""
import numpy as np
import pytest

from oracle import serving
from tests import test_gpu_kv_cache as kv
from tests import test_gpu_rope as rope
from tests._util import from_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,n,hd,rot", [(3, 2, 1024, 256), (2500, 3, 64, 32), (1190, 37, 128, 128), (5000, 1, 256, 16),
                                        (1, 300, 128, 128), (65, 48, 80, 80)])
def test_rope_pieces(layout, dt, T, n, hd, rot):
    import torch
    import token_level_dynamic_b200 as w
    dtype = getattr(torch, dt)
    scaling, amp = rope.SCALINGS[T % 3]
    x, pos = rope._case(T, n, hd, dtype, T + rot)
    xd, p, cfg = x.cuda(), torch.from_numpy(pos).cuda(), rope._cfg(w, rot, layout, scaling, amp)
    got = w.wide_rope(xd, p, cfg)
    rope._check(got, x, pos, rot, layout, scaling, amp, dtype)
    assert w.wide_rope(xd, p, cfg, out=xd) is xd and torch.equal(xd, got)


@pytest.mark.parametrize("rot", [2, 10, 64, 128, 250, 256])
def test_rope_frequencies_of_every_pair(rot):
    """Position 1 shows each pair's frequency itself: cos and sin of f_i."""
    import torch
    import token_level_dynamic_b200 as w
    x = torch.zeros((1, 1, 256), device="cuda")
    x[..., 0:rot // 2] = 1.0
    got = w.wide_rope(x, torch.ones(1, dtype=torch.int32, device="cuda"), w.wide_rope_config(rot, 5e5))[0, 0]
    f = 5e5 ** (-2.0 * np.arange(rot // 2) / rot)
    assert np.max(np.abs(got[:rot // 2].cpu().double().numpy() - np.cos(f))) <= 8 * 2.0 ** -24
    assert np.max(np.abs(got[rot // 2:rot].cpu().double().numpy() - np.sin(f))) <= 8 * 2.0 ** -24


@pytest.mark.parametrize("kind", kv.KINDS)
@pytest.mark.parametrize("n_seq,seq_len,n_kv", [(3, 100, 1), (2, 45, 17), (1, 333, 2), (40, 3, 16), (7, 1, 64)])
def test_append_and_read_in_chunks(kind, n_seq, seq_len, n_kv):
    """Sequences of several chunks of tokens, some of which begin before the
    cache or end past it: those rows are skipped and reported, the others as
    the same rows appended alone."""
    import torch
    import token_level_dynamic_b200 as w
    cap = seq_len + 20
    rng = np.random.default_rng(n_seq)
    k, v = kv._rows(n_seq * seq_len, n_kv, 3, special=False)
    start = rng.integers(-seq_len // 2 - 1, cap - seq_len // 2, n_seq)
    count = rng.integers(0, seq_len + 1, n_seq)
    up = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
    got, want = (w.wide_kv_cache(n_seq, n_kv, cap, kv._dtype(kind)) for _ in range(2))
    w.wide_clear_device_status()
    w.wide_kv_append(k, v, got, up(start), count=up(count))
    out = w.wide_get_device_status()
    ko, vo = (torch.full_like(k, 7.0) for _ in range(2))
    w.wide_clear_device_status()
    w.wide_kv_read(got, up(start), seq_len, count=up(count), k=ko, v=vo)
    assert w.wide_get_device_status() == out
    w.wide_clear_device_status()
    # the rows that have a place, each by itself
    skipped = False
    there = np.zeros((n_seq, seq_len), bool)
    for s in range(n_seq):
        for i in range(count[s]):
            ok = 0 <= start[s] + i < cap
            skipped |= not ok
            there[s, i] = ok
    at = np.flatnonzero(there.reshape(-1))
    assert out == (w.WIDE_DEV_BAD_RANGE if skipped else 0)
    one = {n: t[:1].clone() for n, t in want.items()}
    for t in at[:: max(1, len(at) // 25)]:
        s, i = divmod(int(t), seq_len)
        p = int(start[s]) + i
        w.wide_kv_append(k[t:t + 1], v[t:t + 1], one, up([p]))
        for n in got:
            a, b = got[n][s, :, p].view(torch.uint8), one[n][0, :, p].view(torch.uint8)
            assert torch.equal(a, b), (n, s, p)
        kk, vv = w.wide_kv_read(one, up([p]), 1)
        assert torch.equal(ko[t], kk[0]) and torch.equal(vo[t], vv[0])
    rest = torch.from_numpy(~there.reshape(-1)).cuda()
    assert torch.all(ko[rest] == 7.0) and torch.all(vo[rest] == 7.0)
    # and nothing else in the cache
    for s in range(n_seq):
        used = torch.zeros(cap, dtype=torch.bool)
        used[[int(start[s]) + i for i in range(seq_len) if there[s, i]]] = True
        for n in got:
            assert torch.all(got[n][s][:, ~used].view(torch.uint8) == 0), (n, s)


@pytest.mark.parametrize("rep,N", [(4, 2), (4, 8), (4, 20), (4, 40)])
def test_attention_past_2_to_31_bytes(rep, N):
    """The same sequence in a cache of 3 GB of codes a tensor (heads 200 MB
    apart, the last past 2^31 bytes), in a small one and in one of 2048
    positions, which more than 16 rows of a group take to the large one's
    kernel: the same bits in the same kernel, and each within the bound of
    test_gpu_attn_tree.py."""
    import torch
    import token_level_dynamic_b200 as w
    n_kv, cap, have = 16, 3 << 19, 300
    big = {n: torch.empty((1, n_kv, cap, 128), dtype=torch.int8, device="cuda") for n in ("k", "v")}
    for n in ("k_scale", "v_scale"):
        big[n] = torch.full((1, n_kv, cap, 4), 255, dtype=torch.uint8, device="cuda")
    small = w.wide_kv_cache(1, n_kv, have + N, torch.int8)
    g = torch.Generator(device="cuda").manual_seed(N)
    k, v, q = (torch.randn((have + N if i < 2 else N, n_kv * (1 if i < 2 else rep), 128), generator=g, device="cuda")
               .to(torch.bfloat16) for i in range(3))
    for c in (big, small):
        w.wide_kv_append(k, v, c)
    cl = torch.tensor([have], dtype=torch.int32, device="cuda")
    same = w.wide_kv_cache(1, n_kv, 2048, torch.int8)
    w.wide_kv_append(k, v, same)
    outs = [w.wide_attn_tree(q, c, cl) for c in (big, same, small)]
    assert torch.equal(outs[0], outs[1])
    kd, vd = (from_dev(x).reshape(have + N, n_kv, 128).transpose(1, 0, 2)[None]
              for x in w.wide_kv_read(small, None, have + N))
    qd = from_dev(q).reshape(1, N, n_kv * rep, 128)
    ref, spread, reach = serving.attn_tree(qd, kd, vd, [have], [N], np.tril(np.ones((1, N, N), bool)),
                                           np.ones((1, N, n_kv), bool), 128 ** -0.5, np.zeros(qd.shape))
    e = 128 * 2.0 ** -23 * reach[..., None]
    bound = (2.0 ** -8 + 4 * e + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(ref)
    for out in (outs[0], outs[2]):
        assert np.all(np.abs(from_dev(out).reshape(ref.shape) - ref) <= bound)
