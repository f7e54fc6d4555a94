"""A step with drafted tokens, every operator's part against the fp64 oracle on
the step's inputs: queries and keys rotated by the tokens' depths in their trees,
keys and values in the cache and nowhere else, attention of the queries as the
oracle rotates them over what the cache stands for.

Bounds.  Rotated values: 8 * 2^-24 * A (|a| + |b|) as in test_gpu_rope.py (A = 1
here), then half a step of their format (bf16 2^-8, e4m3 2^-4 of the value or
2^-10 of the scale, int8 2^-1 of the scale).  Attention: the query's own rounding
moves a score by at most d = (2^-8 + 2^-20) * reach (reach = max_p scale *
sum_d |q_d k_pd|, which holds the rotation's 2^-21 as well for q of this size),
fp32 sums by e = 128 * 2^-23 * reach; a weight changes by a factor within
exp(+-2 (d + e)), so the output by (exp(2 (d + e)) - 1) * spread, the weights'
rounding adds 2^-8 * exp(2 (d + e)) * spread, fp32 2^-20 * spread and the last
rounding 2^-8 |out|."""
import numpy as np
import pytest

from oracle import serving
from tests._util import from_dev
from tests.test_gpu_attn_tree import KINDS, Case

pytestmark = pytest.mark.gpu
ROPE = dict(factor=8.0, low=1.0, high=4.0, original=8192)


def _step(kind, draft_len, seed):
    """The cache of an earlier state, the step's fused projection and its positions."""
    import torch
    S, N, n_kv, rep = 3, 7, 4, 4
    c = Case(kind, n_kv, rep, N, [65, 400, 3], draft_len, "random", 0.7, seed=seed)
    depth = c.tree.sum(-1) - 1
    pos = (c.cache_len[:, None] + depth).reshape(-1).astype(np.int32)
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((S * N, (n_kv * rep + 2 * n_kv) * 128), generator=g).to(torch.bfloat16).cuda()

    def heads(first, n):
        return qkv.as_strided((S * N, n, 128), (qkv.stride(0), 128, 1), first * 128)
    return c, pos, heads(0, n_kv * rep), heads(n_kv * rep, n_kv), heads(n_kv * rep + n_kv, n_kv)


def _rotated(x, pos):
    """(the exact rotation, its error in fp32) of rows of whole heads in the half layout."""
    x = from_dev(x)
    m = np.abs(x)
    pair = m[..., :64] + m[..., 64:]
    return serving.rope(x, pos, 128, **ROPE), 8 * 2.0 ** -24 * np.concatenate([pair, pair], -1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("draft_len", [None, [7, 5, 0]])
def test_step_against_the_definition(kind, draft_len):
    import torch
    import token_level_dynamic_b200 as w
    c, pos, q0, k0, v0 = _step(kind, draft_len, 11)
    before = {n: t.clone() for n, t in c.cache.items()}
    old = {n: c.values(n) for n in "kv"}
    p = torch.from_numpy(pos).cuda()
    rope = w.wide_rope_config(128, factor=8.0, low_freq=1.0, high_freq=4.0, original_len=8192)
    w.wide_clear_device_status()
    q = w.wide_rope(q0, p, rope)
    w.wide_kv_append(k0, v0, c.cache, c.cl, count=c.dl, rope=rope, positions=p)
    c.q = q
    got = c.run()
    assert w.wide_get_device_status() == 0

    # queries
    qx, slack = _rotated(q0, pos)
    assert np.all(np.abs(from_dev(q) - qx) <= slack + 2.0 ** -8 * (np.abs(qx) + slack))
    # the cache: new rows as defined, the others as they were
    kx, slack = _rotated(k0, pos)
    new = {n: c.values(n) for n in "kv"}
    for s in range(c.S):
        m, at = int(c.draft_len[s]), int(c.cache_len[s])
        keep = np.ones(c.cache["k"].shape[2], bool)
        keep[at:at + m] = False
        for n in c.cache:
            assert torch.equal(c.cache[n][s][:, keep].view(torch.uint8), before[n][s][:, keep].view(torch.uint8)), n
        for n in "kv":
            assert np.array_equal(new[n][s][:, keep], old[n][s][:, keep])
        rows = slice(s * c.N, s * c.N + m)
        have = new["k"][s, :, at:at + m].transpose(1, 0, 2)
        ref, sl = kx[rows], slack[rows]
        if kind == "bf16":
            bound = sl + 2.0 ** -8 * (np.abs(ref) + sl)
            vx = from_dev(v0)[rows]
        else:
            vx = serving.kv_decode(*serving.kv_encode(from_dev(v0)[rows], kind), kind)
            if m:
                top = np.max((np.abs(ref) + sl).reshape(m, c.n_kv, 4, 32), -1)
                scale = np.repeat(2.0 ** np.ceil(np.log2(top / serving.KV_MAX[kind])), 32, -1)
                half = scale / 2 if kind == "i8" else np.maximum(2.0 ** -4 * (np.abs(ref) + sl), scale * 2.0 ** -10)
                bound = half + sl
        if m:
            assert np.all(np.abs(have - ref) <= bound), float(np.max(np.abs(have - ref) / bound))
        assert np.array_equal(new["v"][s, :, at:at + m].transpose(1, 0, 2), vx)
    # attention of the exactly rotated queries
    out = np.full(qx.shape, 7.0).reshape(c.S, c.N, -1, 128)
    ref, spread, reach = serving.attn_tree(qx.reshape(out.shape), new["k"], new["v"], c.cache_len, c.draft_len,
                                           c.tree, c.heads, 128 ** -0.5, out)
    f = np.exp(2 * (2.0 ** -8 + 2.0 ** -20 + 128 * 2.0 ** -23) * reach)[..., None]
    bound = (f - 1 + 2.0 ** -8 * f + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(ref)
    err = np.abs(from_dev(got).reshape(ref.shape) - ref)
    assert np.all(err <= bound), float(np.max(err / np.maximum(bound, 1e-30)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("given", [True, False])
def test_a_chain_at_once_and_one_token_at_a_time(kind, given):
    """The same bits in the cache, with positions given and with the cache's own."""
    import torch
    import token_level_dynamic_b200 as w
    c, _, _, k0, v0 = _step(kind, None, 12)
    rope = w.wide_rope_config(128, factor=8.0, low_freq=1.0, high_freq=4.0, original_len=8192)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    chain = c.cache_len[:, None] + np.arange(c.N)[None]
    one = {n: t.clone() for n, t in c.cache.items()}
    w.wide_kv_append(k0, v0, c.cache, c.cl, rope=rope, positions=up(chain.reshape(-1)) if given else None)
    for i in range(c.N):
        rows = torch.arange(c.S, device="cuda") * c.N + i
        w.wide_kv_append(k0[rows], v0[rows], one, up(chain[:, i]), rope=rope,
                         positions=up(chain[:, i]) if given else None)
    for n in one:
        assert torch.equal(one[n].view(torch.uint8), c.cache[n].view(torch.uint8)), n
    k, v = w.wide_kv_read(c.cache, c.cl, c.N)
    kx, _ = _rotated(k0, chain.reshape(-1))
    assert torch.any(k != k0) and np.max(np.abs(from_dev(k) - kx)) <= np.max(np.abs(kx)) * 2.0 ** -4
    assert np.max(np.abs(from_dev(v) - from_dev(v0))) <= np.max(np.abs(from_dev(v0))) * 2.0 ** -4
