"""wide_attn_tree on the GPU against the fp64 oracle on the cached values.

Bound, element by element, with p the exact weights: a score is a 128-term
product sum kept to 23 bits or more, so off by at most
e = 128 * 2^-23 * max_p scale * sum_d |q_d k_pd| (the exponent's own product
and the base-2 exponential, 2^-22, are below it); a weight is rounded to bf16
(2^-8) and scaled by its row's sum, both within 2 e: the output is off by
(2^-8 + 4 e + 2^-20) * sum_p p |v_p| and the last rounding, 2^-8 |out|."""
import numpy as np
import pytest

from oracle import serving
from tests._util import from_dev

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "i8"]


def _words(bits):
    n = bits.shape[-1]
    pad = np.zeros(bits.shape[:-1] + (-(-n // 32) * 32,), dtype=np.uint8)
    pad[..., :n] = bits
    return np.packbits(pad, axis=-1, bitorder="little").view(np.uint32)


def _trees(rng, S, N):
    a = np.zeros((S, N, N), dtype=bool)
    for s in range(S):
        for i in range(N):
            p = int(rng.integers(-1, i)) if i else -1
            if p >= 0:
                a[s, i] = a[s, p]
            a[s, i, i] = True
    return a


class Case:
    """A problem on the device and its truth values on the host."""

    def __init__(self, kind, n_kv, rep, N, cache_len, draft_len=None, tree="random", keep=1.0, seed=0,
                 extra=5, peaky=2.0):
        import torch
        import token_level_dynamic_b200 as w
        rng = np.random.default_rng(seed)
        self.cache_len = np.asarray(cache_len, dtype=np.int32)
        S = self.S = len(self.cache_len)
        self.N, self.n_kv, self.rep, self.kind = N, n_kv, rep, kind
        self.draft_len = np.full(S, N, np.int32) if draft_len is None else np.asarray(draft_len, np.int32)
        cap = int(np.max(self.cache_len + self.draft_len)) + extra
        dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[kind]
        self.cache = w.wide_kv_cache(S, n_kv, cap, dt)
        x = rng.standard_normal((2, S * cap, n_kv, 128))
        x[0, :, :, 3::17] *= 5.0
        t = torch.from_numpy(x).to(torch.bfloat16).cuda()
        w.wide_kv_append(t[0], t[1], self.cache)
        self.q = torch.from_numpy(peaky * rng.standard_normal((S * N, n_kv * rep, 128))).to(torch.bfloat16).cuda()
        self.tree = np.tril(np.ones((N, N), bool))[None].repeat(S, 0) if tree == "chain" else \
            _trees(rng, S, N) if tree == "random" else rng.random((S, N, N)) < 0.4
        self.heads = rng.random((S, N, n_kv)) < keep
        self.tm = None if tree == "chain" else self._up(_words(self.tree).reshape(S * N, -1))
        self.hm = None if keep >= 1.0 else self._up(_words(self.heads).reshape(S * N, -1))
        self.cl = torch.from_numpy(self.cache_len).cuda()
        self.dl = None if draft_len is None else torch.from_numpy(self.draft_len).cuda()

    @staticmethod
    def _up(words):
        import torch
        return torch.from_numpy(np.ascontiguousarray(words).view(np.int32)).cuda()

    def run(self, **kw):
        import torch
        import token_level_dynamic_b200 as w
        if "out" not in kw:
            kw["out"] = torch.full_like(self.q, 7.0)
        return w.wide_attn_tree(self.q, self.cache, self.cl, tree_mask=self.tm, head_mask=self.hm,
                                draft_len=self.dl, **kw)

    def values(self, name):
        import token_level_dynamic_b200 as w
        cap = self.cache["k"].shape[2]
        kv = w.wide_kv_read(self.cache, None, cap)
        x = from_dev(kv[0 if name == "k" else 1])
        return x.reshape(self.S, cap, self.n_kv, 128).transpose(0, 2, 1, 3)

    def check(self, got, scale=128 ** -0.5):
        q = from_dev(self.q).reshape(self.S, self.N, self.n_kv * self.rep, 128)
        out = np.full(q.shape, 7.0)
        ref, spread, reach = serving.attn_tree(q, self.values("k"), self.values("v"), self.cache_len,
                                               self.draft_len, self.tree, self.heads, scale, out)
        g = from_dev(got).reshape(ref.shape)
        e = 128 * 2.0 ** -23 * reach[..., None]
        bound = (2.0 ** -8 + 4 * e + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(ref)
        assert np.array_equal(np.isnan(g), np.isnan(ref))
        fine = np.isfinite(ref)
        assert np.array_equal(g[~fine], ref[~fine], equal_nan=True)
        err = np.abs(g[fine] - ref[fine])
        assert np.all(err <= bound[fine]), float(np.max(err / np.maximum(bound[fine], 1e-30)))


@pytest.fixture(autouse=True)
def _status():
    import token_level_dynamic_b200 as w
    w.wide_clear_device_status()
    yield
    assert w.wide_get_device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_kv,rep,N,cache_len,draft_len,tree,keep", [
    (1, 1, 1, [0], None, "chain", 1.0),
    (1, 1, 1, [1], None, "chain", 1.0),
    (8, 4, 1, [2048], None, "chain", 1.0),
    (8, 4, 1, [300, 17, 0, 1], None, "chain", 0.5),
    (2, 3, 5, [63, 64, 65, 127], None, "random", 1.0),
    (2, 3, 5, [128, 129, 0, 59], [5, 0, 3, 1], "random", 0.4),
    (8, 4, 8, [500, 900], None, "random", 0.34),
    (4, 8, 16, [1000], None, "chain", 1.0),
    (3, 2, 33, [77, 10], [33, 31], "random", 0.6),
    (2, 4, 64, [700, 123], None, "random", 1.0),
    (2, 4, 61, [260], None, "random", 0.5),
    (1, 32, 3, [100], None, "chain", 1.0),
    (40, 1, 2, [30, 200], None, "chain", 0.5),
    (1, 5, 130, [40], None, "random", 0.8),
    (1, 1, 1024, [3], None, "chain", 1.0),
    (2, 2, 6, [0, 0], None, "holes", 1.0),
    (2, 2, 40, [0, 9], [40, 37], "holes", 0.7),
])
def test_matches_the_definition(kind, n_kv, rep, N, cache_len, draft_len, tree, keep):
    c = Case(kind, n_kv, rep, N, cache_len, draft_len, tree, keep, seed=N * 31 + n_kv)
    c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences_of_any_length(kind):
    """Units of different lengths share CTAs, runs are split between them."""
    rng = np.random.default_rng(1)
    c = Case(kind, 4, 4, 3, rng.integers(0, 700, 40), rng.integers(0, 4, 40), "random", 0.6, seed=2)
    c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
def test_long_context(kind):
    c = Case(kind, 1, 2, 4, [70001], None, "random", 1.0, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
def test_values_that_are_not_finite(kind):
    """A NaN or infinity in a new token's key or value reaches the rows that
    attend it and no others; one in the context reaches every row; rows past
    the sequence's end reach none."""
    import torch
    import token_level_dynamic_b200 as w
    for rep, N in ((2, 6), (4, 33)):
        c = Case(kind, 2, rep, N, [90], [N - 1], "random", 1.0, seed=4)
        bad = torch.randn(1, 2, 128, device="cuda").to(torch.bfloat16)

        def put(pos, k=None, v=None):
            kk, vv = w.wide_kv_read(c.cache, torch.tensor([pos], dtype=torch.int32, device="cuda"), 1)
            kk, vv = (kk if k is None else k), (vv if v is None else v)
            w.wide_kv_append(kk, vv, c.cache, torch.tensor([pos], dtype=torch.int32, device="cuda"))

        nan = bad.clone()
        nan[0, 0, 70] = float("nan")
        put(90 + N - 1, k=nan, v=nan)            # past the end
        got = c.run()
        assert torch.isfinite(got.view(1, N, -1)[:, :N - 1]).all()
        c.check(got)
        inf = bad.clone()
        inf[0, 0, 33] = float("inf")
        inf[0, 1, 34] = float("-inf")
        put(91, v=inf)                           # new token 1's value
        got = c.run()
        see = c.tree[0, :N - 1, 1]
        fin = torch.isfinite(got.view(1, N, 2, rep, 128)[0, :N - 1]).all(-1).all(-1).cpu().numpy()
        assert np.array_equal(fin[:, 0], ~see) and np.array_equal(fin[:, 1], ~see)
        c.check(got)
        put(92, k=nan)                           # new token 2's key, head 0
        got = c.run()
        g = torch.isnan(got.view(1, N, 2, rep, 128)[0, :N - 1]).all(-1).all(-1).cpu().numpy()
        assert np.array_equal(g[:, 0], c.tree[0, :N - 1, 2])
        put(10, v=nan)                           # the context
        got = c.run().view(1, N, 2, rep, 128)[0, :N - 1]
        assert torch.isnan(got[:, 0, :, 70]).all()


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_extreme_scales(kind):
    """Blocks of very large and very small values (scales from 2^-124 up)."""
    import torch
    import token_level_dynamic_b200 as w
    c = Case(kind, 2, 2, 3, [200], None, "chain", 1.0, seed=5)
    x = torch.randn(203, 2, 128, device="cuda")
    v = x.clone()
    v[:, 0, :32] *= 1e30
    v[:, 0, 32:64] *= 1e-30
    v[:, 1, 64:96] *= 2.0 ** 17
    x[:, 1, 0:32] *= 2.0 ** 20
    c.q[:, 2:, 0:32] *= 2.0 ** -21
    w.wide_kv_append(x.to(torch.bfloat16), v.to(torch.bfloat16), c.cache)
    c.check(c.run())


def test_lengths_out_of_range_are_flagged_and_left_out():
    import torch
    import token_level_dynamic_b200 as w
    c = Case("i8", 2, 2, 4, [10, 20, 30, 40, 50], [4, 4, 4, 4, 4], "chain", 0.5, seed=6)
    ref = c.run()
    c.cl[1], c.dl[2], c.dl[3], c.cl[4] = -1, 5, -2, c.cache["k"].shape[2] - 3
    got = c.run()
    assert w.wide_get_device_status() == w.WIDE_DEV_BAD_RANGE
    w.wide_clear_device_status()
    assert torch.equal(got[:4], ref[:4]) and torch.all(got[4:] == 7.0)


@pytest.mark.parametrize("kind", KINDS)
def test_strided_q_scale_workspace_and_repeat(kind):
    """q inside a wider row, a scale of its own, a caller's workspace full of
    NaN, and the same call twice: bit-equal outputs."""
    import torch
    import token_level_dynamic_b200 as w
    c = Case(kind, 2, 4, 7, [333, 50], None, "random", 0.7, seed=7)
    ref = c.run(scale=0.05)
    c.check(ref, scale=0.05)
    wide = torch.zeros(c.q.shape[0], 8 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    view = wide.as_strided(c.q.shape, (wide.stride(0), 128, 1), 8)
    view.copy_(c.q)
    c.q = view
    need = w.wide_attn_tree_workspace_bytes(c.cache, 7, 8)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((14, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        assert torch.equal(c.run(scale=0.05, workspace=ws, out=out), ref)
    assert torch.all(ws[need:] == 255)


def test_other_stream_and_graph_replay():
    """Captured once, replayed with other lengths, masks and queries; and on a
    stream of its own."""
    import torch
    import token_level_dynamic_b200 as w
    c = Case("e4m3", 4, 4, 6, [900, 300], [6, 4], "random", 0.6, seed=8)
    ref = c.run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out, ws = torch.full_like(c.q, 7.0), torch.empty(w.wide_attn_tree_workspace_bytes(c.cache, 6, 16),
                                                     dtype=torch.uint8, device="cuda")
    c.run(out=out, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, workspace=ws)
    c.cl.copy_(torch.tensor([100, 901], dtype=torch.int32))
    c.dl.copy_(torch.tensor([2, 6], dtype=torch.int32))
    c.q.neg_()
    c.hm.bitwise_not_()
    out.fill_(7.0)
    graph.replay()
    assert torch.equal(out, c.run())
    graph.replay()
    assert torch.equal(out, c.run())


@pytest.mark.parametrize("kind", KINDS)
def test_a_step_with_drafted_tokens(kind):
    """Rotation, append and attention as a step uses them: drafted tokens'
    positions are their depths in the tree; the result equals the oracle on
    the fp64-rotated query over the cached keys, and the bf16 cache agrees
    with a chain appended one token at a time."""
    import torch
    import token_level_dynamic_b200 as w
    S, N, n_kv, rep = 3, 7, 4, 4
    rng = np.random.default_rng(9)
    c = Case(kind, n_kv, rep, N, [65, 400, 3], [7, 5, 7], "random", 0.7, seed=9)
    depth = c.tree.sum(-1) - 1
    pos = torch.from_numpy((c.cache_len[:, None] + depth).reshape(-1).astype(np.int32)).cuda()
    qkv = torch.from_numpy(rng.standard_normal((S * N, (n_kv * rep + 2 * n_kv) * 128))).to(torch.bfloat16).cuda()
    head = lambda a, n: qkv.as_strided((S * N, n, 128), (qkv.stride(0), 128, 1), a * 128)  # noqa: E731
    rope = w.wide_rope_config(128, factor=8.0, low_freq=1.0, high_freq=4.0, original_len=8192)
    q = w.wide_rope(head(0, n_kv * rep), pos, rope)
    w.wide_kv_append(head(n_kv * rep, n_kv), head(n_kv * rep + n_kv, n_kv), c.cache, c.cl, count=c.dl, rope=rope,
                     positions=pos)
    kw = dict(factor=8.0, low=1.0, high=4.0, original=8192)
    assert np.max(np.abs(from_dev(q) - serving.rope(from_dev(head(0, n_kv * rep)), pos.cpu().numpy(), 128, **kw))) \
        <= 2.0 ** -8 * 8
    c.q = q
    c.check(c.run())
