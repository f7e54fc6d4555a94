"""wide_attn_tree at the borders of its row layouts (16, 32, 64, 128, 256 rows
of a run) and of its division of the work: many units, runs split between
CTAs, references that rise with every tile, nothing kept, nothing attended.
Most cases run in a cache just large enough and in one with room for more
positions, which takes the other kernel (checked by the launches' names).
Oracle and bound as in test_gpu_attn_tree.py."""
import numpy as np
import pytest

from tests.test_gpu_attn_tree import KINDS, Case

pytestmark = pytest.mark.gpu
ROOM = ["small", "roomy"]      # caches of the rows kernel and of the tiles kernel


def _roomy(c, room):
    """The case in a cache with so much room that the tiles kernel takes it
    (its rule: blocks of 16 rows and 128 positions of the whole cache)."""
    import token_level_dynamic_b200 as w
    if room == "roomy":
        rows = c.N * c.rep
        rt = next(r for r in (32, 64, 128, 256) if rows <= r or r == 256)
        cap = 128 * (-(-(256 + 5 * rt) // (c.S * c.n_kv * -(-rows // 16))) + 1)
        old, values = c.cache, {n: c.values(n) for n in ("k", "v")}
        c.values = values.get
        if cap > old["k"].shape[2]:
            c.cache = w.wide_kv_cache(c.S, c.n_kv, cap, old["k"].dtype)
            for n in old:
                c.cache[n][:, :, :old[n].shape[2]].copy_(old[n])
    return c


def _launched(call):
    import token_level_dynamic_b200 as w
    w.wide_profile_start(64)
    out = call()
    w.wide_profile_stop()
    return out, [n for n, _ in w.wide_profile_read(64)]


@pytest.fixture(autouse=True)
def _status():
    import token_level_dynamic_b200 as w
    w.wide_clear_device_status()
    yield
    assert w.wide_get_device_status() == 0


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rep,N", [(1, 16), (1, 17), (3, 11), (8, 8), (5, 13), (2, 64), (3, 43), (4, 64),
                                   (1, 257), (32, 17)])
def test_rows_at_the_borders_of_the_layouts(room, kind, rep, N):
    """Runs of up to 16, 32, 64, 128 and 256 rows, and several runs a unit."""
    c = Case(kind, 2, rep, N, [130, 257], [N, max(N - 2, 0)], "random", 1.0, seed=rep * 100 + N)
    c = _roomy(c, room)
    c.check(c.run())


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rep,N", [(4, 1), (4, 8), (4, 16), (4, 32), (4, 64)])
def test_one_token_of_context_to_a_tile_more(room, kind, rep, N):
    """Contexts around the tiles of 128 keys, without and with a tail of new positions."""
    c = Case(kind, 1, rep, N, [0, 1, 127, 128, 129, 255, 256, 383], None, "random", 0.8, seed=N)
    c = _roomy(c, room)
    c.check(c.run())


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rep,N", [(4, 4), (4, 8), (4, 16), (4, 32), (4, 64)])
def test_reference_rises_with_every_tile(room, kind, rep, N):
    """Keys that grow along the context: the running maximum moves in every
    tile, by more than the 2^8 that a reference may lag, and the last keys
    take all of the weight."""
    import torch
    import token_level_dynamic_b200 as w
    c = Case(kind, 1, rep, N, [1500], None, "random", 1.0, seed=N + 1)
    cap = c.cache["k"].shape[2]
    g = torch.Generator(device="cuda").manual_seed(N)
    k = torch.randn((cap, 1, 128), generator=g, device="cuda")
    k[:, :, :32] += 0.02 * torch.arange(cap, device="cuda")[:, None, None]
    c.q[:, :, :32] = c.q[:, :, :32].abs()
    v = torch.randn((cap, 1, 128), generator=g, device="cuda")
    small = c.cache
    for falling in (False, True):
        # rising; then falling: the first tile's reference stays
        c.cache = small
        c.__dict__.pop("values", None)
        kk = k.flip(0).contiguous() if falling else k
        w.wide_kv_append(kk.to(torch.bfloat16), v.to(torch.bfloat16), c.cache)
        _roomy(c, room)
        c.check(c.run())


@pytest.mark.parametrize("kind", ["bf16", "i8"])
@pytest.mark.parametrize("rep,N", [(2, 2), (4, 6), (4, 33)])
def test_more_units_than_a_planning_window(kind, rep, N):
    """2400 units of many lengths, some of no length, shared out to the CTAs."""
    rng = np.random.default_rng(N)
    lens = rng.integers(0, 90, 300)
    lens[rng.random(300) < 0.3] = 0
    new = rng.integers(0, N + 1, 300)
    c = Case(kind, 8, rep, N, lens, new, "random", 0.4, seed=N)
    c.check(c.run())


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("rep,N", [(2, 4), (4, 8), (4, 40)])
def test_nothing_kept_and_nothing_new(room, rep, N):
    """All pairs skipped: zeros for the tokens that there are.  No new tokens: nothing is written."""
    import torch
    c = Case("e4m3", 4, rep, N, [300, 0, 40], [N, N, 0], "random", 0.5, seed=1)
    c.hm.zero_()
    c.heads[:] = False
    c = _roomy(c, room)
    got = c.run()
    assert torch.all(got[:2 * N] == 0) and torch.all(got[2 * N:] == 7.0)
    c.dl.zero_()
    assert torch.all(c.run() == 7.0)


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("kind", KINDS)
def test_infinite_keys(room, kind):
    """An infinite key (a NaN key in 8 bits) of the context makes every row
    NaN that it reaches with a positive score, in every layout."""
    import torch
    import token_level_dynamic_b200 as w
    for rep, N in ((4, 4), (4, 8), (4, 32), (4, 64)):
        c = Case(kind, 1, rep, N, [200], None, "chain", 1.0, seed=2)
        kk, vv = w.wide_kv_read(c.cache, torch.tensor([150], dtype=torch.int32, device="cuda"), 1)
        kk[0, 0, 5] = float("inf")
        w.wide_kv_append(kk, vv, c.cache, torch.tensor([150], dtype=torch.int32, device="cuda"))
        c = _roomy(c, room)
        got = c.run()
        hit = (c.q[:, :, 5] > 0) if kind == "bf16" else torch.ones_like(c.q[:, :, 5], dtype=torch.bool)
        assert torch.isnan(got[hit]).all() and torch.isfinite(got[~hit]).all()


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("rep,N", [(4, 3), (4, 16), (4, 61)])
def test_two_graphs_on_one_workspace(room, rep, N):
    """Two captured calls on one workspace, replayed in turn, give what the
    eager calls gave, bit for bit."""
    import torch
    import token_level_dynamic_b200 as w
    cs = [Case(k, 4, rep, N, [700, 33], [N, N - 1], "random", 0.7, seed=5 + i) for i, k in enumerate(("i8", "i8"))]
    cs = [_roomy(c, room) for c in cs]
    refs = [c.run() for c in cs]
    ws = torch.empty(max(w.wide_attn_tree_workspace_bytes(c.cache, N, 4 * rep) for c in cs),
                     dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.full_like(c.q, 7.0) for c in cs], []
    for c, o in zip(cs, outs):
        c.run(out=o, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, r in zip(outs, refs):
            assert torch.equal(o, r)


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("kind", KINDS)
def test_long_run_repeats_bit_for_bit(room, kind):
    """Long contexts split over all CTAs, run again and again while the parts
    arrive in another order: the same bits, and the device stays clear of
    errors (waits that give up, parts in the wrong place)."""
    import torch
    for rep, N in ((4, 16), (4, 64)):
        c = Case(kind, 2, rep, N, [9000, 2500], None, "random", 0.6, seed=6)
        c = _roomy(c, room)
        ref = c.run()
        c.check(ref)
        for _ in range(20):
            assert torch.equal(c.run(), ref)


@pytest.mark.parametrize("room,rep,N,kernel", [("small", 4, 4, "attn_tree"), ("roomy", 4, 4, "attn_tree"),
                                               ("small", 4, 8, "attn_tree"), ("roomy", 1, 17, "attn_tree_tiles"),
                                               ("roomy", 4, 64, "attn_tree_tiles"), ("small", 4, 64, "attn_tree")])
def test_which_kernel_runs(room, rep, N, kernel):
    c = _roomy(Case("i8", 1, rep, N, [100], None, "chain", 1.0), room)
    out, names = _launched(c.run)
    assert names == [kernel, "attn_tree_join"], names
    c.check(out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rep,N", [(4, 8), (4, 16), (4, 32), (4, 64), (3, 85)])
def test_new_values_that_are_not_finite(kind, rep, N):
    """In the tiles kernel: an infinity or NaN in a new token's value reaches
    the rows that attend it and no others, one past the end none, one in a new
    token's key the rows that attend it."""
    import torch
    import token_level_dynamic_b200 as w
    for which in ("v", "k", "past"):
        c = Case(kind, 2, rep, N, [190], [N - 1], "random", 1.0, seed=7)
        pos = 190 + (N - 1 if which == "past" else 2)
        at = torch.tensor([pos], dtype=torch.int32, device="cuda")
        kk, vv = w.wide_kv_read(c.cache, at, 1)
        x = vv if which != "k" else kk
        x[0, 0, 33] = float("nan") if which == "k" else float("inf")
        x[0, 1, 100] = float("nan")
        w.wide_kv_append(kk, vv, c.cache, at)
        _roomy(c, "roomy")
        got, names = _launched(c.run)
        assert names[0] == "attn_tree_tiles"
        bad = ~torch.isfinite(got.view(N, 2, rep, 128)[:N - 1]).all(-1).all(-1).cpu().numpy()
        sees = c.tree[0, :N - 1, 2] if which != "past" else np.zeros(N - 1, bool)
        assert np.array_equal(bad[:, 0], sees) and np.array_equal(bad[:, 1], sees)
        c.check(got)


@pytest.mark.parametrize("rep,N", [(4, 8), (4, 33), (4, 64)])
def test_replay_with_other_lengths_and_strided_queries(rep, N):
    """In the tiles kernel: a captured call replayed with other lengths, masks
    and queries, which lie inside wider rows; a stream of its own."""
    import torch
    import token_level_dynamic_b200 as w
    c = _roomy(Case("e4m3", 4, rep, N, [900, 300], [N, N - 2], "random", 0.6, seed=8), "roomy")
    ref = c.run()
    c.check(ref)
    wide = torch.zeros(c.q.shape[0], 4 * rep * 128 + 72, dtype=torch.bfloat16, device="cuda")
    view = wide.as_strided(c.q.shape, (wide.stride(0), 128, 1), 8)
    view.copy_(c.q)
    c.q = view
    out = torch.full((c.S * N, 4 * rep, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((w.wide_attn_tree_workspace_bytes(c.cache, N, 4 * rep) + 256,), 255, dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.run(out=out, workspace=ws, stream=st)
    st.synchronize()
    assert torch.equal(out, ref) and torch.all(ws[-256:] == 255)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, workspace=ws)
    for lens, new in (([100, 901], [2, N]), ([0, 0], [N, 1]), ([5, 1200], [0, 3])):
        c.cl.copy_(torch.tensor(lens, dtype=torch.int32))
        c.dl.copy_(torch.tensor(new, dtype=torch.int32))
        c.q.neg_()
        c.hm.bitwise_not_()
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(out, c.run(out=torch.full_like(out, 7.0)))
