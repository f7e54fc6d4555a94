"""wide_attn_tree at the borders of its row layouts (16, 32, 64, 128, 256 rows
of a run) and of its division of the work: many units, runs split between
CTAs, references that rise with every tile, nothing kept, nothing attended.
Oracle and bound as in test_gpu_attn_tree.py."""
import numpy as np
import pytest

from tests.test_gpu_attn_tree import KINDS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status():
    import token_level_dynamic_b200 as w
    w.wide_clear_device_status()
    yield
    assert w.wide_get_device_status() == 0


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rep,N", [(1, 16), (1, 17), (3, 11), (8, 8), (5, 13), (2, 64), (3, 43), (4, 64),
                                   (1, 257), (32, 17)])
def test_rows_at_the_borders_of_the_layouts(kind, rep, N):
    """Runs of up to 16, 32, 64, 128 and 256 rows, and several runs a unit."""
    c = Case(kind, 2, rep, N, [130, 257], [N, max(N - 2, 0)], "random", 1.0, seed=rep * 100 + N)
    c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rep,N", [(4, 1), (4, 8), (4, 16), (4, 32), (4, 64)])
def test_one_token_of_context_to_a_tile_more(kind, rep, N):
    """Contexts around the tiles of 128 keys, without and with a tail of new positions."""
    c = Case(kind, 1, rep, N, [0, 1, 127, 128, 129, 255, 256, 383], None, "random", 0.8, seed=N)
    c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rep,N", [(4, 4), (4, 8), (4, 16), (4, 32), (4, 64)])
def test_reference_rises_with_every_tile(kind, rep, N):
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
    w.wide_kv_append(k.to(torch.bfloat16), v.to(torch.bfloat16), c.cache)
    c.check(c.run())
    # and falling: the first tile's reference stays
    w.wide_kv_append(k.flip(0).to(torch.bfloat16).contiguous(), v.to(torch.bfloat16), c.cache)
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


@pytest.mark.parametrize("rep,N", [(2, 4), (4, 8), (4, 40)])
def test_nothing_kept_and_nothing_new(rep, N):
    """All pairs skipped: zeros for the tokens that there are.  No new tokens: nothing is written."""
    import torch
    c = Case("e4m3", 4, rep, N, [300, 0, 40], [N, N, 0], "random", 0.5, seed=1)
    c.hm.zero_()
    c.heads[:] = False
    got = c.run()
    assert torch.all(got[:2 * N] == 0) and torch.all(got[2 * N:] == 7.0)
    c.dl.zero_()
    assert torch.all(c.run() == 7.0)


@pytest.mark.parametrize("kind", KINDS)
def test_infinite_keys(kind):
    """An infinite key (a NaN key in 8 bits) of the context makes every row
    NaN that it reaches with a positive score, in every layout."""
    import torch
    import token_level_dynamic_b200 as w
    for rep, N in ((4, 4), (4, 8), (4, 32), (4, 64)):
        c = Case(kind, 1, rep, N, [200], None, "chain", 1.0, seed=2)
        kk, vv = w.wide_kv_read(c.cache, torch.tensor([150], dtype=torch.int32, device="cuda"), 1)
        kk[0, 0, 5] = float("inf")
        w.wide_kv_append(kk, vv, c.cache, torch.tensor([150], dtype=torch.int32, device="cuda"))
        got = c.run()
        hit = (c.q[:, :, 5] > 0) if kind == "bf16" else torch.ones_like(c.q[:, :, 5], dtype=torch.bool)
        assert torch.isnan(got[hit]).all() and torch.isfinite(got[~hit]).all()


@pytest.mark.parametrize("rep,N", [(4, 3), (4, 16), (4, 61)])
def test_two_graphs_on_one_workspace(rep, N):
    """Two captured calls on one workspace, replayed in turn, give what the
    eager calls gave, bit for bit."""
    import torch
    import token_level_dynamic_b200 as w
    cs = [Case(k, 4, rep, N, [700, 33], [N, N - 1], "random", 0.7, seed=5 + i) for i, k in enumerate(("i8", "i8"))]
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


@pytest.mark.parametrize("kind", KINDS)
def test_long_run_repeats_bit_for_bit(kind):
    """Long contexts split over all CTAs, run again and again while the parts
    arrive in another order: the same bits, and the device stays clear of
    errors (waits that give up, parts in the wrong place)."""
    import torch
    for rep, N in ((4, 16), (4, 64)):
        c = Case(kind, 2, rep, N, [9000, 2500], None, "random", 0.6, seed=6)
        ref = c.run()
        c.check(ref)
        for _ in range(20):
            assert torch.equal(c.run(), ref)
