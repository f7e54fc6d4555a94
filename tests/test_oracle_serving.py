"""Pins of the serving oracle (CPU): rotation against complex numbers and the
layer oracle's RoPE, cache codes against torch's e4m3 type and brute force,
tree attention against torch and against hand-made cases."""
import numpy as np
import pytest

from oracle import attention, serving


def test_rope_half_equals_the_layer_oracle_and_interleaved_is_its_permutation():
    rng = np.random.default_rng(0)
    x, pos = rng.standard_normal((5, 3, 128)), rng.integers(0, 9000, 5)
    got = serving.rope(x, pos, 128)
    assert np.allclose(got, attention.rope(x.transpose(1, 0, 2), pos, 5e5).transpose(1, 0, 2), atol=1e-12)
    perm = np.concatenate([np.arange(0, 128, 2), np.arange(1, 128, 2)])
    inter = serving.rope(x, pos, 128, layout="interleaved")
    assert np.allclose(inter[..., perm], serving.rope(x[..., perm], pos, 128), atol=1e-12)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_undone_by_the_negative_position_and_rest_copied(layout):
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((4, 2, 96)), rng.integers(-500, 500, 4)
    kw = dict(layout=layout, factor=8.0, low=1.0, high=4.0, original=8192)
    y = serving.rope(x, pos, 36, **kw)
    assert np.array_equal(y[..., 36:], x[..., 36:])
    assert np.allclose(serving.rope(y, -pos, 36, **kw), x, atol=1e-12)
    assert np.allclose(np.sum(y * y, -1), np.sum(x * x, -1), rtol=1e-12)


def test_rope_scaling_ends():
    f = serving.rope_frequencies(128)
    assert np.allclose(serving.rope_frequencies(128, factor=4.0), f / 4)
    g = serving.rope_frequencies(128, factor=4.0, low=1.0, high=4.0, original=8192)
    turns = 8192 * f / (2 * np.pi)
    assert np.allclose(g[turns >= 4], f[turns >= 4]) and np.allclose(g[turns <= 1], f[turns <= 1] / 4)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all(g[mid] < f[mid]) and np.all(g[mid] > f[mid] / 4)


def test_e4m3_codes_equal_torch():
    import torch
    rng = np.random.default_rng(2)
    x = rng.standard_normal((64, 128)) * np.exp(rng.uniform(-20, 20, (64, 1)))
    codes, byte = serving.kv_encode(x, "e4m3")
    y = x.reshape(64, 4, 32) * 2.0 ** (127.0 - byte[..., None])
    assert np.max(np.abs(y)) <= 448 and np.min(np.max(np.abs(y), -1)) > 224
    ref = torch.from_numpy(y).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    # float64 -> float32 first only matters within 2^-24 of a tie
    assert np.mean(ref.reshape(64, 128) != codes) < 1e-3
    v = serving.kv_decode(codes, byte, "e4m3")
    vt = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    assert np.array_equal(v, (vt.reshape(64, 4, 32) * 2.0 ** (byte[..., None] - 127.0)).reshape(64, 128))


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_cache_codes_special_blocks(kind):
    x = np.zeros((1, 128))
    x[0, 32] = np.inf
    x[0, 64] = serving.KV_MAX[kind]                    # exactly the largest: scale 1
    x[0, 96] = np.nextafter(serving.KV_MAX[kind], 1e9)  # just above: scale 2
    codes, byte = serving.kv_encode(x, kind)
    assert byte.tolist() == [[0, 255, 127, 128]]
    v = serving.kv_decode(codes, byte, kind)
    assert np.all(v[0, :32] == 0) and np.all(np.isnan(v[0, 32:64])) and v[0, 64] == x[0, 64]


def test_i8_ties_go_to_even():
    x = np.zeros((1, 128))
    x[0, :6] = [127, 0.5, 1.5, 2.5, -0.5, -1.5]
    codes, byte = serving.kv_encode(x, "i8")
    assert byte[0, 0] == 127 and codes[0, :6].tolist() == [127, 0, 2, 2, 0, -2]


def test_attn_tree_equals_torch_and_skips():
    import torch
    rng = np.random.default_rng(3)
    S, N, n_kv, rep, cap = 2, 4, 2, 3, 20
    q = rng.standard_normal((S, N, n_kv * rep, 128))
    k, v = rng.standard_normal((2, S, n_kv, cap, 128))
    tree = np.tril(np.ones((N, N), bool))[None].repeat(S, 0)
    tree[1, 3] = [True, False, False, True]
    heads = np.ones((S, N, n_kv), bool)
    heads[0, 2, 1] = False
    out = np.full(q.shape, 7.0)
    serving.attn_tree(q, k, v, [9, 0], [4, 3], tree, heads, 0.1, out)
    assert np.all(out[1, 3] == 7.0)                       # past the sequence's tokens: untouched
    assert np.all(out[0, 2, 3:] == 0.0)
    for s, c, m in ((0, 9, 4), (1, 0, 3)):
        see = np.concatenate([np.ones((m, c), bool), tree[s, :m, :m]], 1)
        for h in range(n_kv * rep):
            ref = torch.nn.functional.scaled_dot_product_attention(
                torch.from_numpy(q[s, :m, h])[None], torch.from_numpy(k[s, h // rep, :c + m])[None],
                torch.from_numpy(v[s, h // rep, :c + m])[None],
                attn_mask=torch.from_numpy(see), scale=0.1)[0].numpy()
            rows = [t for t in range(m) if heads[s, t, h // rep]]
            assert np.allclose(out[s, rows, h], ref[rows], atol=1e-12)
    empty = np.full((1, 1, 1, 128), 7.0)
    serving.attn_tree(q[:1, :1, :1], k[:1, :1], v[:1, :1], [0], [1], np.zeros((1, 1, 1), bool),
                      np.ones((1, 1, 1), bool), 0.1, empty)
    assert np.all(empty == 0.0)
