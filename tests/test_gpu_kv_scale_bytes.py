"""Caches that a caller fills: a scale byte b stands for 2^(b - 127) for every
byte of a finite value, 0 among them, whatever the codes; wide_kv_read and both
attention kernels take the same number, code * 2^(b - 127) rounded to bf16."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

N, LAST = 64, 246          # 64 rows of 4 blocks: the bytes 0 .. 246 (448 * 2^(247 - 127) is no bf16 number)


@pytest.fixture(autouse=True)
def _status():
    import token_level_dynamic_b200 as w
    w.wide_clear_device_status()
    yield
    assert w.wide_get_device_status() == 0


def _cache(kind, cap, seed=0):
    """One head, `cap` positions; codes and scale bytes of the first 64 by hand, the rest zeros."""
    import torch
    import token_level_dynamic_b200 as w
    rng = np.random.default_rng(seed)
    dt = torch.float8_e4m3fn if kind == "e4m3" else torch.int8
    cache = w.wide_kv_cache(1, 1, cap, dt)
    want = {}
    for name in ("k", "v"):
        if kind == "e4m3":
            codes = rng.integers(0, 127, (N, 128)).astype(np.uint8) | (rng.integers(0, 2, (N, 128)) << 7).astype(np.uint8)
        else:
            codes = rng.integers(-127, 128, (N, 128)).astype(np.int8).view(np.uint8)
        b = np.minimum(rng.permutation(N * 4), LAST).astype(np.uint8).reshape(N, 4)
        codes, b = torch.from_numpy(codes), torch.from_numpy(b)
        cache[name].view(torch.uint8)[0, 0, :N] = codes.cuda()
        cache[name + "_scale"][0, 0, :N] = b.cuda()
        x = codes.view(dt).double().reshape(N, 4, 32) * torch.exp2(b.double() - 127.0)[..., None]
        want[name] = x.reshape(N, 128).float().to(torch.bfloat16)     # (exact in fp32: 7 bits at most)
    return cache, want


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_read_of_every_scale_byte(kind):
    import torch
    import token_level_dynamic_b200 as w
    cache, want = _cache(kind, N)
    for got, name in zip(w.wide_kv_read(cache, None, N), "kv"):
        assert torch.equal(got[:, 0].cpu(), want[name]), name


@pytest.mark.parametrize("cap", [N, 1 << 17])              # the kernel for few positions, and the other
@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("rep", [1, 2, 3, 8])
def test_attention_multiplies_the_value_read(kind, rep, cap):
    """Each new token attends itself alone with a score of zero: its weight is
    one, its output the value."""
    import torch
    import token_level_dynamic_b200 as w
    cache, want = _cache(kind, cap, seed=rep)
    q = torch.zeros((N, rep, 128), dtype=torch.bfloat16, device="cuda")
    tree = np.zeros((N, 2), dtype=np.uint32)
    tree[np.arange(N), np.arange(N) // 32] = np.uint32(1) << (np.arange(N) % 32).astype(np.uint32)
    out = w.wide_attn_tree(q, cache, torch.zeros(1, dtype=torch.int32, device="cuda"),
                           tree_mask=torch.from_numpy(tree.view(np.int32)).cuda())
    for h in range(rep):
        assert torch.equal(out[:, h].cpu(), want["v"])


@pytest.mark.parametrize("cap", [2 * N, 1 << 17])
@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("n", [4, 8, 16, 32, 64])
@pytest.mark.parametrize("byte", [0, 1, 2, 127])
def test_keys_of_small_scale_bytes(kind, n, byte, cap):
    """Two earlier positions, one with the key 64 * 2^(byte - 127) in one
    element and the value 1, against a query that makes the score
    32 / sqrt(128): the output is the first one's weight.  (64: e4m3 68, i8 40.)"""
    import torch
    import token_level_dynamic_b200 as w
    cache, _ = _cache(kind, cap)
    for t in cache.values():
        t.view(torch.uint8).zero_()
    cache["k"].view(torch.uint8)[0, 0, 0, 5] = 0x68 if kind == "e4m3" else 64
    cache["k_scale"][0, 0, 0, 0] = byte
    cache["v"].view(torch.uint8)[0, 0, 0, :] = 0x38 if kind == "e4m3" else 1
    cache["v_scale"][0, 0, 0, :] = 127
    q = torch.zeros((n, 4, 128), device="cuda")
    q[..., 5] = 2.0 ** (126 - byte)
    tree = torch.zeros((n, (n + 31) // 32), dtype=torch.int32, device="cuda")
    out = w.wide_attn_tree(q.to(torch.bfloat16), cache, torch.full((1,), 2, dtype=torch.int32, device="cuda"),
                           tree_mask=tree)
    p = 1.0 / (1.0 + np.exp(-32.0 / np.sqrt(128.0)))
    # the weights' rounding and the output's, half a step of bf16 each, and 2^-20 for fp32
    assert float((out.double() - p).abs().max()) <= (2 * 2.0 ** -8 + 2.0 ** -20) * p


@pytest.mark.parametrize("cap", [2 * N, 1 << 17])
@pytest.mark.parametrize("kind", ["e4m3", "i8"])
@pytest.mark.parametrize("n", [4, 8, 16, 32, 64])
def test_255_is_nan_whatever_the_codes(kind, n, cap):
    """In a value of the context: NaN in its block of every row; in a key: in every row."""
    import torch
    import token_level_dynamic_b200 as w
    cache, _ = _cache(kind, cap)
    for name in ("k", "v"):
        cache[name + "_scale"].fill_(120)
    q = torch.randn((n, 4, 128), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").to(torch.bfloat16)
    have = torch.full((1,), 40, dtype=torch.int32, device="cuda")
    assert torch.isfinite(w.wide_attn_tree(q, cache, have)).all()
    cache["v_scale"][0, 0, 7, 2] = 255
    bad = torch.zeros(128, dtype=torch.bool, device="cuda")
    bad[64:96] = True
    assert torch.equal(torch.isnan(w.wide_kv_read(cache, None, 40)[1][7, 0]), bad)
    out = w.wide_attn_tree(q, cache, have)
    assert torch.isnan(out[..., bad]).all() and torch.isfinite(out[..., ~bad]).all()
    cache["k_scale"][0, 0, 9, 1] = 255
    assert torch.isnan(w.wide_attn_tree(q, cache, have)).all()
