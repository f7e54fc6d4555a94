"""wide_attn_tree with values near the end of fp32's range: a weight is at most 1,
so a sum is infinite only if the plain sum of weights times values is.  Queries
and keys of one element each make scores whose weights are known."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("n", [1, 4, 8, 16, 32, 64])
def test_a_late_key_with_a_large_value(n, kind):
    """Keys of score 0 and, among the last, one of 7.65 in base 2 (below what
    moves a row's reference) with the value 2^121, in so many sequences that a CTA
    has several tiles of one: the mean is the exact one to the weights' rounding
    and the output's, 2^-8 each, and 2^-16 for the score's."""
    import torch
    import token_level_dynamic_b200 as w
    S, n_kv, have, at = 40, 16, 600, 580
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[kind]
    cache = w.wide_kv_cache(S, n_kv, have + n, dt)
    k, v = (torch.zeros((S, have + n, n_kv, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[:, at, :, 0] = 60.0
    v[:, at, :, 0:64] = 2.0 ** 121
    v[..., 64:] = -2.0 ** 112
    w.wide_kv_append(k.view(-1, n_kv, 128), v.view(-1, n_kv, 128), cache)
    q = torch.zeros((S * n, 4 * n_kv, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    tree = torch.zeros((S * n, (n + 31) // 32), dtype=torch.int32, device="cuda")
    w.wide_clear_device_status()
    out = w.wide_attn_tree(q, cache, torch.full((S,), have, dtype=torch.int32, device="cuda"), tree_mask=tree)
    assert w.wide_get_device_status() == 0
    # (int8 holds 60 as it is, e4m3 too)
    p = np.exp(60.0 / np.sqrt(128.0))
    want = np.zeros(128)
    want[:64] = p / (p + have - 1) * 2.0 ** 121
    want[64:] = -2.0 ** 112
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= (2 * 2.0 ** -8 + 2.0 ** -16) * np.abs(want))


@pytest.mark.parametrize("cap", [400, 1 << 17])            # the kernel for few positions, and the other
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("n", [1, 4, 8, 16, 32, 64])
def test_scores_up_to_2_to_29(n, sign, cap):
    """Scores of +-2^29 at two keys and, elsewhere, of at least 2^21 less: the
    output is the mean of the two values (1 and 3) to the weights' rounding and
    its own, 2^-8 each, and 2^-16 for fp32."""
    import torch
    import token_level_dynamic_b200 as w
    have = 300
    cache = w.wide_kv_cache(1, 1, cap, torch.bfloat16)
    top, rest = (2.0 ** 14, 2.0 ** 14 * (1 - 2.0 ** -8)) if sign > 0 else (-2.0 ** 14, -2.0 ** 14 * (1 + 2.0 ** -7))
    cache["k"][0, 0, :have, 0] = rest
    for i, at in enumerate((10, 290)):
        cache["k"][0, 0, at, 0] = top
        cache["v"][0, 0, at] = 1.0 + 2.0 * i
    cache["v"][0, 0, 100] = 1e30
    q = torch.zeros((n, 4, 128), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 2.0 ** 15
    tree = torch.zeros((n, (n + 31) // 32), dtype=torch.int32, device="cuda")
    out = w.wide_attn_tree(q, cache, torch.full((1,), have, dtype=torch.int32, device="cuda"), tree_mask=tree, scale=1.0)
    assert float((out.double() - 2.0).abs().max()) <= 2 * (2 * 2.0 ** -8 + 2.0 ** -16)
