"""wide_attn_tree over bf16 caches with infinities and NaNs among the values of
the context: weights are positive, so an infinity comes back as that infinity
in its element of every row, whatever its weight rounds to, and only a NaN or
infinities of both signs give NaN.  In every layout of both kernels.  Oracle and
bound as in test_gpu_attn_tree.py."""
import numpy as np
import pytest

from tests.test_gpu_attn_tree import Case
from tests.test_gpu_attn_tree_runs import ROOM, _roomy

pytestmark = pytest.mark.gpu
# up to 16, 32, 64, 128 and 256 rows of a run, and two runs a unit
LAYOUTS = [(4, 1), (4, 4), (4, 8), (4, 16), (4, 32), (3, 43), (4, 64), (4, 100)]


@pytest.fixture(autouse=True)
def _status():
    import token_level_dynamic_b200 as w
    w.wide_clear_device_status()
    yield
    assert w.wide_get_device_status() == 0


def _put(c, pos, v=(), k=()):
    """Elements (head, dim, value) of the value and key rows at a position."""
    for name, what in (("v", v), ("k", k)):
        for head, dim, x in what:
            c.cache[name][0, head, pos, dim] = x


def _check(c, room, some):
    c = _roomy(c, room)
    got = c.run()
    c.check(got)
    f = got.float().cpu().numpy()
    assert np.isinf(f).any() == some[0] and np.isnan(f).any() == some[1]


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("rep,N", LAYOUTS)
@pytest.mark.parametrize("have", [200, 3000])
def test_infinite_values_of_the_context(room, rep, N, have):
    """Infinities at the start, in the middle and in the last tile of the
    context, which for 3000 positions are in several parts of a run."""
    inf = float("inf")
    c = Case("bf16", 2, rep, N, [have], None, "random", 0.8, seed=N)
    small = c.cache
    _put(c, 0, [(0, 0, inf), (0, 77, -inf), (1, 5, inf)])
    _put(c, have // 2, [(0, 31, inf), (1, 127, -inf)])
    _put(c, have - 1, [(0, 0, inf), (1, 64, inf)])
    _check(c, room, (True, False))
    c.cache = small
    c.__dict__.pop("values", None)                        # (the roomy cache's)
    _put(c, 17, [(0, 0, -inf), (1, 64, float("nan"))])    # both signs; a NaN
    _check(c, room, (True, True))


@pytest.mark.parametrize("room", ROOM)
@pytest.mark.parametrize("rep,N", LAYOUTS)
@pytest.mark.parametrize("have", [200, 3000])
def test_infinite_values_of_weights_that_round_to_nothing(room, rep, N, have):
    """Keys so far below the others that fp32 holds no weight for them (e^-280),
    in the context and among the new tokens; and a reference that rises by as
    much after the infinity was added."""
    inf = float("inf")
    c = Case("bf16", 1, rep, N, [have], None, "chain", 1.0, seed=N + 1)
    c.q[:, :, 0] = 4.0
    at = [1, have // 3, have - 2]
    for i, pos in enumerate(at):
        _put(c, pos, [(0, 9 + i, inf), (0, 40 + i, -inf)], [(0, 0, -800.0)])
    new = have + N // 2
    _put(c, new, [(0, 100, inf)], [(0, 0, -800.0)])
    _check(c, room, (True, False))
    # the first position's weight is one until the last one's key comes
    d = Case("bf16", 1, rep, N, [have], None, "chain", 1.0, seed=N + 2)
    d.q[:, :, 0] = 4.0
    _put(d, 0, [(0, 3, inf)])
    _put(d, have - 1, [], [(0, 0, 800.0)])
    _check(d, room, (True, False))
