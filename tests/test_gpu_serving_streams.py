"""wide_rope, wide_kv_read and wide_attn_tree on a stream that is not the
current one, with outputs and workspaces of the call's own: they are made, and
zeroed, on the call's stream, whatever the current stream still has to do."""
import pytest

from tests.test_gpu_attn_tree import Case
from tests.test_gpu_kv_cache import _dtype, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["stream", "handle"])
def stream(request):
    """(what a call is given, the stream itself)"""
    import torch
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    return (st if request.param == "stream" else st.cuda_stream), st


def _watch(monkeypatch):
    """Handles of the streams that tensors are made on, filled in by calls."""
    import torch
    seen = []
    for name in ("empty", "zeros"):
        def made(*args, real=getattr(torch, name), **kwargs):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return real(*args, **kwargs)
        monkeypatch.setattr(torch, name, made)
    return seen


def test_read_with_counts_is_zeroed_on_the_calls_stream(stream):
    """Zeros that waited in the current stream would come after the rows."""
    import torch
    import token_level_dynamic_b200 as w
    given, st = stream
    k, v = _rows(12, 4, 21, special=False)
    cache = w.wide_kv_cache(3, 4, 20, _dtype("e4m3"))
    start, count = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 0, 0], [4, 0, 3]))
    w.wide_kv_append(k, v, cache)
    want = w.wide_kv_read(cache, start, 4, count=count)
    assert not torch.any(want[0][4:8]) and torch.any(want[0][:4])
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    got = w.wide_kv_read(cache, start, 4, count=count, stream=given)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_what_a_call_makes_is_made_on_its_stream(stream, monkeypatch):
    import torch
    import token_level_dynamic_b200 as w
    given, st = stream
    c = Case("i8", 2, 2, 5, [40, 300], [5, 3], "random", 0.6, seed=4)
    x = torch.randn((5, 3, 64), device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    cfg = w.wide_rope_config(64)
    start = torch.zeros(2, dtype=torch.int32, device="cuda")

    def calls(**kw):
        return [w.wide_rope(x, pos, cfg, **kw), *w.wide_kv_read(c.cache, start, 9, **kw),
                w.wide_attn_tree(c.q, c.cache, c.cl, tree_mask=c.tm, head_mask=c.hm, draft_len=c.dl, **kw)]
    want = calls()
    torch.cuda.synchronize()
    seen = _watch(monkeypatch)
    got = calls(stream=given)
    monkeypatch.undo()
    assert len(seen) >= 5 and set(seen) == {st.cuda_stream}
    assert torch.cuda.current_stream().cuda_stream != st.cuda_stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
