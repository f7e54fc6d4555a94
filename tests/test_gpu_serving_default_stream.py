"""wide_rope, wide_kv_read and wide_attn_tree given the default stream by its
handle, 0 or 1 (cudaStreamLegacy), while another one is current: what a call
makes is made there."""
import pytest

from tests.test_gpu_attn_tree import Case
from tests.test_gpu_serving_streams import _watch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [0, 1])
def test_default_stream_by_handle(handle, monkeypatch):
    import torch
    import token_level_dynamic_b200 as w
    c = Case("i8", 2, 2, 5, [40, 300], [5, 3], "random", 0.6, seed=4)
    x = torch.randn((5, 3, 64), device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    cfg = w.wide_rope_config(64)
    start, count = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 0], [9, 4]))

    def calls(**kw):
        return [w.wide_rope(x, pos, cfg, **kw), *w.wide_kv_read(c.cache, start, 9, count=count, **kw),
                w.wide_attn_tree(c.q, c.cache, c.cl, tree_mask=c.tm, head_mask=c.hm, draft_len=c.dl, **kw)]
    want = calls()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        seen = _watch(monkeypatch)
        got = calls(stream=handle)
        monkeypatch.undo()
        assert torch.cuda.current_stream() == st
    assert len(seen) >= 5 and set(seen) == {0}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
