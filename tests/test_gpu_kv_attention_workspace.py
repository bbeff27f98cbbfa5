"""The binding's workspaces: a caller's own is looked at, the binding's own is ready on the stream of the call."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_kv_attention import _cache, _queries, _table

pytestmark = pytest.mark.gpu


def _call(rng, batch=2, n=3000, kvh=2, heads=16, D=128, page=64):
    c, _, _, _ = _cache(rng, 64, page, kvh, D)
    t = torch.from_numpy(rng.integers(0, 64, (batch, -(-n // page))).astype(np.int32)).cuda()
    q = _queries(rng, batch, heads, D, torch.bfloat16, 1.0)[0].cuda()
    return q, c, t, torch.full((batch,), n, dtype=torch.int32, device="cuda")


def test_a_callers_workspace_is_checked():
    args = _call(np.random.default_rng(1))
    need = api.nvfp4_kv_attention_workspace_bytes(2, 2, 16, 2, 128)
    want = api.nvfp4_kv_attention(*args)
    zeros = lambda n, **kw: torch.zeros(n, **{"dtype": torch.uint8, "device": "cuda", **kw})
    for bad in (zeros(need, device="cpu"), zeros(2 * need)[::2], zeros(need, dtype=torch.float32)):
        with pytest.raises(ValueError, match="workspace"):
            api.nvfp4_kv_attention(*args, workspace=bad)
    with pytest.raises(RuntimeError, match="SHAPE"):
        api.nvfp4_kv_attention(*args, workspace=zeros(need - 1))
    assert torch.equal(want, api.nvfp4_kv_attention(*args, workspace=zeros(need)))


def test_a_captured_call_on_a_side_stream_clears_its_workspace_there():
    """The capturing stream is busy with other work and memory when the side stream's call starts."""
    args = _call(np.random.default_rng(2), batch=3, n=6000)
    want = api.nvfp4_kv_attention(*args)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    out = torch.empty_like(want)
    x = torch.randn((4096, 4096), device="cuda")
    y = torch.empty_like(x)
    torch.mm(x, x, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        for _ in range(3):
            torch.mm(x, x, out=y)
        api.nvfp4_kv_attention(*args, out=out, stream=side)
        junk = [torch.full((20 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        main.wait_stream(side)
        del junk
    for _ in range(5):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert api.device_status() == 0


def test_the_workspace_of_a_capturing_side_stream_is_the_graphs_own(monkeypatch):
    """Host side alone: where the workspace of a call comes from, and on which stream it is cleared."""
    seen = []
    real = api._new_attention_workspace

    def spy(need, device):
        seen.append((torch.cuda.current_stream().cuda_stream, torch.cuda.is_current_stream_capturing()))
        return real(need, device)
    monkeypatch.setattr(api, "_new_attention_workspace", spy)
    args = _call(np.random.default_rng(3))
    out = torch.empty_like(args[0])
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.nvfp4_kv_attention(*args, out=out, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        api.nvfp4_kv_attention(*args, out=out, stream=side)
        main.wait_stream(side)
    assert seen == [(side.cuda_stream, False), (side.cuda_stream, True)]
