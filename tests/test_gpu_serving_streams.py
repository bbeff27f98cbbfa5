"""Outputs that the serving operators' bindings make for a call on another stream: memory in which the current stream
may still be at work is not taken, and what the call's stream still writes is not handed out again."""
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api

pytestmark = pytest.mark.gpu

N = 3 << 20          # bytes; every output is made that large


def _calls():
    c = api.NVFP4KVCache.empty(64, 64, 2, 128)
    c.pages.zero_()
    i32 = lambda *s, v=0: torch.full(s, v, dtype=torch.int32, device="cuda")
    tokens = N // (2 * 128 * 2)
    slots = i32(tokens, v=-1)
    q = torch.zeros((N // (8 * 128 * 2), 8, 128), dtype=torch.bfloat16, device="cuda")
    table, lens = i32(q.shape[0], 1), i32(q.shape[0], v=9)
    logits = torch.zeros((4, N // 16), device="cuda")
    stack, count = i32(64), i32(1)
    ctx = i32(4)
    return {"read": lambda s: api.nvfp4_kv_read(c, slots, stream=s)[0],
            "attention": lambda s: api.nvfp4_kv_attention(q, c, table, lens, stream=s),
            "logits": lambda s: api.nvfp4_process_logits(logits, stream=s),
            "plan": lambda s: api.nvfp4_kv_plan(ctx, ctx, i32(4, 2), stack, count, 64, N // 4, stream=s).slots}


@pytest.mark.parametrize("name", ["read", "attention", "logits", "plan"])
def test_outputs_of_calls_on_another_stream(name):
    call, side = _calls()[name], torch.cuda.Stream()
    call(side)                                                   # whatever is made once
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    made = torch.empty(N, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(100_000_000)                               # the current stream is at work ...
    made.fill_(1)
    at = made.data_ptr()
    del made                                                     # ... in memory that the host has given back
    out = call(side)
    assert out.untyped_storage().nbytes() == N and not at <= out.data_ptr() < at + N
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    out = call(side)
    at = out.data_ptr()
    del out                                                      # the side stream has yet to write it
    for _ in range(4):
        again = torch.empty(N, dtype=torch.uint8, device="cuda")
        assert not at <= again.data_ptr() < at + N
    torch.cuda.synchronize()
    out, want = call(side), call(None)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    torch.cuda._sleep(100_000_000)
    copy = out.clone()                                           # the current stream has yet to read it
    at = out.data_ptr()
    del out
    with torch.cuda.stream(side):
        for _ in range(4):
            again = torch.empty(N, dtype=torch.uint8, device="cuda")
            assert not at <= again.data_ptr() < at + N
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
