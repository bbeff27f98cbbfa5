"""Page tables and slot maps on the GPU against the one-request-after-the-other oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, to_np

pytestmark = pytest.mark.gpu


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def _case(rng, batch, page, most_ctx, most_new, extra, width=None):
    ctx = rng.integers(0, most_ctx + 1, batch)
    new = rng.integers(0, most_new + 1, batch)
    used = -(-ctx // page)
    need = int((-(-(ctx + new) // page) - used).sum())
    width = width or int((-(-(ctx + new) // page)).max()) + 1
    total = int(used.sum()) + need + 40
    ids = rng.permutation(total)
    table = np.full((batch, width), -1)
    at = 0
    for b in range(batch):
        n = min(int(used[b]), width)
        table[b, :n] = ids[at:at + n]
        at += n
    count = max(0, need + extra)
    stack = np.full(max(total, count), -9)
    stack[:min(count, total - at)] = ids[at:at + min(count, total - at)]
    return ctx, new, table, stack, min(count, total - at)


def _check(ctx, new, table, stack, count, page, most, in_place=False):
    want = S.kv_plan(ctx, new, table, stack, count, page, most)
    t, cnt = _dev(table), _dev([count])
    guards = [Guarded((n,), torch.int32) for n in (max(most, 1), max(most, 1), len(ctx) + 1, len(ctx), 1, 2)]
    out = api.KVPlan(*[g.t for g in guards])
    out.slots, out.positions = out.slots[:most], out.positions[:most]
    if in_place:
        out.free_count = cnt
    api.nvfp4_kv_plan(_dev(ctx), _dev(new), t, _dev(stack), cnt, page, out=out)
    got = [to_np(x) for x in (t, out.slots, out.positions, out.cu_q, out.kv_lens, out.free_count, out.info)]
    for g, w, name in zip(got, want, ("table", "slots", "positions", "cu_q", "kv_lens", "free_count", "info")):
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), name
    for g in guards:
        g.check("plan output")


@pytest.mark.parametrize("batch", [1, 2, 8, 255, 256, 257, 1000, 1024, 1025, 2500])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_plan_matches_oracle(batch, page):
    rng = np.random.default_rng(batch * 100 + page)
    for most_ctx, most_new, extra in ((0, 1, 0), (300, 1, 3), (500, 70, 0), (3 * page, 2 * page, -(batch // 2))):
        ctx, new, table, stack, count = _case(rng, batch, page, most_ctx, most_new, extra)
        total = int(new.sum())
        for most in {total, total + 37, max(0, total - 5), 0}:
            _check(ctx, new, table, stack, count, page, most)
        _check(ctx, new, table, stack, count, page, total, in_place=True)


def test_plan_long_prompts_take_many_pages():
    rng = np.random.default_rng(5)
    ctx, new, table, stack, count = _case(rng, 3, 16, 10, 1, 0)
    new = np.array([40000, 0, 3])
    width = 3000
    table = np.full((3, width), -1)
    table[:, 0] = [5, 6, 7]
    stack = rng.permutation(4000) + 10
    _check(np.minimum(ctx, 16), new, table, stack, 4000, 16, int(new.sum()) + 3, in_place=True)


def test_plan_refuses_bad_lengths_and_full_tables():
    table = np.full((6, 2), -1)
    table[:, 0] = np.arange(6)
    ctx = np.array([-3, 5, 16, 30, 16, 2 ** 31 - 20])
    new = np.array([4, -2, 17, 2, 16, 19])
    _check(ctx, new, table, np.arange(10, 30), 20, 16, 60)


def test_release_then_plan_chain():
    """Ended requests' pages are what the next plan hands out, over several steps, counts in place."""
    rng = np.random.default_rng(9)
    batch, page, width, pool = 300, 16, 20, 3000
    ids = rng.permutation(pool)
    table, lens = np.full((batch, width), -1), np.zeros(batch, np.int64)
    stack, count = ids.copy(), pool
    t_dev, s_dev, c_dev = _dev(table), _dev(stack), _dev([count])
    for step in range(5):
        ended = (rng.random(batch) < 0.3).astype(np.uint8)
        stack, count = S.kv_release(lens, ended, table, stack, count, page)
        api.nvfp4_kv_release(_dev(lens), _dev(ended, torch.uint8), t_dev, s_dev, c_dev, page)
        assert int(c_dev) == count and np.array_equal(to_np(s_dev)[:count], stack[:count])
        ctx = np.where(ended, 0, lens)
        new = rng.integers(0, 40, batch)
        table, slots, pos, cu, kv, count, info = S.kv_plan(ctx, new, table, stack, count, page, int(new.sum()))
        out = api.nvfp4_kv_plan(_dev(ctx), _dev(new), t_dev, s_dev, c_dev, page, max_tokens=int(new.sum()))
        assert out.free_count is c_dev
        for g, w in ((t_dev, table), (out.slots, slots), (out.positions, pos), (out.cu_q, cu), (out.kv_lens, kv),
                     (c_dev, [count]), (out.info, info)):
            assert np.array_equal(to_np(g).reshape(-1), np.asarray(w).reshape(-1))
        lens = kv
    assert api.device_status() == 0


def test_release_large_and_bounds():
    """Many pages (several CTAs), both count forms; a stack too small drops what does not fit."""
    rng = np.random.default_rng(11)
    batch, width, page = 64, 300, 16
    table = rng.permutation(batch * width).reshape(batch, width)
    lens = rng.integers(-5, width * page + 100, batch)
    ended = (rng.random(batch) < 0.8).astype(np.uint8)
    for cap, count in ((batch * width + 10, 7), (1000, 990), (0, 0)):
        stack = np.arange(cap) + 10 ** 6
        want, n = S.kv_release(lens, ended, table, stack, count, page)
        for in_place in (False, True):
            s, c = _dev(stack), _dev([count])
            o = c if in_place else _dev([-1])
            api.nvfp4_kv_release(_dev(lens), _dev(ended, torch.uint8), _dev(table), s, c, page, free_count_out=o)
            assert int(o) == n and np.array_equal(to_np(s), want)


def test_plan_in_a_graph():
    """One decode step's plan captured with the count in place: each replay takes the next pages."""
    page, batch = 16, 4
    table = torch.full((batch, 8), -1, dtype=torch.int32, device="cuda")
    stack, count = torch.arange(32, dtype=torch.int32, device="cuda"), torch.tensor([32], dtype=torch.int32, device="cuda")
    lens, one = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.ones(batch, dtype=torch.int32, device="cuda")
    out = api.KVPlan.empty(batch, batch, free_count=count)
    api.nvfp4_kv_plan(lens, one, table.clone(), stack, torch.tensor([32], dtype=torch.int32, device="cuda"), page,
                      out=api.KVPlan.empty(batch, batch))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.nvfp4_kv_plan(lens, one, table, stack, count, page, out=out)
        lens.copy_(out.kv_lens)
    for step in range(40):
        g.replay()
        assert to_np(lens).tolist() == [step + 1] * batch
        assert int(count) == 32 - batch * (step // page + 1)
        t = to_np(table)
        assert to_np(out.slots).tolist() == [int(t[b, step // page]) * page + step % page for b in range(batch)]
