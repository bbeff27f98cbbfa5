"""ServingStep over requests that come and go: a request's tokens do not depend on what its row, or an empty row, held
before."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from nvfp4_w4a4_decode_gemv_gb300.serving_step import ServingStep
from tests.gpu_util import to_np
from tests.test_gpu_serving_step import D, KVH, LAYERS, M, PAGE, VOCAB, _feed, _step

pytestmark = pytest.mark.gpu


class Request:
    def __init__(self, seed, n):
        rng = np.random.default_rng(seed)
        self.ids = torch.from_numpy(rng.integers(0, VOCAB, n).astype(np.int32)).cuda()
        self.k, self.v = ([torch.from_numpy(rng.standard_normal((n, KVH, D)).astype(np.float32)).to(torch.bfloat16).cuda()
                           for _ in range(LAYERS)] for _ in range(2))
        self.feeds = [(torch.from_numpy(rng.standard_normal(512).astype(np.float32)).cuda(), float(np.float32(rng.random())))
                      for _ in range(16)]


def _start(st, requests: dict):
    rows = sorted(requests)
    return st.start({r: requests[r].ids for r in rows},
                    *[[torch.cat([getattr(requests[r], what)[layer] for r in rows]) for layer in range(LAYERS)]
                      for what in "kv"])


def _run(st, feeds: dict):
    """One step; what comes out of the rows in `feeds`."""
    for r, (h, u) in feeds.items():
        st.h_in[r] = h
        st.u[r] = u
    st.run()
    return {r: [to_np(t[r]).copy() for t in (st.sampler.token, st.sampler.H, st.sampler.T, st.logits)] for r in feeds}


def _same(a, b):
    for x, y in zip(a, b):
        assert np.array_equal(x, y), (x, y)


def _end(st, *rows):
    st.end(torch.tensor([int(r in rows) for r in range(M)], dtype=torch.uint8, device="cuda"))


def test_a_request_in_a_used_row_is_like_one_in_a_fresh_step():
    """Row 0 has had a request and some idle steps; the idle rows hold large hidden states."""
    rng = np.random.default_rng(1)
    used, fresh = _step(), _step()
    _start(used, {r: Request(10 + r, n) for r, n in enumerate((40, 15, 3))})
    for _ in range(3):
        _feed(used, rng)
        used.run()
    _end(used, 0, 1, 2)
    used.h_in.mul_(100)
    for _ in range(2):
        used.run()
    want, mine = Request(20, 33), Request(20, 33)
    for st, req in ((used, want), (fresh, mine)):
        _start(st, {0: req})
    for i in range(12):                                             # past the window of 8 entropies
        _same(_run(used, {0: want.feeds[i]})[0], _run(fresh, {0: mine.feeds[i]})[0])
    assert api.device_status() == 0


def test_empty_rows_keep_their_state_and_outputs():
    rng = np.random.default_rng(2)
    st = _step()
    _start(st, {1: Request(30, 20)})
    _feed(st, rng)
    before, token = st.sampler.state.clone(), st.sampler.token.clone()
    st.run()
    stride = before.numel() // M
    same = (st.sampler.state == before).view(M, stride).all(1).cpu().tolist()
    assert same == [True, False, True]
    assert torch.equal(st.sampler.token[[0, 2]], token[[0, 2]])


def test_a_refused_token_is_retried_as_if_nothing_had_been():
    """No page for row 0's token: its sampler stays, the other row's result is as without it, and the retry gives what
    the first try would have given."""
    a, b = Request(40, 16), Request(41, 20)
    st = _step(num_pages=3)                                         # 1 + 2 pages, none left
    _start(st, {0: a, 1: b})
    out = _run(st, {0: a.feeds[0], 1: b.feeds[0]})
    assert to_np(st.plan.info).tolist() == [1, 2] and to_np(st.lens).tolist() == [16, 21, 0]
    alone = _step()
    _start(alone, {1: b})
    _same(out[1], _run(alone, {1: b.feeds[0]})[1])
    _end(st, 1)
    ref = _step()
    _start(ref, {0: a})
    for i in range(3):
        _same(_run(st, {0: a.feeds[i]})[0], _run(ref, {0: a.feeds[i]})[0])
    assert to_np(st.n_tokens).tolist() == [19, 0, 0] and api.device_status() == 0


def test_captured_step_with_empty_and_reused_rows():
    """The same in a captured graph."""
    def play(captured):
        st = _step()
        _start(st, {0: Request(50, 18), 2: Request(51, 7)})
        if captured:
            warm = _step()
            _start(warm, {0: Request(50, 18)})
            warm.run()
            torch.cuda.synchronize()
            graph = st.capture()
        out, req = [], Request(52, 9)
        rng = np.random.default_rng(3)
        for i in range(8):
            if i == 3:
                _end(st, 0)
            if i == 5:
                _start(st, {0: req})
            _feed(st, rng)
            graph.replay() if captured else st.run()
            out.append([to_np(t).copy() for t in (st.sampler.token, st.sampler.H, st.sampler.T, st.lens, st.tokens)])
        return out
    for x, y in zip(play(False), play(True)):
        _same(x, y)


def test_a_refused_prompt_leaves_its_row_empty():
    """A pool too small for the second of three prompts: its row has no request, takes no page when one comes free,
    and can be started again."""
    big, small, other = Request(60, 40), Request(61, 5), Request(62, 16)
    st = _step(num_pages=3)
    plan = _start(st, {0: small, 1: big, 2: other})                  # 1 + 3 + 1 pages of 3: rows 1 and 2 (behind it) refused
    assert to_np(plan.info).tolist()[0] == 2 and to_np(plan.kv_lens).tolist() == [5, 0, 0]
    assert to_np(st.lens).tolist() == [5, 0, 0] and to_np(st.active).tolist() == [1, 0, 0]
    assert to_np(st.n_tokens).tolist() == [5, 0, 0] and to_np(st.n_prompt).tolist() == [5, 0, 0]
    _run(st, {0: small.feeds[0]})
    _end(st, 0)
    assert int(st.free_count) == 3
    st.run()
    assert int(st.free_count) == 3 and to_np(st.lens).tolist() == [0, 0, 0] and not to_np(st.n_tokens).any()
    _start(st, {1: big})
    ref = _step()
    _start(ref, {1: Request(60, 40)})
    for i in range(3):
        _same(_run(st, {1: big.feeds[i]})[1], _run(ref, {1: big.feeds[i]})[1])
    assert api.device_status() == 0


def test_prompts_that_do_not_fit_a_row_are_refused_before_anything_is_taken():
    st = _step()
    held = [t.clone() for t in (st.lens, st.n_tokens, st.active, st.free_count, st.table, st.tokens)]
    too_long, fine = Request(70, 201), Request(71, 200)              # max_len 200, pages for 208
    with pytest.raises(ValueError, match="max_len"):
        _start(st, {0: Request(72, 3), 2: too_long})
    with pytest.raises(ValueError, match="row"):
        _start(st, {M: Request(72, 3)})
    with pytest.raises(ValueError, match="row"):
        _start(st, {-1: Request(72, 3)})
    for t, x in zip((st.lens, st.n_tokens, st.active, st.free_count, st.table, st.tokens), held):
        assert torch.equal(t, x)
    _start(st, {2: fine})
    assert to_np(st.lens).tolist() == [0, 0, 200]


def test_a_row_with_a_request_takes_no_other():
    st = _step()
    _start(st, {0: Request(80, 20)})
    free, lens = int(st.free_count), to_np(st.lens).copy()
    with pytest.raises(ValueError, match="has a request"):
        _start(st, {0: Request(81, 4), 1: Request(82, 4)})
    assert int(st.free_count) == free and np.array_equal(to_np(st.lens), lens) and to_np(st.active).tolist() == [1, 0, 0]


def test_a_full_history_ends_the_row():
    """max_len tokens: no page, no key and no token more, though the last page has room; the history stays."""
    st = _step()
    _start(st, {0: Request(90, 199), 1: Request(91, 10)})
    req = Request(92, 1)
    _run(st, {0: req.feeds[0], 1: req.feeds[1]})
    assert to_np(st.n_tokens).tolist() == [200, 11, 0] and to_np(st.lens).tolist() == [200, 11, 0]
    history, state = to_np(st.tokens)[0].copy(), st.sampler.state.view(M, -1)[0].clone()
    for i in range(2):
        _run(st, {0: req.feeds[2 + i], 1: req.feeds[4 + i]})
    assert to_np(st.n_tokens).tolist() == [200, 13, 0] and to_np(st.lens).tolist() == [200, 13, 0]
    assert np.array_equal(to_np(st.tokens)[0], history) and torch.equal(st.sampler.state.view(M, -1)[0], state)
