"""The attention kernels where work is plenty: tiles of 16 rows, full-size units, segments in many pieces.

The bounds are those of tests/test_gpu_kv_attention.py.  Tables may name a page many times, so a small cache gives
long contexts; a few kv heads and rows of each case are compared.
"""
import numpy as np
import pytest
import torch

from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, to_np
from tests.test_gpu_kv_attention import _check, _queries

pytestmark = pytest.mark.gpu


class Pool:
    """A cache of random pages (scales of all magnitudes around 1) and its values, a kv head at a time."""

    def __init__(self, rng, num_pages, page, heads, D, kg=0.25, vg=0.05):
        self.page, self.D, self.kg, self.vg = page, D, kg, vg
        self.c = api.NVFP4KVCache.empty(num_pages, page, heads, D, kg, vg)
        p = rng.integers(0, 256, self.c.pages.shape).astype(np.uint8)
        for at in (8 * D, 17 * D):
            p[..., at:at + D] = rng.integers(40, 72, p.shape[:-1] + (D,))
        self.pages = p
        self.c.pages.copy_(torch.from_numpy(p))

    def values(self, table_row, n, head):
        at = np.arange(n)
        slots = table_row[at // self.page].astype(np.int64) * self.page + at % self.page
        kc, ks, vc, vs = S.read_slots(self.pages[:, head:head + 1], slots, self.page, self.D)
        return S.dequantize_rows(kc, ks, self.kg), S.dequantize_rows(vc, vs, self.vg)


def _run(seed, lens, rows, heads, kvh, D, page, width=None, window=0, dtype=torch.bfloat16, max_q=None, pool=200, looked=4):
    rng = np.random.default_rng(seed)
    p = Pool(rng, pool, page, kvh, D)
    need = max(-(-n // page) for n in lens)
    table = np.full((len(lens), width or max(1, need)), -1, np.int32)
    for b, n in enumerate(lens):
        table[b, :-(-n // page)] = rng.integers(0, pool, -(-n // page))
    total, group = sum(rows), heads // kvh
    q, q64 = _queries(rng, total, heads, D, dtype, 1.0)
    g, gl = Guarded((total, heads, D), torch.bfloat16), Guarded((total, heads), torch.float32)
    cu = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    args = (q.cuda(), p.c, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
            None if all(r == 1 for r in rows) else torch.from_numpy(cu).cuda())
    api.nvfp4_kv_attention(*args, max_q=max_q, window=window, out=g.t, lse=gl.t)
    g.check("attention out")
    gl.check("attention lse")
    again = api.nvfp4_kv_attention(*args, max_q=max_q, window=window)
    assert torch.equal(again, g.t)
    spots = [(b, h) for b in range(len(lens)) for h in range(kvh) if rows[b]]
    for i in rng.permutation(len(spots))[:looked]:
        b, h = spots[i]
        k, v = p.values(table[b], lens[b], h)
        hs = np.arange(h * group, (h + 1) * group)
        at = slice(int(cu[b]), int(cu[b + 1]))
        _check(g.t[at][:, hs].contiguous(), gl.t[at][:, hs].contiguous(), 0, q64[at][:, hs], k, v, D ** -0.5, window)
    assert api.device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,rows,lens", [(24, (1, 1, 1, 1), (0, 1, 700, 3001)), (20, (2, 1, 2), (1, 64, 1500)),
                                             (8, (4, 6, 0, 3, 1), (70, 5, 9, 2000, 129)), (33, (1, 1), (17, 400)),
                                             (48, (1,), (800,)), (5, (9, 7), (4, 333))])
@pytest.mark.parametrize("window", [0, 100])
def test_sixteen_row_tiles(D, group, rows, lens, window):
    """17 to 48 rows a kv head in tables with room for more than 2^18 keys."""
    kvh, page = 2, 32
    width = (1 << 18) // (kvh * page * len(lens)) + 1
    _run(group + D, list(lens), list(rows), group * kvh, kvh, D, page, width, window, max_q=max(rows),
         dtype=torch.float32 if group == 20 else torch.bfloat16, looked=20)


@pytest.mark.parametrize("D,kvh,lens", [(128, 8, [2000 + 7 * i for i in range(64)]), (64, 16, [3500 - 13 * i for i in range(64)]),
                                        (128, 16, [1, 0, 30000, 17, 25000, 64, 9999, 16000])])
@pytest.mark.parametrize("group", [1, 8])
def test_full_size_units(D, kvh, lens, group):
    """Eight rounds and more for every warp: units of 64 keys (D = 128) and 128 (D = 64)."""
    _run(D + kvh + group, lens, [1] * len(lens), group * kvh, kvh, D, 64)


@pytest.mark.parametrize("D", [64, 128])
def test_full_size_units_of_sixteen_row_tiles(D):
    lens = [4000 - 31 * i for i in range(32)]
    _run(D, lens, [4] * 32, 64, 8, D, 64, max_q=4)
    _run(D + 1, lens, [3] * 32, 64, 8, D, 48, window=1500, max_q=3, dtype=torch.float32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [10001, 16000, 131000])
def test_many_pieces_of_a_segment(D, n):
    """More than 16 pieces: the square root of the keys."""
    _run(n + D, [n], [1], 64, 8, D, 64, pool=500, looked=2)
    _run(n + D + 1, [n], [4], 64, 8, D, 64, max_q=4, pool=500, looked=1)


def test_small_and_large_calls_share_a_workspace():
    """Every variant leaves the workspace ready for the others."""
    rng = np.random.default_rng(5)
    p = Pool(rng, 100, 64, 8, 128)
    ws = torch.zeros(api.nvfp4_kv_attention_workspace_bytes(64, 512, 64, 8, 128), dtype=torch.uint8, device="cuda")
    calls = []
    for batch, rows, n in ((64, 1, 2000), (1, 1, 16000), (16, 4, 3000), (2, 128, 900), (1, 4, 131000), (3, 1, 5)):
        table = torch.from_numpy(rng.integers(0, 100, (batch, -(-n // 64))).astype(np.int32)).cuda()
        q = _queries(rng, batch * rows, 64, 128, torch.bfloat16, 1.0)[0].cuda()
        cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * rows
        calls.append((q, p.c, table, torch.full((batch,), n, dtype=torch.int32, device="cuda"), cu, rows))
    alone = [api.nvfp4_kv_attention(*c) for c in calls]
    for order in (range(6), reversed(range(6)), (3, 0, 3, 4, 1, 5, 2)):
        for i in order:
            assert torch.equal(alone[i], api.nvfp4_kv_attention(*calls[i], workspace=ws))
    assert not to_np(ws[:api.ATTENTION_WS_ZEROED]).view(np.uint32)[:642].any()
    assert api.device_status() == 0
