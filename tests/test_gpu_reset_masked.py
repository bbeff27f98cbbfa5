"""The sampler on what grammar masks leave: whole chunks of -inf, rows without any token, masked tails.

Logits of -inf have probability 0 on every path (rows of up to 262144 logits take one cluster, longer ones several
launches).  Bounds as in tests/test_gpu_reset.py: H within 1e-4 relative, the token within 4e-6 Z of u Z.
"""
import numpy as np
import pytest
import torch

from oracle import reset as R
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_reset import _token_ok

pytestmark = pytest.mark.gpu

LONG = 262208


def _logits(V, M, seed):
    return torch.from_numpy((np.random.default_rng(seed).standard_normal((M, V)) * 3).astype(np.float32))


@pytest.mark.parametrize("V", [1000, 151936, LONG, 300007])
@pytest.mark.parametrize("top_p", [1.0, 0.9])
def test_masked_chunks_have_no_mass(V, top_p):
    M = 5
    x = _logits(V, M, V)
    x[0, :V // 2] = -np.inf                                    # the first half
    x[1, V // 3:] = -np.inf                                    # all but the first third
    x[2] = -np.inf
    x[2, [7, V // 2, V - 1]] = torch.tensor([1.0, 2.0, 1.5])   # three tokens of far-apart chunks
    x[3, :V - 1] = -np.inf                                     # one token
    s = api.ResetSampler(M, V, top_p=top_p)
    states = [R.RowState(w=8) for _ in range(M)]
    p = R.ResetParams(tau0=float(np.float32(0.6)), t_low=float(np.float32(0.3)), t_high=1.0, w=8,
                      top_p=float(np.float32(top_p)))
    xd = x.cuda()
    for u in (0.0, 0.37, 0.999):
        tok, H, T = (to_np(t) for t in s(xd, None, torch.full((M,), u, device="cuda")))
        for r in range(M):
            ln = x[r].double().numpy()
            Hr = R.token_entropy(ln)
            res = R.reset_update(states[r], Hr, False, p)
            assert abs(H[r] - Hr) <= 1e-4 * max(Hr, 1e-6), (r, H[r], Hr)
            assert R.temperature_is_ambiguous(res, p) or T[r] == np.float32(res.T)
            assert np.isfinite(ln[tok[r]]) and _token_ok(ln, float(T[r]), float(np.float32(u)), int(tok[r]), p.top_p)
    assert api.device_status() == 0


@pytest.mark.parametrize("V", [1000, 30011, 151936, LONG])
def test_uniforms_next_to_one_never_give_a_masked_token(V):
    """u = 1 - 2^-24: u Z rounds past the last partial sums now and then; the token is then the last one with mass."""
    M = 64 if V < 10 ** 5 else 16
    s = api.ResetSampler(M, V)
    u = torch.full((M,), 1 - 2.0 ** -24, device="cuda")
    rng = np.random.default_rng(V)
    for i in range(40):
        x = _logits(V, M, 1000 * V + i).cuda()
        cut = torch.from_numpy(rng.integers(1, V, M)).cuda()
        x[torch.arange(V, device="cuda")[None] >= cut[:, None]] = -np.inf
        x[:, 3::7] = -np.inf
        x[:, 0] = 0.0
        tok, _, _ = s(x, None, u)
        assert torch.isfinite(x.gather(1, tok.long()[:, None])).all(), i
    assert api.device_status() == 0


@pytest.mark.parametrize("V", [1000, 151936, LONG])
@pytest.mark.parametrize("top_p", [1.0, 0.9])
def test_rows_without_a_distribution_give_no_token_and_keep_their_state(V, top_p):
    """A row of -inf alone, one with NaN, one with +inf: token -1, reported, and the row goes on afterwards as if the
    call had not been; the other rows do not notice."""
    M = 4
    a, b = api.ResetSampler(M, V, top_p=top_p), api.ResetSampler(M, V, top_p=top_p)
    u = torch.tensor([0.1, 0.5, 0.9, 0.3], device="cuda")
    good = _logits(V, M, 5).cuda()
    for s in (a, b):
        s(good, None, u)
    bad = _logits(V, M, 6).cuda()
    bad[0] = -np.inf
    bad[1, V // 2] = np.nan
    bad[3, V - 1] = np.inf
    before = a.state.clone()
    assert api.device_status() == 0
    tok, H, T = (to_np(t).copy() for t in a(bad, None, u))
    assert tok[[0, 1, 3]].tolist() == [-1, -1, -1] and tok[2] >= 0
    assert np.all(H[[0, 1, 3]] == 0) and np.all(T[[0, 1, 3]] == np.float32(a.params.t_high))
    assert api.device_status() == api.DEVERR_NO_TOKEN
    stride = a.state.numel() // M
    same = (a.state == before).view(M, stride).all(1).cpu().tolist()
    assert same == [True, True, False, True]
    other = bad.clone()
    other[[0, 1, 3]] = good[[0, 1, 3]]
    tb, Hb, Tb = (to_np(t) for t in b(other, None, u))
    assert tb[2] == tok[2] and Hb[2] == H[2] and Tb[2] == T[2]
    b.state.view(M, stride)[[0, 1, 3]] = before.view(M, stride)[[0, 1, 3]]
    after = _logits(V, M, 7).cuda()
    for x, y in zip(a(after, None, u), b(after, None, u)):
        assert torch.equal(x, y)
    assert api.device_status() == 0


def test_no_alloc_rows_without_a_distribution():
    V, M = LONG, 2
    s = api.ResetSampler(M, V)
    x = _logits(V, M, 8).cuda()
    x[1] = -np.inf
    api.reset_sample_noalloc(x, None, torch.tensor([0.5, 0.5], device="cuda"), s.state, s.params, s.token, s.H, s.T)
    assert to_np(s.token)[0] >= 0 and to_np(s.token)[1] == -1 and api.device_status() == api.DEVERR_NO_TOKEN
