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
