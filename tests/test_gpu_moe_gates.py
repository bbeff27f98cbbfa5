"""SiLU of large gates: each gate is one product of a code and a scale, so that it is known to one FP32 rounding.

h = g / (1 + exp(-g)) u: a gate off by 2^-24 |g| shifts exp(-g) by as much, exp is off by 2 + 1.173 |g| ulp and the quotient
by 2: below 2^-15 for |g| < 105; BF16 rounds by 2^-8.  Where FP32's exp(-g) overflows (g < -88.72) h is 0.
"""
import numpy as np
import pytest
import torch

from oracle import nvfp4 as Q
from oracle.formats import e2m1_decode, e4m3_decode
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import bits

pytestmark = pytest.mark.gpu


def _gates():
    """64 (code, scale) of |code * scale| in 80 .. 104: every other one negative."""
    found = {}
    for c in range(1, 8):
        for s in range(1, 0x7F):
            v = float(e2m1_decode(np.array([c], np.uint8))[0] * e4m3_decode(np.array([s], np.uint8))[0])
            if 80 <= v <= 104:
                found.setdefault(v, (c, s))
    pick = [found[v] for v in sorted(found)]
    return [(pick[i // 2 % len(pick)][0] | (8 if i % 2 else 0), pick[i // 2 % len(pick)][1]) for i in range(64)]


# few places: one CTA an item, K split over a cluster; many places
@pytest.mark.parametrize("T,K", [(3, 64), (3, 512), (70, 64)])
def test_large_gates(T, K):
    factors = np.array([1.0, 0.9978, 0.9921, 1.0031, 1.0069], np.float32)      # the experts' global scales
    E, I = len(factors), 64
    codes, scales = np.zeros((E, 2 * I, K // 2), np.uint8), np.full((E, 2 * I, K // 16), 0x38, np.uint8)
    for i, (c, s) in enumerate(_gates()):
        codes[:, i, 0], scales[:, i, 0] = c, s
    codes[:, I:, 0], scales[:, I:, 0] = 7, 0x7E                                # u = 6 * 448
    w = api.nvfp4_moe_pack_weights(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(),
                                   torch.from_numpy(factors).cuda(), gated=True)
    x = np.zeros((T, K // 2), np.uint8)
    x[:, 0] = 2                                                                # 1.0
    xt = api.NVFP4Tensor(torch.from_numpy(x).cuda(), torch.full((T, K // 16), 0x38, dtype=torch.uint8, device="cuda"),
                         torch.ones(1, device="cuda"))
    r = api.nvfp4_moe_plan(torch.arange(E, dtype=torch.int32, device="cuda").repeat(T, 1), E)
    got = Q.bf16_bits_to_f32(bits(api.nvfp4_moe_gate_up(xt, w, r))).astype(np.float64).reshape(E, T, I)
    f = factors.astype(np.float64)[:, None, None]
    code = codes[:, :I, 0].astype(np.uint8)
    g = np.broadcast_to((e2m1_decode(code) * e4m3_decode(scales[:, :I, 0])).astype(np.float64)[:, None, :] * f, got.shape)
    want = g / (1.0 + np.exp(-g)) * (2688.0 * f)
    assert ((g < -87.4) & (g > -88.6)).any() and (g < -89).any() and (g > 89).any()
    normal, gone = g > -88.67, g < -88.77
    assert np.all(np.abs(got - want)[normal] <= np.abs(want)[normal] * (2.0 ** -8 + 2.0 ** -15))
    assert not got[gone].any()
    assert api.device_status() == 0
