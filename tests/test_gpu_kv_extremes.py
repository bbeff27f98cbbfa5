"""Rows that no scale of the cache reaches: codes, scales and signs equal to the quantizer's recipe."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_kv_cache import _bf16_values, _cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("glob", [1.0, 0.37, 2.0 ** -9, 2.0 ** -60, 2.0 ** -100, 2.0 ** 90, 3e-38])
@pytest.mark.parametrize("heads,tokens", [(1, 5), (300, 60)])
def test_extreme_values_of_both_signs(glob, heads, tokens):
    """Quotients that overflow FP32 saturate with the value's own sign, as infinities do; a NaN takes the largest code
    and its sign, and the block's scale is that of the other values.  Both ways of the append."""
    D, page = 128, 16
    assert (tokens * heads * D > 1 << 21) == (heads == 300)
    rng = np.random.default_rng(heads)
    x = rng.standard_normal((tokens, heads, D)).astype(np.float32)
    mag = rng.choice([0.0, 1e-44, 1e-30, 1.0, 400.0, 1e10, 1e30, 3e38, np.inf], (tokens, heads, D // 16))
    with np.errstate(all="ignore"):
        x = np.where(rng.random(x.shape) < 0.3, np.copysign(np.repeat(mag, 16, -1), x), x * np.float32(glob)).astype(np.float32)
    x[0, 0, :16] = [-3e38, 1, -1, 0, -0.0, 2, 3, -np.inf, np.inf, -4, 5, 6, 7, -8, 9, -10]
    k = torch.from_numpy(x).to(torch.bfloat16)
    v = torch.from_numpy(-x[::-1].copy()).to(torch.bfloat16)
    n_pages = -(-tokens // page)
    c = _cache(n_pages, page, heads, D, glob, glob)
    slots = np.arange(tokens, dtype=np.int32)
    api.nvfp4_kv_append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), c)
    got = S.read_slots(to_np(c.pages), slots.astype(np.int64), page, D)
    for rows, codes, scales in ((k, got[0], got[1]), (v, got[2], got[3])):
        # by the recipe, on the host: the scale's argument may be infinite, the codes saturate at +-6
        b = _bf16_values(rows).reshape(tokens, heads, D // 16, 16)
        g = np.float32(glob)
        with np.errstate(all="ignore"):
            t = (np.abs(b).max(-1) / (np.float32(6) * g)).astype(np.float32)
        s = S.e4m3_encode_nonneg(np.minimum(t, np.float32(448)))
        assert np.array_equal(scales, s)
        with np.errstate(all="ignore"):
            step = (S.e4m3_decode(s).astype(np.float32) * g)[..., None]
            q = np.where(step > 0, b / np.where(step > 0, step, np.float32(1)), np.copysign(np.float32(0), b))
            q = np.copysign(np.minimum(np.abs(q), np.float32(6)), b).astype(np.float32)
        want = S.e2m1_encode(q).reshape(codes.shape)
        assert np.array_equal(codes, want), np.argwhere(codes != want)[:3]


def test_nan_takes_its_sign_and_no_scale():
    x = torch.zeros((1, 1, 64), dtype=torch.float32)
    x[0, 0, :4] = torch.tensor([1.0, -2.0, 6.0, 3.0])
    x[0, 0, 4] = np.nan
    x.view(torch.int32)[0, 0, 5] = -0x400000                    # a NaN with the sign bit
    c = _cache(1, 16, 1, 64, 1.0, 1.0)
    k = x.to(torch.bfloat16)
    k.view(torch.int16)[0, 0, 5] = -0x40                         # (whatever the cast made of it)
    api.nvfp4_kv_append(k.cuda(), k.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), c)
    codes = S.read_slots(to_np(c.pages), np.array([0]), 16, 64)[0][0, 0]
    assert codes[:6].tolist() == [2, 8 + 4, 7, 5, 7, 15]
