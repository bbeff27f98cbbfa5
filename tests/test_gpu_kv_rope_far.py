"""Far positions: q's bits and the cache's bytes at positions up to 131071, by the kernel for few tokens and by windows."""
import numpy as np
import pytest
import torch

from tests.test_gpu_kv_rope import _case, _windows

pytestmark = pytest.mark.gpu

LIMIT = 131072


@pytest.mark.parametrize("style", ["halves", "pairs"])
@pytest.mark.parametrize("D,rotated", [(64, 32), (128, 128)])
def test_few_tokens(D, rotated, style):
    rng = np.random.default_rng(D)
    positions = np.concatenate([np.linspace(0, LIMIT - 1, 60).astype(np.int64), LIMIT - 4 + np.arange(8)])   # 4 outside
    _case(68, 3, 2, D, rotated, style, torch.float32, rng.permutation(128)[:68], positions, 64, 2, limit=LIMIT)


@pytest.mark.parametrize("style", ["halves", "pairs"])
def test_many_tokens(style):
    slots, positions, n_pages = _windows(4200, 64, 0, np.random.default_rng(6))
    _case(4200, 2, 4, 128, 128, style, torch.bfloat16, slots, positions + LIMIT - 1600, 64, n_pages, limit=LIMIT)
