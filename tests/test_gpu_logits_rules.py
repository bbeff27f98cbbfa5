"""Rules on the logits against FP64.  Each of at most five steps (penalty, two subtractions, the product
frequency * count, bias) is one FP32 rounding, 2^-24 of what it yields, and no intermediate is larger than the sum
of the magnitudes added up: |y - ref| <= 6 * 2^-24 * size (one step in reserve for the products' roundings)."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, to_np

pytestmark = pytest.mark.gpu


def _inputs(rng, M, V, hist, nb, masks, dtype=torch.float32):
    x = torch.from_numpy((rng.standard_normal((M, V)) * 4).astype(np.float32)).to(dtype)
    d = {}
    if hist:
        d["tokens"] = rng.integers(-2, V + 2, (M, hist)).astype(np.int32)
        d["tokens"][:, ::3] = rng.integers(0, min(V, 9), d["tokens"][:, ::3].shape)
        d["n_tokens"] = rng.integers(-1, hist + 3, M).astype(np.int32)
        d["n_prompt"] = rng.integers(-1, hist + 3, M).astype(np.int32)
        d["repetition"] = rng.uniform(0.7, 1.6, M).astype(np.float32)
        d["presence"] = rng.uniform(-1, 2, M).astype(np.float32)
        d["frequency"] = rng.uniform(-0.5, 0.5, M).astype(np.float32)
    if nb:
        d["bias_ids"] = rng.integers(-1, V + 1, (M, nb)).astype(np.int32)
        d["bias_ids"][:, nb // 2:] = d["bias_ids"][:, : nb - nb // 2]                 # repeated ids: the last holds
        d["bias_values"] = (rng.standard_normal((M, nb)) * 5).astype(np.float32)
    if masks:
        d["mask"] = rng.integers(-2 ** 31, 2 ** 31, (masks, (V + 31) // 32)).astype(np.int32)
        d["mask_rows"] = rng.integers(-2, masks + 1, M).astype(np.int32)
    return x, d


def _check(x, d, got, **kw):
    ref, size = S.process_logits(x.double().numpy(), **d, **kw)
    got = got.astype(np.float64)
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine])
    assert np.all(np.abs(got - np.where(fine, ref, 0))[fine] <= (6 * 2.0 ** -24 * size)[fine])


def _dev(d):
    return {k: torch.from_numpy(v).cuda() for k, v in d.items()}


@pytest.mark.parametrize("V", [1, 3, 31, 33, 1000, 4096, 4097, 32000, 151936])
@pytest.mark.parametrize("M,hist,nb,masks", [(1, 0, 0, 0), (3, 40, 0, 0), (2, 0, 9, 0), (3, 0, 0, 2), (5, 700, 30, 3),
                                             (1, 5000, 3, 1)])
def test_rules(V, M, hist, nb, masks):
    rng = np.random.default_rng(V + M * 7 + hist)
    x, d = _inputs(rng, M, V, hist, nb, masks)
    g = Guarded((M, V), torch.float32)
    api.nvfp4_process_logits(x.cuda(), out=g.t, **_dev(d))
    g.check("logits out")
    _check(x, d, to_np(g.t))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,V", [(64, 20000), (7, 151936), (100, 513), (300, 100)])
def test_batches_types_and_strides(dtype, M, V):
    rng = np.random.default_rng(M)
    x, d = _inputs(rng, M, V, 200, 20, 5, dtype)
    _check(x, d, to_np(api.nvfp4_process_logits(x.cuda(), **_dev(d))))
    wide = torch.zeros((M, V + 7), dtype=dtype, device="cuda")
    wide[:, 3:V + 3] = x.cuda()
    _check(x, d, to_np(api.nvfp4_process_logits(wide[:, 3:V + 3], **_dev(d))))


def test_in_place_and_parts():
    rng = np.random.default_rng(1)
    x, d = _inputs(rng, 4, 5000, 60, 8, 4)
    y = x.cuda()
    api.nvfp4_process_logits(y, out=y, **_dev(d))
    _check(x, d, to_np(y))
    for leave in ("n_prompt", "repetition", "presence", "frequency", "mask_rows"):
        part = {k: v for k, v in d.items() if k != leave}
        _check(x, part, to_np(api.nvfp4_process_logits(x.cuda(), **_dev(part))))


def test_infinities_nan_fill_and_empty_masks():
    V = 200
    x = torch.linspace(-3, 3, V).repeat(3, 1)
    x[:, 5], x[:, 6], x[:, 7] = -np.inf, np.inf, np.nan
    d = {"tokens": np.tile(np.arange(0, 20, dtype=np.int32), (3, 1)), "n_tokens": np.full(3, 20, np.int32),
         "n_prompt": np.full(3, 0, np.int32), "repetition": np.full(3, 1.5, np.float32),
         "mask": np.zeros((2, 7), np.int32), "mask_rows": np.array([0, 1, -1], np.int32)}
    d["mask"][1, 0] = 0b11100001
    y = to_np(api.nvfp4_process_logits(x.cuda(), **_dev(d)))
    assert np.all(np.isneginf(y[0]))                                    # nothing allowed
    assert np.isneginf(y[1, 5]) and np.isposinf(y[1, 6]) and np.isnan(y[1, 7]) and np.isneginf(y[1, 1:5]).all()
    assert np.isneginf(y[2, 5]) and np.isposinf(y[2, 6]) and np.isnan(y[2, 7]) and np.isfinite(y[2, 8:]).all()
    low = torch.finfo(torch.float32).min
    z = to_np(api.nvfp4_process_logits(x.cuda(), fill=low, **_dev(d)))
    assert np.all(z[0] == np.float32(low)) and np.all(z[1, 8:] == np.float32(low))


def test_counts_are_exact_for_many_repeats():
    """One token repeated 20000 times among others: its count is exact, and repeats give the same bits."""
    V, n = 3001, 20001
    tok = np.full((1, n), 77, np.int32)
    tok[0, ::2] = np.arange(n // 2 + 1) % V
    x = torch.zeros((1, V))
    d = {"tokens": tok, "n_tokens": np.array([n], np.int32), "frequency": np.array([0.5], np.float32)}
    y = api.nvfp4_process_logits(x.cuda(), **_dev(d))
    want = -0.5 * np.bincount(tok[0], minlength=V)
    assert np.array_equal(to_np(y)[0].astype(np.float64), want)
    assert torch.equal(y, api.nvfp4_process_logits(x.cuda(), **_dev(d)))


def test_into_the_sampler():
    """A grammar that allows one token a row, then the ReSET sampler: it samples that token."""
    M, V = 4, synth_vocab()
    allowed = [5, 31, 32, V - 1]
    mask = np.zeros((M, (V + 31) // 32), np.uint32)
    for r, t in enumerate(allowed):
        mask[r, t // 32] = np.uint32(1) << np.uint32(t % 32)
    x = torch.from_numpy(np.random.default_rng(2).standard_normal((M, V)).astype(np.float32)).cuda()
    y = api.nvfp4_process_logits(x, mask=torch.from_numpy(mask.view(np.int32)).cuda())
    tok, H, T = api.ResetSampler(M, V)(y, None, torch.tensor([0.0, 0.3, 0.9, 0.999]).cuda())
    assert to_np(tok).tolist() == allowed and np.all(to_np(H) == 0)
    assert api.device_status() == 0


def synth_vocab():
    from nvfp4_w4a4_decode_gemv_gb300 import synth
    return synth.LM_HEAD_VOCAB


def test_graph_capture():
    rng = np.random.default_rng(3)
    x, d = _inputs(rng, 2, 3000, 50, 4, 2)
    dev, xd = _dev(d), x.cuda()
    out = api.nvfp4_process_logits(xd, **dev)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.nvfp4_process_logits(xd, out=out, **dev)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)
