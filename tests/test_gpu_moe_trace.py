"""A traced step with experts holds what the step computed: rows by place in place of the dense gate and up products."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_moe_step import _start, _step
from tests.test_gpu_serving_step import _feed

pytestmark = pytest.mark.gpu


def test_trace():
    rng = np.random.default_rng(3)
    st = _step(layers=2)
    _start(st, rng, {0: 9, 1: 3})
    _feed(st, rng)
    trace = []
    st.run(trace=trace)
    assert len(trace) == 3 and not any("y_gu" in t for t in trace)
    assert torch.equal(trace[1]["h_mid"], st.h_mid) and not torch.equal(trace[0]["h_mid"], st.h_mid)
    for t in trace[:2]:                                            # the quantized rows are h_mid's
        xq = api.nvfp4_quantize_act(t["h_mid"])
        assert np.array_equal(to_np(xq.codes), to_np(t["xq_d"][0])) and np.array_equal(to_np(xq.scales), to_np(t["xq_d"][1]))
