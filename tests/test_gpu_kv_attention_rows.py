"""The attention tests again, by the kernel for many query rows: a max_q that promises millions of rows chooses it
whatever the shapes are."""
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.test_gpu_kv_attention import (  # noqa: F401  (collected here with the fixture below)
    test_bad_pages_and_lengths_are_skipped_and_reported, test_cache_beyond_four_gigabytes, test_decode_groups,
    test_decode_lengths, test_decode_pages_and_ragged_batch, test_flat_and_peaked_weights, test_growing_scores,
    test_growing_scores_of_many_rows, test_many_rows_few_tiles_are_cut_and_merged,
    test_many_rows_of_more_requests_than_a_warp_has_lanes, test_many_rows_of_unequal_lengths, test_prefill_chunks,
    test_prompt_rows_of_many_requests, test_queries_of_very_different_magnitudes, test_repeat_streams_and_graph,
    test_row_ranges_outside_the_rows_are_skipped, test_several_rows_a_request, test_strided_queries_and_shared_output,
    test_windows)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def many_rows(monkeypatch):
    call = api.nvfp4_kv_attention

    def forced(q, cache, table, lens, starts=None, max_q=None, **kw):
        if starts is None:
            starts = torch.arange(q.shape[0] + 1, dtype=torch.int32, device=q.device)
        return call(q, cache, table, lens, starts, max_q=10 ** 6, **kw)

    monkeypatch.setattr(api, "nvfp4_kv_attention", forced)
