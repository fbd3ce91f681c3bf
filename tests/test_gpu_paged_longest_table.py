"""The tests of the paged calls again, with page tables that have room for more than
131,072 keys: they then take the kernel whose parts may be of several runs."""
import pytest

import test_gpu_paged as paged
from test_gpu_paged import (  # noqa: F401
    test_single_row, test_head_groups, test_chunks, test_empty_sequences_and_masked_rows,
    test_rows_before_and_behind_are_left_alone, test_prefix_single_rows, test_prefix_chunks,
    test_second_query_tile_of_few_rows, test_nothing_but_the_rows_is_written, test_large_scores,
    test_repeats_are_bit_identical, test_another_stream_and_two_at_once,
    test_two_captured_calls_in_turn, test_row_ranges_out_of_order_stay_inside,
    test_drawn_batches, test_calls_one_after_another_share_a_workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def longest_table(monkeypatch):
    monkeypatch.setattr(paged, "LEAST_KEYS", 140000)
