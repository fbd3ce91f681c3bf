"""The tests of the paged calls again, with page tables that have room for many
keys: short batches then take the kernel of long ones."""
import pytest

import test_gpu_paged as paged
from test_gpu_paged import (  # noqa: F401
    test_single_row, test_head_groups, test_chunks, test_many_sequences_of_one_key,
    test_empty_sequences_and_masked_rows, test_rows_before_and_behind_are_left_alone,
    test_prefix_single_rows, test_prefix_chunks, test_second_query_tile_of_few_rows,
    test_a_page_in_several_places, test_many_sequences, test_nothing_but_the_rows_is_written,
    test_large_scores, test_equal_keys_give_the_mean_of_the_values, test_strided_rows, test_scale,
    test_repeats_are_bit_identical, test_another_stream_and_two_at_once,
    test_captured_calls_follow_the_device_arrays, test_two_captured_calls_in_turn,
    test_append_rows_without_a_place, test_short_chunks,
    test_row_ranges_out_of_order_stay_inside, test_offsets_past_32_bits, test_drawn_batches,
    test_calls_one_after_another_share_a_workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def long_table(monkeypatch):
    monkeypatch.setattr(paged, "LEAST_KEYS", 12000)


def test_lengths_and_pages_out_of_range_are_bounded(h3lib):
    # as with short tables: lengths past the table are taken as the table's; pages
    # outside the pool read as zero keys and values
    n, page = 12032, 64
    P = paged.Paged([n, n], 2, page)
    q = paged.rnd(paged.gen(8), 2, 4, paged.DH)
    want = paged.attend(h3lib, q, P, [0, 1, 2])
    paged.check_attention(want, q, P, [0, 1, 2], False, paged.DH ** -0.5)
    c = h3lib.kv_cache(P.k, P.v)
    ws = paged.torch.empty(h3lib.attention_paged_workspace_bytes(2, 4), dtype=paged.torch.uint8,
                           device="cuda")
    o = paged.torch.empty_like(q)
    h3lib.attention_paged(q, o, c, h3lib.kv_batch(paged.i32([0, 1, 2]),
                                                  paged.i32([2 ** 31 - 1, n]), P.table, 2), ws)
    h3lib.check_device_error()
    assert paged.torch.equal(o, want)
    # where the keys are split goes by all lengths: another sum order for row 1
    h3lib.attention_paged(q, o, c, h3lib.kv_batch(paged.i32([0, 1, 2]), paged.i32([-5, n]),
                                                  P.table, 2), ws)
    h3lib.check_device_error()
    E = paged.Paged([0, n], 2, page)
    E.k, E.v, E.table = P.k, P.v, P.table
    paged.check_attention(o, q, E, [0, 1, 2], False, paged.DH ** -0.5, "no keys")
    for bad in (-1, P.pages, 2 ** 31 - 1, -2 ** 31):
        table = P.table.clone()
        table[0, 1] = bad
        b = h3lib.kv_batch(paged.i32([0, 1, 2]), paged.i32([n, n]), table, 2)
        h3lib.attention_paged(q, o, c, b, ws)
        h3lib.check_device_error()
        Z = paged.Paged([n], 2, page)
        k, v = (x.to(paged.torch.bfloat16).clone() for x in P.keys(0))
        k[page:2 * page], v[page:2 * page] = 0, 0
        Z.put(Z.table[0], k, v)
        paged.check_attention(o[:1], q[:1], Z, [0, 1], False, paged.DH ** -0.5, f"page {bad}")
        assert paged.torch.equal(o[1], want[1])
